"""CPU checks of attention's binding and statuses beside tests/test_attend_cpu.py."""

import pytest

import fp8_quant_gb300 as kv
from fp8_quant_gb300 import build as kvbuild


@pytest.fixture(scope="module", autouse=True)
def lib():
    kvbuild.build()
    return kv.load_library()


def test_status_of_a_wait():
    assert kv.kv_status_str(5) == "KV_ERR_WAIT" and kv.KVStatus(5).name == "ERR_WAIT"


def test_a_workspace_is_contiguous(monkeypatch):
    import torch
    monkeypatch.setattr(kv.raw, "kv_attend", lambda *a: pytest.fail("called"))
    q, kc = (torch.zeros(s, dtype=torch.bfloat16) for s in ((2, 8, 64), (4, 16, 2, 64)))
    with pytest.raises(ValueError, match="contiguous"):
        kv.kv_attend(q, kc, kc, torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                     work=torch.zeros(4096, dtype=torch.uint8)[::2], err=torch.zeros(2, dtype=torch.int64))


def test_rotated_queries_belong_to_the_caches_device(monkeypatch):
    """Queries may be page-locked host memory; a result on the host beside them would be refused."""
    import torch
    monkeypatch.setattr(kv.raw, "kv_store_rope", lambda *a: 0)
    monkeypatch.setattr(kv, "_stream_handle", lambda stream, device: 0)
    q, k = torch.zeros(3, 8, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    cache = torch.zeros(16, 2, 64, dtype=torch.bfloat16, device="meta")
    out = kv.kv_store_rope(k, k, cache, cache, torch.arange(3), torch.arange(3), torch.zeros(9, 64), q=q,
                           err=torch.zeros(2, dtype=torch.int64))
    assert out.device == cache.device and out.shape == q.shape


@pytest.mark.parametrize("shape,page_size", [((64, 2, 64), 0), ((64, 2, 64), -16), ((4, 0, 2, 64), None), ((64, 0, 64), 16)])
def test_empty_pages_and_caches_are_refused(shape, page_size, monkeypatch):
    import torch
    monkeypatch.setattr(kv.raw, "kv_attend", lambda *a: pytest.fail("called"))
    q, kc = torch.zeros(2, 8, 64, dtype=torch.bfloat16), torch.zeros(shape, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        kv.kv_attend(q, kc, kc, torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), page_size=page_size,
                     work=torch.zeros(256, dtype=torch.uint8), err=torch.zeros(2, dtype=torch.int64))
