"""Tensors in pageable host memory, where the kernels want device memory: refused before anything is launched."""

import pytest

torch = pytest.importorskip("torch")

from attncheck import AttendProblem, rope_table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    yield


def refused(call, args, name):
    import fp8_quant_gb300 as kv
    call(**args)
    torch.cuda.synchronize()
    with pytest.raises((kv.KVError, TypeError, ValueError)) as e:
        call(**dict(args, **{name: args[name].cpu()}))
    assert getattr(e.value, "status", kv.KVStatus.ERR_INVALID_ARG) == kv.KVStatus.ERR_INVALID_ARG
    call(**args)
    torch.cuda.synchronize()


@pytest.mark.parametrize("fmt,names", [
    (None, ["k", "v", "k_cache", "v_cache", "indices", "positions", "cos_sin", "q", "q_out", "err"]),
    ("e4m3fn", ["cos_sin", "inv_k_scale", "inv_v_scale"]), ("e2m1", ["k_cache", "k_scales", "v_scales", "inv_v_scale"])])
def test_host_memory_in_an_append(fmt, names):
    import fp8_quant_gb300 as kv
    T, HQ, H, D, dev = 5, 4, 2, 64, "cuda"
    a = dict(indices=torch.arange(T, device=dev), positions=torch.arange(T, device=dev),
             cos_sin=torch.from_numpy(rope_table(16, D)).to(dev), err=kv.error_record(), fmt=fmt)
    for n, h in (("q", HQ), ("q_out", HQ), ("k", H), ("v", H)):
        a[n] = torch.ones(T, h, D, dtype=torch.bfloat16, device=dev)
    width = D // 2 if fmt == "e2m1" else D
    for n in ("k_cache", "v_cache"):
        a[n] = torch.zeros(32, H, width, dtype=torch.uint8 if fmt else torch.bfloat16, device=dev)
    if fmt:
        a["inv_k_scale"], a["inv_v_scale"] = (torch.ones(1, device=dev) for _ in range(2))
    if fmt == "e2m1":
        a["k_scales"], a["v_scales"] = (torch.zeros(32, H, D // 16, dtype=torch.uint8, device=dev) for _ in range(2))
    for name in names:
        refused(kv.kv_store_rope, a, name)


@pytest.mark.parametrize("name", ["k_cache", "v_cache", "k_scales", "v_scales", "k_out", "v_out", "indices", "k_scale", "err"])
def test_host_memory_in_a_gather(name):
    import fp8_quant_gb300 as kv
    T, H, D, dev = 5, 2, 64, "cuda"
    a = dict(indices=torch.arange(T, device=dev), err=kv.error_record(), k_scale=torch.ones(1, device=dev))
    for n in ("k_cache", "v_cache"):
        a[n] = torch.zeros(32, H, D // 2, dtype=torch.uint8, device=dev)
    for n in ("k_scales", "v_scales"):
        a[n] = torch.zeros(32, H, D // 16, dtype=torch.uint8, device=dev)
    for n in ("k_out", "v_out"):
        a[n] = torch.zeros(T, H, D, dtype=torch.bfloat16, device=dev)
    refused(kv.kv_gather_fp4, a, name)


@pytest.mark.parametrize("fmt,names", [
    (None, ["q", "k_cache", "v_cache", "page_table", "seq_lens", "q_start", "out", "lse", "work", "err"]),
    ("e4m3fn", ["k_scale", "v_scale"]), ("e2m1", ["v_cache", "k_scales", "v_scales", "k_scale"])])
def test_host_memory_in_attention(fmt, names):
    import fp8_quant_gb300 as kv
    p = AttendProblem([40, 3], [2, 1], 4, 2, 64, fmt=fmt, page=16, seed=81)
    d = p.tensors(torch.device("cuda"))
    a = dict(q=d["q"], k_cache=d["kc"].contiguous(), v_cache=d["vc"].contiguous(), page_table=d["table"], seq_lens=d["lens"],
             q_start=d["q_start"], out=torch.empty_like(d["q"]), lse=torch.empty(3, 4, device="cuda"),
             work=torch.zeros(1 << 20, dtype=torch.uint8, device="cuda"), err=kv.error_record(), fmt=fmt,
             k_scale=d.get("k_scale"), v_scale=d.get("v_scale"), k_scales=d.get("ks"), v_scales=d.get("vs"))
    for name in names:
        refused(kv.kv_attend, a, name)
