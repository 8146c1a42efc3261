"""Rotated appends whose query heads do not fill whole passes of a warp, so that one warp holds rows of Q, K
and V side by side, some written as they are and some quantised."""

import pytest

pytest.importorskip("torch")

from test_gpu_rope import run

pytestmark = pytest.mark.gpu

FMTS = (None, "e4m3fn", "e2m1")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    yield


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("HQ,H,D,R", [(14, 2, 64, 64), (14, 2, 64, 32), (3, 1, 128, 128), (7, 3, 128, 96), (5, 5, 128, 64),
                                      (9, 3, 96, 96), (1, 2, 32, 32), (25, 5, 64, 0), (3, 3, 256, 192)])
@pytest.mark.parametrize("T", [1, 700])
def test_rows_of_all_kinds_in_a_warp(T, HQ, H, D, R, interleaved, fmt):
    run(T, HQ, H, D, R, "bf16", fmt, interleaved=interleaved, seed=9)


def test_pinned_queries_without_an_output():
    import torch
    import fp8_quant_gb300 as kv
    from attncheck import rope_table
    T, HQ, H, D = 30, 4, 2, 64
    q, k, v = (torch.randn(T, h, D).to(torch.bfloat16) for h in (HQ, H, H))
    tab, pos = torch.from_numpy(rope_table(64, 64)).cuda(), torch.arange(T, device="cuda")
    got = []
    for put in (lambda x: x.cuda(), lambda x: x.pin_memory()):
        kc, vc = (torch.zeros(32, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        got.append(kv.kv_store_rope(put(k), put(v), kc, vc, pos, pos, tab, q=put(q)))
        torch.cuda.synchronize()
    assert got[1].is_cuda and torch.equal(*got)
