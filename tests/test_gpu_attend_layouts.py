"""Attention over caches of every layout that the kernels for long page tables meet, and calls side by side.

A page table much wider than its sequences stands for a large cache, so that short sequences
take the kernels that long ones do.
"""

import pytest

torch = pytest.importorskip("torch")

from attncheck import AttendProblem

pytestmark = pytest.mark.gpu

FMTS = (None, "e4m3fn", "e2m1")
WIDE = 60000    # tokens that a table row has room for

LENS, NQ1, NQ3 = [1, 15, 16, 17, 63, 64, 65, 127, 333, 1100, 0], [1] * 11, [1, 3, 2, 1, 3, 3, 1, 2, 3, 3, 0]


def widened(p):
    d = p.tensors(torch.device("cuda"))
    t = d["table"]
    wide = torch.full((t.shape[0], max(WIDE // p.page, t.shape[1])), -1, dtype=torch.int32, device="cuda")
    wide[:, :t.shape[1]] = t
    d["table"] = wide
    return d


def run(p, **kw):
    d = widened(p)
    lse = torch.empty(sum(p.nqs), p.HQ, device="cuda")
    err = torch.zeros(2, dtype=torch.int64, device="cuda")
    p.check(p.attend(d, lse=lse, err=err, **kw), lse)
    assert err[0].item() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("HQ,H", [(1, 1), (4, 2), (6, 3), (10, 5), (16, 8), (12, 12), (16, 2)])
@pytest.mark.parametrize("D", [32, 64, 96, 128])
def test_heads_and_dims(D, HQ, H, fmt):
    """KV heads that share 128 bytes of a slot and heads that do not; scales in one run and not."""
    run(AttendProblem(LENS, NQ1, HQ, H, D, fmt=fmt, page=32, seed=41))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("page", [16, 48, 64, 80, 128, 8, 20])
@pytest.mark.parametrize("D", [64, 128])
def test_pages(D, page, fmt):
    """Pages of whole tiles, of a tile's part, and of neither."""
    run(AttendProblem(LENS, NQ3, 8, 4, D, fmt=fmt, page=page, seed=42))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("layout", [dict(hnd=True), dict(pad=16), dict(pad=3), dict(q_gap=8), dict(hnd=True, pad=16)])
@pytest.mark.parametrize("D", [64, 128])
def test_strides(D, layout, fmt):
    run(AttendProblem(LENS, NQ1, 8, 4, D, fmt=fmt, page=16, seed=43, **layout))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (64, 4), (100, 33), (700, 0)])
def test_windows(window, sinks, fmt, dtype):
    run(AttendProblem(LENS, NQ3, 8, 2, 128, dtype=dtype, fmt=fmt, page=16, window=window, sinks=sinks, seed=44))


@pytest.mark.parametrize("fmt", FMTS)
def test_two_streams_at_once(fmt):
    """Calls on two streams, each with its workspace, and the record's counts of both."""
    p = AttendProblem([3000, 700, 2100, 5], [1] * 4, 16, 4, 128, fmt=fmt, page=16, seed=45)
    d = widened(p)
    want = p.attend(d)
    p.check(want)
    streams = [torch.cuda.Stream() for _ in range(2)]
    works = [torch.zeros(8 << 20, dtype=torch.uint8, device="cuda") for _ in streams]
    outs = [[torch.empty_like(want) for _ in range(20)] for _ in streams]
    torch.cuda.synchronize()
    for i in range(20):
        for s, w, o in zip(streams, works, outs):
            p.attend(d, out=o[i], work=w, stream=s)
    torch.cuda.synchronize()
    # another number of shares joins in another grouping of the sums: the call with its own workspace size
    # is the reference for its bytes, the 64-bit definition for its values
    for o in outs:
        p.check(o[0])
        for x in o[1:]:
            assert torch.equal(x, outs[0][0])


@pytest.mark.parametrize("fmt", FMTS)
def test_tensors_made_on_another_stream(fmt):
    """Outputs and workspace left to the call belong to the stream that it runs on."""
    p = AttendProblem([300, 40], [1, 1], 8, 2, 128, fmt=fmt, page=16, seed=46)
    d = widened(p)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = [p.attend(d, stream=s) for _ in range(5)]
    trash = [torch.full((1 << 20,), 7.0, device="cuda") for _ in range(8)]   # on the current stream
    s.synchronize()
    torch.cuda.synchronize()
    assert len(trash) == 8
    for o in outs:
        p.check(o)
