"""Attention over the paged cache (kv_attend) against its definition in 64 bits: head layouts,
lengths from zero to several thousand, windows and sinks, page sizes that end inside a tile,
strides, NaN in every place that no row sees, and bad tables and lengths. Bounds are derived in
``attncheck.AttendProblem.reference``."""

import numpy as np
import pytest

from attncheck import AttendProblem

pytestmark = pytest.mark.gpu

FMTS = (None, "e4m3fn", "e2m1")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    yield


def run(p, **kw):
    import torch
    import fp8_quant_gb300 as kv
    dev = torch.device("cuda")
    d = p.tensors(dev)
    T = sum(p.nqs)
    err = torch.zeros(2, dtype=torch.int64, device=dev)
    lse = torch.full((T, p.HQ), 123.0, device=dev)
    out = torch.full((T, p.HQ, p.D), 55.0, dtype=d["q"].dtype, device=dev)
    p.attend(d, out=out, lse=lse, err=err, **kw)
    st, n, first = kv.kv_error_poll(err)
    assert (st, n) == (0, 0)
    p.check(out, lse, kw.get("sm_scale"))
    return d, out, lse


# decode-sized and prefill-sized batches: (lens, queries)
BATCHES = {
    "one_key": ([1], [1]),
    "decode_ragged": ([1, 17, 300, 64, 129, 15], [1] * 6),
    "decode_long": ([5000, 70], [1, 1]),
    "speculative": ([90, 4, 333], [4, 4, 2]),
    "whole_prompts": ([33, 130, 257], [33, 130, 257]),
    "chunks": ([700, 129, 1000], [65, 128, 311]),
    "mixed": ([512, 1, 300, 640], [1, 1, 300, 2]),
}
HEADS = {"gqa4": (8, 2), "mha": (3, 3), "mqa8": (8, 1), "gqa5": (10, 2), "mqa20": (20, 1)}


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("batch", BATCHES)
def test_batches(batch, fmt):
    lens, nqs = BATCHES[batch]
    run(AttendProblem(lens, nqs, 8, 2, 128, fmt=fmt, seed=11))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("batch", ["decode_ragged", "speculative", "chunks"])
def test_heads(heads, batch, fmt):
    HQ, H = HEADS[heads]
    lens, nqs = BATCHES[batch]
    run(AttendProblem(lens, nqs, HQ, H, 64, dtype="f16", fmt=fmt, seed=12))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 4), (100, 0), (64, 33), (4096, 4), (7, 1000)])
@pytest.mark.parametrize("batch", ["decode_ragged", "speculative", "chunks", "whole_prompts"])
def test_windows(batch, window, sinks, fmt):
    lens, nqs = BATCHES[batch]
    run(AttendProblem(lens, nqs, 8, 2, 64, fmt=fmt, window=window, sinks=sinks, seed=13))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [16, 48, 64, 80, 96, 112, 128, 160, 192, 256, 320])
@pytest.mark.parametrize("batch", ["decode_ragged", "chunks"])
def test_head_dims(batch, D, fmt):
    lens, nqs = BATCHES[batch]
    run(AttendProblem(lens, nqs, 4, 2, D, fmt=fmt, window=90, sinks=3, seed=14))


@pytest.mark.parametrize("fmt", [None, "e4m3fn"])
@pytest.mark.parametrize("D", [1, 7, 40, 72, 100, 576])
def test_head_dims_of_the_general_kernel(D, fmt):
    run(AttendProblem([1, 50, 77], [1, 3, 20], 4, 2, D, fmt=fmt, window=40, sinks=2, seed=15))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("page", [1, 3, 16, 24, 64, 256])
@pytest.mark.parametrize("batch", ["decode_ragged", "chunks"])
def test_page_sizes(batch, page, fmt):
    lens, nqs = BATCHES[batch]
    run(AttendProblem(lens, nqs, 4, 1, 128, fmt=fmt, page=page, window=200, sinks=5, seed=16))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("batch", ["decode_ragged", "chunks"])
@pytest.mark.parametrize("layout", [dict(hnd=True), dict(pad=3), dict(q_gap=8), dict(q_gap=3),
                                    dict(hnd=True, pad=1, q_gap=16)])
def test_strides(layout, batch, fmt):
    lens, nqs = BATCHES[batch]
    run(AttendProblem(lens, nqs, 8, 4, 64, dtype="f16", fmt=fmt, seed=17, **layout))


@pytest.mark.parametrize("fmt", FMTS)
def test_cache_offset_by_one_element(fmt):
    """Bases off their 16-byte alignment take the general kernel and give the same rows."""
    import torch
    p = AttendProblem([40, 3], [1, 2], 4, 2, 64, fmt=fmt, seed=18)
    d = p.tensors(torch.device("cuda"))
    for n in ("kc", "vc"):
        big = torch.empty(d[n].numel() + 1, dtype=d[n].dtype, device="cuda")
        moved = big[1:].view(d[n].shape)
        moved.copy_(d[n])
        d[n] = moved
    p.check(p.attend(d))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("batch", [([0, 5, 0], [1, 1, 1]), ([0, 3, 2], [4, 7, 2]), ([20, 0], [90, 70]),
                                   ([30, 8, 9], [0, 8, 0])])
def test_rows_that_see_nothing(batch, fmt):
    """Empty sequences and rows before the first token: zeros, and lse -inf."""
    lens, nqs = batch
    d, out, lse = run(AttendProblem(lens, nqs, 4, 2, 64, fmt=fmt, window=3, seed=19))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("batch", ["speculative", "chunks", "whole_prompts"])
def test_nan_reaches_only_rows_that_see_it(batch, fmt):
    """A NaN value row inside the sequences: rows whose mask hides it are as if it were not there."""
    lens, nqs = BATCHES[batch]
    p = AttendProblem(lens, nqs, 4, 2, 64, fmt=fmt, window=24, sinks=2, seed=20)
    for b, n in enumerate(lens):
        for j in (n - 1, max(0, n - 30)):
            pg, off = p.table[b, j // p.page], j % p.page
            p.value[1][pg, off, 0, :] = np.nan
            if fmt is None:
                p.cache[1][pg, off, 0, :] = 0x7FC0
            elif fmt == "e4m3fn":
                p.cache[1][pg, off, 0, :] = 0x7F
            else:
                p.scales[1][pg, off, 0, :] = 0x7F
    run(p)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("batch", ["decode_ragged", "chunks"])
def test_infinite_keys_hidden_or_weightless(batch, dtype):
    """Keys whose scores are -inf weigh nothing; the type's largest values do no harm."""
    lens, nqs = BATCHES[batch]
    p = AttendProblem(lens, nqs, 4, 2, 64, dtype=dtype, seed=21)
    big = 0x7F7F if dtype == "bf16" else 0x7BFF
    low = 0xFF7F if dtype == "bf16" else 0xFBFF
    p.q[:] = np.abs(p.q.view(np.int16)).astype(np.uint16) & 0x7FFF   # positive queries
    for b, n in enumerate(lens):
        if n > 2:
            pg, off = p.table[b, 0], 1
            p.cache[0][pg, off] = low              # the lowest finite value
            p.cache[1][pg, off] = big              # never weighed
            p.value[0][pg, off] = -1e30
            p.value[1][pg, off] = 1.0
    import torch
    d = p.tensors(torch.device("cuda"))
    out = p.attend(d)
    assert torch.isfinite(out).all()
    p.check(out)


@pytest.mark.parametrize("fmt", FMTS)
def test_queries_of_any_size(fmt):
    """Queries near the top of bf16's range over small keys (the quantised caches are multiplied in
    fp16 after a power of two per row)."""
    p = AttendProblem([300, 70], [1, 40], 8, 2, 64, fmt=fmt, seed=22, scale=2.0 ** 60)
    run(p, sm_scale=2.0 ** -63)
    p = AttendProblem([300, 70], [1, 40], 8, 2, 64, fmt=fmt, seed=22, scale=2.0 ** -60)
    run(p, sm_scale=2.0 ** 57)


@pytest.mark.parametrize("batch", ["decode_long", "decode_ragged", "chunks"])
@pytest.mark.parametrize("fmt", FMTS)
def test_workspace_sizes_and_repeats(batch, fmt):
    """Any workspace will do, none included; the same call gives the same bytes."""
    import torch
    import fp8_quant_gb300 as kv
    lens, nqs = BATCHES[batch]
    p = AttendProblem(lens, nqs, 8, 2, 128, fmt=fmt, seed=23)
    d = p.tensors(torch.device("cuda"))
    for size in (256, 1 << 16, 1 << 20, 6 << 20, kv.ATTEND_WORK_BYTES):
        work = torch.randint(0, 256, (size,), dtype=torch.uint8, device="cuda")
        work[:kv.ATTEND_HEAD_BYTES] = 0
        a = p.attend(d, work=work)
        p.check(a)
        for _ in range(3):
            assert torch.equal(p.attend(d, work=work).view(torch.int16), a.view(torch.int16))
        assert not work[:kv.ATTEND_HEAD_BYTES].any()
    T = sum(nqs)
    out = torch.empty_like(a)
    err = kv.error_record()
    st = (d["q"].stride(0) * 2, d["q"].stride(1) * 2, out.stride(0) * 2, out.stride(1) * 2)
    eb = d["kc"].element_size()
    st += tuple(x * eb for x in d["kc"].stride()[:3]) + tuple(x * eb for x in d["vc"].stride()[:3])
    sc = None
    if fmt == "e2m1":
        sc = (d["ks"].data_ptr(), d["vs"].data_ptr(), *d["ks"].stride()[:3], *d["vs"].stride()[:3])
    rc = kv.raw.kv_attend(
        d["q"].data_ptr(), out.data_ptr(), None, d["kc"].data_ptr(), d["vc"].data_ptr(),
        d["table"].data_ptr(), p.width, p.width, d["lens"].data_ptr(), d["q_start"].data_ptr(),
        len(lens), T, p.HQ, p.H, p.D, 1, st, p.page, p.num_pages, {None: 0, "e4m3fn": 1, "e2m1": 2}[fmt],
        d["k_scale"].data_ptr() if fmt else None, d["v_scale"].data_ptr() if fmt else None, sc,
        128 ** -0.5, 0, 0, None, 0, err.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    p.check(out)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("sm_scale", [0.0, -0.3, 2.0])
@pytest.mark.parametrize("batch", ["speculative", "chunks"])
def test_score_scales(batch, sm_scale, fmt):
    """Any finite scale: 0 weighs all visible keys alike, a negative one turns the order round."""
    lens, nqs = BATCHES[batch]
    run(AttendProblem(lens, nqs, 4, 2, 64, fmt=fmt, window=40, sinks=1, seed=28, scale=0.25), sm_scale=sm_scale)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("nq", [1, 30])
def test_bad_pages_and_lengths(nq, fmt):
    """Keys of a page id out of range are not visible; a length out of range counts as 0; both are
    counted, and the other sequences are as ever."""
    import torch
    import fp8_quant_gb300 as kv
    p = AttendProblem([100, 90, 80], [nq] * 3, 4, 2, 64, fmt=fmt, seed=24)
    d = p.tensors(torch.device("cuda"))
    table = d["table"].clone()
    table[0, 2] = p.num_pages                         # keys 32 .. 47 of sequence 0
    table[0, 3] = -1                                  # keys 48 .. 63
    lens = d["lens"].clone()
    lens[1] = p.width * p.page + 1
    d2 = dict(d, table=table, lens=lens)
    err = kv.error_record()
    lse = torch.empty((3 * nq, 4), device="cuda")
    out = p.attend(d2, lse=lse, err=err)
    st, n, first = kv.kv_error_poll(err)
    assert st == kv.KVStatus.ERR_INDEX_OOB and n >= 2 and first == 0
    hide = np.ones((nq, 100), bool)
    hide[:, 32:64] = False
    see = p.visible
    p.visible = lambda b: see(b) & hide if b == 0 else see(b)
    p.lens[1] = 0
    p.check(out, lse)


@pytest.mark.parametrize("fmt", FMTS)
def test_many_long_sequences(fmt):
    """Enough keys that CTAs take several shares and items are cut anywhere."""
    lens = [9000 - 517 * i for i in range(16)]
    run(AttendProblem(lens, [1] * 16, 16, 8, 64, fmt=fmt, page=32, seed=29))
    run(AttendProblem(lens, [3] * 16, 2, 1, 128, fmt=fmt, page=64, window=3000, sinks=40, seed=30))


def test_q_start_is_clamped_and_gaps_are_left_alone():
    import torch
    p = AttendProblem([40, 40], [3, 2], 4, 2, 64, seed=25)
    d = p.tensors(torch.device("cuda"))
    out = torch.full_like(d["q"], 7.0)
    p.attend(d, q_start=torch.tensor([1, 3, 99], dtype=torch.int32, device="cuda"), out=out)
    assert (out[0] == 7.0).all()
    full = out.clone()
    p.attend(d, q_start=torch.tensor([-4, -1, -1], dtype=torch.int32, device="cuda"), out=out)
    assert torch.equal(out, full)


def test_stream_and_graph():
    """On a side stream, with its own workspace, and captured in a CUDA graph."""
    import torch
    p = AttendProblem([900, 33], [1, 1], 8, 2, 128, fmt="e4m3fn", seed=26)
    d = p.tensors(torch.device("cuda"))
    ref = p.attend(d)
    p.check(ref)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = p.attend(d, stream=s)
    s.synchronize()
    assert torch.equal(got, ref)
    out = torch.empty_like(ref)
    work = torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")
    p.attend(d, out=out, work=work)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.attend(d, out=out, work=work)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        p.check(out)


def test_cache_beyond_32_bits():
    """Rows whose byte offsets pass 2^32 (a 6 GB cache, pages at its end)."""
    import torch
    import fp8_quant_gb300 as kv
    ps, H, D, n = 64, 8, 128, 1000
    pages = (6 << 30) // (ps * H * D * 2)
    kc = torch.empty((pages, ps, H, D), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    p = AttendProblem([n, n], [1, 40], 16, H, D, page=ps, seed=27)
    d = p.tensors(torch.device("cuda"))
    first = pages - p.num_pages
    kc[first:], vc[first:] = d["kc"], d["vc"]
    table = torch.where(d["table"] >= 0, d["table"] + first, d["table"])
    out = kv.kv_attend(d["q"], kc, vc, table, d["lens"], q_start=d["q_start"])
    p.check(out)
