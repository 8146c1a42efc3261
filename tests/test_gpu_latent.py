"""The append to a cache of latent rows (kv_store_latent) and its gather (kv_gather_latent) against their definitions:
dims, layouts, formats, rotations, bad slots and positions, the bytes around the rows, streams and graphs."""

import numpy as np
import pytest

from attncheck import E4M3_ALL, bits_to_f32
from latentcheck import StoreProblem, to_bits

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

FMTS = (None, "e4m3fn")
DIMS = [(512, 64), (256, 64), (256, 32), (128, 64), (8, 16), (24, 48), (1008, 16), (960, 64), (512, 512), (504, 0), (7, 6), (100, 0), (1, 2),
        (33, 64), (64, 24)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    yield


def run(p, skip=(), bad=0, **layout):
    import fp8_quant_gb300 as kv
    d = p.tensors("cuda", **layout)
    q_out = p.call(d)
    st, n, first = kv.kv_error_poll(d["err"])
    assert n == bad and (st == kv.KVStatus.ERR_INDEX_OOB) == (bad > 0)
    p.check(d, skip)
    if p.HQ:
        p.check_q(q_out)
    return d, first


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("L,R", DIMS)
def test_dims(L, R, norm, dtype, fmt):
    run(StoreProblem(37, L, R, HQ=3 if R else 0, dtype=dtype, fmt=fmt, norm=norm, seed=5))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T", [1, 2, 255, 2000])
@pytest.mark.parametrize("HQ", [1, 5, 32, 70])
def test_batches_and_heads(T, HQ, fmt):
    run(StoreProblem(T, 256, 64, HQ=HQ, fmt=fmt, seed=6, interleaved=HQ == 5, idx=np.int32 if T == 255 else np.int64))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("R,rot", [(64, 64), (64, 32), (64, 0), (16, 16), (48, 48), (6, 4), (512, 512)])
def test_rotations(R, rot, inter, fmt):
    run(StoreProblem(19, 128, R, HQ=4, fmt=fmt, rot=rot, interleaved=inter, dtype="f16", seed=7))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("layout", [dict(fused=True), dict(fused=True, gap=8), dict(fused=True, gap=1), dict(pad=64), dict(pad=3)])
def test_strides(layout, fmt):
    run(StoreProblem(50, 512, 64, HQ=2, fmt=fmt, seed=8), **layout)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("page", [1, 3, 64])
def test_pages(page, fmt):
    run(StoreProblem(130, 128, 32, fmt=fmt, page=page, seed=9))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("L", [256, 33])
def test_bad_slots_and_positions(L, fmt):
    """Tokens 3 and 11 have no slot, token 7 no position: two rows of queries are rotated all the same, one is left."""
    import fp8_quant_gb300 as kv
    p = StoreProblem(20, L, 64, HQ=2, fmt=fmt, seed=10)
    d = p.tensors("cuda")
    d["indices"][3], d["indices"][11], d["positions"][7] = -1, p.pages * p.page, p.max_pos
    d["q_out"] = torch.full_like(d["q"], 9.0)
    p.call(d)
    assert kv.kv_error_poll(d["err"]) == (kv.KVStatus.ERR_INDEX_OOB, 3, 3)
    p.check(d, [3, 7, 11])
    p.check_q(d["q_out"], [7])
    assert bool((d["q_out"][7] == 9.0).all())


@pytest.mark.parametrize("fmt", FMTS)
def test_queries_in_place_and_into_whole_rows(fmt):
    p = StoreProblem(33, 512, 64, HQ=6, fmt=fmt, seed=11)
    d = p.tensors("cuda")
    whole = torch.full((33, 6, 576), 3.0, dtype=torch.bfloat16, device="cuda")
    d["q_out"] = whole[..., 512:]
    p.call(d)
    p.check_q(d["q_out"])
    assert bool((whole[..., :512] == 3.0).all())
    d["q_out"] = d["q"]
    p.call(d)
    p.check_q(d["q"])
    p.check(d)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("L", [256, 33])
def test_rows_of_zeros_and_of_odd_values(L, fmt):
    """A row of zeros (its scale 1), a row with NaN, one with infinity: other rows do not notice."""
    p = StoreProblem(6, L, 64, norm=False, fmt=fmt, seed=12)
    p.c[1], p.r[1] = 0, 0
    p.c[2, 3], p.c[4, 5] = 0x7FC0, 0x7F80
    d = p.tensors("cuda")
    p.call(d)
    flat = d["cache"].reshape(-1, L + 64)
    rows = flat[torch.from_numpy(p.slots).cuda()]
    keep = [0, 1, 3, 5]
    if fmt is None:
        assert np.array_equal(to_bits(rows)[:, :L], p.c)
    else:
        sc = d["scales"][torch.from_numpy(p.slots).cuda(), 0].cpu().numpy()
        assert sc[1] == 1.0 and np.isfinite(sc[2]) and np.isinf(sc[4])
        codes = rows.cpu().numpy()
        # (zeros turned by a negative cosine are (+0)(-c) - (+0)s = -0)
        assert (codes[1, :L] == 0).all() and (codes[1] & 0x7F == 0).all() and codes[2, 3] == 0x7F and codes[4, 5] == 0x7F and (codes[4, 6:L] & 0x7F == 0).all()
        want, _ = p.rows()
        got = E4M3_ALL[codes[keep]] * sc[keep, None]
        assert (np.abs(got - want[keep]) <= 2.0 ** -4 * np.abs(want[keep]) * 1.001 + sc[keep, None] * 2.0 ** -10).all()


def test_norm_of_large_and_small_rows():
    """Squares near fp32's ends, and eps against a row of zeros."""
    p = StoreProblem(4, 512, 64, norm=True, seed=13)
    p.c[0] = 0
    p.c[1] = (p.c[1] & 0x8000) | 0x5F00     # 2^63 and a bit: their squares sum to 2^136 of fp32's 2^128
    p.c[2] = (p.c[2] & 0x8000) | 0x2000     # 2^-63: far below eps
    p.c[3] = (p.c[3] & 0x8000) | 0x5A00     # 2^53: sum 2^115
    d = p.tensors("cuda")
    p.call(d)
    rows = bits_to_f32(to_bits(d["cache"].reshape(-1, 576)[torch.from_numpy(p.slots).cuda()]), "bf16")
    want, off = p.rows()
    assert (rows[0, :512] == 0).all() and (rows[1, :512] == 0).all()   # the mean overflows: 1 / sqrt(inf)
    for i in (2, 3):
        assert (np.abs(rows[i] - want[i]) <= 2.0 ** -8 * np.abs(want[i]) + off[i] * 2 + 2.0 ** -130).all()


# -- the gather -------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("L,R,pad,page", [(512, 64, 0, 16), (512, 64, 64, 32), (256, 32, 0, 1), (8, 16, 8, 3), (7, 6, 0, 16), (100, 0, 4, 64),
                                          (960, 64, 2, 5)])
@pytest.mark.parametrize("T", [1, 33, 700])
def test_gather(T, L, R, pad, page, dtype, fmt):
    import fp8_quant_gb300 as kv
    p = StoreProblem(T, L, R, dtype=dtype, fmt=fmt, page=page, norm=False, seed=14, idx=np.int32 if T == 33 else np.int64)
    d = p.tensors("cuda", pad=pad)
    p.call(d)
    out = torch.full((T + 1, L + R + 5 if T == 33 else L + R), 4.0, dtype=d["c"].dtype, device="cuda")
    rows = out[:, :L + R]
    at = d["indices"].clone()
    if T > 5:
        at[2], at[5] = -3, p.pages * page
    err = torch.zeros(2, dtype=torch.int64, device="cuda")
    kv.kv_gather_latent(d["cache"], rows, at, page_size=page, fmt=fmt, scales=d.get("scales"), err=err)
    st, n, first = kv.kv_error_poll(err)
    assert (n, first) == ((2, 2) if T > 5 else (0, -1))
    keep = np.setdiff1d(np.arange(T), [2, 5] if T > 5 else [])
    flat = d["cache"].reshape(-1, L + R)[torch.from_numpy(p.slots[keep].astype(np.int64)).cuda()]
    if fmt is None:
        assert np.array_equal(to_bits(rows)[keep], to_bits(flat))
    else:
        sc = d["scales"][:, 0].cpu().numpy()[p.slots[keep].astype(np.int64)]
        want = torch.from_numpy((E4M3_ALL[flat.cpu().numpy()].astype(np.float32) * sc[:, None]).astype(np.float32)).to(out.dtype)
        assert torch.equal(rows[torch.from_numpy(keep).cuda()].cpu(), want)
    assert bool((out[T] == 4.0).all()) and (out.shape[1] == L + R or bool((out[:, L + R:] == 4.0).all()))
    if T > 5:
        assert bool((rows[2] == 4.0).all()) and bool((rows[5] == 4.0).all())


@pytest.mark.parametrize("fmt", FMTS)
def test_pinned_host_memory(fmt):
    """Inputs, slot ids and positions of an append, and a gather's rows, in page-locked host memory."""
    import fp8_quant_gb300 as kv
    p = StoreProblem(40, 512, 64, HQ=2, fmt=fmt, seed=15)
    d = p.tensors("cuda")
    for n in ("c", "r", "q", "indices", "positions"):
        d[n] = d[n].cpu().pin_memory()
    q = p.call(d)
    assert q.is_cuda
    p.check(d)
    p.check_q(q)
    out = torch.empty((40, 576), dtype=torch.bfloat16).pin_memory()
    kv.kv_gather_latent(d["cache"], out, d["indices"], page_size=p.page, fmt=fmt, scales=d.get("scales"), err=d["err"])
    dev = torch.empty_like(out, device="cuda")
    kv.kv_gather_latent(d["cache"], dev, d["indices"], page_size=p.page, fmt=fmt, scales=d.get("scales"), err=d["err"])
    torch.cuda.synchronize()
    assert torch.equal(out, dev.cpu())


@pytest.mark.parametrize("fmt", FMTS)
def test_graph_and_streams(fmt):
    """An append and a gather captured together, replayed over new inputs; and on a stream of their own."""
    import fp8_quant_gb300 as kv
    ps = [StoreProblem(64, 512, 64, HQ=4, fmt=fmt, seed=s) for s in (16, 17)]
    ds = [p.tensors("cuda") for p in ps]
    d = ps[0].tensors("cuda")
    d["q_out"] = torch.empty_like(d["q"])
    out = torch.empty((64, 576), dtype=torch.bfloat16, device="cuda")

    def both(stream=None):
        ps[0].call(d, stream=stream)
        kv.kv_gather_latent(d["cache"], out, d["indices"], page_size=16, fmt=fmt, scales=d.get("scales"), err=d["err"], stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    both(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for p, new in zip(ps[::-1], ds[::-1]):
        for n in ("c", "r", "q", "indices", "positions"):
            d[n].copy_(new[n])
        d["weight"].copy_(new["weight"])
        d["store"].fill_(7.0 if fmt is None else 0x55)
        if fmt:
            d["scales"].fill_(-3.0)
        graph.replay()
        p.check(d)
        p.check_q(d["q_out"])
        slots = torch.from_numpy(p.slots).cuda()
        want = d["cache"].reshape(-1, 576)[slots]
        if fmt:
            want = (want.view(torch.float8_e4m3fn).float() * d["scales"][slots]).to(out.dtype)
        assert torch.equal(out, want)


def test_many_slots_and_far_pages():
    """Byte offsets beyond 2^32: the last page of a 6 GB cache."""
    import fp8_quant_gb300 as kv
    pages, page = 45000, 64
    cache = torch.zeros((pages, page, 1, 576 + 512), dtype=torch.bfloat16, device="cuda")[..., :576]
    p = StoreProblem(64, 512, 64, page=page, seed=18)
    d = p.tensors("cuda")
    at = torch.arange(64, device="cuda") + (pages - 1) * page
    kv.kv_store_latent(d["c"], d["r"], cache, at, d["positions"], d["cos_sin"], weight=d["weight"], page_size=page, err=d["err"])
    out = torch.zeros((64, 576), dtype=torch.bfloat16, device="cuda")
    kv.kv_gather_latent(cache, out, at, page_size=page, err=d["err"])
    want, off = p.rows()
    got = out.double().cpu().numpy()
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + off * 2).all()
    assert torch.equal(out, cache[-1, :, 0])
    assert kv.kv_error_poll(d["err"])[1] == 0
