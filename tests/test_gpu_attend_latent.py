"""Attention over a paged cache of latent rows (kv_attend_latent) against its definition in 64 bits. Bounds are derived in
``latentcheck.LatentProblem.reference``."""

import numpy as np
import pytest

from latentcheck import LatentProblem, NAN16

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

FMTS = (None, "e4m3fn")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    yield


def run(p, bad=0, **kw):
    import fp8_quant_gb300 as kv
    d = p.tensors("cuda")
    T = sum(p.nqs)
    err = torch.zeros(2, dtype=torch.int64, device="cuda")
    lse = torch.full((T, p.HQ), 123.0, device="cuda")
    out = torch.full((T, p.HQ, p.L), 55.0, dtype=d["q"].dtype, device="cuda")
    p.attend(d, out=out, lse=lse, err=err, **kw)
    st, n, first = kv.kv_error_poll(err)
    assert (n > 0) == (bad > 0) and st in (kv.KVStatus.OK, kv.KVStatus.ERR_INDEX_OOB)
    p.check(out, lse, kw.get("sm_scale"))
    return d, out, lse


BATCHES = {
    "one_key": ([1], [1]),
    "decode_ragged": ([1, 17, 300, 64, 129, 15, 63, 65], [1] * 8),
    "decode_long": ([5000, 70], [1, 1]),
    "speculative": ([90, 4, 333, 64], [4, 4, 2, 3]),
    "whole_prompts": ([33, 130, 257], [33, 130, 257]),
    "chunks": ([700, 129, 1000], [65, 128, 311]),
    "mixed": ([512, 1, 300, 640], [1, 1, 300, 2]),
}


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("batch", BATCHES)
def test_batches(batch, dtype, fmt):
    lens, nqs = BATCHES[batch]
    run(LatentProblem(lens, nqs, 8, 512, 64, dtype=dtype, fmt=fmt, seed=11))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("HQ", [1, 3, 5, 12, 24, 32, 33, 48, 64, 65, 130])
@pytest.mark.parametrize("batch", ["decode_ragged", "speculative"])
def test_heads(batch, HQ, fmt):
    lens, nqs = BATCHES[batch]
    run(LatentProblem(lens, nqs, HQ, 128, 64, dtype="f16", fmt=fmt, seed=12))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("L,R", [(512, 64), (256, 64), (256, 32), (128, 64), (64, 0), (576, 0), (16, 16), (8, 8), (40, 24), (264, 8), (512, 16),
                                 (200, 56), (384, 192), (504, 72), (512, 0)])
@pytest.mark.parametrize("batch", ["decode_ragged", "chunks"])
def test_dims(batch, L, R, fmt):
    lens, nqs = BATCHES[batch]
    if L > 512:
        L, R = 448, L + R - 448
    run(LatentProblem(lens, nqs, 6, L, R, fmt=fmt, seed=13))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("L,R", [(1, 0), (1, 1), (7, 6), (100, 12), (300, 20), (513, 64), (960, 64), (576, 0), (33, 64)])
def test_dims_of_the_general_kernel(L, R, fmt):
    run(LatentProblem([1, 50, 77], [1, 3, 20], 4, L, R, fmt=fmt, seed=14))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("page", [1, 3, 8, 16, 24, 32, 64, 128, 256])
@pytest.mark.parametrize("batch", ["decode_ragged", "chunks"])
def test_page_sizes(batch, page, fmt):
    lens, nqs = BATCHES[batch]
    run(LatentProblem(lens, nqs, 12, 256, 64, fmt=fmt, page=page, seed=15))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("batch", ["decode_ragged", "chunks"])
@pytest.mark.parametrize("layout", [dict(pad=3), dict(slot_pad=64), dict(slot_pad=8), dict(slot_pad=3), dict(q_gap=8), dict(q_gap=3),
                                    dict(pad=1, slot_pad=16, q_gap=16)])
def test_strides(layout, batch, fmt):
    lens, nqs = BATCHES[batch]
    run(LatentProblem(lens, nqs, 8, 128, 64, dtype="f16", fmt=fmt, seed=16, **layout))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("batch", [([0, 5, 0], [1, 1, 1]), ([0, 3, 2], [4, 7, 2]), ([20, 0], [90, 70]), ([30, 8, 9], [0, 8, 0])])
def test_rows_that_see_nothing(batch, fmt):
    """Empty sequences and rows before the first token: zeros, and lse -inf."""
    lens, nqs = batch
    run(LatentProblem(lens, nqs, 4, 128, 64, fmt=fmt, seed=17))


@pytest.mark.parametrize("what", [np.nan, np.inf])
@pytest.mark.parametrize("batch", ["speculative", "chunks", "whole_prompts"])
def test_nan_reaches_only_rows_that_see_it(batch, what):
    """A NaN or infinite value at a sequence's last key: only its last query sees it."""
    lens, nqs = BATCHES[batch]
    p = LatentProblem(lens, nqs, 4, 256, 64, seed=18)
    for b, n in enumerate(lens):
        pg, off = p.table[b, (n - 1) // p.page], (n - 1) % p.page
        p.cache[pg, off, 3] = NAN16["bf16"] if np.isnan(what) else 0x7F80
        p.value[pg, off, 3] = what
    d = p.tensors("cuda")
    out = p.attend(d)
    ref, bound, _, _ = p.reference()
    got = out.double().cpu().numpy()
    rows = np.ones(got.shape[0], bool)
    rows[p.q_start[1:][np.array(nqs) > 0] - 1] = False
    assert np.isfinite(got[rows]).all() and (np.abs(got[rows] - ref[rows]) <= bound[rows]).all()
    assert np.isnan(got[~rows]).any(axis=(1, 2)).all() or np.isinf(what)


def test_nan_scales_and_codes_reach_only_rows_that_see_them():
    lens, nqs = BATCHES["chunks"]
    p = LatentProblem(lens, nqs, 4, 256, 64, fmt="e4m3fn", seed=19)
    for b, n in enumerate(lens):
        pg, off = p.table[b, (n - 1) // p.page], (n - 1) % p.page
        p.scales[pg, off] = np.nan
        p.value[pg, off] = np.nan
    p.check(p.attend(p.tensors("cuda")))


@pytest.mark.parametrize("batch", ["decode_long", "chunks"])
def test_rows_of_very_different_scales(batch):
    """Rows whose scales differ by up to 2^60 from one another, zeros among them."""
    lens, nqs = BATCHES[batch]
    p = LatentProblem(lens, nqs, 8, 256, 64, fmt="e4m3fn", seed=20, scale_spread=8.0, scale=2.0 ** -9)
    pg, off = p.table[0, 1], 3
    p.scales[pg, off] = 0.0
    p.value[pg, off] = 0.0
    run(p)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("sm_scale", [0.0, -0.3, 2.0, 1e-3])
@pytest.mark.parametrize("batch", ["decode_ragged", "chunks"])
def test_scales_of_scores(batch, sm_scale, fmt):
    lens, nqs = BATCHES[batch]
    run(LatentProblem(lens, nqs, 8, 128, 64, fmt=fmt, seed=21, dtype="f16"), sm_scale=sm_scale)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("fmt", FMTS)
def test_growing_scores(dtype, fmt):
    """Scores that grow by far more than a weight's range from one tile of keys to the next."""
    p = LatentProblem([1000, 400], [3, 200], 8, 256, 64, dtype=dtype, fmt=fmt, seed=22, scale=20.0)
    run(p)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("batch", ["decode_ragged", "chunks"])
def test_bad_pages_and_lengths(batch, fmt):
    """Keys of pages out of range are not seen, a bad length counts as 0; both are counted."""
    import fp8_quant_gb300 as kv
    lens, nqs = BATCHES[batch]
    p = LatentProblem(lens, nqs, 8, 128, 64, fmt=fmt, seed=23)
    d = p.tensors("cuda")
    b = 2
    hidden = [1, 3]
    for page, bad in zip(hidden, (-1, p.num_pages)):
        d["table"][b, page] = bad
    d["lens"][1] = p.width * p.page + 1
    err = torch.zeros(2, dtype=torch.int64, device="cuda")
    lse = torch.zeros((sum(nqs), 8), device="cuda")
    out = p.attend(d, err=err, lse=lse)
    st, n, first = kv.kv_error_poll(err)
    assert st == kv.KVStatus.ERR_INDEX_OOB and first == 1 and n >= 2
    # the definition without the hidden keys
    rows = slice(p.q_start[b], p.q_start[b + 1])
    keys = np.array([j for j in range(lens[b]) if j // p.page not in hidden])
    from attncheck import UNIT, bits_to_f32
    k = p.value[p.table[b, keys // p.page], keys % p.page]
    q = bits_to_f32(p.q[rows], p.dtype).astype(np.float64)
    s = np.einsum("thd,nd->thn", q, k) / np.sqrt(p.D)
    s = np.where(keys[None, None] <= (lens[b] - nqs[b] + np.arange(nqs[b]))[:, None, None], s, -np.inf)
    some = np.isfinite(s).any(-1)
    w = np.exp(s - np.where(some, s.max(-1), 0.0)[..., None])
    w = w / np.maximum(w.sum(-1, keepdims=True), 1e-300)
    want = w @ k[:, :p.L]
    a = w @ np.abs(k[:, :p.L])
    got = out[rows].double().cpu().numpy()
    assert (np.abs(got - want) <= UNIT[p.dtype] * (np.abs(want) + a) * 1.1 + 1e-4).all()
    assert bool((out[p.q_start[1]:p.q_start[2]] == 0).all()) and bool(torch.isneginf(lse[p.q_start[1]:p.q_start[2]]).all())
    others = [i for i in range(len(lens)) if i not in (1, b)]
    ref, bound, _, _ = p.reference()
    for i in others:
        at = slice(p.q_start[i], p.q_start[i + 1])
        assert (np.abs(out[at].double().cpu().numpy() - ref[at]) <= bound[at]).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_behind_the_last_sequence_are_left(fmt):
    p = LatentProblem([40, 70], [3, 5], 8, 128, 64, fmt=fmt, seed=24)
    d = p.tensors("cuda")
    big = torch.cat((d["q"], torch.full((4, 8, 192), float("nan"), dtype=torch.bfloat16, device="cuda")))
    out = torch.full((12, 8, 128), 55.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((12, 8), 44.0, device="cuda")
    p.attend(dict(d, q=big), out=out, lse=lse)
    p.check(out[:8], lse[:8])
    assert bool((out[8:] == 55.0).all()) and bool((lse[8:] == 44.0).all())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("work", [None, 256, 1 << 20, 1 << 22])
def test_workspaces(work, fmt):
    """None and too small a one, too: the same rows; its head is zero after every call."""
    import fp8_quant_gb300 as kv
    p = LatentProblem([3000, 1, 777, 2048], [1, 1, 2, 1], 32, 512, 64, fmt=fmt, seed=25)
    d = p.tensors("cuda")
    w = None
    if work:
        w = torch.full((work,), 0x5A, dtype=torch.uint8, device="cuda")
        w[:kv.ATTEND_HEAD_BYTES] = 0
    for _ in range(2):
        p.check(p.attend(d, work=w))
        if w is not None:
            assert not bool(w[:kv.ATTEND_HEAD_BYTES].any())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("batch", ["decode_long", "chunks"])
def test_same_bits_again(batch, fmt):
    lens, nqs = BATCHES[batch]
    p = LatentProblem(lens, nqs, 32, 512, 64, fmt=fmt, seed=26)
    d = p.tensors("cuda")
    outs = [p.attend(d) for _ in range(4)]
    assert all(torch.equal(outs[0], o) for o in outs[1:])


@pytest.mark.parametrize("fmt", FMTS)
def test_graph_over_growing_sequences_and_a_stream_of_its_own(fmt):
    p = LatentProblem([900, 64, 1500], [1, 1, 1], 16, 512, 64, fmt=fmt, seed=27)
    d = p.tensors("cuda")
    work = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
    out = torch.empty((3, 16, 512), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    p.attend(d, out=out, work=work, q_start=None, stream=side)
    side.synchronize()
    p.check(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.attend(d, out=out, work=work, q_start=None)
    for lens in ([900, 64, 1500], [10, 1, 1499], [0, 64, 333]):
        d["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        p.lens = lens
        graph.replay()
        p.check(out)


def test_two_calls_at_once():
    """Two streams, a workspace each."""
    ps = [LatentProblem([4000, 2000], [1, 1], 32, 512, 64, seed=s) for s in (28, 29)]
    ds = [p.tensors("cuda") for p in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    outs = [None, None]
    works = [torch.zeros(1 << 24, dtype=torch.uint8, device="cuda") for _ in ps]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, (p, d) in enumerate(zip(ps, ds)):
            outs[i] = torch.empty((2, 32, 512), dtype=torch.bfloat16, device="cuda") if outs[i] is None else outs[i]
            p.attend(d, out=outs[i], work=works[i], stream=streams[i])
    torch.cuda.synchronize()
    for p, o in zip(ps, outs):
        p.check(o)


def test_offsets_beyond_32_bits():
    """Pages of a 7 GB cache, the last of them in use; scales behind 2^22 slots."""
    import fp8_quant_gb300 as kv
    p = LatentProblem([200, 64], [1, 2], 8, 512, 64, seed=30, page=64)
    d = p.tensors("cuda")
    pages = 46000
    cache = torch.zeros((pages, 64, 1, 576 + 640), dtype=torch.bfloat16, device="cuda")[..., :576]
    cache[-p.num_pages:] = d["cache"]
    d["cache"] = cache
    d["table"] = torch.where(d["table"] >= 0, d["table"] + (pages - p.num_pages), d["table"]).to(torch.int32)
    p.check(p.attend(d))
    del cache, d
    p = LatentProblem([200, 64], [1, 2], 8, 512, 64, seed=31, page=64, fmt="e4m3fn")
    d = p.tensors("cuda")
    cache = torch.zeros((pages, 64, 1, 576 + 1024), dtype=torch.uint8, device="cuda")[..., :576]
    cache[-p.num_pages:] = d["cache"]
    scales = torch.full((pages * 64, 1), float("nan"), device="cuda")
    scales[-p.num_pages * 64:] = d["scales"]
    d["cache"], d["scales"] = cache, scales
    d["table"] = torch.where(d["table"] >= 0, d["table"] + (pages - p.num_pages), d["table"]).to(torch.int32)
    p.check(p.attend(d))


@pytest.mark.parametrize("fmt", FMTS)
def test_an_append_and_the_attention_that_reads_it(fmt):
    """Prompts, then single tokens, as a server runs them: rows appended, then attended over, against 64 bits."""
    import fp8_quant_gb300 as kv
    from fp8_quant_gb300.examples import latent_layer as ex
    layer, outs, inputs = ex.generate((5, 130, 300), 4, fmt=fmt)
    want = torch.stack([ex.plain_attention(layer, x) for x in inputs])
    off = (outs[-1].double() - want).square().sum().sqrt() / want.square().sum().sqrt()
    # 16-bit rows, queries and weights: a few roundings of 2^-9 (rms); e4m3fn rows: codes 2^-5 off (rms, at most 2^-4) both as
    # keys and as values
    assert off.item() <= (2.0 ** -6 if fmt is None else 2.0 ** -3)
    assert kv.kv_error_poll(layer.err)[1] == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("HQ", [16, 32, 64])
def test_many_short_items_a_share(HQ, fmt):
    """Shares that hold the end of one sequence, whole ones of a tile, and the beginning of another; call after call. A warp
    that is late with an item's outputs must find the next items' scores."""
    rng = np.random.default_rng(5)
    lens = [int(n) for pair in zip(rng.integers(900, 2500, 20), rng.integers(0, 70, 20)) for n in pair]
    p = LatentProblem(lens, [1] * len(lens), HQ, 512, 64, fmt=fmt, seed=40, page=64)
    d = p.tensors("cuda")
    work = torch.zeros(1 << 25, dtype=torch.uint8, device="cuda")
    first = p.attend(d, work=work, q_start=None)
    p.check(first)
    for _ in range(50):
        outs = [p.attend(d, work=work, q_start=None) for _ in range(4)]
        assert all(torch.equal(first, o) for o in outs)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("nqs", [[1, 1], [20, 20]])
def test_a_split_call_that_lost_a_part_gives_nan(nqs, fmt):
    """The mark that a CTA leaves in the workspace's head, set beforehand: no row is made of parts that may be missing."""
    import fp8_quant_gb300 as kv
    p = LatentProblem([3000, 700], nqs, 8, 512, 64, fmt=fmt, seed=41)
    d = p.tensors("cuda")
    work = torch.zeros(kv.ATTEND_WORK_BYTES, dtype=torch.uint8, device="cuda")
    lse = torch.zeros(sum(nqs), 8, device="cuda")
    p.check(p.attend(d, work=work, lse=lse), lse)
    work.view(torch.int32)[1] = 1
    assert p.attend(d, work=work, lse=lse).isnan().all() and lse.isnan().all()
    work[:kv.ATTEND_HEAD_BYTES] = 0
    p.check(p.attend(d, work=work, lse=lse), lse)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("long", [90_000, 160_000])
def test_no_wait_runs_out_while_rows_are_done_again(long, fmt):
    """A NaN that one sequence's last token sees has its 64 rows done key by key, for seconds: longer than any wait may last.
    The CTA's next item waits all that time, and so does the other CTA of a pair, whose rows are the token's before.
    (Items enough that none is split.)"""
    import fp8_quant_gb300 as kv
    B = 700
    lens = [64] * B
    lens[150] = long
    p = LatentProblem(lens, [2] * B, 64, 128, 64, fmt=fmt, seed=42, page=64)
    at = p.table[150, (long - 1) // 64], (long - 1) % 64
    p.value[at[0], at[1], :] = np.nan
    p.cache[at[0], at[1], :] = 0x7F if fmt else NAN16[p.dtype]
    d = p.tensors("cuda")
    err = kv.error_record()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    out = p.attend(d, err=err)
    start.record()
    out = p.attend(d, out=out, err=err)
    end.record()
    assert kv.kv_error_poll(err) == (kv.KVStatus.OK, 0, -1)
    assert bool(out[301].isnan().all()) and not bool(out[:301].isnan().any()) and not bool(out[302:].isnan().any())
    if long > 100_000 and fmt is None:
        assert start.elapsed_time(end) > 2300      # it did take longer than a wait may


def _refused(call, args, name):
    import fp8_quant_gb300 as kv
    call(**args)
    torch.cuda.synchronize()
    with pytest.raises((kv.KVError, TypeError, ValueError)) as e:
        call(**dict(args, **{name: args[name].cpu()}))
    assert getattr(e.value, "status", kv.KVStatus.ERR_INVALID_ARG) == kv.KVStatus.ERR_INVALID_ARG
    call(**args)
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", ["q", "cache", "page_table", "seq_lens", "q_start", "scales", "out", "lse", "work", "err"])
def test_host_memory_is_refused(name):
    """Pageable host memory, before anything is launched."""
    import fp8_quant_gb300 as kv
    p = LatentProblem([40, 3], [2, 1], 4, 64, 64, fmt="e4m3fn", seed=43)
    d = p.tensors("cuda")
    a = dict(q=d["q"], cache=d["cache"], page_table=d["table"], seq_lens=d["lens"], q_start=d["q_start"], scales=d["scales"], fmt="e4m3fn",
             out=torch.empty(3, 4, 64, dtype=d["q"].dtype, device="cuda"), lse=torch.empty(3, 4, device="cuda"), latent_dim=64,
             work=torch.zeros(1 << 20, dtype=torch.uint8, device="cuda"), err=kv.error_record())
    _refused(kv.kv_attend_latent, a, name)


def test_two_graphs_with_one_workspace():
    ps = [LatentProblem([4000, 200], [1, 1], 32, 512, 64, seed=s) for s in (44, 45)]
    ds = [p.tensors("cuda") for p in ps]
    work = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
    outs = [torch.empty((2, 32, 512), dtype=torch.bfloat16, device="cuda") for _ in ps]
    graphs = []
    for p, d, o in zip(ps, ds, outs):
        p.attend(d, out=o, work=work)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            p.attend(d, out=o, work=work)
        graphs.append(g)
    for _ in range(3):
        for g, o in zip(graphs, outs):
            o.zero_()
            g.replay()
    torch.cuda.synchronize()
    for p, o in zip(ps, outs):
        p.check(o)
