"""Attention at the edges of what its layouts may be: far strides, pages that no row needs, bytes next to a row's own."""

import pytest

torch = pytest.importorskip("torch")

from attncheck import AttendProblem

pytestmark = pytest.mark.gpu

FMTS = (None, "e4m3fn", "e2m1")
WIDE = 60000    # tokens that a table row has room for: short sequences then take the kernels of long ones


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    yield


def tensors(p, wide):
    d = p.tensors(torch.device("cuda"))
    if wide:
        t = d["table"]
        d["table"] = torch.full((t.shape[0], WIDE // p.page), -1, dtype=torch.int32, device="cuda")
        d["table"][:, :t.shape[1]] = t
    return d


SLOT = (1 << 28) + (1 << 26)    # 7 and 8 of them pass 2^31


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("wide,nq", [(False, 1), (False, 3), (True, 1), (False, 40)])
def test_slot_strides_beyond_28_bits(wide, nq, fmt):
    """A slot-major cache ([page_size, pages, H, D]): rows of one page lie 320 MB apart."""
    p = AttendProblem([90, 33, 17], [nq, 1, nq], 8, 4, 64, fmt=fmt, seed=51)
    d = tensors(p, wide)
    big = torch.empty(p.page * SLOT, dtype=torch.uint8, device="cuda")
    at = 0
    for n in ("kc", "vc"):
        t = d[n]
        eb, (pages, _, H, W) = t.element_size(), t.shape
        d[n] = big.view(t.dtype).as_strided(t.shape, (H * W, SLOT // eb, W, 1), at // eb)
        d[n].copy_(t)
        at += pages * H * W * eb
    assert at <= SLOT
    p.check(p.attend(d))


@pytest.mark.parametrize("wide,nq", [(False, 1), (True, 1), (True, 3), (False, 40)])
@pytest.mark.parametrize("D,H", [(32, 8), (96, 8), (96, 16), (80, 4), (112, 2), (48, 2), (160, 4)])
def test_block_scales_next_to_a_row(D, H, wide, nq):
    """NaN scales of another head or of a slot that no row sees leave every other row's bits as they are."""
    p = AttendProblem([333, 64, 50, 1], [nq, 1, nq, 1], 2 * H, H, D, fmt="e2m1", page=32, seed=52)
    d = tensors(p, wide)
    want = p.attend(d)
    p.check(want)
    used = torch.from_numpy(p.used).cuda()[..., None, None]
    clean = dict(d, ks=torch.where(used, d["ks"], 0), vs=torch.where(used, d["vs"], 0))
    assert torch.equal(p.attend(clean).view(torch.int16), want.view(torch.int16))
    dirty = dict(d, ks=d["ks"].clone(), vs=d["vs"].clone())
    for n in ("ks", "vs"):
        dirty[n][:, :, 1] = 0x7F
    got = p.attend(dirty)
    others = [h for h in range(2 * H) if h // 2 != 1]
    assert torch.equal(got[:, others].view(torch.int16), want[:, others].view(torch.int16))
    assert got[:, 2:4].isnan().all()


def check_without_unseen_pages(p, wide):
    """A window's freed pages: no count in the record, and the bits of a whole table. They hold NaN, too."""
    d = tensors(p, wide)
    err = torch.zeros(2, dtype=torch.int64, device="cuda")
    want = p.attend(d, err=err)
    table, gone = d["table"].clone(), 0
    bare = {n: d[n].clone() for n in ("kc", "vc", "ks", "vs") if n in d}
    for b, n in enumerate(p.lens):
        seen = p.visible(b).any(0)
        for i in range(-(-n // p.page)):
            if not seen[i * p.page:(i + 1) * p.page].any():
                table[b, i] = -1
                gone += 1
                for x in bare.values():
                    x[p.table[b, i]] = float("nan") if x.dtype.is_floating_point else 0x7F
    assert gone > 3
    p.check(want)
    got = p.attend(dict(d, table=table), err=err)
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    assert not err.any()
    assert torch.equal(p.attend(dict(d, **bare), err=err).view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page,window,sinks", [(16, 100, 4), (16, 40, 20), (32, 300, 1), (16, 64, 0), (64, 65, 70), (8, 33, 3)])
@pytest.mark.parametrize("nq", [1, 3, 40])
def test_pages_that_no_row_sees_may_be_gone(nq, page, window, sinks, D, fmt):
    check_without_unseen_pages(AttendProblem([1000, 333, 64, 450], [nq, 1, 2, nq], 8, 4, D, fmt=fmt, page=page, window=window,
                                             sinks=sinks, seed=53), False)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("page,window,sinks", [(16, 1040, 4), (16, 1041, 20), (32, 1100, 1), (48, 1077, 0), (64, 1030, 70)])
@pytest.mark.parametrize("B,H,nq", [(64, 1, 1), (20, 8, 3)])
def test_pages_of_long_windows_may_be_gone(B, H, nq, page, window, sinks, fmt):
    """Windows of 8 MB and more together, of few rows each, as the TMA-fed kernels take them."""
    lens = [1500 - 19 * (i % 23) for i in range(B)]
    p = AttendProblem(lens, [nq, 1] * (B // 2), 2 * H if H == 1 else H, H, 128, fmt=fmt, page=page, window=window, sinks=sinks, seed=54)
    check_without_unseen_pages(p, True)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("B,nq,wide", [(200, 40, False), (200, 1, True)])
def test_a_bad_page_is_its_own_sequences_matter(B, nq, wide, fmt):
    """Sequences without a bad page keep their bits, whatever a CTA met before them; the others' keys there are hidden."""
    import numpy as np
    import fp8_quant_gb300 as kv
    p = AttendProblem([64 + i % 3 for i in range(B)], [nq] * B, 4, 1, 128, fmt=fmt, page=16, seed=55)
    d = tensors(p, wide)
    want = p.attend(d)
    bad = list(range(0, B, 3)) + list(range(104, 152))      # first items of CTAs that have two, among them
    table = d["table"].clone()
    table[bad, 1] = -1
    err = kv.error_record()
    got = p.attend(dict(d, table=table), err=err)
    status, n, first = kv.kv_error_poll(err)
    assert status == kv.KVStatus.ERR_INDEX_OOB and n >= len(set(bad)) and first == 0
    good = [i for i in range(B) if i not in bad]
    assert torch.equal(got.view(B, nq, 4, 128)[good].view(torch.int16), want.view(B, nq, 4, 128)[good].view(torch.int16))
    see = p.visible
    hide = lambda n: (np.arange(n) < 16) | (np.arange(n) >= 32)   # noqa: E731
    p.visible = lambda b: see(b) & hide(p.lens[b]) if b in bad else see(b)
    p.check(got)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("nq,wide", [(1, False), (3, True), (40, False)])
def test_rows_done_again_are_written_last(nq, wide, fmt):
    """Rows that a hidden NaN touched: their second result and its lse stay, call after call."""
    p = AttendProblem([500, 333, 64], [nq] * 3, 8, 2, 64, fmt=fmt, page=16, window=70, sinks=2, seed=56)
    d = tensors(p, wide)
    for b, n in enumerate(p.lens):      # the window's page holds hidden keys in front of it, NaN now
        j = n - nq - 70
        if j > 2:
            at = p.table[b, j // 16], j % 16
            x = d["vc"] if fmt is None else d["ks"] if fmt == "e2m1" else d["vc"]
            x[at] = float("nan") if fmt is None else 0x7F
    first = lse = None
    for i in range(10):
        out, l = torch.full_like(d["q"], 7.0), torch.full((3 * nq, 8), 7.0, device="cuda")
        p.attend(d, out=out, lse=l)
        if i == 0:
            p.check(out, l)
            first, lse = out, l
        assert torch.equal(out.view(torch.int16), first.view(torch.int16)) and torch.equal(l, lse)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("B,nq,n,page", [(48, 4, 3000, 64), (48, 4, 3000, 32), (96, 2, 1500, 16), (64, 1, 4000, 64)])
def test_long_calls_repeat_themselves(B, nq, n, page, fmt):
    """Enough shares that the copies run into the next one while a warp still multiplies: the same bits thirty times."""
    import fp8_quant_gb300 as kv
    HQ, H, D, dev = 32, 8, 128, "cuda"
    g = torch.Generator(device=dev).manual_seed(57)
    lens = torch.tensor([n - 11 * i for i in range(B)], dtype=torch.int32, device=dev)
    need = -(-n // page)
    pages = B * need
    table = torch.randperm(pages, generator=g, device=dev).to(torch.int32).view(B, need)
    a = dict(fmt=fmt, q_start=torch.arange(0, B * nq + 1, nq, dtype=torch.int32, device=dev))
    if fmt is None:
        kc, vc = (torch.randn(pages, page, H, D, generator=g, device=dev, dtype=torch.bfloat16) for _ in range(2))
    else:
        width = D // 2 if fmt == "e2m1" else D
        kc, vc = (torch.randint(0, 256, (pages, page, H, width), generator=g, device=dev, dtype=torch.uint8) for _ in range(2))
        if fmt == "e4m3fn":
            kc, vc = (x & 0xB7 for x in (kc, vc))          # finite, at most 1.875
        else:
            a["k_scales"], a["v_scales"] = (torch.randint(0x28, 0x30, (pages, page, H, D // 16), generator=g, device=dev,
                                                          dtype=torch.uint8) for _ in range(2))
    q = torch.randn(B * nq, HQ, D, generator=g, device=dev, dtype=torch.bfloat16)
    work = torch.zeros(kv.ATTEND_WORK_BYTES, dtype=torch.uint8, device=dev)
    first = kv.kv_attend(q, kc, vc, table, lens, work=work, **a)
    assert first.isfinite().all()
    for _ in range(30):
        assert torch.equal(kv.kv_attend(q, kc, vc, table, lens, work=work, **a).view(torch.int16), first.view(torch.int16))
