"""The rotated append (kv_store_rope) and the 4-bit gather (kv_gather_fp4), byte for byte against
float32 steps rounded one by one (numpy) and 64-bit code tables, and within their roundings of the
rotation in 64 bits."""

import numpy as np
import pytest

import workloads as wl
from attncheck import (E4M3_ALL, UNIT, bits_to_f32, e4m3_codes, fp4_rows, fp4_values, rope_table,
                       rotated)

pytestmark = pytest.mark.gpu

FMTS = (None, "e4m3fn", "e2m1")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build()
    yield


def same16(got, want, dtype):
    """Equal bytes; any NaN for a NaN."""
    gn, wn = (np.isnan(bits_to_f32(x, dtype)) for x in (got, want))
    return np.array_equal(gn, wn) and np.array_equal(got[~gn], want[~wn])


def problem(T, HQ, H, D, dtype, seed, fused=False, special=False):
    n = (HQ + 2 * H) * D
    x = wl.to_bits(wl.normal(seed, T * n) * np.float32(2.0), dtype).reshape(T, n)
    if special:   # infinities, NaN, the largest values, subnormals and zeros of either sign
        pats = [0x7F80, 0xFF80, 0x7FC1, 0x7F7F, 0xFF7F, 0x0001, 0x8001, 0x0000, 0x8000] if dtype == "bf16" \
            else [0x7C00, 0xFC00, 0x7E01, 0x7BFF, 0xFBFF, 0x0001, 0x8001, 0x0000, 0x8000]
        at = wl.splitmix64(seed + 5, 0, x.size // 7) % np.uint64(x.size)
        x.reshape(-1)[at.astype(np.int64)] = np.resize(np.array(pats, np.uint16), at.size)
        x[0] = 0
    return x


def run(T, HQ, H, D, R, dtype="bf16", fmt=None, page=16, interleaved=False, idx=np.int64, pdt=np.int64,
        seed=3, fused=True, q="out", bad=(), bad_pos=(), pad=0, special=False, hnd=False, scales=True,
        table_pad=0, gather=True):
    import torch
    import fp8_quant_gb300 as kv
    dev = torch.device("cuda")
    dt = torch.bfloat16 if dtype == "bf16" else torch.float16
    x = problem(T, HQ, H, D, dtype, seed, fused, special)
    max_pos = 4096
    table = rope_table(max_pos, R)
    pos = (wl.splitmix64(seed + 1, 0, T) % np.uint64(max_pos)).astype(pdt)
    pages = -(-(T + 40) // page)
    slots = wl.distinct_slots(seed + 2, pages * page, T).astype(idx)
    for t, s in bad:
        slots[t] = s if s < 0 else pages * page + s
    for t, s in bad_pos:
        pos[t] = s if s < 0 else max_pos + s
    width = {None: D, "e4m3fn": D, "e2m1": D // 2}[fmt]
    w = torch.from_numpy(x.view(np.int16)).to(dev).view(dt)
    tq, tk, tv = w.split((HQ * D, H * D, H * D), 1)
    if not fused:
        tq, tk, tv = tq.contiguous(), tk.contiguous(), tv.contiguous()
    tq, tk, tv = (t.unflatten(1, (-1, D)) for t in (tq, tk, tv))
    xq, xk, xv = (a.reshape(T, -1, D) for a in np.split(x, [HQ * D, (HQ + H) * D], 1))

    def cache(w, dtype, fill):
        shape = (pages, H, page + pad, w) if hnd else (pages, page + pad, H, w)
        c = torch.full(shape, fill, dtype=dtype, device=dev)
        return (c.transpose(1, 2) if hnd else c)[:, :page]
    cdt, fill = (torch.int16, 0x7A5A) if fmt is None else (torch.uint8, 0x5A)
    kc, vc = cache(width, cdt, fill), cache(width, cdt, fill)
    ks, vs = (cache(D // 16, torch.uint8, 0x5B) for _ in range(2)) if fmt == "e2m1" else (None, None)
    inv = np.array([13.7, 0.31], np.float32) if scales and fmt else None
    tinv = None if inv is None else torch.from_numpy(inv).to(dev)
    ttab = torch.zeros((max_pos, R + table_pad), device=dev)
    ttab[:, :R] = torch.from_numpy(table).to(dev)
    err = kv.error_record()
    tq_out = None
    if q == "out":
        tq_out = torch.full((T, HQ, D), 3.0, dtype=dt, device=dev)
    elif q == "in_place":
        tq_out = tq
    res = kv.kv_store_rope(
        tk, tv, kc.view(dt) if fmt is None else kc, vc.view(dt) if fmt is None else vc,
        torch.from_numpy(slots).to(dev), torch.from_numpy(pos).to(dev), ttab[:, :R],
        q=None if q is None else tq, q_out=tq_out, page_size=page, interleaved=interleaved, fmt=fmt,
        inv_k_scale=None if inv is None else tinv[0:1], inv_v_scale=None if inv is None else tinv[1:2],
        k_scales=ks, v_scales=vs, err=err)
    st, n, first = kv.kv_error_poll(err)
    skipped = sorted({t for t, _ in bad} | {t for t, _ in bad_pos})
    assert n == len(skipped) and first == (skipped[0] if skipped else -1)

    pos_ok = (pos >= 0) & (pos < max_pos)
    ok = pos_ok & (slots >= 0) & (slots < pages * page)
    p = np.where(pos_ok, pos, 0).astype(np.int64)
    f32 = {n: bits_to_f32(a, dtype) for n, a in (("q", xq), ("k", xk), ("v", xv))}
    rot = {n: rotated(f32[n], table, p, interleaved) for n in "qk"}
    to16 = lambda a: wl.to_bits(a, dtype).reshape(a.shape)   # noqa: E731
    if q is not None:
        got = res.view(torch.int16).cpu().numpy().view(np.uint16)
        want = to16(rot["q"])
        want[..., R:] = xq[..., R:]
        if q == "in_place":
            want[~pos_ok] = xq[~pos_ok]
        else:
            want[~pos_ok] = wl.to_bits(np.float32([3.0]), dtype)[0]
        assert same16(got, want, dtype)
        if not special:   # the rotation in 64 bits, within its roundings
            z = table.astype(np.float64)[p, None]
            ia, ib = (np.arange(0, R, 2), np.arange(1, R, 2)) if interleaved else (
                np.arange(R // 2), np.arange(R // 2, R))
            a, b = (f32["q"][..., i].astype(np.float64) for i in (ia, ib))
            e = np.array(f32["q"], np.float64)
            e[..., ia], e[..., ib] = a * z[..., :R // 2] - b * z[..., R // 2:], b * z[..., :R // 2] + a * z[..., R // 2:]
            mag = np.zeros_like(e)
            mag[..., ia] = mag[..., ib] = np.abs(a) + np.abs(b)
            lim = UNIT[dtype] * np.abs(e) * 1.001 + mag * 2.0 ** -22 + 2.0 ** -25
            assert (np.abs(bits_to_f32(got, dtype) - e)[pos_ok] <= lim[pos_ok]).all()
    else:
        assert res is None
    rows = slots[ok].astype(np.int64)
    with np.errstate(invalid="ignore", over="ignore"):
        for side, c, sc, i in (("k", kc, ks, 0), ("v", vc, vs, 1)):
            y = rot["k"] if side == "k" else f32["v"]
            flat = c.cpu().numpy()
            flat = flat.reshape(pages * page, H, -1)
            if fmt is None:
                want = np.full((pages * page, H, D), 0x7A5A, np.uint16)
                v16 = to16(y)
                raw_ = xk if side == "k" else xv
                keep = R if side == "k" else 0
                v16[..., keep:] = raw_[..., keep:]
                want[rows] = v16[ok]
                assert same16(flat.view(np.uint16), want, dtype)
                continue
            y = (y * (np.float32(1.0) if inv is None else inv[i])).astype(np.float32)
            want = np.full((pages * page, H, width), 0x5A, np.uint8)
            if fmt == "e4m3fn":
                want[rows] = e4m3_codes(y)[ok]
            else:
                codes, bs = fp4_rows(y)
                want[rows] = codes[ok]
                wsc = np.full((pages * page, H, D // 16), 0x5B, np.uint8)
                wsc[rows] = bs[ok]
                assert np.array_equal(sc.cpu().numpy().reshape(wsc.shape), wsc)
            assert np.array_equal(flat, want)
    if fmt == "e2m1" and gather:
        gk = torch.full((T, H, D), 9.0, dtype=dt, device=dev)
        gv = gk.clone()
        fwd = torch.tensor([0.13, 2.7], dtype=torch.float32, device=dev)
        kv.kv_gather_fp4(kc, vc, ks, vs, gk, gv, torch.from_numpy(slots).to(dev), page_size=page,
                         k_scale=fwd[0:1], v_scale=None, err=err)
        st, n, first = kv.kv_error_poll(err)
        slot_bad = ~((slots >= 0) & (slots < pages * page))
        assert n == int(slot_bad.sum())
        at = np.where(slot_bad, 0, slots).astype(np.int64)
        for out, c, sc, g in ((gk, kc, ks, np.float32(0.13)), (gv, vc, vs, np.float32(1.0))):
            val = fp4_values(c.cpu().numpy().reshape(pages * page, H, -1)[at],
                             sc.cpu().numpy().reshape(pages * page, H, -1)[at]).astype(np.float32)
            want = to16((val * g).astype(np.float32))
            want[slot_bad] = wl.to_bits(np.float32([9.0]), dtype)[0]
            assert same16(out.view(torch.int16).cpu().numpy().view(np.uint16), want, dtype)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T", [1, 2, 63, 500])
def test_sizes(T, dtype, fmt):
    run(T, 8, 2, 128, 128, dtype, fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(64, 64), (64, 32), (128, 64), (128, 96), (96, 48), (48, 48), (80, 80), (128, 2),
                                 (128, 0), (16, 16), (256, 128), (192, 64), (32, 10), (576, 64)])
def test_head_and_rotary_dims(D, R, interleaved, fmt):
    run(37, 3, 2, D, R, "bf16", fmt, interleaved=interleaved)


@pytest.mark.parametrize("fmt", [None, "e4m3fn"])
@pytest.mark.parametrize("D,R", [(1, 0), (7, 6), (20, 20), (45, 30), (72, 40)])
def test_odd_head_dims(D, R, fmt):
    run(21, 2, 3, D, R, "f16", fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("kw", [dict(fused=False), dict(q=None), dict(q="in_place"), dict(q="in_place", interleaved=True),
                                dict(pad=2), dict(hnd=True), dict(page=1), dict(page=7), dict(idx=np.int32),
                                dict(pdt=np.int32), dict(scales=False), dict(table_pad=3), dict(table_pad=8)])
def test_forms(kw, fmt):
    run(90, 8, 4, 64, 64, "bf16", fmt, **kw)


@pytest.mark.parametrize("heads", [(1, 1), (5, 5), (32, 8), (40, 1), (7, 1)])
@pytest.mark.parametrize("fmt", FMTS)
def test_head_counts(heads, fmt):
    run(33, *heads, 128, 128, "bf16", fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_large(fmt):
    run(5001, 32, 8, 128, 128, "bf16", fmt, page=64, idx=np.int32)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("R", [0, 64])
def test_special_values(R, dtype, fmt):
    run(64, 2, 2, 64, R, dtype, fmt, special=True)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 40])
@pytest.mark.parametrize("q", ["out", "in_place", None])
def test_out_of_range_slots_and_positions(q, D, fmt):
    if fmt == "e2m1" and D == 40:
        D = 48
    run(50, 4, 2, D, 32, "bf16", fmt, q=q, bad=[(3, -1), (9, 0), (20, 1 << 20)], bad_pos=[(9, -5), (10, 0), (49, 77)])


def test_misaligned_views():
    """Rows one element off 16-byte alignment."""
    import torch
    import fp8_quant_gb300 as kv
    T, H, D = 20, 2, 64
    big = torch.randn(3, T * H * D + 1, dtype=torch.bfloat16, device="cuda")
    q, k, v = (big[i, 1:].view(T, H, D) for i in range(3))
    tab = torch.from_numpy(rope_table(64, 64)).cuda()
    pos = torch.arange(T, device="cuda")
    out = []
    for a, b, c in ((q, k, v), (q.clone(), k.clone(), v.clone())):
        kc = torch.zeros(32, H, D, dtype=torch.bfloat16, device="cuda")
        vc = torch.zeros_like(kc)
        qo = kv.kv_store_rope(b, c, kc, vc, pos, pos, tab, q=a)
        out.append((qo, kc, vc))
    for x, y in zip(*out):
        assert torch.equal(x, y)


def test_pinned_host_inputs():
    import torch
    import fp8_quant_gb300 as kv
    T, H, D = 30, 2, 64
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(T, H, D, generator=g).to(torch.bfloat16) for _ in range(3))
    tab = torch.from_numpy(rope_table(64, 64)).cuda()
    pos = torch.arange(T)
    got = []
    for put in (lambda x: x.cuda(), lambda x: x.pin_memory()):
        kc = torch.zeros(32, H, D, dtype=torch.uint8, device="cuda")
        vc = torch.zeros_like(kc)
        qo = torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda")
        kv.kv_store_rope(put(k), put(v), kc, vc, put(pos), put(pos), tab, q=put(q), q_out=qo, fmt="e4m3fn")
        torch.cuda.synchronize()
        got.append((qo, kc, vc))
    for x, y in zip(*got):
        assert torch.equal(x, y)


def test_every_e2m1_code_and_scale():
    """All 256 code bytes under all block scales decode exactly; NaN scales give NaN."""
    import torch
    import fp8_quant_gb300 as kv
    codes = np.tile(np.arange(256, dtype=np.uint8), (256, 1)).reshape(256, 1, 256)
    scales = np.repeat(np.arange(256, dtype=np.uint8), 32).reshape(256, 1, 32)
    put = lambda a: torch.from_numpy(a.copy()).cuda()   # noqa: E731
    k = torch.empty(256, 1, 512, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    kv.kv_gather_fp4(put(codes), put(codes), put(scales), put(scales), k, v, torch.arange(256, device="cuda"))
    with np.errstate(invalid="ignore"):
        want = fp4_values(codes, scales)
    got = k.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~np.isnan(want)], want[~np.isnan(want)])   # at most 6 significant bits
    assert torch.equal(k.view(torch.int16), v.view(torch.int16))
    assert E4M3_ALL.size == 256


def test_duplicate_slots_do_no_harm_to_others():
    import torch
    import fp8_quant_gb300 as kv
    T, H, D = 64, 2, 64
    k = torch.randn(T, H, D, dtype=torch.bfloat16, device="cuda")
    tab = torch.from_numpy(rope_table(64, 64)).cuda()
    slots = torch.arange(T, device="cuda")
    slots[10:20] = 5
    kc = torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    kv.kv_store_rope(k, k, kc, vc, slots, torch.zeros_like(slots), tab)
    keep = [i for i in range(T) if i != 5 and not 10 <= i < 20]
    assert torch.equal(vc[keep], k[keep]) and (vc[10:20] == 0).all()
    assert all(any(torch.equal(vc[5, h, d], k[t, h, d]) for t in [5, *range(10, 20)])
               for h in range(H) for d in range(0, D, 16))
