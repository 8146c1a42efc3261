"""Problems and 64-bit references for the rotated append, the 4-bit cache and attention.

The references are written from the formulas in ``include/kvstore.h`` with numpy, in float64
(attention) or in float32 steps whose every operation IEEE rounds once (the append, whose bytes
are compared exactly; the roundings to codes go through float64 tables).
"""

from __future__ import annotations

import math

import numpy as np

import workloads as wl

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _e4m3_table():
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m * 2.0 ** -9, (1 + m / 8.0) * 2.0 ** (e - 7.0))


E4M3 = _e4m3_table()
E4M3_ALL = np.concatenate((E4M3, [np.nan], -E4M3, [np.nan]))   # by code


def nearest_code(mag, table):
    """Index of the table value nearest to each magnitude, ties to the even index, saturating."""
    mid = (table[1:] + table[:-1]) / 2
    n = np.searchsorted(mid, mag, side="left")
    m = np.minimum(n, mid.size - 1)
    return n + ((n < mid.size) & (mag == mid[m]) & (n % 2 == 1))


def e4m3_codes(y):
    """float32 -> e4m3fn codes: nearest even, saturating, NaN -> 0x7F."""
    with np.errstate(invalid="ignore"):
        y = np.asarray(y, np.float64)
    c = nearest_code(np.minimum(np.abs(np.nan_to_num(y, nan=0.0, posinf=1e9, neginf=-1e9)), 448.0), E4M3)
    return np.where(np.isnan(y), 0x7F, c + 128 * np.signbit(y)).astype(np.uint8)


def e2m1_codes(y):
    """float32 -> e2m1 codes (one per byte): nearest even, saturating, NaN -> +6."""
    y = np.asarray(y, np.float64)
    c = nearest_code(np.minimum(np.abs(np.nan_to_num(y, nan=0.0, posinf=1e9, neginf=-1e9)), 6.0), E2M1)
    return np.where(np.isnan(y), 7, c + 8 * np.signbit(y)).astype(np.uint8)


def fp4_rows(y):
    """float32 rows [..., D] -> packed codes [..., D / 2], block scale codes [..., D / 16]."""
    y = np.asarray(y, np.float32)
    b = y.reshape(y.shape[:-1] + (-1, 16))
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        amax = np.fmax.reduce(np.abs(b), axis=-1, initial=np.float32(0.0))
        s = e4m3_codes((amax * np.float32(1.0 / 6.0)).astype(np.float32))
        f = E4M3[s].astype(np.float32)
        r = np.where(f > 0, np.float32(1.0) / f, np.float32(0.0)).astype(np.float32)
        c = e2m1_codes((b * r[..., None]).astype(np.float32)).reshape(y.shape)
    return (c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8), s


def fp4_values(codes, scales):
    """float64 values of packed codes and block scales (exact)."""
    c = np.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[:-1] + (-1,))
    v = np.where(c > 7, -E2M1[c & 7], E2M1[c & 7])
    return (v.reshape(scales.shape + (16,)) * E4M3_ALL[scales][..., None]).reshape(v.shape)


def bits_to_f32(bits, dtype):
    if dtype == "bf16":
        return (bits.astype(np.uint32) << 16).view(np.float32)
    return bits.view(np.float16).astype(np.float32)


def rotated(x, table, pos, interleaved):
    """float32 rows [T, h, D] rotated by their positions, each operation rounded once."""
    R = table.shape[1]
    c, s = table[pos, None, :R // 2], table[pos, None, R // 2:]
    out = np.array(x, np.float32)
    ia, ib = (np.arange(0, R, 2), np.arange(1, R, 2)) if interleaved else (
        np.arange(R // 2), np.arange(R // 2, R))
    a, b = x[..., ia], x[..., ib]
    with np.errstate(invalid="ignore", over="ignore"):
        out[..., ia] = (a * c).astype(np.float32) - (b * s).astype(np.float32)
        out[..., ib] = (b * c).astype(np.float32) + (a * s).astype(np.float32)
    return out


def rope_table(max_pos, R):
    f = 10000.0 ** (-np.arange(0, R, 2) / max(R, 1))
    a = np.arange(max_pos)[:, None] * f
    return np.concatenate((np.cos(a), np.sin(a)), 1).astype(np.float32)


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------

UNIT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}    # largest relative rounding error


class AttendProblem:
    """Ragged queries over a paged cache, host side (numpy), every unwritten cache byte a NaN.

    ``lens`` / ``nqs``: tokens and queries of each sequence. ``hnd``: [pages, H, page_size, D]
    storage; ``pad``: spare slots behind each page.
    """

    def __init__(self, lens, nqs, HQ, H, D, dtype="bf16", fmt=None, page=16, window=0, sinks=0,
                 seed=1, hnd=False, pad=0, q_gap=0, scale=1.0):
        self.lens, self.nqs, self.HQ, self.H, self.D = list(lens), list(nqs), HQ, H, D
        self.dtype, self.fmt, self.page, self.window, self.sinks = dtype, fmt, page, window, sinks
        self.hnd, self.pad, self.q_gap = hnd, pad, q_gap
        self._known = {}
        B = len(lens)
        need = [max(1, -(-max(n, 0) // page)) for n in lens]
        self.width = max(need) + 1
        self.num_pages = sum(need) + 2
        perm = np.argsort(wl.splitmix64(seed, 0, self.num_pages), kind="stable")
        self.table = np.full((B, self.width), -7, np.int32)     # unused entries: no page
        k = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[k:k + n]
            k += n
        T = sum(nqs)
        self.q_start = np.concatenate(([0], np.cumsum(nqs))).astype(np.int32)
        self.q = wl.to_bits(wl.normal(seed + 1, T * HQ * D) * np.float32(1.5 * scale), dtype).reshape(T, HQ, D)
        shape = (self.num_pages, page + pad, H)
        rows = [wl.to_bits(wl.normal(seed + 2 + i, int(np.prod(shape)) * D), dtype).reshape(shape + (D,))
                for i in range(2)]
        used = np.zeros(shape[:2], bool)
        for b, n in enumerate(lens):
            j = np.arange(max(n, 0))
            used[self.table[b, j // page], j % page] = True
        self.used = used
        nan16 = 0x7FC0 if dtype == "bf16" else 0x7E00
        self.kv_scale = (1.0, 1.0)
        self.scales = None
        if fmt is None:
            self.cache = [np.where(used[..., None, None], r, nan16).astype(np.uint16) for r in rows]
            self.value = [bits_to_f32(c, dtype).astype(np.float64) for c in self.cache]
        else:
            self.kv_scale = (np.float32(0.021), np.float32(0.034))
            f32 = [bits_to_f32(r, dtype) / s for r, s in zip(rows, self.kv_scale)]
            if fmt == "e4m3fn":
                self.cache = [np.where(used[..., None, None], e4m3_codes(x), 0x7F).astype(np.uint8) for x in f32]
                self.value = [E4M3_ALL[c] * float(s) for c, s in zip(self.cache, self.kv_scale)]
            else:
                enc = [fp4_rows(x) for x in f32]
                self.cache = [c for c, _ in enc]
                self.scales = [np.where(used[..., None, None], s, 0x7F).astype(np.uint8) for _, s in enc]
                self.value = [fp4_values(c, s) * float(g)
                              for c, s, g in zip(self.cache, self.scales, self.kv_scale)]

    def visible(self, b):
        """[nq, len] truth values of sequence b."""
        n, nq = max(self.lens[b], 0), self.nqs[b]
        p = n - nq + np.arange(nq)[:, None]
        j = np.arange(n)[None]
        see = j <= p
        if self.window:
            see &= (j > p - self.window) | (j < self.sinks)
        return see

    def reference(self, sm_scale=None):
        """(out, bound, lse, lse_bound) in float64: the definition, and how far a right kernel
        may be from it. With u the rounding of the 16-bit type, A = sum p |v| and d the error of a
        score (fp32 sums of D products, each sum off by at most 2^-22 of the products' magnitudes;
        queries of the quantised caches rounded at 2^-25 of their row's largest):
            |out' - out| <= u |out| + (u + 2 d) A + n 2^-24 max|v|,
        the last term for weights below the smallest normal fp16."""
        sm = 1.0 / math.sqrt(self.D) if sm_scale is None else sm_scale
        T, G, u = sum(self.nqs), self.HQ // self.H, UNIT[self.dtype]
        out = np.zeros((T, self.HQ, self.D))
        bound = np.zeros_like(out)
        lse = np.full((T, self.HQ), -np.inf)
        lse_bound = np.zeros((T, self.HQ))
        q = bits_to_f32(self.q, self.dtype).astype(np.float64)
        for b, n in enumerate(self.lens):
            n = max(n, 0)
            if n == 0 or self.nqs[b] == 0:
                continue
            j = np.arange(n)
            pg, off = self.table[b, j // self.page], j % self.page
            see = self.visible(b)
            rows = slice(self.q_start[b], self.q_start[b + 1])
            for h in range(self.HQ):
                k, v = self.value[0][pg, off, h // G], self.value[1][pg, off, h // G]
                x = q[rows, h]
                with np.errstate(invalid="ignore"):
                    s = np.where(see, (x @ k.T) * sm, -np.inf)
                    mag = (np.abs(x) @ np.abs(np.nan_to_num(k)).T) * abs(sm)
                    d = mag.max(-1) * 2.0 ** -22 * 4 + self.D * 2.0 ** -25 * np.abs(x).max(-1) * \
                        np.abs(np.nan_to_num(k)).max() * abs(sm) + 2.0 ** -20
                    top = s.max(-1, keepdims=True)
                    some = see.any(-1)
                    w = np.where(see, np.exp(s - np.where(np.isfinite(top), top, 0.0)), 0.0)
                    tot = w.sum(-1, keepdims=True)
                    w = np.divide(w, tot, out=np.zeros_like(w), where=tot > 0)
                    o = np.zeros((see.shape[0], self.D))
                    bad = ~np.isfinite(v)
                    o = w @ np.where(bad, 0.0, v)
                    o[(see @ bad.astype(np.float64)) > 0] = np.nan
                    a = w @ np.abs(np.nan_to_num(v))
                out[rows, h] = np.where(some[:, None], o, 0.0)
                bound[rows, h] = u * np.abs(o) + (u + 2 * d[:, None]) * a + \
                    n * 2.0 ** -24 * np.abs(np.nan_to_num(v)).max() + 2.0 ** -24
                with np.errstate(divide="ignore"):
                    lse[rows, h] = np.where(some, top[:, 0] + np.log(tot[:, 0]), -np.inf)
                lse_bound[rows, h] = d + 2.0 ** -21 * (1 + np.abs(np.where(some, lse[rows, h], 0.0)))
        return out, bound, lse, lse_bound

    # -- the device side --------------------------------------------------------------------

    def tensors(self, dev):
        import torch
        dt = torch.bfloat16 if self.dtype == "bf16" else torch.float16

        def paged(a, view=None):
            t = torch.from_numpy(np.ascontiguousarray(a.transpose(0, 2, 1, 3) if self.hnd else a)).to(dev)
            t = t.view(view) if view is not None else t
            t = t.transpose(1, 2) if self.hnd else t
            return t[:, :self.page]
        d = dict(table=torch.from_numpy(self.table).to(dev),
                 lens=torch.tensor(self.lens, dtype=torch.int32, device=dev),
                 q_start=torch.from_numpy(self.q_start).to(dev))
        q = torch.from_numpy(self.q.view(np.int16)).to(dev).view(dt)
        if self.q_gap:   # rows and heads with room between them
            big = torch.full((q.shape[0], self.HQ, self.D + self.q_gap), float("nan"), dtype=dt, device=dev)
            big[..., :self.D] = q
            q = big[..., :self.D]
        d["q"] = q
        if self.fmt is None:
            d["kc"], d["vc"] = (paged(c.view(np.int16), dt) for c in self.cache)
        else:
            d["kc"], d["vc"] = (paged(c) for c in self.cache)
            d["k_scale"], d["v_scale"] = (torch.tensor([s], dtype=torch.float32, device=dev) for s in self.kv_scale)
        if self.scales is not None:
            d["ks"], d["vs"] = (paged(s) for s in self.scales)
        return d

    def attend(self, d, **kw):
        import fp8_quant_gb300 as kv
        return kv.kv_attend(d["q"], d["kc"], d["vc"], d["table"], d["lens"],
                            q_start=kw.pop("q_start", d["q_start"]), page_size=self.page,
                            window=self.window, sinks=self.sinks, fmt=self.fmt,
                            k_scale=d.get("k_scale"), v_scale=d.get("v_scale"),
                            k_scales=d.get("ks"), v_scales=d.get("vs"), **kw)

    def check(self, out, lse=None, sm_scale=None):
        ref, bound, rl, lb = self.reference(sm_scale)
        got = out.double().cpu().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(ref)), "NaN in other places"
        err = np.abs(np.nan_to_num(got) - np.nan_to_num(ref))
        worst = np.nanmax(np.where(np.isnan(ref), 0.0, err / np.where(bound > 0, bound, 1e-30))) if err.size else 0.0
        if worst > 1.0:
            at = np.unravel_index(np.nanargmax(np.where(np.isnan(ref), 0.0, err / bound)), err.shape)
            raise AssertionError(f"out is {worst:.3g} times its bound off at {at}: {got[at]} for {ref[at]}")
        if lse is not None:
            l = lse.double().cpu().numpy()
            assert np.array_equal(np.isneginf(l), np.isneginf(rl))
            fin = np.isfinite(rl)
            assert np.array_equal(np.isfinite(l), fin) or np.isnan(rl).any()
            w = np.max(np.abs(l[fin] - rl[fin]) / lb[fin], initial=0.0)
            assert w <= 1.0, f"lse is {w:.3g} times its bound off"
        return worst
