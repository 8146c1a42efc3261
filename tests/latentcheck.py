"""Problems and 64-bit references for the cache of latent rows: its append, its gather and attention over it.

Written from the formulas in ``include/kvstore.h`` with numpy in float64, apart from the library.
"""

from __future__ import annotations

import math

import numpy as np

import workloads as wl
from attncheck import E4M3_ALL, UNIT, bits_to_f32, e4m3_codes, rope_table, rotated

NAN16 = {"bf16": 0x7FC0, "f16": 0x7E00}


def to_tensor(bits, dtype, dev):
    import torch
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).to(dev).view(
        torch.bfloat16 if dtype == "bf16" else torch.float16)


def to_bits(t):
    import torch
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


class StoreProblem:
    """Inputs of an append and what the cache holds after it."""

    def __init__(self, T, L, R, HQ=0, dtype="bf16", fmt=None, page=16, pages=None, norm=True, rot=None, interleaved=False,
                 idx=np.int64, seed=1, eps=1e-6, spread=1.5):
        self.T, self.L, self.R, self.HQ, self.dtype, self.fmt, self.page = T, L, R, HQ, dtype, fmt, page
        self.norm, self.interleaved, self.eps = norm, interleaved, eps
        self.rot = R if rot is None else rot
        self.pages = pages or -(-T // page) + 2
        slots = self.pages * page
        self.slots = np.argsort(wl.splitmix64(seed, 0, slots), kind="stable")[:T].astype(idx)
        self.max_pos = 5000
        self.pos = (wl.splitmix64(seed + 1, 0, max(T, 1))[:T] % np.uint64(self.max_pos)).astype(idx)
        self.table = rope_table(self.max_pos, self.rot)
        bits = lambda s, n, f=spread: wl.to_bits(wl.normal(seed + s, max(n, 1))[:n] * np.float32(f), dtype)  # noqa: E731
        self.c = bits(2, T * L).reshape(T, L)
        self.r = bits(3, T * R).reshape(T, R)
        self.q = bits(4, T * HQ * R).reshape(T, HQ, R)
        self.w = wl.to_bits(1 + np.float32(0.2) * wl.normal(seed + 5, L), dtype) if norm else None

    def turned(self, bits):
        """(float32 rows with every operation rounded once, sum of a pair's magnitudes) of rotary dims [T, h, R]."""
        x = bits_to_f32(bits, self.dtype)
        mag = np.abs(x).astype(np.float64)
        R = self.rot
        ia, ib = (np.arange(0, R, 2), np.arange(1, R, 2)) if self.interleaved else (np.arange(R // 2), np.arange(R // 2, R))
        both = mag[..., ia] + mag[..., ib]
        mag[..., ia] = mag[..., ib] = both
        return rotated(x, self.table, self.pos, self.interleaved), mag

    def rows(self):
        """(float64 rows [T, L + R], how far an fp32 form of them may be)."""
        c = bits_to_f32(self.c, self.dtype).astype(np.float64)
        r, _ = self.turned(self.r[:, None])
        off = np.zeros((self.T, self.L + self.R))
        if self.norm:
            with np.errstate(invalid="ignore", over="ignore"):
                c = c / np.sqrt(np.mean(c * c, -1, keepdims=True) + self.eps) * bits_to_f32(self.w, self.dtype).astype(np.float64)
            off[:, :self.L] = np.abs(c) * (2.0 ** -18 + 3 * 2.0 ** -24) + 2.0 ** -140
        return np.concatenate((c, r[:, 0].astype(np.float64)), 1), off

    def tensors(self, dev, pad=0, fused=False, gap=0):
        """The call's tensors; ``pad``: spare elements behind a slot, ``gap``: between rows of the inputs."""
        import torch
        d = dict(positions=torch.from_numpy(self.pos).to(dev), cos_sin=torch.from_numpy(self.table).to(dev),
                 indices=torch.from_numpy(self.slots).to(dev), err=torch.zeros(2, dtype=torch.int64, device=dev))
        c, r = to_tensor(self.c, self.dtype, dev), to_tensor(self.r, self.dtype, dev)
        if fused or gap:
            big = torch.full((self.T, self.L + self.R + gap), float("nan"), dtype=c.dtype, device=dev)
            big[:, :self.L], big[:, self.L:self.L + self.R] = c, r
            c, r = big[:, :self.L], big[:, self.L:self.L + self.R]
        d["c"], d["r"] = c, r
        if not self.R:
            for n in ("r", "positions", "cos_sin"):
                d[n] = None
        D = self.L + self.R
        if self.fmt is None:
            store = torch.full((self.pages, self.page, 1, D + pad), 7.0, dtype=c.dtype, device=dev)
        else:
            store = torch.full((self.pages, self.page, 1, D + pad), 0x55, dtype=torch.uint8, device=dev)
            d["scales"] = torch.full((self.pages * self.page, 1), -3.0, device=dev)
        d["store"], d["cache"] = store, store[..., :D]
        d["weight"] = to_tensor(self.w, self.dtype, dev) if self.norm else None
        if self.HQ:
            d["q"] = to_tensor(self.q, self.dtype, dev)
        return d

    def call(self, d, **kw):
        import fp8_quant_gb300 as kv
        a = {n: d.get(n) for n in ("weight", "q", "q_out", "scales", "err")}
        a.update(page_size=self.page, interleaved=self.interleaved, fmt=self.fmt, eps=self.eps, **kw)
        return kv.kv_store_latent(d["c"], d["r"], d["cache"], d["indices"], d["positions"], d["cos_sin"], **a)

    def check_q(self, got, skip=()):
        want, _ = self.turned(self.q)
        keep = np.setdiff1d(np.arange(self.T), skip)
        have = to_bits(got)[keep]
        assert np.array_equal(have, wl.to_bits(want, self.dtype).reshape(want.shape)[keep]), "rotated queries differ"

    def check(self, d, skip=()):
        """The whole cache and the scales: rows within their bounds, everything else as it was. ``skip``: tokens not written."""
        keep = np.setdiff1d(np.arange(self.T), skip)
        store = d["store"]
        D, u = self.L + self.R, UNIT[self.dtype]
        slots = self.slots[keep]
        flat = store.reshape(self.pages * self.page, -1)
        import torch
        mask = np.ones(flat.shape[0], bool)
        mask[slots] = False
        fill = 7.0 if self.fmt is None else 0x55
        assert bool((flat[torch.from_numpy(mask).to(flat.device)] == fill).all()), "an untouched slot changed"
        assert bool((flat[:, D:] == fill).all()), "padding changed"
        want, off = self.rows()
        want, off = want[keep], off[keep]
        rows = flat[torch.from_numpy(slots.astype(np.int64)).to(flat.device)][:, :D]
        if self.fmt is None:
            got = bits_to_f32(to_bits(rows), self.dtype).astype(np.float64)
            bound = u * np.abs(want) + off * (1 + u) + 2.0 ** -25
            exact = slice(self.L, D) if self.norm else slice(0, D)
            with np.errstate(over="ignore"):
                bits = wl.to_bits(want.astype(np.float32), self.dtype).reshape(want.shape)
            assert np.array_equal(to_bits(rows)[:, exact], bits[:, exact]), "bytes differ"
            assert (np.abs(got - want) <= bound).all(), f"off by {np.max(np.abs(got - want) / bound)} bounds"
            return
        sc = d["scales"][:, 0].cpu().numpy()
        assert (sc[mask] == -3.0).all(), "an untouched scale changed"
        top = np.abs(want).max(1)
        ws = np.where(top > 0, top / 448.0, 1.0)
        gs = sc[slots].astype(np.float64)
        assert (np.abs(gs - ws) <= ws * (2.0 ** -17)).all(), "scales"
        got = E4M3_ALL[rows.cpu().numpy()] * gs[:, None]
        if not self.norm:   # every step is one IEEE operation: the codes themselves
            with np.errstate(divide="ignore"):
                inv = np.where(top > 0, np.float32(448.0) / top.astype(np.float32), np.float32(1.0)).astype(np.float32)
            assert np.array_equal(rows.cpu().numpy(), e4m3_codes((want.astype(np.float32) * inv[:, None]).astype(np.float32)))
        bound = 2.0 ** -4 * np.abs(want) * (1 + 2.0 ** -12) + 2.0 ** -10 * ws[:, None] * (1 + 2.0 ** -12) + off * 2
        assert (np.abs(got - want) <= bound).all(), f"off by {np.max(np.abs(got - want) / bound)} bounds"


class LatentProblem:
    """Ragged queries over a paged cache of latent rows, host side; every unwritten cache row (and its scale) a NaN."""

    def __init__(self, lens, nqs, HQ, L, R, dtype="bf16", fmt=None, page=16, seed=1, pad=0, slot_pad=0, q_gap=0, scale=1.0,
                 scale_spread=0.0):
        self.lens, self.nqs, self.HQ, self.L, self.D = list(lens), list(nqs), HQ, L, L + R
        self.dtype, self.fmt, self.page, self.pad, self.slot_pad, self.q_gap = dtype, fmt, page, pad, slot_pad, q_gap
        need = [max(1, -(-max(n, 0) // page)) for n in lens]
        self.width = max(need) + 1
        self.num_pages = sum(need) + 2
        perm = np.argsort(wl.splitmix64(seed, 0, self.num_pages), kind="stable")
        self.table = np.full((len(lens), self.width), -7, np.int32)     # unused entries: no page
        k = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[k:k + n]
            k += n
        T = sum(nqs)
        self.q_start = np.concatenate(([0], np.cumsum(nqs))).astype(np.int32)
        self.q = wl.to_bits(wl.normal(seed + 1, max(T, 1) * HQ * self.D)[:T * HQ * self.D] * np.float32(1.5 * scale),
                            dtype).reshape(T, HQ, self.D)
        shape = (self.num_pages, page)
        rows = wl.normal(seed + 2, int(np.prod(shape)) * self.D).reshape(shape + (self.D,)).astype(np.float32)
        if scale_spread:  # rows of very different magnitudes
            rows = rows * np.exp2(scale_spread * wl.normal(seed + 3, int(np.prod(shape))).reshape(shape + (1,))).astype(np.float32)
        used = np.zeros(shape, bool)
        for b, n in enumerate(lens):
            j = np.arange(max(n, 0))
            used[self.table[b, j // page], j % page] = True
        self.scales = None
        if fmt is None:
            self.cache = np.where(used[..., None], wl.to_bits(rows, dtype).reshape(rows.shape), NAN16[dtype]).astype(np.uint16)
            self.value = bits_to_f32(self.cache, dtype).astype(np.float64)
        else:
            top = np.abs(rows).max(-1)
            self.scales = np.where(used, top / np.float32(448.0), np.nan).astype(np.float32)
            self.cache = np.where(used[..., None], e4m3_codes((rows * (np.float32(448.0) / top)[..., None]).astype(np.float32)),
                                  0x7F).astype(np.uint8)
            self.value = E4M3_ALL[self.cache] * self.scales.astype(np.float64)[..., None]

    def reference(self, sm_scale=None):
        """(out, bound, lse, lse_bound) in float64. With u the rounding of the 16-bit type, A = sum p |v| and d the error of
        a score (fp32 sums of D products, each sum off by at most 2^-22 of the products' magnitudes; queries over 8-bit rows
        rounded at 2^-25 of their row's largest):
            |out' - out| <= u |out| + (u + 2 d) A + n 2^-24 max|v|,
        weights being rounded once (u) and those below the smallest fp16 lost (the last term)."""
        sm = 1.0 / math.sqrt(self.D) if sm_scale is None else sm_scale
        T, u, L = sum(self.nqs), UNIT[self.dtype], self.L
        out, bound = np.zeros((T, self.HQ, L)), np.zeros((T, self.HQ, L))
        lse, lse_bound = np.full((T, self.HQ), -np.inf), np.zeros((T, self.HQ))
        q = bits_to_f32(self.q, self.dtype).astype(np.float64)
        for b, n in enumerate(self.lens):
            n, nq = max(n, 0), self.nqs[b]
            if n == 0 or nq == 0:
                continue
            j = np.arange(n)
            k = self.value[self.table[b, j // self.page], j % self.page]
            see = j[None] <= n - nq + np.arange(nq)[:, None]
            some = see.any(-1)
            for h in range(self.HQ):
                x = q[self.q_start[b]:self.q_start[b] + nq, h]
                kf = np.nan_to_num(k, posinf=0.0, neginf=0.0)
                with np.errstate(invalid="ignore"):
                    s = np.where(see, (x @ k.T) * sm, -np.inf)
                    d = (np.abs(x) @ np.abs(kf).T * abs(sm)).max(-1) * 2.0 ** -20 + self.D * 2.0 ** -25 * np.abs(x).max(-1) * \
                        np.abs(kf).max() * abs(sm) + 2.0 ** -20
                    top = s.max(-1, keepdims=True)
                    w = np.where(see, np.exp(s - np.where(np.isfinite(top), top, 0.0)), 0.0)
                    tot = w.sum(-1, keepdims=True)
                    w = np.divide(w, tot, out=np.zeros_like(w), where=~(tot <= 0))
                v = k[:, :L]
                bad = ~np.isfinite(v)
                o = w @ np.where(bad, 0.0, v)
                o[(see @ bad.astype(np.float64)) > 0] = np.nan
                o = np.where(np.isnan(w).any(-1)[:, None], np.nan, o)
                a = w @ np.abs(kf[:, :L])
                at = slice(self.q_start[b], self.q_start[b] + nq)
                out[at, h] = np.where(some[:, None], o, 0.0)
                bound[at, h] = u * np.abs(o) + (u + 2 * d[:, None]) * a + n * 2.0 ** -24 * np.abs(kf).max() + 2.0 ** -24
                with np.errstate(divide="ignore", invalid="ignore"):
                    lse[at, h] = np.where(some, top[:, 0] + np.log(tot[:, 0]), -np.inf)
                lse_bound[at, h] = d + 2.0 ** -21 * (1 + np.abs(np.where(some, lse[at, h], 0.0)))
        return out, bound, lse, lse_bound

    def tensors(self, dev):
        import torch
        d = dict(table=torch.from_numpy(self.table).to(dev), lens=torch.tensor(self.lens, dtype=torch.int32, device=dev),
                 q_start=torch.from_numpy(self.q_start).to(dev))
        q = to_tensor(self.q, self.dtype, dev)
        if self.q_gap:   # heads with room between them
            big = torch.full((q.shape[0], self.HQ, self.D + self.q_gap), float("nan"), dtype=q.dtype, device=dev)
            big[..., :self.D] = q
            q = big[..., :self.D]
        d["q"] = q
        kind = q.dtype if self.fmt is None else torch.uint8
        big = torch.zeros((self.num_pages, self.page + self.pad, 1, self.D + self.slot_pad), dtype=kind, device=dev)
        if self.fmt is None:
            big.fill_(float("nan"))
        cache = big[:, :self.page, :, :self.D]
        cache.copy_((to_tensor(self.cache, self.dtype, dev) if self.fmt is None else torch.from_numpy(self.cache).to(dev))[:, :, None])
        d["cache"] = cache
        d["scales"] = None if self.scales is None else torch.from_numpy(self.scales.reshape(-1, 1)).to(dev)
        return d

    def attend(self, d, **kw):
        import fp8_quant_gb300 as kv
        return kv.kv_attend_latent(d["q"], d["cache"], d["table"], d["lens"], latent_dim=self.L, q_start=kw.pop("q_start", d["q_start"]),
                                   page_size=self.page, fmt=self.fmt, scales=d["scales"], **kw)

    def check(self, out, lse=None, sm_scale=None):
        ref, bound, rl, lb = self.reference(sm_scale)
        got = out.double().cpu().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(ref)), "NaN in other places"
        fine = ~np.isnan(ref)
        err = np.abs(got[fine] - ref[fine]) / np.where(bound[fine] > 0, bound[fine], 1e-30)
        assert np.max(err, initial=0.0) <= 1.0, f"out is {np.max(err):.3g} times its bound off"
        if lse is not None:
            l = lse.double().cpu().numpy()
            assert np.array_equal(np.isneginf(l), np.isneginf(rl))
            fin = np.isfinite(rl)
            assert np.max(np.abs(l[fin] - rl[fin]) / lb[fin], initial=0.0) <= 1.0, "lse"
