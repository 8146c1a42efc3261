"""Cases of the cache-append and attention operators.

Three operators over one paged KV cache:

* ``append``      K/V rows rotated by position and written at their slots (and the rotated q rows
                  out), into a cache of the rows' own type, of e4m3fn codes with per-tensor scales,
                  or of e2m1 codes with one e4m3fn scale per 16 dims (read back dequantised).
* ``attend``      attention of ragged queries over a paged 16-bit or e4m3fn cache, causal, with an
                  optional sliding window and first tokens that stay visible.
* ``attend_fp4``  the same over the e2m1 cache.

Sizes follow the library's own workloads: 32 query heads over 8 KV heads of 128 (the fused QKV
rows of 6,144), 2 heads of 64, pages of 16, 32 and 64, batches of 256, 8,192 and 32,768 tokens.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# --------------------------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------------------------

def _append(name, T, HQ, H, D, dtype, fmt, page, rot, interleaved, fused, slots, index, max_pos):
    return dict(name=name, op="append", T=T, HQ=HQ, H=H, D=D, dtype=dtype, fmt=fmt, page=page,
                rot=rot, interleaved=interleaved, fused=fused, slots=slots, index=index,
                max_pos=max_pos)


def _attend(name, op, fmt, dtype, B, q_min, q_max, len_min, len_max, HQ, H, D, page, window, sinks):
    return dict(name=name, op=op, fmt=fmt, dtype=dtype, B=B, q_min=q_min, q_max=q_max,
                len_min=len_min, len_max=len_max, HQ=HQ, H=H, D=D, page=page, window=window,
                sinks=sinks)


def listed():
    return [
        # one sequence generating one token: what a call costs at least
        _append("append_one", 1, 32, 8, 128, "bf16", "same", 16, 128, False, False, 1 << 16, "i64", 32768),
        # a decode step of 256 sequences into an FP8 cache
        _append("append_decode_fp8", 256, 32, 8, 128, "bf16", "e4m3fn", 32, 128, False, True, 1 << 18, "i64", 32768),
        # a prefill whose q, k and v are column views of one projection's output
        _append("append_prefill", 32768, 32, 8, 128, "f16", "same", 64, 128, False, True, 1 << 16, "i32", 32768),
        # a mid-size prefill into the 4-bit cache, half of each head rotated in interleaved pairs
        _append("append_fp4", 8191, 32, 8, 128, "bf16", "e2m1", 32, 64, True, False, 1 << 15, "i64", 16384),
        # a small model's step: a few short sequences, small heads
        _attend("attend_small", "attend", "same", "f16", 3, 1, 1, 90, 1000, 8, 2, 64, 16, 256, 4),
        # serving long conversations with a window and sinks, one token each
        _attend("attend_decode_window", "attend", "same", "bf16", 128, 1, 1, 3000, 16384, 32, 8, 128, 64, 4096, 4),
        # the same step without a window over an FP8 cache
        _attend("attend_decode_fp8", "attend", "e4m3fn", "bf16", 32, 1, 1, 16000, 32768, 32, 8, 128, 32, 0, 0),
        # prompts of odd lengths joining sequences that already have a context, windowed
        _attend("attend_prefill_window", "attend", "same", "bf16", 2, 2500, 4095, 5000, 8190, 32, 8, 128, 64, 1024, 4),
        # one whole prompt, causal
        _attend("attend_prefill_full", "attend", "same", "f16", 1, 8192, 8192, 8192, 8192, 32, 8, 128, 64, 0, 0),
        # a decode step of many long sequences over the 4-bit cache
        _attend("fp4_decode", "attend_fp4", "e2m1", "bf16", 64, 1, 1, 16000, 32768, 32, 8, 128, 64, 0, 0),
        # one very long sequence: the key axis is the only one to split
        _attend("fp4_long", "attend_fp4", "e2m1", "bf16", 1, 1, 1, 131071, 131071, 32, 8, 128, 16, 0, 0),
        # chunks of prompts over a long 4-bit context, windowed
        _attend("fp4_chunk", "attend_fp4", "e2m1", "f16", 3, 400, 1000, 9000, 16380, 32, 8, 128, 32, 4096, 16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "attend", "attend_fp4"))
    H = rng.choice((1, 2, 4, 8))
    G = rng.choice((1, 2, 4, 5, 8) if H < 8 else (1, 2, 4))
    D = rng.choice((64, 96, 128, 128))
    dtype = rng.choice(("bf16", "f16"))
    page = rng.choice((16, 32, 64))
    if op == "append":
        T = _log(rng, 1, 32768)
        rot = rng.choice((D, D, D // 2))
        slots = page * max(1, -(-2 * T // page))
        fused = rng.random() < 0.5
        return dict(op=op, T=T, HQ=H * G, H=H, D=D, dtype=dtype,
                    fmt=rng.choice(("same", "e4m3fn", "e2m1")), page=page, rot=rot,
                    interleaved=rng.random() < 0.3, fused=fused, slots=slots,
                    index=rng.choice(("i32", "i64")), max_pos=32768)
    fmt = "e2m1" if op == "attend_fp4" else rng.choice(("same", "same", "e4m3fn"))
    window = rng.choice((0, 0, _log(rng, 64, 8192)))
    sinks = rng.choice((0, 4, _log(rng, 1, 128))) if window else 0
    if rng.random() < 0.6:      # decode: one query, or the few of a speculative step
        B = _log(rng, 1, 128)
        L = _log(rng, 64, min(65536, (1 << 20) // B))
        q_max = rng.choice((1, 1, 1, rng.randint(2, 6)))
        q_min = 1
    else:                       # prefill, whole or a chunk
        B = rng.randint(1, 4)
        L = _log(rng, 128, 8192)
        q_max = _log(rng, 16, max(16, min(L, 4096 // B)))
        q_min = max(1, q_max // 3)
    return dict(op=op, fmt=fmt, dtype=dtype, B=B, q_min=q_min, q_max=min(q_max, L),
                len_min=max(min(q_max, L), L // 4), len_max=L, HQ=H * G, H=H, D=D, page=page,
                window=window, sinks=sinks)


def _spread(lo, hi, n):
    """n whole numbers from hi down to lo, evenly spread."""
    return [hi if n == 1 else hi - (hi - lo) * i // (n - 1) for i in range(n)]


def _lengths(case):
    """(queries, length) of each sequence of the batch, before the seed's shuffle."""
    lens = _spread(case["len_min"], case["len_max"], case["B"])
    qs = _spread(case["q_min"], case["q_max"], case["B"])
    return [(min(q, n), n) for q, n in zip(qs, lens)]


def _row_bytes(fmt, D):
    """Bytes of one cached head row, its block scales included."""
    return {"same": 2 * D, "e4m3fn": D, "e2m1": D // 2 + D // 16}[fmt]


def work(case):
    HQ, H, D = case["HQ"], case["H"], case["D"]
    if case["op"] == "append":
        T = case["T"]
        ib = 4 if case["index"] == "i32" else 8
        rows = T * (2 * HQ * D * 2 + 2 * H * D * 2 + 2 * H * _row_bytes(case["fmt"], D) + 2 * ib)
        rows += min(T, case["max_pos"]) * case["rot"] * 4
        if case["fmt"] == "e2m1":   # read back: codes and scales in, rows out
            rows += T * (2 * H * _row_bytes("e2m1", D) + 2 * H * D * 2 + ib)
        return {"bytes": rows, "flops": T * (HQ + H) * case["rot"] * 3 + 2 * T * H * D}
    seen = pairs = tokens = 0
    for nq, n in _lengths(case):
        p = np.arange(n - nq, n, dtype=np.int64)
        W, S = case["window"] or n, case["sinks"]
        lo = np.maximum(0, p - W + 1)
        pairs += int(np.sum(p + 1 - lo + np.minimum(lo, S)))
        seen += int(n - lo[0] + min(lo[0], S))
        tokens += nq
    by = 2 * seen * H * _row_bytes(case["fmt"], D) + 2 * tokens * HQ * D * 2
    by += 4 * (2 * case["B"] + 1) + 4 * sum(-(-n // case["page"]) for _, n in _lengths(case))
    return {"bytes": by, "flops": 4 * D * HQ * pairs}


# --------------------------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) & 0x7FFFFFFF)
    return g


def _normal(shape, g, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _table(max_pos, rot):
    """[max_pos, rot] fp32: the cosines of a row's rot / 2 angles, then their sines."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    a = torch.arange(max_pos, device="cuda", dtype=torch.float64)[:, None] * f
    return torch.cat((a.cos(), a.sin()), 1).float().contiguous()


def _fp8(y):
    return y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _fp4(y):
    """fp32 rows [..., D] -> packed e2m1 codes [..., D / 2], e4m3fn block scales [..., D / 16]:
    a block's scale is its largest magnitude / 6; codes round to nearest, ties to even."""
    b = y.unflatten(-1, (-1, 16))
    s = _fp8(b.abs().amax(-1, keepdim=True) * (1.0 / 6.0))
    f = s.float()
    z = b * torch.where(f > 0, 1.0 / f, 0.0)
    m = z.abs()
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    code = (code + 8 * (z.signbit())).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), s.squeeze(-1)


def _unfp4(codes, scales):
    """The fp32 values of packed e2m1 codes and their block scales. The magnitude of code m is
    piecewise linear: m / 2 up to 3, m - 2 up to 5, 2 m - 8 above."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    m = (c & 7).float()
    x = torch.maximum(torch.maximum(m * 0.5, m - 2.0), 2.0 * m - 8.0)
    x = torch.where(c > 7, -x, x)
    return (x.unflatten(-1, (-1, 16)) * scales.float().unsqueeze(-1)).flatten(-2)


def _prepare_append(case, seed):
    g = _gen(seed)
    T, HQ, H, D, dt = case["T"], case["HQ"], case["H"], case["D"], DTYPES[case["dtype"]]
    it = torch.int32 if case["index"] == "i32" else torch.int64
    if case["fused"]:
        qkv = _normal((T, (HQ + 2 * H) * D), g, dt, 1.5)
        q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split((HQ * D, H * D, H * D), 1))
    else:
        q, k, v = (_normal((T, h, D), g, dt, 1.5) for h in (HQ, H, H))
    # a prompt's tokens fill whole pages in turn, the pages anywhere in the cache
    n_pages = case["slots"] // case["page"]
    pages = torch.randperm(n_pages, generator=g, device="cuda")
    t = torch.arange(T, device="cuda")
    slots = (pages[t // case["page"]] * case["page"] + t % case["page"]).to(it)
    start = torch.randint(0, case["max_pos"] - min(T, case["max_pos"]) + 1, (1,), generator=g, device="cuda")
    pos = ((start + t) % case["max_pos"]).to(it)
    st = dict(case=case, q=q, k=k, v=v, slots=slots, pos=pos, table=_table(case["max_pos"], case["rot"]),
              q_out=torch.empty((T, HQ, D), device="cuda", dtype=dt), err=torch.zeros(2, dtype=torch.int64, device="cuda"))
    shape = (n_pages, case["page"], H)
    if case["fmt"] == "same":
        st["kc"], st["vc"] = (torch.zeros(shape + (D,), device="cuda", dtype=dt) for _ in range(2))
    elif case["fmt"] == "e4m3fn":
        st["kc"], st["vc"] = (torch.zeros(shape + (D,), device="cuda", dtype=torch.uint8) for _ in range(2))
        st["inv"] = 60.0 + 4.0 * torch.rand(2, generator=g, device="cuda")
    else:
        st["kc"], st["vc"] = (torch.zeros(shape + (D // 2,), device="cuda", dtype=torch.uint8) for _ in range(2))
        st["ks"], st["vs"] = (torch.zeros(shape + (D // 16,), device="cuda", dtype=torch.uint8) for _ in range(2))
        st["inv"] = 32.0 + 4.0 * torch.rand(2, generator=g, device="cuda")
        st["fwd"] = 1.0 / st["inv"]
        st["k_rows"], st["v_rows"] = (torch.empty((T, H, D), device="cuda", dtype=dt) for _ in range(2))
    return st


def _prepare_attend(case, seed):
    g = _gen(seed)
    B, HQ, H, D, ps, dt = case["B"], case["HQ"], case["H"], case["D"], case["page"], DTYPES[case["dtype"]]
    order = torch.randperm(B, generator=torch.Generator().manual_seed(int(seed) & 0x7FFFFFFF)).tolist()
    pairs = [_lengths(case)[i] for i in order]
    need = [-(-n // ps) for _, n in pairs]
    n_pages, width = sum(need) + 3, max(need)
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    first = torch.tensor([0] + np.cumsum(need).tolist()[:-1], device="cuda")
    col = torch.arange(width, device="cuda")
    used = col[None] < torch.tensor(need, device="cuda")[:, None]
    table = torch.where(used, perm[torch.where(used, first[:, None] + col[None], 0)], 0).to(torch.int32)
    nq = sum(q for q, _ in pairs)
    st = dict(case=case, table=table.contiguous(), lens=torch.tensor([n for _, n in pairs], dtype=torch.int32, device="cuda"),
              q_start=torch.tensor([0] + np.cumsum([q for q, _ in pairs]).tolist(), dtype=torch.int32, device="cuda"),
              q=_normal((nq, HQ, D), g, dt, 1.5), out=torch.empty((nq, HQ, D), device="cuda", dtype=dt),
              work=torch.zeros(1 << 26, dtype=torch.uint8, device="cuda"), err=torch.zeros(2, dtype=torch.int64, device="cuda"))
    # keys with a few strong channels, as rotated keys have, and values without
    ch = torch.where(torch.rand((H, D), generator=g, device="cuda") < 0.04, 4.0, 0.8)
    shape = (n_pages, ps, H, D)
    kc, vc = torch.empty(shape, device="cuda", dtype=dt), torch.empty(shape, device="cuda", dtype=dt)
    kc.normal_(0.0, 1.0, generator=g).mul_(ch.to(dt))
    vc.normal_(0.0, 1.0, generator=g)
    if case["fmt"] == "same":
        st["kc"], st["vc"] = kc, vc
        return st
    st["fwd"] = torch.rand(2, generator=g, device="cuda") * 0.01 + 0.03
    parts = []
    for x, s in ((kc, st["fwd"][0]), (vc, st["fwd"][1])):
        step = max(1, (1 << 27) // (ps * H * D))   # the fp32 copy stays small
        enc = _fp8 if case["fmt"] == "e4m3fn" else _fp4
        got = [enc(x[i:i + step].float() / s) for i in range(0, n_pages, step)]
        parts.append([torch.cat([r.view(torch.uint8) for r in c]) for c in zip(*got)] if enc is _fp4
                     else [torch.cat([c.view(torch.uint8) for c in got])])
    st["kc"], st["vc"] = parts[0][0], parts[1][0]
    if case["fmt"] == "e2m1":
        st["ks"], st["vs"] = parts[0][1], parts[1][1]
    return st


def prepare(case, seed):
    return _prepare_append(case, seed) if case["op"] == "append" else _prepare_attend(case, seed)


# --------------------------------------------------------------------------------------------
# One pass: the plain forms and the library's calls
# --------------------------------------------------------------------------------------------

def _rotate(x, cos, sin, rot, interleaved):
    """fp32 rows [T, h, D]; cos, sin [T, 1, rot / 2]."""
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])
    a, b = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((r, x[..., rot:]), -1)


def _plain_append(st):
    case = st["case"]
    rot, dt, slots = case["rot"], DTYPES[case["dtype"]], st["slots"].long()
    cos, sin = st["table"][st["pos"].long()].unsqueeze(1).split(rot // 2, -1)
    q, k = (_rotate(st[n].float(), cos, sin, rot, case["interleaved"]) for n in ("q", "k"))
    v = st["v"].float()
    st["q_out"].copy_(q.to(dt))
    if case["fmt"] == "same":
        st["kc"].flatten(0, 1)[slots] = k.to(dt)
        st["vc"].flatten(0, 1)[slots] = v.to(dt)
        return st["q_out"], st["kc"], st["vc"]
    k, v = k * st["inv"][0], v * st["inv"][1]
    if case["fmt"] == "e4m3fn":
        st["kc"].flatten(0, 1)[slots] = _fp8(k).view(torch.uint8)
        st["vc"].flatten(0, 1)[slots] = _fp8(v).view(torch.uint8)
        return st["q_out"], st["kc"].view(torch.float8_e4m3fn), st["vc"].view(torch.float8_e4m3fn)
    kc, vc, ks, vs = (st[n].flatten(0, 1) for n in ("kc", "vc", "ks", "vs"))
    (kc[slots], a), (vc[slots], b) = _fp4(k), _fp4(v)
    ks[slots], vs[slots] = a.view(torch.uint8), b.view(torch.uint8)
    st["k_rows"].copy_((_unfp4(kc[slots], ks[slots].view(torch.float8_e4m3fn)) * st["fwd"][0]).to(dt))
    st["v_rows"].copy_((_unfp4(vc[slots], vs[slots].view(torch.float8_e4m3fn)) * st["fwd"][1]).to(dt))
    return st["q_out"], st["k_rows"], st["v_rows"]


def _own_append(st):
    import fp8_quant_gb300 as kv
    case = st["case"]
    fmt = None if case["fmt"] == "same" else case["fmt"]
    inv = st.get("inv")
    kv.kv_store_rope(st["k"], st["v"], st["kc"], st["vc"], st["slots"], st["pos"], st["table"], q=st["q"],
                     q_out=st["q_out"], page_size=case["page"], interleaved=case["interleaved"], fmt=fmt,
                     inv_k_scale=None if inv is None else inv[0:1], inv_v_scale=None if inv is None else inv[1:2],
                     k_scales=st.get("ks"), v_scales=st.get("vs"), err=st["err"])
    if fmt is None:
        return st["q_out"], st["kc"], st["vc"]
    if fmt == "e4m3fn":
        return st["q_out"], st["kc"].view(torch.float8_e4m3fn), st["vc"].view(torch.float8_e4m3fn)
    kv.kv_gather_fp4(st["kc"], st["vc"], st["ks"], st["vs"], st["k_rows"], st["v_rows"], st["slots"],
                     page_size=case["page"], k_scale=st["fwd"][0:1], v_scale=st["fwd"][1:2], err=st["err"])
    return st["q_out"], st["k_rows"], st["v_rows"]


def _rows(st, which, at):
    """fp32 cache rows [..., H, D] of the slots `at`."""
    fmt = st["case"]["fmt"]
    x = st[which + "c"].flatten(0, 1)[at]
    if fmt == "same":
        return x.float()
    s = st["fwd"][0 if which == "k" else 1]
    if fmt == "e4m3fn":
        return x.view(torch.float8_e4m3fn).float() * s
    return _unfp4(x, st[which + "s"].flatten(0, 1)[at].view(torch.float8_e4m3fn)) * s


def _plain_attend(st):
    case = st["case"]
    HQ, H, D, ps, L, Q = case["HQ"], case["H"], case["D"], case["page"], case["len_max"], case["q_max"]
    lens, start = st["lens"].long(), st["q_start"].long()
    j = torch.arange(L, device="cuda")
    at = st["table"].long()[:, j // ps] * ps + j % ps                        # [B, L]
    i = torch.arange(Q, device="cuda")
    row = (start[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)             # [B, Q]
    p = (lens - (start[1:] - start[:-1]))[:, None] + i                       # positions
    see = (j <= p[..., None]) & (j < lens[:, None, None])
    if case["window"]:
        see &= (j > p[..., None] - case["window"]) | (j < case["sinks"])
    see = see[:, None, None]                                                 # [B, 1, 1, Q, L]
    q = st["q"].float()[row].unflatten(2, (H, HQ // H)).permute(0, 2, 3, 1, 4)   # [B, H, G, Q, D]
    k = _rows(st, "k", at).permute(0, 2, 3, 1)                               # [B, H, D, L]
    s = (q.flatten(2, 3) @ k).unflatten(2, (HQ // H, Q)) * (1.0 / math.sqrt(D))
    del k
    s = torch.where(see, s, float("-inf"))
    s = torch.exp(s - s.amax(-1, keepdim=True))
    total = s.sum(-1, keepdim=True)
    v = _rows(st, "v", at).transpose(1, 2)                                   # [B, H, L, D]
    o = (s.flatten(2, 3) @ v).unflatten(2, (HQ // H, Q)) / total
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)                               # [B, Q, HQ, D]
    t = torch.arange(st["q"].shape[0], device="cuda")
    b = (t[:, None] >= start[1:]).sum(1)
    st["out"].copy_(o[b, t - start[b]].to(st["out"].dtype))
    return st["out"]


def _own_attend(st):
    import fp8_quant_gb300 as kv
    case = st["case"]
    fwd = st.get("fwd")
    return kv.kv_attend(st["q"], st["kc"], st["vc"], st["table"], st["lens"],
                        q_start=None if case["q_max"] == 1 else st["q_start"], window=case["window"],
                        sinks=case["sinks"], fmt=None if case["fmt"] == "same" else case["fmt"],
                        k_scale=None if fwd is None else fwd[0:1], v_scale=None if fwd is None else fwd[1:2],
                        k_scales=st.get("ks"), v_scales=st.get("vs"), out=st["out"], work=st["work"], err=st["err"])


def run(state):
    if state["case"]["op"] == "append":
        return _own_append(state) if own else _plain_append(state)
    return _own_attend(state) if own else _plain_attend(state)


# --------------------------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------------------------

def _near(x, grid):
    """Index of the value of `grid` (ascending, from 0) nearest to each |x|; ties to the even index."""
    g = np.asarray(grid, dtype=np.float64)
    mid = (g[1:] + g[:-1]) / 2
    m = np.abs(x)
    n = np.searchsorted(mid, m, side="left")                 # a tie stays below ...
    tie = (n < mid.size) & (m == mid[np.minimum(n, mid.size - 1)]) & (n % 2 == 1)
    return n + tie                                           # ... unless the index above is the even one


def _e4m3_values():
    """The 127 finite magnitudes of e4m3fn, by code."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m * 2.0 ** -9, (1 + m / 8.0) * 2.0 ** (e - 7.0))


def _exact_append(case, seed):
    st = _prepare_append(case, seed)
    T, H, D, R = case["T"], case["H"], case["D"], case["rot"]
    host = {n: st[n].double().cpu().numpy() for n in ("q", "k", "v", "table")}
    pos, slots = st["pos"].cpu().numpy().astype(np.int64), st["slots"].cpu().numpy().astype(np.int64)
    z = host["table"][pos, :R // 2] + 1j * host["table"][pos, R // 2:]      # a rotation is a product in C
    if case["interleaved"]:
        ia, ib = np.arange(0, R, 2), np.arange(1, R, 2)
    else:
        ia, ib = np.arange(R // 2), np.arange(R // 2, R)
    for n in ("q", "k"):
        w = (host[n][:, :, ia] + 1j * host[n][:, :, ib]) * z[:, None]
        host[n][:, :, ia], host[n][:, :, ib] = w.real, w.imag
    if case["fmt"] == "same":
        kc, vc = (np.zeros((case["slots"], H, D)) for _ in range(2))
        kc[slots], vc[slots] = host["k"], host["v"]
        shape = tuple(st["kc"].shape)
        return host["q"], kc.reshape(shape), vc.reshape(shape)
    inv = st["inv"].double().cpu().numpy()
    e4 = _e4m3_values()
    out = []
    for n, s in (("k", inv[0]), ("v", inv[1])):
        y = host[n] * s
        if case["fmt"] == "e4m3fn":
            c = np.zeros((case["slots"], H, D))
            c[slots] = np.copysign(e4[_near(y, e4)], y)
            out.append(c.reshape(tuple(st["kc"].shape)))
        else:
            b = y.reshape(T, H, D // 16, 16)
            sc = e4[_near(np.abs(b).max(-1, keepdims=True) / 6.0, e4)]
            u = np.divide(b, sc, out=np.zeros_like(b), where=sc > 0)
            f = st["fwd"].double().cpu().numpy()[len(out)]
            out.append((np.copysign(np.asarray(E2M1)[_near(u, E2M1)], u) * sc * f).reshape(T, H, D))
    return host["q"], out[0], out[1]


def _decoded(st, which, slots):
    """float64 cache rows of one sequence's slots, on the device."""
    case = st["case"]
    x = st[which + "c"].view(-1, *st[which + "c"].shape[2:])[slots]
    if case["fmt"] == "same":
        return x.double()
    s = float(st["fwd"].double()[0 if which == "k" else 1])
    val = torch.tensor(np.concatenate((_e4m3_values(), [np.nan])), device="cuda")
    val = torch.cat((val, -val))
    if case["fmt"] == "e4m3fn":
        return val[x.int()] * s
    four = torch.tensor(np.concatenate((E2M1, np.negative(E2M1))), device="cuda")
    d = torch.empty(x.shape[:-1] + (case["D"],), dtype=torch.float64, device="cuda")
    d[..., 0::2], d[..., 1::2] = four[(x % 16).int()], four[(x // 16).int()]
    block = val[st[which + "s"].view(-1, *st[which + "s"].shape[2:])[slots].int()]
    return d * block.repeat_interleave(16, -1) * s


def _exact_attend(case, seed):
    st = _prepare_attend(case, seed)
    st["case"] = case
    HQ, H, D, ps = case["HQ"], case["H"], case["D"], case["page"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lens, start, table = st["lens"].tolist(), st["q_start"].tolist(), st["table"].long()
    for b, n in enumerate(lens):
        j = torch.arange(n, device="cuda")
        slots = table[b, torch.div(j, ps, rounding_mode="floor")] * ps + j.remainder(ps)
        k, v = _decoded(st, "k", slots), _decoded(st, "v", slots)
        nq = start[b + 1] - start[b]
        for i0 in range(0, nq, 1024):                       # blocks of queries
            i = torch.arange(i0, min(nq, i0 + 1024), device="cuda")
            at = i + (n - nq)
            hidden = j[None] > at[:, None]
            if case["window"]:
                hidden |= (at[:, None] - j[None] >= case["window"]) & (j[None] >= case["sinks"])
            x = st["q"][start[b] + i].double()
            for h in range(HQ):
                w = x[:, h] @ k[:, h // (HQ // H)].T / math.sqrt(D)
                w = torch.softmax(w.masked_fill(hidden, float("-inf")), -1)
                out[start[b] + i, h] = w @ v[:, h // (HQ // H)]
    return out


def exact(case, seed):
    if case["op"] == "append":
        return _exact_append(case, seed)
    if work(case)["flops"] > 4e12:      # the 64-bit products would take too long
        return None
    return _exact_attend(case, seed)
