"""Serving one attention layer from a paged KV cache: rotated appends and the attention that reads them.

``python -m fp8_quant_gb300.examples.attention_layer --fmt e2m1`` admits a ragged batch of
prompts, then generates tokens with the whole step (append, attention, the lengths) in one
CUDA graph, and prints the step's time and how far the last outputs are from the attention of
the unquantised keys and values in 64 bits.
"""

from __future__ import annotations

import argparse
import math

import torch

import fp8_quant_gb300 as kv


def rope_table(max_position, rot, device, base=10000.0):
    """fp32 [max_position, rot]: the cosines of a row's rot / 2 angles, then their sines."""
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(max_position, dtype=torch.float64)[:, None] * f
    return torch.cat((a.cos(), a.sin()), 1).float().to(device)


class AttentionLayer:
    """The cache of one layer and its two passes. ``fmt`` as in :func:`kv.kv_store_rope`.

    One stream at a time: the workspace and the error record belong to the layer.
    """

    def __init__(self, q_heads, kv_heads, dim, *, pages, page_size, max_position, rot=None,
                 fmt=None, dtype=torch.bfloat16, window=0, sinks=0, device="cuda"):
        self.HQ, self.H, self.D, self.page_size, self.fmt = q_heads, kv_heads, dim, page_size, fmt
        self.window, self.sinks, self.dtype = window, sinks, dtype
        device = torch.device(device, torch.cuda.current_device())
        shape = (pages, page_size, kv_heads)
        width, kind = {None: (dim, dtype), "e4m3fn": (dim, torch.uint8),
                       "e2m1": (dim // 2, torch.uint8)}[fmt]
        self.k_cache, self.v_cache = (torch.zeros(shape + (width,), dtype=kind, device=device) for _ in range(2))
        self.k_scales = self.v_scales = None
        if fmt == "e2m1":
            self.k_scales, self.v_scales = (torch.zeros(shape + (dim // 16,), dtype=torch.uint8, device=device)
                                            for _ in range(2))
        self.forward_scale = self.inverse_scale = (None, None)   # K's and V's
        self.cos_sin = rope_table(max_position, dim if rot is None else rot, device)
        self.work = torch.zeros(kv.ATTEND_WORK_BYTES, dtype=torch.uint8, device=device)
        self.err = kv.error_record(device)
        self.free = list(range(pages))

    def calibrate(self, k, v):
        """Tensor scales from some rows, with room for a rotated pair (sqrt 2) and for rows to come."""
        if self.fmt is not None:
            inv = kv.kv_absmax_inv(k, v, fp8_max=224.0)[2:]
            fwd = 1.0 / inv
            self.inverse_scale, self.forward_scale = (inv[0:1], inv[1:2]), (fwd[0:1], fwd[1:2])

    def admit(self, lengths):
        """Pages for sequences that may grow to ``lengths`` tokens: their page table."""
        need = [-(-n // self.page_size) for n in lengths]
        if sum(need) > len(self.free):
            raise RuntimeError(f"{sum(need)} pages wanted, {len(self.free)} free")
        table = torch.full((len(need), max(need)), -1, dtype=torch.int32)
        for b, n in enumerate(need):
            table[b, :n] = torch.tensor([self.free.pop() for _ in range(n)], dtype=torch.int32)
        return table.to(self.k_cache.device)

    def slots(self, table, seq, positions):
        """The cache slots of `positions` of the sequences `seq`."""
        page = table[seq, positions // self.page_size]
        return page.long() * self.page_size + positions % self.page_size

    def __call__(self, qkv, table, seq_lens, slots, positions, q_start=None, q_rot=None, out=None):
        """The attention of new tokens. ``qkv``: [tokens, (HQ + 2 H) D], a projection's output."""
        q, k, v = (x.unflatten(1, (-1, self.D))
                   for x in qkv.split((self.HQ * self.D, self.H * self.D, self.H * self.D), 1))
        q_rot = kv.kv_store_rope(k, v, self.k_cache, self.v_cache, slots, positions, self.cos_sin, q=q,
                                 q_out=q_rot, page_size=self.page_size, fmt=self.fmt,
                                 inv_k_scale=self.inverse_scale[0], inv_v_scale=self.inverse_scale[1],
                                 k_scales=self.k_scales, v_scales=self.v_scales, err=self.err)
        return kv.kv_attend(q_rot, self.k_cache, self.v_cache, table, seq_lens, q_start=q_start,
                            window=self.window, sinks=self.sinks, fmt=self.fmt,
                            k_scale=self.forward_scale[0], v_scale=self.forward_scale[1],
                            k_scales=self.k_scales, v_scales=self.v_scales, out=out, work=self.work, err=self.err)

    def prefill(self, qkv, table, lengths):
        """All tokens of prompts of `lengths`, one after the other in `qkv`."""
        device = qkv.device
        n = torch.tensor(lengths, device=device)
        q_start = torch.cat((n.new_zeros(1), n.cumsum(0))).to(torch.int32)
        seq = torch.repeat_interleave(torch.arange(len(lengths), device=device), n)
        positions = torch.arange(qkv.shape[0], device=device) - q_start[seq]
        return self(qkv, table, n.to(torch.int32), self.slots(table, seq, positions), positions, q_start)


class DecodeStep:
    """One token for each sequence, captured once: fill ``qkv``, replay, read ``out``."""

    def __init__(self, layer, table, lengths, graph=True):
        B, device = table.shape[0], table.device
        self.layer, self.table = layer, table
        self.qkv = torch.zeros(B, (layer.HQ + 2 * layer.H) * layer.D, dtype=layer.dtype, device=device)
        self.q_rot, self.out = (torch.empty(B, layer.HQ, layer.D, dtype=layer.dtype, device=device) for _ in range(2))
        self.lengths = torch.tensor(lengths, dtype=torch.int32, device=device)
        self.seq = torch.arange(B, device=device)
        self.graph = None
        if graph:
            self.graph = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(self.graph):
                self._step()

    def _step(self):
        positions = self.lengths.long()
        self.lengths += 1
        self.layer(self.qkv, self.table, self.lengths, self.layer.slots(self.table, self.seq, positions),
                   positions, q_rot=self.q_rot, out=self.out)

    def __call__(self):
        self._step() if self.graph is None else self.graph.replay()
        return self.out


def plain_attention(layer, qkv, q_heads):
    """One sequence's last token in 64 bits, from all its tokens' q, k and v."""
    n, R = qkv.shape[0], layer.cos_sin.shape[1]
    q, k, v = (x.unflatten(1, (-1, layer.D)).double()
               for x in qkv.split((q_heads * layer.D, layer.H * layer.D, layer.H * layer.D), 1))

    def rotate(x, pos):
        c, s = layer.cos_sin[pos].double().unsqueeze(1).split(R // 2, -1)
        a, b = x[..., :R // 2], x[..., R // 2:R]
        return torch.cat((a * c - b * s, b * c + a * s, x[..., R:]), -1)

    pos = torch.arange(n, device=qkv.device)
    keys = rotate(k, pos).repeat_interleave(q_heads // layer.H, 1)
    scores = torch.einsum("hd,nhd->hn", rotate(q[-1:], pos[-1:])[0], keys) / math.sqrt(layer.D)
    if layer.window:
        scores.masked_fill_((pos <= n - 1 - layer.window) & (pos >= layer.sinks), -math.inf)
    return torch.einsum("hn,nhd->hd", scores.softmax(-1), v.repeat_interleave(q_heads // layer.H, 1))


def generate(prompts=(1, 77, 300, 1023), steps=8, q_heads=32, kv_heads=8, dim=128, page_size=16, fmt=None,
             window=0, sinks=0, dtype=torch.bfloat16, graph=True, seed=1):
    """Prompts, then `steps` tokens each. Returns the layer, its decode step, all outputs and the inputs
    per sequence. The projections' outputs are random, so the steps do not depend on one another's results."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    ends = [n + steps for n in prompts]
    pages = sum(-(-n // page_size) for n in ends) + 1
    layer = AttentionLayer(q_heads, kv_heads, dim, pages=pages, page_size=page_size, max_position=max(ends),
                           fmt=fmt, dtype=dtype, window=window, sinks=sinks)
    width = (q_heads + 2 * kv_heads) * dim
    rows = [torch.randn(n, width, generator=g, device="cuda").to(dtype) for n in ends]
    table = layer.admit(ends)
    first = torch.cat([r[:n] for r, n in zip(rows, prompts)])
    k, v = first[:, q_heads * dim:].split(kv_heads * dim, 1)
    layer.calibrate(k.unflatten(1, (-1, dim)), v.unflatten(1, (-1, dim)))
    outs = [layer.prefill(first, table, prompts)]
    step = DecodeStep(layer, table, prompts, graph)
    for i in range(steps):
        step.qkv.copy_(torch.stack([r[n + i] for r, n in zip(rows, prompts)]))
        outs.append(step().clone())
    status, bad, _ = kv.kv_error_poll(layer.err)
    if status != kv.KVStatus.OK or bad:
        raise RuntimeError(f"{kv.kv_status_str(status)}: {bad} tokens or sequences out of range")
    return layer, step, outs, rows


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--fmt", choices=("same", "e4m3fn", "e2m1"), default="same")
    ap.add_argument("--prompts", type=int, nargs="+", default=[4000] * 16 + [37, 1])
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--window", type=int, default=0)
    ap.add_argument("--sinks", type=int, default=0)
    args = ap.parse_args()
    layer, step, outs, rows = generate(args.prompts, args.steps, fmt=None if args.fmt == "same" else args.fmt,
                                       window=args.window, sinks=args.sinks)
    err = ref = 0.0
    for b, r in enumerate(rows):
        want = plain_attention(layer, r, layer.HQ)
        err += (outs[-1][b].double() - want).square().sum().item()
        ref += want.square().sum().item()
    step.lengths -= args.steps   # the same steps once more, timed
    events = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    events[0].record()
    for _ in range(args.steps):
        step()
    events[1].record()
    torch.cuda.synchronize()
    print(f"{len(rows)} sequences, {sum(args.prompts)} prompt tokens, {args.steps} steps, cache {args.fmt}: "
          f"{events[0].elapsed_time(events[1]) * 1e3 / args.steps:.1f} us a step, "
          f"relative error {math.sqrt(err / ref):.4f}")


if __name__ == "__main__":
    main()
