"""Serving one attention layer from a paged cache of latent rows: appends and the attention that reads them.

``python -m fp8_quant_gb300.examples.latent_layer --fmt e4m3fn`` admits a ragged batch of prompts, then
generates tokens with the whole step (append, attention, the lengths) in one CUDA graph, and prints the step's
time and how far the last outputs are from the attention of the unquantised rows in 64 bits.

A token's projections give its latent and rotary dims, [L + R], and its queries [HQ, L + R], the first L of which
already carry the keys' up-projection; the outputs [HQ, L] go to the values' up-projection. The scores are those of the
heads as they were before that, of `head_dim` dims, and so is their scale.
"""

from __future__ import annotations

import argparse
import math

import torch

import fp8_quant_gb300 as kv
from fp8_quant_gb300.examples.attention_layer import rope_table

EPS = 1e-6


class LatentLayer:
    """The cache of one layer and its two passes. ``fmt`` as in :func:`kv.kv_store_latent`. ``head_dim``: dims of a head's
    queries and keys before the keys' up-projection went into the queries, rotary ones included.

    One stream at a time: the workspace and the error record belong to the layer.
    """

    def __init__(self, heads, latent, rotary, *, head_dim, pages, page_size, max_position, weight=None, fmt=None,
                 dtype=torch.bfloat16, device="cuda"):
        self.HQ, self.L, self.R, self.page_size, self.fmt, self.dtype = heads, latent, rotary, page_size, fmt, dtype
        self.weight, self.sm_scale = weight, 1.0 / math.sqrt(head_dim)
        device = torch.device(device, torch.cuda.current_device())
        self.cache = torch.zeros((pages, page_size, 1, latent + rotary), dtype=torch.uint8 if fmt else dtype, device=device)
        self.scales = torch.zeros((pages * page_size, 1), device=device) if fmt else None
        self.cos_sin = rope_table(max_position, rotary, device)
        self.work = torch.zeros(kv.ATTEND_WORK_BYTES, dtype=torch.uint8, device=device)
        self.err = kv.error_record(device)
        self.free = list(range(pages))

    def admit(self, lengths):
        """Pages for sequences that may grow to ``lengths`` tokens: their page table."""
        need = [-(-n // self.page_size) for n in lengths]
        if sum(need) > len(self.free):
            raise RuntimeError(f"{sum(need)} pages wanted, {len(self.free)} free")
        table = torch.full((len(need), max(need)), -1, dtype=torch.int32)
        for b, n in enumerate(need):
            table[b, :n] = torch.tensor([self.free.pop() for _ in range(n)], dtype=torch.int32)
        return table.to(self.cache.device)

    def slots(self, table, seq, positions):
        """The cache slots of `positions` of the sequences `seq`."""
        return table[seq, positions // self.page_size].long() * self.page_size + positions % self.page_size

    def __call__(self, rows, q, table, seq_lens, slots, positions, q_start=None, out=None):
        """The attention of new tokens. ``rows``: [tokens, L + R]; ``q``: [tokens, HQ, L + R], whose rotary dims are
        rotated in place."""
        turn = q[..., self.L:]
        kv.kv_store_latent(rows[:, :self.L], rows[:, self.L:], self.cache, slots, positions, self.cos_sin, weight=self.weight,
                           eps=EPS, q=turn, q_out=turn, page_size=self.page_size, fmt=self.fmt, scales=self.scales, err=self.err)
        return kv.kv_attend_latent(q, self.cache, table, seq_lens, latent_dim=self.L, q_start=q_start, sm_scale=self.sm_scale,
                                   fmt=self.fmt, scales=self.scales, out=out, work=self.work, err=self.err)

    def prefill(self, rows, q, table, lengths):
        """All tokens of prompts of `lengths`, one after the other."""
        n = torch.tensor(lengths, device=rows.device)
        q_start = torch.cat((n.new_zeros(1), n.cumsum(0))).to(torch.int32)
        seq = torch.repeat_interleave(torch.arange(len(lengths), device=rows.device), n)
        positions = torch.arange(rows.shape[0], device=rows.device) - q_start[seq]
        return self(rows, q, table, n.to(torch.int32), self.slots(table, seq, positions), positions, q_start)

    def rows_of(self, table, b, n):
        """The first `n` rows of sequence `b` as the cache holds them, for a projection back to heads."""
        positions = torch.arange(n, device=table.device)
        out = torch.empty((n, self.L + self.R), dtype=self.dtype, device=table.device)
        kv.kv_gather_latent(self.cache, out, self.slots(table, torch.full_like(positions, b), positions),
                            page_size=self.page_size, fmt=self.fmt, scales=self.scales, err=self.err)
        return out


class DecodeStep:
    """One token for each sequence, captured once: fill ``rows`` and ``q``, replay, read ``out``."""

    def __init__(self, layer, table, lengths, graph=True):
        B, device = table.shape[0], table.device
        self.layer, self.table = layer, table
        self.rows = torch.zeros(B, layer.L + layer.R, dtype=layer.dtype, device=device)
        self.q = torch.zeros(B, layer.HQ, layer.L + layer.R, dtype=layer.dtype, device=device)
        self.out = torch.empty(B, layer.HQ, layer.L, dtype=layer.dtype, device=device)
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
        self.layer(self.rows, self.q, self.table, self.lengths, self.layer.slots(self.table, self.seq, positions), positions,
                   out=self.out)

    def __call__(self):
        self._step() if self.graph is None else self.graph.replay()
        return self.out


def plain_attention(layer, inputs):
    """One sequence's last token in 64 bits, from all its tokens' rows and its last queries."""
    rows, q = inputs[0].double(), inputs[1][-1].double()
    n, L = rows.shape[0], layer.L
    latent = rows[:, :L]
    if layer.weight is not None:
        latent = latent / (latent.square().mean(-1, keepdim=True) + EPS).sqrt() * layer.weight.double()

    def rotate(x, c, s):
        a, b = x.split(layer.R // 2, -1)
        return torch.cat((a * c - b * s, b * c + a * s), -1)

    c, s = layer.cos_sin[:n].double().split(layer.R // 2, -1)
    keys = torch.cat((latent, rotate(rows[:, L:], c, s)), -1)
    q = torch.cat((q[:, :L], rotate(q[:, L:], c[-1], s[-1])), -1)
    return (q @ keys.T * layer.sm_scale).softmax(-1) @ keys[:, :L]


def generate(prompts=(1, 77, 300, 1023), steps=8, heads=32, latent=512, rotary=64, head_dim=128 + 64, page_size=16, fmt=None,
             dtype=torch.bfloat16, graph=True, seed=1):
    """Prompts, then `steps` tokens each. Returns the layer, all outputs and the inputs per sequence. The projections'
    outputs are random, so the steps do not depend on one another's results."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    ends = [n + steps for n in prompts]
    weight = (1 + 0.2 * torch.randn(latent, generator=g, device="cuda")).to(dtype)
    layer = LatentLayer(heads, latent, rotary, head_dim=head_dim, pages=sum(-(-n // page_size) for n in ends) + 1,
                        page_size=page_size, max_position=max(ends), weight=weight, fmt=fmt, dtype=dtype)
    D = latent + rotary
    inputs = [(torch.randn(n, D, generator=g, device="cuda").to(dtype), torch.randn(n, heads, D, generator=g, device="cuda").to(dtype))
              for n in ends]
    table = layer.admit(ends)
    first = [torch.cat([x[i][:n] for x, n in zip(inputs, prompts)]) for i in (0, 1)]
    outs = [layer.prefill(*first, table, prompts)]
    step = DecodeStep(layer, table, prompts, graph)
    for i in range(steps):
        step.rows.copy_(torch.stack([x[0][n + i] for x, n in zip(inputs, prompts)]))
        step.q.copy_(torch.stack([x[1][n + i] for x, n in zip(inputs, prompts)]))
        outs.append(step().clone())
    status, bad, _ = kv.kv_error_poll(layer.err)
    if status != kv.KVStatus.OK or bad:
        raise RuntimeError(f"{kv.kv_status_str(status)}: {bad} tokens or sequences out of range")
    layer.table, layer.step = table, step
    return layer, outs, inputs


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--fmt", choices=("same", "e4m3fn"), default="same")
    ap.add_argument("--prompts", type=int, nargs="+", default=[4000] * 16 + [37, 1])
    ap.add_argument("--steps", type=int, default=16)
    args = ap.parse_args()
    layer, outs, inputs = generate(args.prompts, args.steps, fmt=None if args.fmt == "same" else args.fmt)
    err = ref = 0.0
    for b, x in enumerate(inputs):
        want = plain_attention(layer, x)
        err += (outs[-1][b].double() - want).square().sum().item()
        ref += want.square().sum().item()
    step = layer.step
    step.lengths -= args.steps   # the same steps once more, timed
    events = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    events[0].record()
    for _ in range(args.steps):
        step()
    events[1].record()
    torch.cuda.synchronize()
    print(f"{len(inputs)} sequences, {sum(args.prompts)} prompt tokens, {args.steps} steps, cache {args.fmt}: "
          f"{events[0].elapsed_time(events[1]) * 1e3 / args.steps:.1f} us a step, relative error {math.sqrt(err / ref):.4f}")


if __name__ == "__main__":
    main()
