"""A byte encoder of gated-delta mixer blocks in serving, in front of the H-Net chunker and a global model.

Prompts of ragged length go through the blocks in one call each, leaving every
stream's states in a pool; H-Net routing and compaction then cut the rows into
chunks.  The global model attends over the chunks, whose keys and values stay
in 8-bit pages, and its rows go back to bytes.  After that each stream takes one
byte at a time through the recurrent form, in place in its slot of the pool, and
one chunk at a time through the global model.  Weights are random; the point is
the path and its calls:

  rmsnorm_q8 -> linear_i8 -> gated_delta | gated_delta_step -> rmsnorm_q8 -> linear_i8
  ... -> rmsnorm -> route_fused -> compact
  rmsnorm_q8 -> linear_i8 -> kv_write -> attention | attention_step -> rmsnorm_q8 -> linear_i8
  ... -> rmsnorm -> dechunk_ema

    python examples/mixer_serving.py [--streams 16] [--longest 2048] [--steps 32] [--layers 2]
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import byte_level_lm_amd as B  # noqa: E402
from synthdata import event_bytes  # noqa: E402

D, HEADS, WIDTH = 512, 4, 128  # rows, heads and head width of the encoder
KV_HEADS, PAGE = 2, 64         # of the global model: heads of keys and values, positions of a page


class Block:
    """One mixer block: 8-bit projections, norm weights and the gates' bias."""

    def __init__(self, gen):
        def weight(n, k):  # in 8 bits, once
            return B.quant_rows_q8(torch.randn(n, k, device="cuda", generator=gen) / k ** 0.5)

        self.qkv = 3 * HEADS * WIDTH
        self.w_in, self.s_in = weight(self.qkv + 2 * HEADS, D)  # q, k, v, then the two gates
        self.w_out, self.s_out = weight(D, HEADS * WIDTH)
        self.norm_in = torch.ones(D, device="cuda", dtype=torch.bfloat16)
        self.norm_out = torch.ones(HEADS * WIDTH, device="cuda", dtype=torch.bfloat16)
        self.decay = torch.exp(torch.linspace(-4.0, -1.0, HEADS, device="cuda"))

    def __call__(self, x, residual, mix):
        """mix(q, k, v, g, beta) is the rule over a prompt or its step; returns (y, residual)."""
        codes, scale, residual = B.rmsnorm_q8(x, self.norm_in, residual=residual)
        rows = B.linear_i8(codes, scale, self.w_in, self.s_in)
        q, k, v = (rows[:, i * HEADS * WIDTH:(i + 1) * HEADS * WIDTH].unflatten(1, (HEADS, WIDTH)) for i in range(3))
        gates = rows[:, self.qkv:].float()
        g = -torch.nn.functional.softplus(gates[:, :HEADS]) * self.decay
        o = mix(q, k, v, g, torch.sigmoid(gates[:, HEADS:]))
        codes, scale, _ = B.rmsnorm_q8(o.flatten(1), self.norm_out)
        return B.linear_i8(codes, scale, self.w_out, self.s_out), residual


class Encoder:
    def __init__(self, layers, streams, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.embed = torch.randn(256, D, device="cuda", generator=gen).to(torch.bfloat16)
        self.blocks = [Block(gen) for _ in range(layers)]
        self.norm = torch.ones(D, device="cuda", dtype=torch.bfloat16)
        self.wq, self.wk = ((torch.randn(D, D, device="cuda", generator=gen) / D ** 0.5).to(torch.bfloat16)
                            for _ in range(2))
        # a pool of states by layer; streams come and go by their slot
        self.pool = [torch.zeros(streams, HEADS, WIDTH, WIDTH, device="cuda") for _ in range(layers)]

    def _run(self, data, mix):
        x, residual = self.embed[data], torch.zeros(len(data), D, device="cuda", dtype=torch.bfloat16)
        for i, block in enumerate(self.blocks):
            x, residual = block(x, residual, lambda *a, i=i: mix(i, *a))
        return B.rmsnorm(x, self.norm, residual=residual)[0]

    def prompt(self, data, offsets, slots):
        """Rows [total, D] of the packed prompts; their states go to the pool's slots."""
        def mix(i, *a):
            o, state = B.gated_delta(*a, offsets)
            self.pool[i][slots.long()] = state
            return o
        return self._run(data, mix)

    def step(self, data, slots):
        """Rows [streams, D] of one byte of each stream."""
        return self._run(data, lambda i, *a: B.gated_delta_step(*a, self.pool[i], slots=slots)[0])

    def chunks(self, h, offsets):
        """H-Net routing and compaction of the encoder's rows."""
        p, b, _ = B.route_fused(h, self.wq, self.wk, offsets, threshold=0.5)
        return B.compact(b, offsets, rows=h, p=p)


class AttentionBlock:
    """One block of the global model: 8-bit projections, norm weights and the pages of its keys and values."""

    def __init__(self, gen, npages):
        def weight(n, k):
            return B.quant_rows_q8(torch.randn(n, k, device="cuda", generator=gen) / k ** 0.5)

        self.heads = (HEADS, KV_HEADS, KV_HEADS)  # of q, k and v
        self.w_in, self.s_in = weight(sum(self.heads) * WIDTH, D)
        self.w_out, self.s_out = weight(D, HEADS * WIDTH)
        self.norm_in = torch.ones(D, device="cuda", dtype=torch.bfloat16)
        self.norm_out = torch.ones(HEADS * WIDTH, device="cuda", dtype=torch.bfloat16)
        self.pages = [torch.zeros(npages, KV_HEADS, PAGE, WIDTH, device="cuda", dtype=torch.int8) for _ in range(2)]
        self.scales = {x: torch.zeros(npages, KV_HEADS, PAGE, device="cuda") for x in ("k_scale", "v_scale")}

    def __call__(self, x, residual, attend):
        """attend(block, q, k, v) writes the keys and values and attends; returns (y, residual)."""
        codes, scale, residual = B.rmsnorm_q8(x, self.norm_in, residual=residual)
        rows = B.linear_i8(codes, scale, self.w_in, self.s_in)
        parts = rows.split([h * WIDTH for h in self.heads], 1)
        o = attend(self, *(part.unflatten(1, (-1, WIDTH)) for part in parts))
        codes, scale, _ = B.rmsnorm_q8(o.flatten(1), self.norm_out)
        return B.linear_i8(codes, scale, self.w_out, self.s_out), residual


class GlobalModel:
    """Attention over every stream's chunks, with room for `longest` of each."""

    def __init__(self, layers, streams, longest, seed=1):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        cols = -(-longest // PAGE)
        self.blocks = [AttentionBlock(gen, streams * cols) for _ in range(layers)]
        self.norm = torch.ones(D, device="cuda", dtype=torch.bfloat16)
        self.table = torch.arange(streams * cols, device="cuda", dtype=torch.int32).view(streams, cols)
        self.lengths = torch.zeros(streams, device="cuda", dtype=torch.int32)  # chunks of each stream so far
        self.slopes = 2.0 ** -torch.arange(1, HEADS + 1, device="cuda", dtype=torch.float32)  # order through the distance

    def _run(self, x, attend):
        residual = torch.zeros_like(x)
        for block in self.blocks:
            x, residual = block(x, residual, attend)
        return B.rmsnorm(x, self.norm, residual=residual)[0]

    def prompt(self, rows, offsets, slots):
        """Rows [chunks, D] of the packed chunks of new streams."""
        at, table = slots.long(), self.table[slots.long()]

        def attend(block, q, k, v):
            B.kv_write(k, v, *block.pages, table, offsets=offsets, **block.scales)
            return B.attention(q, k, v, offsets, slopes=self.slopes)
        y = self._run(rows, attend)
        self.lengths[at] = offsets.diff().to(torch.int32)
        return y

    def step(self, rows, slots):
        """Rows [streams, D] of one chunk of each stream."""
        at, table = slots.long(), self.table[slots.long()]
        start = self.lengths[at]
        now = start + 1

        def attend(block, q, k, v):
            B.kv_write(k, v, *block.pages, table, start=start, **block.scales)
            return B.attention_step(q, *block.pages, table, now, slopes=self.slopes, **block.scales)
        y = self._run(rows, attend)
        self.lengths[at] = now
        return y


def streams_of_bytes(rng, count, longest):
    return [event_bytes(rng, longest // 32 + 1).reshape(-1)[:int(n)]
            for n in rng.integers(max(longest // 4, 1), longest + 1, count)]


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--streams", type=int, default=16)
    ap.add_argument("--longest", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--layers", type=int, default=2)
    a = ap.parse_args()
    data = streams_of_bytes(np.random.default_rng(0), a.streams, a.longest)
    offsets = torch.from_numpy(np.cumsum([0] + [len(d) for d in data])).cuda()
    packed = torch.from_numpy(np.concatenate(data).astype(np.int64)).cuda()
    encoder = Encoder(a.layers, a.streams + 4)
    slots = torch.randperm(a.streams + 4, device="cuda")[:a.streams].to(torch.int32)

    def clock(f):
        f()
        torch.cuda.synchronize()
        t = time.perf_counter()
        out = f()
        torch.cuda.synchronize()
        return out, (time.perf_counter() - t) * 1e3

    h, ms = clock(lambda: encoder.prompt(packed, offsets, slots))
    (idx, chunk_offsets, rows, p, status), ms_c = clock(lambda: encoder.chunks(h, offsets))
    print(f"prompts: {len(packed)} bytes of {a.streams} streams through {a.layers} blocks in {ms:.3f} ms, "
          f"{int(chunk_offsets[-1])} chunks in {ms_c:.3f} ms")
    n = int(chunk_offsets[-1])
    model = GlobalModel(a.layers, a.streams + 4, a.longest + a.steps + 1)
    y, ms = clock(lambda: model.prompt(rows[:n], chunk_offsets, slots))
    out, ms_d = clock(lambda: B.dechunk_ema(y, p, idx, chunk_offsets, offsets, len(packed)))
    print(f"global model: {n} chunks through {a.layers} blocks in {ms:.3f} ms, back to {out.shape[0]} bytes in {ms_d:.3f} ms")
    nxt = torch.randint(0, 256, (a.steps, a.streams), device="cuda")
    _, ms = clock(lambda: [encoder.step(nxt[i], slots) for i in range(a.steps)])
    print(f"steps: {a.steps} bytes of each stream in {ms:.3f} ms, {ms / a.steps * 1e3:.0f} us a byte of all streams")
    chunks = torch.randn(a.steps, a.streams, D, device="cuda").to(torch.bfloat16)
    _, ms = clock(lambda: [model.step(chunks[i], slots) for i in range(a.steps // 2)])
    print(f"global steps: {ms / max(a.steps // 2, 1) * 1e3:.0f} us a chunk of all streams")


if __name__ == "__main__":
    main()
