"""Transformer blocks on 4-bit weights over the 8-bit paged cache: prompts of different lengths in
one ragged batch, then single tokens from a captured graph.  Random weights.

    python examples/decode_kv8.py [--batch 8 --prompt 1000 --steps 64 --layers 2]

A block is eight calls and no kernel from elsewhere: the norm kernel adds the branch to the residual
stream and writes the INT8 rows that the GEMM reads; the rotary kernel turns the queries where
they lie in the projection's output and appends keys and values; attention reads the cache;
SwiGLU is part of the last linear layer's activation preparation.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import rotated_bit_linear_amd as rbl  # noqa: E402


class Block:
    def __init__(self, hidden, ffn, Hq, Hkv, D, gen, device="cuda"):
        def weight(n, k):
            return rbl.quant_weight_w4((torch.randn(n, k, generator=gen) * k ** -0.5).to(torch.bfloat16).to(device))

        def gain(n):
            return (1 + 0.1 * torch.randn(n, generator=gen)).to(device)

        self.qkv, self.o = weight((Hq + 2 * Hkv) * D, hidden), weight(hidden, Hq * D)
        self.up, self.down = weight(2 * ffn, hidden), weight(hidden, ffn)
        self.norm1, self.norm2, self.q_norm, self.k_norm = gain(hidden), gain(hidden), gain(D), gain(D)
        self.ffn, self.Hq, self.D = ffn, Hq, D
        self.freq, self.axis = rbl.rope_table(D, device=device)

    def _linear(self, q, s, w):
        y = torch.empty(q.shape[0], w[0].shape[0], dtype=torch.bfloat16, device=q.device)
        rbl.cr_gemm_s8s4_rowscale(q, s, *w, y)
        return y

    def __call__(self, branch, stream, cache, batch, max_new, max_kv):
        """Adds `branch` (the block before's) to the residual stream in place; returns this block's."""
        cu, kv_lens, table, pos = batch
        q, s, _ = rbl.quant_act_rmsnorm(branch, self.norm1, residual=stream, sum=stream)
        qkv = self._linear(q, s, self.qkv)
        n = self.Hq * self.D
        q = rbl.rope_append_kv8(qkv, cache, cu, kv_lens, table, max_new, self.Hq, pos, self.freq, self.axis,
                                self.q_norm, self.k_norm, out=qkv[:, :n])
        a = rbl.attn_kv8(q, cache, cu, kv_lens, table, max_new, max_kv, self.Hq)
        branch = rbl.linear_w4a8(a, *self.o, n)
        q, s, _ = rbl.quant_act_rmsnorm(branch, self.norm2, residual=stream, sum=stream)
        return rbl.linear_w4a8(self._linear(q, s, self.up), *self.down, self.ffn, swiglu=True)


class Model:
    """Blocks, one cache for each, and the pages that each sequence may come to fill."""

    def __init__(self, layers, hidden, ffn, Hq, Hkv, D, batch, max_kv, seed=0, device="cuda"):
        gen = torch.Generator().manual_seed(seed)
        self.blocks = [Block(hidden, ffn, Hq, Hkv, D, gen, device) for _ in range(layers)]
        pages = -(-max_kv // rbl.KV8_PAGE)
        self.caches = [rbl.Kv8Cache.empty(batch * pages, Hkv, D, device) for _ in range(layers)]
        self.table = torch.randperm(batch * pages, generator=gen).int().view(batch, pages).to(device)
        self.max_kv = max_kv

    def forward(self, x, batch, max_new):
        branch, stream = torch.zeros_like(x), x.clone()
        for block, cache in zip(self.blocks, self.caches):
            branch = block(branch, stream, cache, batch, max_new, self.max_kv)
        return stream + branch

    def prompt(self, x, lengths):
        """x [sum of lengths, hidden]; fills the caches from their first token."""
        d = x.device
        n = torch.tensor(lengths, dtype=torch.int32)
        cu = torch.cat([torch.zeros(1, dtype=torch.int32), n.cumsum(0).int()]).to(d)
        pos = torch.cat([torch.arange(k, dtype=torch.int32) for k in lengths])[:, None].to(d)
        self.kv_lens = n.to(d)
        return self.forward(x, (cu, self.kv_lens, self.table, pos), max(lengths))

    def single(self, x):
        """The next token of every sequence; x [batch, hidden].  Lengths live on the device, so the
        same captured launches serve every step."""
        B = x.shape[0]
        if not hasattr(self, "cu1"):
            self.cu1 = torch.arange(B + 1, dtype=torch.int32, device=x.device)
        pos = self.kv_lens[:, None].clone()
        self.kv_lens += 1
        return self.forward(x, (self.cu1, self.kv_lens, self.table, pos), 1)


def main():
    p = argparse.ArgumentParser()
    for name, value in dict(batch=8, prompt=1000, steps=64, layers=2, hidden=5376, ffn=14336, heads=32, kv_heads=8).items():
        p.add_argument("--" + name.replace("_", "-"), type=int, default=value)
    a = p.parse_args()
    model = Model(a.layers, a.hidden, a.ffn, a.heads, a.kv_heads, 128, a.batch, a.prompt + a.steps + 2)
    lengths = [max(1, a.prompt - 37 * b) for b in range(a.batch)]
    x = torch.randn(sum(lengths), a.hidden, dtype=torch.bfloat16, device="cuda")
    model.prompt(x, lengths)
    model.kv_lens.copy_(torch.tensor(lengths))
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    y = model.prompt(x, lengths)
    torch.cuda.synchronize()
    t1 = time.perf_counter()
    last = y[torch.tensor(lengths).cumsum(0) - 1].clone()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        model.single(last)                     # the first step eagerly
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        last.copy_(model.single(last))
    torch.cuda.synchronize()
    t2 = time.perf_counter()
    for _ in range(a.steps):
        graph.replay()
    torch.cuda.synchronize()
    t3 = time.perf_counter()
    assert torch.isfinite(last).all().item()
    print(f"{a.layers} blocks of {a.hidden}, {a.batch} sequences: prompts of {sum(lengths)} tokens {1e3 * (t1 - t0):.2f} ms, "
          f"single tokens {1e3 * (t3 - t2) / a.steps:.3f} ms a step")


if __name__ == "__main__":
    main()
