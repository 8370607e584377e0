"""A decoder of 4-bit weights and a 4-bit key/value cache, end to end on one GPU.

Prompts are read in chunks, each sequence is forked into branches that share
its pages, the branches decode together, the cache is compacted on the way.
Every step of a layer is one library call:

    q, k, v   w4a16_gemv / w4a16_gemm on one [q + 2 kv heads, hidden] weight
    q, k      qk_norm_rope (norms of each head, rotation by position)
    k, v      kv4_append
    o         kv4_attention (window and sinks optional)
    y         w4a16_gemv / w4a16_gemm

Weights and inputs are random, so the figures are times and not text:

    python examples/kv4_decode.py --sequences 16 --branches 4 --prompt 4000 --steps 32
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_matmul_quantize_amd as qmm  # noqa: E402


def project(weight, x):
    """x [T, K] times a 4-bit weight, by the kernel for the number of tokens."""
    return (qmm.w4a16_gemv if x.shape[0] <= 8 else qmm.w4a16_gemm)(*weight, x)


class Decoder:
    """Attention layers with residuals (no feed-forward part) over one paged cache."""

    def __init__(self, layers=4, hidden=4096, q_heads=32, kv_heads=8, head_dim=128, pages=1024, page=64, group=64,
                 window=0, sinks=0, rows=32768, seed=0, dtype=torch.bfloat16):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.hq, self.hk, self.D, self.window, self.sinks = q_heads, kv_heads, head_dim, window, sinks

        def weight(n, k):
            w = torch.randn((n, k), generator=g, device="cuda") * k ** -0.5
            return qmm.quantize_groupwise(w.to(dtype))

        self.layers = [dict(qkv=weight((q_heads + 2 * kv_heads) * head_dim, hidden), out=weight(hidden, q_heads * head_dim),
                            qw=torch.rand(head_dim, generator=g, device="cuda").add(0.5).to(dtype),
                            kw=torch.rand(head_dim, generator=g, device="cuda").add(0.5).to(dtype)) for _ in range(layers)]
        self.table = qmm.rope_table(rows, *qmm.rope_frequencies(head_dim))
        self.cache = qmm.kv4_cache(pages, kv_heads, head_dim, page, group, layers=layers)
        self.pages = qmm.KvPages(pages, page)

    def copy(self, src, dst):
        if len(src):
            qmm.kv4_copy_pages(self.cache, src.cuda(), dst.cuda())

    def step(self, seqs, x, counts):
        """x [T, hidden]: the next counts[i] tokens of each sequence seqs[i], through every layer."""
        start = [self.pages.length(s) for s in seqs]
        slots, src, dst = self.pages.extend(seqs, counts)
        self.copy(src, dst)                                  # pages that a fork shares and this step writes
        table, context = (t.cuda() for t in self.pages.table(seqs))
        positions = torch.cat([torch.arange(a, a + n) for a, n in zip(start, counts)]).cuda()
        slots = slots.cuda()
        ragged = {}
        if any(n != 1 for n in counts):
            ends = torch.tensor([0] + list(counts)).cumsum(0).int().cuda()
            ragged = dict(cu_q=ends, max_q=max(counts))
        T = x.shape[0]
        for layer, cache in zip(self.layers, self.cache):
            h = x * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6).to(x.dtype)
            q, k, v = project(layer["qkv"], h).view(T, -1, self.D).split([self.hq, self.hk, self.hk], 1)
            q, k = qmm.qk_norm_rope(q, k, positions, self.table, layer["qw"], layer["kw"])
            qmm.kv4_append(k, v, slots, cache)
            o = qmm.kv4_attention(q, cache, table, context, window=self.window, sinks=self.sinks, **ragged)
            x = x + project(layer["out"], o.view(T, -1))
        if self.window:
            for s in seqs:
                self.pages.forget(s, self.window, self.sinks)
        return x


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in dict(layers=4, hidden=4096, q_heads=32, kv_heads=8, head_dim=128, page=64, group=64, window=0,
                            sinks=0, sequences=16, branches=4, prompt=4000, chunk=1024, steps=32, seed=0).items():
        p.add_argument("--" + name.replace("_", "-"), type=int, default=value)
    a = p.parse_args(argv)
    most = -(-(a.prompt + a.steps) // a.page) + 1
    model = Decoder(a.layers, a.hidden, a.q_heads, a.kv_heads, a.head_dim, a.sequences * (most + 2 * a.branches) + 8,
                    a.page, a.group, a.window, a.sinks, a.prompt + a.steps, a.seed)
    g = torch.Generator(device="cuda").manual_seed(a.seed + 1)
    rows = lambda n: torch.randn((n, a.hidden), generator=g, device="cuda").bfloat16()

    def timed(f):
        torch.cuda.synchronize()
        t = time.perf_counter()
        y = f()
        torch.cuda.synchronize()
        return y, time.perf_counter() - t

    seqs = [model.pages.add() for _ in range(a.sequences)]

    def prefill():
        for s in seqs:
            for at in range(0, a.prompt, a.chunk):
                n = min(a.chunk, a.prompt - at)
                model.step([s], rows(n), [n])

    _, t = timed(prefill)
    print(f"prompts: {a.sequences} x {a.prompt} tokens, {a.layers} layers, {t * 1e3:.1f} ms", flush=True)
    heads = [s if b == 0 else model.pages.fork(s) for s in seqs for b in range(a.branches)]
    x = rows(len(heads))
    for _ in range(2):                                       # the first writes copy the shared pages
        x = model.step(heads, x, [1] * len(heads))
    model.copy(*model.pages.compact())

    def decode(x):
        for _ in range(a.steps - 2):
            x = model.step(heads, x, [1] * len(heads))
        return x

    x, t = timed(lambda: decode(x))
    print(f"decode: {len(heads)} branches on {model.pages.pages - model.pages.free_pages} pages, "
          f"{t * 1e3 / max(1, a.steps - 2):.2f} ms a step", flush=True)
    return x


if __name__ == "__main__":
    main()
