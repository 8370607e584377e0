"""Attention over the 4-bit cache in fp64, row by row, with what the kernels'
arithmetic may cost each result (u = 2^-24; S = sum |q|; sk, sv the largest
scale of the visible keys and, of a channel's group, values):

  scores  products q (16 + c) with 16 + c <= 31, summed in fp32: in a group at
          most four chained matrix instructions, the sum of q, one operation
          a group, the base and the exponential; 16 roundings of at most
          31 S sk |scale|:                    dx = 16 u 31 S sk |scale|
  lse     dx + 8 u (1 + |lse|)
  out     2 dx mass, mass = sum p |v| (numerator and sum);
          a probability times its scale is binary16: 2^-11 mass, twice that
          where the kernel for chunks rounds bf16 rows' probabilities first;
          below 2^-14 a step of 2^-24, where the row's largest probability is
          at least 2^7 and its largest scale at least 2^-3 (or kept as it is):
          n 15 2^-32 max(8 sv, 1) for the products and 15 2^-25 max(8 sv, 1)
          for the scales;
          fp32 sums of n keys, 32 an instruction, of codes (and zero-points)
          with 64 added, at most 79 each: (n / 16 + 32) u 158 sv;
          the output's own rounding.

Over the bound are probabilities rounded to bf16 (2^-8 each) where a row sees
some tens of keys, and a missing value of more than about 2^-10 of the weight.
"""
from __future__ import annotations

import math

import numpy as np

U = 2.0 ** -24


def visible(ctx, n, i, window=0, sinks=0, here=None):
    """Keys that query i of a sequence's n sees."""
    pos, j = ctx - n + i, np.arange(ctx)
    seen = j <= pos
    if window:
        seen &= (j > pos - window) | (j < sinks)
    return seen if here is None else seen & here


def hidden(ctx, n, window, sinks):
    """Keys inside the context that none of a sequence's n queries sees."""
    seen = np.zeros(ctx, bool)
    for i in range(n):
        seen |= visible(ctx, n, i, window, sinks)
    return ~seen


def attention(q, k, v, k_scale, v_scale, lens, queries, scale, window=0, sinks=0, here=None, roundings=1,
              rounded=lambda p: p):
    """q [T, Hq, D]; of each sequence k, v fp64 [context, Hkv, D] and their scales [context, Hkv, groups].
    `rounded`: what becomes of the probabilities (a mistake to plant).  Returns out, lse, their bounds (without the
    output's rounding) and the rows' visible counts."""
    T, hq, D = q.shape
    out, b_out = np.zeros((T, hq, D)), np.zeros((T, hq, D))
    lse, b_lse, count = np.full((T, hq), -math.inf), np.zeros((T, hq)), np.zeros(T, int)
    row = 0
    for b, (n, ctx) in enumerate(zip(queries, lens)):
        for i in range(n):
            seen = visible(ctx, n, i, window, sinks, None if here is None else here[b])
            m = count[row] = seen.sum()
            if m:
                kr, vr, sk, sv = (x[b][seen] for x in (k, v, k_scale, v_scale))
                ratio = hq // kr.shape[1]
                for h in range(hq):
                    g = h // ratio
                    x = kr[:, g] @ q[row, h].astype(np.float64) * scale
                    p = np.exp(x - x.max())
                    lse[row, h] = x.max() + math.log(p.sum())
                    total = p.sum()
                    p = rounded(p) / total
                    out[row, h] = p @ vr[:, g]
                    mass = p @ np.abs(vr[:, g])
                    dx = 16 * U * 31 * np.abs(q[row, h]).sum() * sk[:, g].max() * abs(scale)
                    s = np.repeat(sv[:, g].max(0), D // sv.shape[2])
                    small = np.maximum(8 * s, 1) * (m * 15 * 2.0 ** -32 + 15 * 2.0 ** -25)
                    b_out[row, h] = (roundings * 2.0 ** -11 + 2 * dx) * mass + small + (m / 16 + 32) * U * 158 * s
                    b_lse[row, h] = dx + 8 * U * (1 + abs(lse[row, h]))
            row += 1
    return out, lse, b_out, b_lse, count
