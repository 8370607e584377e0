"""Plain implementations (numpy) of the 4-bit paged key/value cache and its
attention: the quantization rule in fp32, the record layout place by place,
the attention in fp64."""
from __future__ import annotations

import math

import numpy as np

f32 = np.float32


def quantize(x: np.ndarray, group: int):
    """x [..., D] fp32 -> codes [..., D], zero-points and binary16-valued scales [..., D/g]."""
    x = x.astype(f32).reshape(*x.shape[:-1], x.shape[-1] // group, group)
    with np.errstate(over="ignore", divide="ignore", invalid="ignore"):
        lo = np.minimum(np.fmin.reduce(x, -1), f32(0))
        hi = np.maximum(np.fmax.reduce(x, -1), f32(0))
        s = ((hi - lo) / f32(15)).astype(f32)
        s = np.minimum(s, f32(65504)).astype(np.float16).astype(f32)
        s = np.where(s == 0, f32(1), s)
        z = np.clip(np.rint((-lo / s).astype(f32)), 0, 15)
        c = np.rint((x / s[..., None]).astype(f32)) + z[..., None]
    c = np.where(np.isnan(c), 0, np.clip(c, 0, 15))
    return c.reshape(*c.shape[:-2], c.shape[-2] * group).astype(np.uint32), z.astype(np.uint32), s


def values(c, z, s):
    """fp64 values (c - z) s."""
    g = c.shape[-1] // z.shape[-1]
    rep = lambda a: np.repeat(a.astype(np.float64), g, -1)
    return (c.astype(np.float64) - rep(z)) * rep(s)


def _nibble(e: int) -> int:
    return 4 * (e // 2) + 16 * (e % 2)


def words(c):
    """Code words [..., D/8] of codes [..., D]."""
    c = c.reshape(*c.shape[:-1], -1, 8)
    out = np.zeros(c.shape[:-1], np.uint32)
    for e in range(8):
        out |= c[..., e] << np.uint32(_nibble(e))
    return out


def store(cache: np.ndarray, k: np.ndarray, v: np.ndarray, slots) -> None:
    """cache uint8 [pages, heads, page, token]; k, v fp32 [T, heads, D]; slots outside are skipped."""
    pages, heads, page, token = cache.shape
    D = k.shape[-1]
    G = (token - D) // 8
    rec = cache.view(np.uint32).reshape(pages, heads, -1)
    half = page * D // 8
    for x, keys in ((k, True), (v, False)):
        c, z, s = quantize(x, D // G)
        w = words(c)
        param = s.astype(np.float16).view(np.uint16).astype(np.uint32) | (z << np.uint32(16))
        for i, slot in enumerate(slots):
            if not 0 <= slot < pages * page:
                continue
            p, t = divmod(int(slot), page)
            for j in range(D // 8):
                at = t * (D // 8) + (j % 4) * (D // 32) + j // 4 if keys else half + (t // 4) * (D // 2) + 4 * j + t % 4
                rec[p, :, at] = w[i, :, j]
            for g in range(G):
                rec[p, :, 2 * half + (0 if keys else G * page) + g * page + t] = param[i, :, g]


def attention(q, k_val, v_val, lens, queries, scale, window=0, sinks=0, here=None):
    """fp64 attention.  q [T, Hq, D]; k_val, v_val: per sequence fp64 [context, Hkv, D]; here: per sequence bool
    [context], whether the token's page is in the table.  Returns out, lse and what the error bounds need:
    mass = sum p |v| per channel, and the rows' visible counts."""
    T, hq, D = q.shape
    out = np.zeros((T, hq, D))
    mass = np.zeros((T, hq, D))
    lse = np.full((T, hq), -math.inf)
    count = np.zeros(T, int)
    row = 0
    for b, (n, ctx) in enumerate(zip(queries, lens)):
        for i in range(n):
            pos = ctx - n + i
            j = np.arange(ctx)
            seen = j <= pos
            if window:
                seen &= (j > pos - window) | (j < sinks)
            if here is not None:
                seen &= here[b]
            count[row] = seen.sum()
            if seen.any():
                ks, vs = k_val[b][seen], v_val[b][seen]
                ratio = hq // ks.shape[1]
                for h in range(hq):
                    x = ks[:, h // ratio] @ q[row, h].astype(np.float64) * scale
                    m = x.max()
                    p = np.exp(x - m)
                    lse[row, h] = m + math.log(p.sum())
                    p /= p.sum()
                    out[row, h] = p @ vs[:, h // ratio]
                    mass[row, h] = p @ np.abs(vs[:, h // ratio])
            row += 1
    return out, lse, mass, count
