"""Norms of queries and keys with the rotation by position, against fp64.

Bound: y is rounded once to the output type; before that at most D/8 + 12 fp32
roundings of the sum of squares and about 8 of the products, each relative to
the pair it is made of: |err| <= half an ulp |y| + 32 u hypot(a, b) (u = 2^-24;
a, b the normed pair), and half the type's smallest step."""
import math

import numpy as np
import pytest
import torch

import quantized_matmul_quantize_amd as qmm
from gpu_util import OUT_HALF_ULP, note

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -24


def rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def half(x, dtype):
    return torch.from_numpy(np.asarray(x, np.float32)).to(dtype)


def reference(x, w, positions, table, eps, interleaved):
    x = x.double().numpy()
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w.double().numpy()
    y, size = x.copy(), np.abs(x)
    if table is not None:
        cs = table.double().numpy()[positions.numpy()][:, None]
        r = 2 * cs.shape[2]
        a_at = np.arange(0, r, 2) if interleaved else np.arange(r // 2)
        b_at = a_at + (1 if interleaved else r // 2)
        a, b = x[..., a_at], x[..., b_at]
        y[..., a_at] = a * cs[..., 0] - b * cs[..., 1]
        y[..., b_at] = b * cs[..., 0] + a * cs[..., 1]
        size[..., a_at] = size[..., b_at] = np.hypot(a, b)
    return y, size


def check(got, x, w, positions, table, eps, interleaved):
    y, size = reference(x, w, positions, table, eps, interleaved)
    tiny = 2.0 ** -25 if got.dtype == F16 else 2.0 ** -134
    bound = OUT_HALF_ULP[got.dtype] * np.abs(y) + 32 * U * size + tiny
    err = np.abs(got.double().cpu().numpy() - y)
    assert (err <= bound).all(), f"worst {(err / bound).max()} of its bound"


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "interleaved"])
@pytest.mark.parametrize("D,rot", [(64, 64), (64, 16), (80, 32), (96, 96), (128, 128), (128, 64), (128, 48), (256, 256),
                                   (256, 32), (512, 512), (8, 0), (24, 16)])
@pytest.mark.parametrize("norm", ["both", "none", "q", "f32"])
def test_norm_and_rotation(dtype, interleaved, D, rot, norm):
    if rot == 0 and norm == "none":
        pytest.skip("nothing to compute")
    note(f"qk_norm_rope D={D} rot={rot} interleaved={interleaved} norm={norm} {dtype}")
    g = rng(D + rot)
    T, hq, hk = 13, 5, 2
    q, k = half(g.standard_normal((T, hq, D)) * 3, dtype), half(g.standard_normal((T, hk, D)) * 0.01, dtype)
    q[3], k[4] = 0, 0                                       # a head of zeros: eps alone
    wt = F32 if norm == "f32" else dtype
    qw = half(1 + 0.3 * g.standard_normal(D), wt) if norm != "none" else None
    kw = half(1 + 0.3 * g.standard_normal(D), wt) if norm in ("both", "f32") else None
    rows = 50
    table = qmm.rope_table(rows, qmm.rope_frequencies(rot)[0]) if rot else None
    pos = torch.from_numpy(g.integers(0, rows, T)) if rot else None
    pos_d = None if pos is None else pos.cuda()
    cuda = lambda t: None if t is None else t.cuda()
    qo, ko = qmm.qk_norm_rope(q.cuda(), k.cuda(), pos_d, table, cuda(qw), cuda(kw), eps=1e-5, interleaved=interleaved)
    tab = None if table is None else table.cpu()
    check(qo, q, qw, pos, tab, 1e-5, interleaved)
    check(ko, k, kw, pos, tab, 1e-5, interleaved)
    # queries alone, and in place
    q2 = q.cuda()
    qo2, none = qmm.qk_norm_rope(q2, None, pos_d, table, cuda(qw), eps=1e-5, interleaved=interleaved, q_out=q2)
    assert none is None and qo2.data_ptr() == q2.data_ptr() and torch.equal(qo2, qo)


@pytest.mark.parametrize("T,hq,hk", [(1, 1, 1), (1, 32, 8), (3, 7, 7), (700, 16, 2)])
def test_views_of_a_projection(T, hq, hk):
    D = 128
    qkv = half(rng(T).standard_normal((T, (hq + 2 * hk) * D)), BF16).cuda()
    q = qkv[:, :hq * D].view(T, hq, D)
    k = qkv[:, hq * D:(hq + hk) * D].view(T, hk, D)
    table = qmm.rope_table(1000, qmm.rope_frequencies(D)[0])
    pos = torch.from_numpy(rng(T + 1).integers(0, 1000, T))
    qo, ko = qmm.qk_norm_rope(q, k, pos.cuda(), table)
    check(qo, q.cpu(), None, pos, table.cpu(), 0, False)
    check(ko, k.cpu(), None, pos, table.cpu(), 0, False)


def test_positions_outside_the_table_are_not_a_number():
    q = half(rng(1).standard_normal((4, 2, 64)), BF16).cuda()
    table = qmm.rope_table(10, qmm.rope_frequencies(32)[0])
    for inter in (False, True):
        out, _ = qmm.qk_norm_rope(q, None, torch.tensor([3, -1, 10, 2 ** 40], device="cuda"), table, interleaved=inter)
        assert out[0].isfinite().all()
        assert out[1:, :, :32].isnan().all() and torch.equal(out[1:, :, 32:], q[1:, :, 32:])


def test_no_tokens():
    x = torch.empty((0, 2, 64), dtype=F16, device="cuda")
    table = qmm.rope_table(4, qmm.rope_frequencies(64)[0])
    qo, ko = qmm.qk_norm_rope(x, x, torch.empty(0, dtype=torch.int64, device="cuda"), table)
    assert qo.shape == ko.shape == (0, 2, 64)


@pytest.mark.parametrize("kw", [dict(), dict(base=500000.0), dict(scaling="linear", factor=4.0),
                                dict(scaling="wavelength", base=500000.0, factor=8.0, original=8192),
                                dict(scaling="yarn", factor=16.0, original=4096)])
def test_table_in_64_bits(kw):
    """Cosines and sines of angles past 10^5: fp64 rounded once (2^-24 of a magnitude m, and fp64's own 10^5 2^-52)."""
    f, m = qmm.rope_frequencies(128, **kw)
    rows = 140001
    got = qmm.rope_table(rows, f, m).cpu().double().numpy()
    for p in (0, 1, 77, 65535, rows - 1):
        want = np.stack([m * np.cos(p * np.array(f)), m * np.sin(p * np.array(f))], -1)
        assert np.abs(got[p] - want).max() <= m * (U + 1e-9)


@pytest.mark.parametrize("dtype,eps", [(BF16, 0.0), (BF16, 1e-40)])
def test_heads_whose_squares_are_subnormal(dtype, eps):
    """Channels of 5e-20: a mean square of 2.5e-39, below fp32's normal numbers, still has a square root."""
    q = half(rng(2).standard_normal((9, 3, 64)) * 5e-20, dtype)
    w = half(1 + 0.3 * rng(3).standard_normal(64), dtype)
    out, _ = qmm.qk_norm_rope(q.cuda(), None, q_weight=w.cuda(), eps=eps)
    check(out, q, w, None, None, eps, False)
