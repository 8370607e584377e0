"""Norms, rotation and append in one pass.

The queries are bit for bit those of qk_norm_rope.  The keys are compared as
cache bytes with the formulas in fp64, rounded once to fp32, and the cache's
rule on those: fp64 values that differ in the order of a sum alone (2^-52) fall
on different sides of a border with a probability of about 2^-26 a key here, so
the bytes of these fixed inputs are the same."""
import numpy as np
import pytest
import torch

import kv4_reference as ref
import quantized_matmul_quantize_amd as qmm
from gpu_util import note

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def half(x, dtype):
    return torch.from_numpy(np.asarray(x, np.float32)).to(dtype)


def cuda(x):
    return None if x is None else x.cuda()


def dirty(pages, heads, D, page, group):
    cache = qmm.kv4_cache(pages, heads, D, page, group)
    cache.fill_(255)
    return cache


def key(x, w, positions, table, eps, interleaved):
    """fp64 key, rounded once to fp32."""
    x = x.double().numpy()
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + np.float64(np.float32(eps))) * w.double().numpy()
    y = x.copy()
    if table is not None:
        rows = table.double().numpy()
        cs = np.full((len(positions), rows.shape[1], 2), np.nan)
        ok = (positions.numpy() >= 0) & (positions.numpy() < len(rows))
        cs[ok] = rows[positions.numpy()[ok]]
        cs, r = cs[:, None], 2 * rows.shape[1]
        a_at = np.arange(0, r, 2) if interleaved else np.arange(r // 2)
        b_at = a_at + (1 if interleaved else r // 2)
        a, b = x[..., a_at], x[..., b_at]
        with np.errstate(invalid="ignore"):
            y[..., a_at] = a * cs[..., 0] - b * cs[..., 1]
            y[..., b_at] = b * cs[..., 0] + a * cs[..., 1]
    with np.errstate(over="ignore"):
        return y.astype(np.float32)


def compare(q, k, v, slots, positions, table, qw, kw, eps, interleaved, page, group, pages, q_out=None, cache=None):
    T, heads, D = k.shape
    cache = dirty(pages, heads, D, page, group) if cache is None else cache
    want = cache.cpu().numpy().copy()
    got_q = qmm.kv4_rope_append(cuda(q), k.cuda(), v.cuda(), slots.cuda(), cache, cuda(positions), cuda(table), cuda(qw),
                                cuda(kw), eps, interleaved, q_out=q_out)
    keys = key(k, kw, positions, table, eps, interleaved)
    # the range of a group is that of its numbers and 0: NaN alone are as zeros, code 0 (numpy's minimum would be NaN)
    groups = keys.reshape(T, heads, -1, group)
    groups[np.isnan(groups).all(-1)] = 0
    ref.store(want, keys, v.float().numpy(), slots.tolist())
    got = cache.cpu().numpy()
    assert np.array_equal(got, want), f"{(got != want).sum()} bytes differ"
    if q is not None:
        want_q, _ = qmm.qk_norm_rope(q.cuda(), None, cuda(positions), cuda(table), cuda(qw), None, eps, interleaved)
        assert torch.equal(got_q.view(torch.int16), want_q.view(torch.int16))
    return got_q


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "interleaved"])
@pytest.mark.parametrize("D,group,page,rot", [(64, 32, 16, 64), (64, 64, 32, 16), (128, 32, 64, 128), (128, 64, 128, 64),
                                              (128, 128, 256, 48), (256, 32, 16, 256), (256, 64, 64, 32),
                                              (256, 128, 32, 0)])
@pytest.mark.parametrize("norm", ["both", "none", "k", "f32"])
def test_formats(dtype, interleaved, D, group, page, rot, norm):
    note(f"kv4_rope_append D={D} group={group} page={page} rot={rot} interleaved={interleaved} norm={norm} {dtype}")
    g = rng(D + group + rot)
    T, hq, hk, rows = 13, 6, 3, 40
    q, k, v = (half(g.standard_normal((T, h, D)) * s, dtype) for h, s in ((hq, 3.0), (hk, 0.5), (hk, 20.0)))
    k[3], v[4] = 0, 0                                       # a head of zeros: eps alone
    wt = F32 if norm == "f32" else dtype
    qw = half(1 + 0.3 * g.standard_normal(D), wt) if norm in ("both", "f32") else None
    kw = half(1 + 0.3 * g.standard_normal(D), wt) if norm != "none" else None
    table = torch.from_numpy(g.standard_normal((rows, rot // 2, 2)).astype(np.float32)) if rot else None
    positions = torch.from_numpy(g.integers(0, rows, T)) if rot else None
    slots = torch.from_numpy(g.permutation(4 * page)[:T].astype(np.int64))
    slots[2], slots[5] = -1, 4 * page                       # queries without a place in the cache
    compare(q, k, v, slots, positions, table, qw, kw, 1e-5, interleaved, page, group, 4)


@pytest.mark.parametrize("T,hq,hk,D", [(1, 1, 1, 128), (3, 17, 1, 64), (5, 0, 2, 256), (700, 40, 8, 128), (2049, 3, 3, 64),
                                       (1300, 32, 32, 64)])
def test_tokens_and_heads(T, hq, hk, D):
    note(f"kv4_rope_append T={T} heads={hq}/{hk} D={D}")
    g = rng(T + hq)
    page, group = 64, 64
    pages = -(-T // page) + 1
    q, k, v = (half(g.standard_normal((T, h, D)), BF16) if h else None for h in (hq, hk, hk))
    table = qmm.rope_table(T + 7, qmm.rope_frequencies(D)[0]).cpu()
    slots = torch.from_numpy(g.permutation(pages * page)[:T].astype(np.int64))
    qw, kw = half(1 + 0.1 * g.standard_normal(D), BF16), half(1 + 0.1 * g.standard_normal(D), BF16)
    compare(q, k, v, slots, torch.arange(T) + 3, table, qw if hq else None, kw, 1e-6, False, page, group, pages)


def test_views_of_a_projection_queries_in_place_and_the_last_slots_of_a_large_cache():
    T, hq, hk, D, page, group, pages = 21, 8, 2, 128, 64, 64, 240000
    g = rng(6)
    qkv = half(g.standard_normal((T, (hq + 2 * hk) * D)), F16).cuda()
    q, k, v = qkv.view(T, -1, D).split([hq, hk, hk], 1)
    cache = qmm.kv4_cache(pages, hk, D, page, group)
    assert cache.numel() > 2 ** 32
    slots = torch.arange(pages * page - T, pages * page, device="cuda")
    table = qmm.rope_table(T, qmm.rope_frequencies(D)[0])
    at = torch.arange(T, device="cuda")
    out = qmm.kv4_rope_append(q, k, v, slots, cache, at, table)
    want, _ = qmm.qk_norm_rope(q, None, at, table)
    assert torch.equal(out, want)
    dense = q.contiguous()
    assert qmm.kv4_rope_append(dense, k, v, slots, cache, at, table, q_out=dense) is dense and torch.equal(dense, want)
    kr, vr = qmm.kv4_read(cache, slots, D, dtype=F32)
    for x, y in ((key(k.cpu(), None, at.cpu(), table.cpu(), 0, False), kr), (v.float().cpu().numpy(), vr)):
        assert np.array_equal(y.cpu().numpy(), ref.values(*ref.quantize(x, group)).astype(np.float32))


def test_positions_outside_the_table_and_what_is_not_finite():
    g = rng(8)
    T, hq, hk, D, page, group = 9, 2, 2, 128, 16, 32
    q, k, v = (half(g.standard_normal((T, h, D)), BF16) for h in (hq, hk, hk))
    k[0, 0, 100], k[1, 1, 70], v[2, 0, 3], v[2, 1, 40] = np.inf, np.nan, -np.inf, np.nan
    positions = torch.arange(T)
    positions[4], positions[5] = -1, 50
    table = torch.from_numpy(g.standard_normal((50, 16, 2)).astype(np.float32))
    for interleaved in (False, True):
        out = compare(q, k, v, torch.arange(T), positions, table, None, None, 1e-6, interleaved, page, group, 1)
        assert out[4, :, :32].isnan().all() and out[4, :, 32:].isfinite().all() and out[6].isfinite().all()


def test_keys_of_any_size():
    """Heads whose mean square is far below and far above eps, and bf16 near its ends."""
    g = rng(9)
    T, D = 8, 64
    size = np.array([1e-38, 1e-30, 1e-20, 1e-10, 1.0, 1e10, 1e18, 1e30])[:, None, None]
    k = half(g.standard_normal((T, 2, D)) * size, BF16)
    v = half(g.standard_normal((T, 2, D)), BF16)
    table = torch.from_numpy(g.standard_normal((T, 16, 2)).astype(np.float32))
    for eps in (1e-6, 0.0):
        compare(None, k, v, torch.arange(T), torch.arange(T), table, None, half(np.ones(D), F32), eps, False, 16, 32, 1)


def test_no_tokens_another_stream_and_a_replayed_graph():
    D, heads = 64, 2
    cache = dirty(2, heads, D, 16, 32)
    none = torch.empty((0, heads, D), dtype=BF16, device="cuda")
    assert qmm.kv4_rope_append(none, none, none, torch.empty(0, dtype=torch.int64, device="cuda"), cache).shape == (0, heads, D)
    assert (cache == 255).all()

    g = rng(11)
    q, k, v = (half(g.standard_normal((5, heads, D)), BF16).cuda() for _ in range(3))
    slots, at = torch.arange(5, device="cuda"), torch.arange(5, device="cuda")
    table = qmm.rope_table(64, qmm.rope_frequencies(D)[0])
    want = dirty(2, heads, D, 16, 32)
    want_q = qmm.kv4_rope_append(q, k, v, slots, want, at, table)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = qmm.kv4_rope_append(q, k, v, slots, cache, at, table)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want_q) and torch.equal(cache, want)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = qmm.kv4_rope_append(q, k, v, slots, cache, at, table)
    for turn in range(3):
        k.copy_(half(g.standard_normal((5, heads, D)), BF16))
        slots.add_(5)
        at.add_(7)
        graph.replay()
        want_q = qmm.kv4_rope_append(q, k, v, slots, want, at, table)
        torch.cuda.synchronize()
        assert torch.equal(out, want_q) and torch.equal(cache, want)
