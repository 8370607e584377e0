"""The 4-bit key/value cache, its attention and the rotation without a GPU:
argument errors found on the host before any launch, sizes, frequencies, and
the reference implementation itself against differences from its definition."""
import ctypes
import math

import numpy as np
import pytest
import torch

import kv4_bounds as bounds
import kv4_reference as ref
import quantized_matmul_quantize_amd as qmm

OK, EINVAL, EUNSUP, EALIGN, EWS, EHIP, ERANGE = 0, -1, -2, -3, -4, -5, -6
P = 0x7F0000000000          # 16-byte aligned stand-in for a device pointer
MIS = P + 2
BF16, F16, F32, I32 = qmm.BF16, qmm.F16, qmm.F32, qmm.I32
bf16, f16, f32, u8, i32, i64 = torch.bfloat16, torch.float16, torch.float32, torch.uint8, torch.int32, torch.int64


def t(shape, dtype):
    return torch.zeros(shape, dtype=dtype)


def raises(fn, match):
    with pytest.raises(ValueError, match=match):
        fn()


# ---------------------------------------------------------------------------
# C ABI.
# ---------------------------------------------------------------------------
def test_page_bytes():
    f = qmm.lib().kv4_page_bytes
    assert f(8, 128, 64, 64) == 8 * 64 * (128 + 16)
    assert f(1, 64, 16, 32) == 16 * (64 + 16) and f(2, 256, 256, 128) == 2 * 256 * (256 + 16)
    for bad in [(0, 128, 64, 64), (8, 96, 64, 32), (8, 128, 48, 64), (8, 128, 512, 64), (8, 128, 64, 16), (8, 64, 64, 128),
                (-1, 128, 64, 64), (8, 128, 64, 0)]:
        assert f(*bad) == 0, bad


def append_args(**k):
    g = k.get
    return [g("k", P), g("kts", 1024), g("khs", 128), g("v", P), g("vts", 1024), g("vhs", 128), g("dt", BF16), g("T", 4),
            g("slots", P), g("cache", P), g("pages", 10), g("heads", 8), g("D", 128), g("page", 64), g("group", 64), None]


def test_append_and_read_errors():
    f = qmm.lib().kv4_append
    a = append_args
    assert f(*a(T=0, k=None)) == OK                        # nothing to append
    for kw in [dict(k=None), dict(v=None), dict(slots=None), dict(cache=None), dict(T=-1), dict(dt=7), dict(pages=0),
               dict(heads=0), dict(D=0), dict(page=0), dict(group=0)]:
        assert f(*a(**kw)) == EINVAL, kw
    for kw in [dict(dt=F32), dict(dt=I32), dict(D=96), dict(page=24), dict(group=48), dict(D=64, group=128)]:
        assert f(*a(**kw)) == EUNSUP, kw
    for kw in [dict(T=1 << 25), dict(T=1 << 31), dict(pages=1 << 31), dict(heads=5000), dict(kts=1 << 26), dict(vts=-(1 << 26))]:
        assert f(*a(**kw)) == ERANGE, kw
    for kw in [dict(k=MIS), dict(v=MIS), dict(cache=MIS), dict(slots=P + 4), dict(kts=1020), dict(vhs=4)]:
        assert f(*a(**kw)) == EALIGN, kw
    r = qmm.lib().kv4_read
    args = lambda **k: [k.get("c", P), 10, 8, k.get("D", 128), 64, 64, k.get("s", P), k.get("T", 4), k.get("k", P),
                        k.get("v", P), k.get("dt", BF16), None]
    assert r(*args(T=0)) == OK and r(*args(c=None)) == EINVAL and r(*args(v=None)) == EINVAL and r(*args(dt=9)) == EINVAL
    assert r(*args(dt=I32)) == EUNSUP and r(*args(D=80)) == EUNSUP and r(*args(T=1 << 31)) == ERANGE
    assert r(*args(k=MIS)) == EALIGN and r(*args(s=P + 4)) == EALIGN


def test_copy_errors():
    f = qmm.lib().kv4_copy_pages
    assert f(P, 1, 4, 64, P, P, 0, None) == OK
    assert f(None, 1, 4, 64, P, P, 1, None) == EINVAL and f(P, 0, 4, 64, P, P, 1, None) == EINVAL
    assert f(P, 1, 4, 0, P, P, 1, None) == EINVAL and f(P, 1, 4, 64, P, P, -1, None) == EINVAL
    assert f(P, 1, 4, 72, P, P, 1, None) == EALIGN and f(MIS, 1, 4, 64, P, P, 1, None) == EALIGN
    assert f(P, 1, 4, 64, P + 4, P, 1, None) == EALIGN
    assert f(P, 70000, 4, 64, P, P, 1, None) == ERANGE and f(P, 1, 4, 64, P, P, 1 << 24, None) == ERANGE


def attention_args(**k):
    g = k.get
    return [g("q", P), g("qts", 4096), g("qhs", 128), g("dt", BF16), g("T", 4), g("hq", 32), g("cu", None), g("seqs", 4),
            g("max_q", 1), g("context", P), g("table", P), g("width", 20), g("stride", 20), g("cache", P), g("pages", 100),
            g("hk", 8), g("D", 128), g("page", 64), g("group", 64), ctypes.c_float(g("scale", 0.1)), g("window", 0),
            g("sinks", 0), g("out", P), None, g("ws", P), g("wsb", 10 ** 9), None]


def test_attention_errors():
    f = qmm.lib().kv4_attention
    a = attention_args
    assert f(*a(T=0)) == OK
    for kw in [dict(q=None), dict(context=None), dict(table=None), dict(cache=None), dict(out=None), dict(T=-1),
               dict(seqs=0), dict(T=5), dict(max_q=0), dict(width=0), dict(stride=19), dict(window=-1), dict(sinks=-1),
               dict(scale=float("nan")), dict(hq=33), dict(hq=0), dict(hk=0), dict(dt=8), dict(pages=0)]:
        assert f(*a(**kw)) == EINVAL, kw
    for kw in [dict(dt=F32), dict(D=96), dict(page=8), dict(group=16)]:
        assert f(*a(**kw)) == EUNSUP, kw
    for kw in [dict(T=1 << 31, cu=P), dict(seqs=70000, T=70000), dict(width=1 << 25, stride=1 << 25),
               dict(hq=80000, hk=8), dict(T=1 << 27, cu=P)]:
        assert f(*a(**kw)) == ERANGE, kw
    for kw in [dict(q=MIS), dict(out=MIS), dict(cache=P + 8), dict(qts=4100), dict(qhs=4), dict(table=P + 2),
               dict(context=P + 1), dict(cu=P + 2)]:
        assert f(*a(**kw)) == EALIGN, kw
    need = qmm.kv4_attention_workspace_bytes(4, 4, 1, 32, 8, 128, 64, 20 * 64)
    wide = qmm.kv4_attention_workspace_bytes(4, 4, 1, 32, 8, 128, 64, 2000 * 64)
    assert need == 0 or need < wide
    assert wide > 0 and wide % (4 * 32 * 4) == 0
    assert f(*a(width=2000, stride=2000, ws=None)) == EWS
    assert f(*a(width=2000, stride=2000, wsb=wide - 1)) == EWS
    assert f(*a(width=2000, stride=2000, ws=MIS)) == EALIGN


def test_attention_workspace():
    w = qmm.kv4_attention_workspace_bytes
    assert w(64, 64, 1, 32, 8, 128, 128, 4096) == 0                   # rows and heads fill the chip
    assert w(1, 1, 1, 32, 8, 128, 64, 512) == 0                       # too short to split
    one = w(1, 1, 1, 32, 8, 128, 64, 65536)
    assert one > 0 and one % (32 * (128 + 2) * 4) == 0                # partial sums, maxima and sums of every chunk
    assert w(1, 1, 1, 32, 8, 128, 64, 65536, 1024, 4) < one           # a window needs fewer chunks
    for bad in [(0, 1, 1, 32, 8, 128, 64, 512), (1, 0, 1, 32, 8, 128, 64, 512), (1, 1, 1, 33, 8, 128, 64, 512),
                (1, 1, 1, 32, 8, 128, 64, 0), (1, 1, 0, 32, 8, 128, 64, 512), (1, 1, 1, 32, 8, 128, 0, 512)]:
        assert w(*bad) == 0


def test_rope_errors():
    f = qmm.lib().qk_norm_rope
    a = lambda **k: [k.get("q", P), k.get("qts", 4096), 128, k.get("hq", 32), k.get("k", P), k.get("kts", 1024), 128,
                     k.get("hk", 8), k.get("dt", BF16), k.get("T", 4), k.get("D", 128), k.get("pos", P), k.get("table", P),
                     k.get("rows", 100), k.get("rot", 128), 0, k.get("qw", P), k.get("kw", P), k.get("wdt", BF16),
                     ctypes.c_float(k.get("eps", 1e-6)), k.get("qo", P), k.get("ko", P), None]
    assert f(*a(T=0)) == OK
    for kw in [dict(q=None), dict(qo=None), dict(k=None), dict(ko=None), dict(hq=0), dict(hk=-1), dict(T=-1), dict(D=0),
               dict(rot=-16), dict(pos=None), dict(table=None), dict(rows=0), dict(eps=-1.0), dict(eps=float("nan")),
               dict(dt=5), dict(wdt=6)]:
        assert f(*a(**kw)) == EINVAL, kw
    for kw in [dict(dt=F32), dict(wdt=F16), dict(D=132), dict(D=520, rot=16), dict(rot=24), dict(rot=144)]:
        assert f(*a(**kw)) == EUNSUP, kw
    assert f(*a(T=1 << 24)) == ERANGE and f(*a(hq=70000)) == ERANGE
    for kw in [dict(q=MIS), dict(ko=MIS), dict(qw=MIS), dict(table=P + 8), dict(pos=P + 4), dict(qts=4100), dict(kts=1028)]:
        assert f(*a(**kw)) == EALIGN, kw
    g = qmm.lib().rope_table
    host = ctypes.cast((ctypes.c_double * 2)(1.0, 0.1), ctypes.c_void_p)
    d = ctypes.c_double(1.0)
    assert g(None, 2, 4, d, P, None) == EINVAL and g(host, 0, 4, d, P, None) == EINVAL and g(host, 2, 0, d, P, None) == EINVAL
    assert g(host, 257, 4, d, P, None) == EUNSUP and g(host, 2, 1 << 30, d, P, None) == ERANGE
    assert g(host, 2, 4, d, MIS, None) == EALIGN


# ---------------------------------------------------------------------------
# Binding.
# ---------------------------------------------------------------------------
def cache(pages=4, heads=2, D=128, page=16, group=64):
    return qmm.kv4_cache(pages, heads, D, page, group, device="cpu")


def test_cache_shapes():
    c = qmm.kv4_cache(5, 3, 128, 32, 32, layers=2, device="cpu")
    assert c.shape == (2, 5, 3, 32, 128 + 32) and c.dtype == u8
    assert c[0, 0].numel() == qmm.kv4_page_bytes(3, 128, 32, 32)
    raises(lambda: qmm.kv4_cache(5, 3, 100), "unsupported")
    raises(lambda: qmm.kv4_cache(5, 3, 128, page=17), "unsupported")


def test_append_and_read_checks():
    k, s, c = t((3, 2, 128), bf16), t((3,), i64), cache()
    raises(lambda: qmm.kv4_append(k.float(), k, s, c), "k has dtype")
    raises(lambda: qmm.kv4_append(k, k.half(), s, c), "v has dtype")
    raises(lambda: qmm.kv4_append(k, k[:2], s, c), "v has shape")
    raises(lambda: qmm.kv4_append(k[0], k, s, c), "k must have 3 dimensions")
    raises(lambda: qmm.kv4_append(t((3, 1, 128), bf16), t((3, 1, 128), bf16), s, c), "heads")
    raises(lambda: qmm.kv4_append(k, k, s.int(), c), "slots has dtype")
    raises(lambda: qmm.kv4_append(k, k, s[:2], c), "slots has shape")
    raises(lambda: qmm.kv4_append(k, k, s, c.to(torch.int8)), "cache has dtype")
    raises(lambda: qmm.kv4_append(k, k, s, c[..., :129]), "cache has shape")
    raises(lambda: qmm.kv4_append(t((3, 2, 256), bf16)[..., ::2], k, s, c), "channels consecutive")
    raises(lambda: qmm.kv4_append(t((3, 2, 132), bf16)[..., :128], k, s, c), "multiples of 8")
    raises(lambda: qmm.kv4_append(k, k, s, c), "device tensors")
    raises(lambda: qmm.kv4_read(c, s, 128, dtype=i32), "output dtype")
    raises(lambda: qmm.kv4_read(c, s.int(), 128), "slots has dtype")
    raises(lambda: qmm.kv4_read(c, s, 128), "device tensors")


def test_copy_checks():
    c = cache()
    raises(lambda: qmm.kv4_copy_pages(c[0], t((1,), i64), t((1,), i64)), "4 dimensions")
    raises(lambda: qmm.kv4_copy_pages(c, t((1,), i32), t((1,), i64)), "src has dtype")
    raises(lambda: qmm.kv4_copy_pages(c, t((1,), i64), t((2,), i64)), "dst has shape")
    raises(lambda: qmm.kv4_copy_pages(c, t((1,), i64), t((1,), i64)), "device tensors")


def test_attention_checks():
    q, c, tab, ctx = t((3, 4, 128), bf16), cache(), t((3, 2), i32), t((3,), i32)
    f = qmm.kv4_attention
    raises(lambda: f(q.float(), c, tab, ctx), "q has dtype")
    raises(lambda: f(t((3, 3, 128), bf16), c, tab, ctx), "multiple of the cache's")
    raises(lambda: f(t((3, 4, 64), bf16), c[..., :80], tab[:, :1].long(), ctx), "page_table has dtype")
    raises(lambda: f(q, c, tab, ctx.long()), "context has dtype")
    raises(lambda: f(q, c, tab, ctx[:2]), "context has shape")
    raises(lambda: f(q, c, t((2, 2), i32), t((2,), i32)), "without cu_q")
    raises(lambda: f(q, c, tab, ctx, cu_q=t((3,), i32)), "cu_q has shape")
    raises(lambda: f(q, c, t((2, 3), i32).t(), ctx), "consecutive rows")
    raises(lambda: f(q, c, tab, ctx, window=-1), "window")
    raises(lambda: f(q, c, tab, ctx, sinks=-2), "sinks")
    raises(lambda: f(q, c, tab, ctx, out=t((3, 4, 128), f16)), "out has dtype")
    raises(lambda: f(q, c, tab, ctx), "device tensors")


def test_rope_checks():
    q, k, pos, tab, w = t((3, 4, 128), bf16), t((3, 2, 128), bf16), t((3,), i64), t((9, 64, 2), f32), t((128,), bf16)
    f = qmm.qk_norm_rope
    raises(lambda: f(q.float(), k, pos, tab), "q has dtype")
    raises(lambda: f(q, k.half(), pos, tab), "k has dtype")
    raises(lambda: f(q, t((2, 2, 128), bf16), pos, tab), "k has shape")
    raises(lambda: f(q, None, pos, tab, k_weight=w), "need k")
    raises(lambda: f(q, k, pos.int(), tab), "positions has dtype")
    raises(lambda: f(q, k, pos, None), "need a table")
    raises(lambda: f(q, k, pos, tab.double()), "table has dtype")
    raises(lambda: f(q, k, pos, t((9, 65, 2), f32)), "rotates")
    raises(lambda: f(q, k, pos, tab, w.half()), "q_weight has dtype")
    raises(lambda: f(q, k, pos, tab, w, w.float()), "k_weight has dtype")
    raises(lambda: f(q, k, pos, tab, w[:64]), "q_weight has shape")
    raises(lambda: f(q, k, pos, tab, eps=-1.0), "eps")
    raises(lambda: f(q, k, pos, tab, q_out=t((3, 4, 64), bf16)), "q_out has shape")
    raises(lambda: f(q, k, pos, tab), "device tensors")
    raises(lambda: qmm.rope_table(0, [1.0]), "at least one row")
    raises(lambda: qmm.rope_table(4, [1.0] * 257), "256 frequencies")


# ---------------------------------------------------------------------------
# Frequencies.
# ---------------------------------------------------------------------------
def test_frequencies():
    f, m = qmm.rope_frequencies(8, base=10000.0)
    assert m == 1.0 and np.allclose(f, [1.0, 0.1, 0.01, 0.001], rtol=1e-15)
    lin, _ = qmm.rope_frequencies(8, scaling="linear", factor=4.0)
    assert np.allclose(lin, np.array(f) / 4, rtol=1e-15)
    # ntk: the slowest pair interpolated by the factor, the fastest kept
    ntk, _ = qmm.rope_frequencies(8, scaling="ntk", factor=4.0)
    assert ntk[0] == f[0] and math.isclose(ntk[-1], f[-1] / 4, rel_tol=1e-12) and all(a <= b for a, b in zip(ntk, f))
    # by wavelength: pairs of many turns keep their frequency, of few are interpolated, monotonic between
    full, _ = qmm.rope_frequencies(128, base=500000.0)
    w, m = qmm.rope_frequencies(128, base=500000.0, scaling="wavelength", factor=8.0, original=8192, low=1.0, high=4.0)
    turns = 8192 * np.array(full) / (2 * math.pi)
    ratio = np.array(w) / np.array(full)
    assert m == 1.0 and np.allclose(ratio[turns >= 4], 1.0) and np.allclose(ratio[turns <= 1], 1 / 8)
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and np.allclose(ratio[mid], 1 / 8 + 7 / 8 * (turns[mid] - 1) / 3)
    y, m = qmm.rope_frequencies(128, scaling="yarn", factor=16.0, original=4096)
    r = np.array(y) / np.array(qmm.rope_frequencies(128)[0])
    assert math.isclose(m, 0.1 * math.log(16) + 1) and r[0] == 1.0 and math.isclose(r[-1], 1 / 16)
    assert (np.diff(r) <= 1e-15).all()
    assert qmm.rope_frequencies(128, scaling="yarn", factor=1.0)[1] == 1.0
    for bad in [dict(rot=7), dict(rot=0), dict(rot=8, base=0.0), dict(rot=8, factor=-1.0), dict(rot=8, scaling="x"),
                dict(rot=2, scaling="ntk"), dict(rot=8, scaling="yarn", low=4.0, high=2.0)]:
        with pytest.raises(ValueError):
            qmm.rope_frequencies(**bad)


# ---------------------------------------------------------------------------
# The reference itself.
# ---------------------------------------------------------------------------
def test_reference_quantizer():
    g = np.random.Generator(np.random.PCG64(1))
    x = g.standard_normal((50, 2, 128)).astype(np.float16).astype(np.float32)
    c, z, s = ref.quantize(x, 32)
    v = ref.values(c, z, s)
    step = np.repeat(s, 32, -1)
    assert (np.abs(v - x) <= step * (0.5 + 2.0 ** -10)).all()          # nearest code; the scale is rounded
    assert c.max() == 15 and c.min() == 0
    zero = ref.quantize(np.zeros((1, 128), np.float32), 64)
    assert (zero[2] == 1).all() and (ref.values(*zero) == 0).all()


def test_reference_layout_reads_back():
    g = np.random.Generator(np.random.PCG64(2))
    D, group, page = 128, 64, 16
    c = np.full((3, 2, page, D + 8 * D // group), 255, np.uint8)
    k, v = (g.standard_normal((5, 2, D)).astype(np.float32) for _ in range(2))
    slots = [3, 17, 40, -1, 47]
    ref.store(c, k, v, slots)
    w = c.view(np.uint32).reshape(3, 2, -1)
    for x, keys in ((k, True), (v, False)):
        code, z, s = ref.quantize(x, group)
        for i, slot in enumerate(slots):
            if slot < 0:
                continue
            p, tt = divmod(slot, page)
            for h in range(2):
                for d in (0, 1, 37, 64, 127):
                    j, e = divmod(d, 8)
                    at = tt * 16 + (j % 4) * 4 + j // 4 if keys else page * 16 + (tt // 4) * 64 + 4 * j + tt % 4
                    assert (w[p, h, at] >> (4 * (e // 2) + 16 * (e % 2))) & 15 == code[i, h, d]
                    par = w[p, h, page * 32 + (0 if keys else 2 * page) + (d // group) * page + tt]
                    assert np.uint16(par & 0xFFFF).view(np.float16) == s[i, h, d // group] and par >> 16 == z[i, h, d // group]


def test_reference_attention_against_sums_of_one_key():
    """One visible key gives its value; two of equal score their mean; masks in hand-written places."""
    q = np.ones((3, 1, 4))
    k = np.zeros((1, 1, 4)).repeat(4, 0)
    v = np.arange(16.0).reshape(4, 1, 4)
    out, lse, mass, n = ref.attention(q, [k], [v], [4], [3], 1.0)
    assert n.tolist() == [2, 3, 4] and np.allclose(out[0, 0], v[:2].mean(0)[0]) and np.allclose(lse[:, 0], np.log([2, 3, 4]))
    out, lse, _, n = ref.attention(q, [k], [v], [4], [3], 1.0, window=1, sinks=1)
    assert n.tolist() == [2, 2, 2] and np.allclose(out[2, 0], (v[0, 0] + v[3, 0]) / 2)
    out, lse, _, n = ref.attention(q, [k], [v], [4], [3], 1.0, here=[np.array([False] * 4)])
    assert n.tolist() == [0, 0, 0] and (out == 0).all() and np.isneginf(lse).all()


def test_blocks_are_the_calls():
    """<name>_block: the same statuses for the same arguments, a word each; floating-point ones as double."""
    lib = qmm.lib()
    value = lambda x: 0 if x is None else getattr(x, "value", x)
    calls = {"kv4_append": [append_args(), append_args(T=0, k=None), append_args(D=96), append_args(k=MIS), append_args(T=-1)],
             "kv4_attention": [attention_args(T=0), attention_args(D=96), attention_args(q=MIS), attention_args(hq=33),
                               attention_args(scale=float("nan")), attention_args(width=2000, stride=2000, ws=None)],
             "kv4_read": [[P, 10, 8, 96, 64, 64, P, 4, P, P, BF16, None], [P, 10, 8, 128, 64, 64, P, 4, MIS, P, BF16, None]],
             "kv4_copy_pages": [[P, 1, 4, 72, P, P, 1, None], [P, 0, 4, 64, P, P, 1, None], [P, 1, 4, 64, P, P, 0, None]],
             "qk_norm_rope": [[P, 4096, 128, 32, P, 1024, 128, 8, BF16, 4, 128, P, P, 100, 24, 0, P, P, BF16,
                               ctypes.c_float(1e-6), P, P, None],
                              [P, 4096, 128, 32, P, 1024, 128, 8, BF16, 4, 128, P, P, 100, 128, 0, P, P, BF16,
                               ctypes.c_float(-1.0), P, P, None]]}
    launched = {("kv4_append", 0)}                   # valid, so it would launch: nothing to compare without a GPU
    for name, lists in calls.items():
        block = getattr(lib, name + "_block")
        assert block(None) == EINVAL
        for i, args in enumerate(lists):
            if (name, i) not in launched:
                want = getattr(lib, name)(*args)
                assert block(qmm._BLOCKS[name].pack(*map(value, args))) == want, (name, i)


@pytest.mark.parametrize("kw", [dict(base=10000.0, original=131072), dict(base=500000.0, original=4 * 10 ** 6),
                                dict(base=10000.0, original=4096), dict(base=500000.0, original=8192)])
def test_yarn_ramp_is_linear_between_its_ends(kw):
    """Also where every pair turns more than `low` times in the original context, so that the ramp's end lies past the
    last pair (a ramp held to the last pair would divide it fully)."""
    rot, factor, low, high = 128, 8.0, 1.0, 32.0
    y, _ = qmm.rope_frequencies(rot, scaling="yarn", factor=factor, low=low, high=high, **kw)
    f = np.array(qmm.rope_frequencies(rot, base=kw["base"])[0])
    # f_i turns original f_i / 2 pi times: i of a given number of turns, to whole pairs outwards
    at = lambda turns: rot / 2 * math.log(kw["original"] / (2 * math.pi * turns)) / math.log(kw["base"])
    first, last = max(math.floor(at(high)), 0), math.ceil(at(low))
    keep = 1 - np.clip((np.arange(rot // 2) - first) / (last - first), 0, 1)
    assert np.allclose(y, f * (keep + (1 - keep) / factor), rtol=1e-13)
    assert last < 64 or (y[-1] > 1.01 * f[-1] / factor)


def test_workspace_of_one_query_each_whatever_the_hint():
    """Without cu_q a call needs what the size query says for the same arguments, the hint included."""
    f, w = qmm.lib().kv4_attention, qmm.lib().kv4_attention_workspace_bytes
    differ = 0
    for seqs, width in [(4, 2000), (16, 500), (64, 2000), (8, 100)]:
        for max_q in (1, 3, 16, 64):
            need = w(seqs, seqs, max_q, 32, 8, 128, 64, width * 64, 0, 0)
            differ += need != w(seqs, seqs, 1, 32, 8, 128, 64, width * 64, 0, 0)
            args = dict(T=seqs, seqs=seqs, max_q=max_q, width=width, stride=width, ws=MIS)
            if need:
                assert f(*attention_args(wsb=need, **args)) == EALIGN      # enough, were it aligned
                assert f(*attention_args(wsb=need - 1, **args)) == EWS
    assert differ > 0


def test_bounds_notice_coarser_probabilities_and_missing_values():
    """The bounds that the kernels are held to: binary16 probabilities are within them, bf16 ones are not where a row
    sees some tens of keys, and the value of no key of a context of 200 with more than 2^-9 of the weight goes missing."""
    g = np.random.Generator(np.random.PCG64(4))
    D, lens = 128, [5, 33, 200]
    q = g.standard_normal((3, 4, D)).astype(np.float16).astype(np.float32)
    parts = [[], [], [], []]
    for n in lens:
        for i, x in enumerate((g.standard_normal((n, 2, D)), g.standard_normal((n, 2, D)))):
            c, z, s = ref.quantize(x.astype(np.float16).astype(np.float32), 64)
            parts[i].append(ref.values(c, z, s))
            parts[2 + i].append(s.astype(np.float64))
    run = lambda rounded=lambda p: p: bounds.attention(q, *parts, lens, [1, 1, 1], D ** -0.5, rounded=rounded)
    out, lse, b_out, b_lse, count = run()
    want = ref.attention(q, parts[0], parts[1], lens, [1, 1, 1], D ** -0.5)
    assert np.allclose(out, want[0], rtol=1e-12) and np.allclose(lse, want[1], rtol=1e-12) and (count == want[3]).all()
    bound = b_out + 2.0 ** -11 * np.abs(out)
    err = lambda rounded: np.abs(run(rounded)[0] - out)
    assert (err(lambda p: (128 * p).astype(np.float16) / 128.0) <= b_out).all()
    coarse = lambda p: torch.from_numpy(p).bfloat16().double().numpy()
    assert (err(coarse) > bound)[:2].any((1, 2)).all()          # (over 200 keys their roundings cancel)
    missed = []
    for j in range(200):
        weight = []

        def without(p):
            if len(p) == 200:
                weight.append(p[j] / p.sum())
                p = np.where(np.arange(200) == j, 0, p)
            return p
        over = (err(without) > bound)[2].any(-1)
        missed += [w for w, seen in zip(weight, over) if not seen]
    assert max(missed, default=0) < 2.0 ** -9
