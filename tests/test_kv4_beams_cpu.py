"""Decoding several continuations of a prompt, without a GPU: argument errors found on the host before any launch,
and the host's bookkeeping of the beams' pages."""
import ctypes

import pytest
import torch

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
# Append with norms and rotation.
# ---------------------------------------------------------------------------
def rope_append_args(**k):
    g = k.get
    return [g("q", P), g("qts", 4096), g("qhs", 128), g("hq", 32), g("k", P), g("kts", 1024), g("khs", 128), g("v", P),
            g("vts", 1024), g("vhs", 128), g("dt", BF16), g("T", 4), g("pos", P), g("table", P), g("rows", 100),
            g("rot", 128), g("inter", 0), g("qw", P), g("kw", P), g("wdt", BF16), ctypes.c_float(g("eps", 1e-6)),
            g("slots", P), g("cache", P), g("pages", 10), g("hk", 8), g("D", 128), g("page", 64), g("group", 64),
            g("out", P), None]


def test_rope_append_errors():
    f, a = qmm.lib().kv4_rope_append, rope_append_args
    assert f(*a(T=0, k=None)) == OK
    for kw in [dict(k=None), dict(v=None), dict(slots=None), dict(cache=None), dict(q=None), dict(out=None), dict(T=-1),
               dict(hq=-1), dict(rot=-16), dict(dt=9), dict(eps=-1.0), dict(eps=float("nan")), dict(pos=None),
               dict(table=None), dict(rows=0), dict(wdt=11), dict(pages=0), dict(hk=0), dict(D=0), dict(page=0),
               dict(group=0)]:
        assert f(*a(**kw)) == EINVAL, kw
    for kw in [dict(dt=F32), dict(dt=I32), dict(wdt=F16), dict(wdt=I32), dict(D=96, rot=96), dict(page=24),
               dict(group=48), dict(D=64, rot=64, group=128), dict(rot=24), dict(rot=144)]:
        assert f(*a(**kw)) == EUNSUP, kw
    for kw in [dict(T=1 << 24), dict(T=1 << 40), dict(hq=70000), dict(hk=5000), dict(pages=1 << 31),
               dict(T=(1 << 24) - 1, hq=4096)]:
        assert f(*a(**kw)) == ERANGE, kw
    for kw in [dict(q=MIS), dict(k=MIS), dict(v=MIS), dict(cache=P + 8), dict(slots=P + 4), dict(qw=MIS), dict(kw=MIS),
               dict(pos=P + 4), dict(table=P + 8), dict(out=MIS), dict(qts=4100), dict(khs=4), dict(vts=1020)]:
        assert f(*a(**kw)) == EALIGN, kw


def test_rope_append_checks():
    q, k, v, slots = t((4, 8, 128), bf16), t((4, 2, 128), bf16), t((4, 2, 128), bf16), t(4, i64)
    cache, pos, table = t((3, 2, 64, 144), u8), t(4, i64), t((9, 64, 2), f32)
    f = qmm.kv4_rope_append
    raises(lambda: f(q, k.float(), v, slots, cache), "k has dtype")
    raises(lambda: f(q, k, v.half(), slots, cache), "v has dtype")
    raises(lambda: f(q, k, v[:3], slots, cache), "v has shape")
    raises(lambda: f(q.half(), k, v, slots, cache), "q has dtype")
    raises(lambda: f(q[:3], k, v, slots, cache), "q has shape")
    raises(lambda: f(q[..., :64], k, v, slots, cache), "q has shape")
    raises(lambda: f(q, k, v, slots[:3], cache), "slots has shape")
    raises(lambda: f(q, k, v, slots.int(), cache), "slots has dtype")
    raises(lambda: f(q, k, v, slots, cache[:, :1].contiguous()), "heads")
    raises(lambda: f(q, k, v, slots, t((3, 2, 64, 137), u8)), "token of head_dim")
    raises(lambda: f(q, k, v, slots, cache, pos), "positions need a table")
    raises(lambda: f(q, k, v, slots, cache, None, table), "positions")
    raises(lambda: f(q, k, v, slots, cache, pos.int(), table), "positions has dtype")
    raises(lambda: f(q, k, v, slots, cache, pos, t((9, 65, 2), f32)), "table rotates")
    raises(lambda: f(q, k, v, slots, cache, pos, table.double()), "table has dtype")
    raises(lambda: f(q, k, v, slots, cache, q_weight=t(128, f16)), "q_weight has dtype")
    raises(lambda: f(q, k, v, slots, cache, q_weight=t(128, f32), k_weight=t(128, bf16)), "k_weight has dtype")
    raises(lambda: f(q, k, v, slots, cache, k_weight=t(64, bf16)), "k_weight has shape")
    raises(lambda: f(None, k, v, slots, cache, q_weight=t(128, bf16)), "need q")
    raises(lambda: f(q, k, v, slots, cache, eps=-1.0), "eps")
    raises(lambda: f(q, k, v, slots, cache, q_out=t((4, 8, 64), bf16)), "q_out has shape")
    raises(lambda: f(q, k.transpose(1, 2).contiguous().transpose(1, 2), v, slots, cache), "channels consecutive")
    raises(lambda: f(q, k, v, slots, cache), "device tensors")
