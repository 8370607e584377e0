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


# ---------------------------------------------------------------------------
# Selection and reordering.
# ---------------------------------------------------------------------------
def select_args(**k):
    g = k.get
    return [g("x", P), g("dt", BF16), g("stride", 1000), g("seqs", 2), g("beams", 4), g("v", 1000), g("scores", P),
            g("finished", None), g("pad", 0), g("k", 4), g("o", P), g("tok", P), g("par", P), g("ws", P), g("wsb", 10 ** 9),
            None]


def test_select_errors():
    f, a = qmm.lib().beam_select, select_args
    assert f(*a(seqs=0, x=None)) == OK
    for kw in [dict(x=None), dict(scores=None), dict(o=None), dict(tok=None), dict(par=None), dict(seqs=-1), dict(beams=0),
               dict(v=0), dict(k=0), dict(k=-3), dict(stride=999), dict(pad=-1), dict(pad=1000), dict(dt=8)]:
        assert f(*a(**kw)) == EINVAL, kw
    for kw in [dict(dt=I32), dict(beams=65), dict(k=65)]:
        assert f(*a(**kw)) == EUNSUP, kw
    for kw in [dict(v=1 << 30, stride=1 << 30), dict(v=1 << 40, stride=1 << 40), dict(seqs=1 << 22), dict(seqs=1 << 62),
               dict(seqs=1 << 18, v=1 << 20, stride=1 << 20)]:
        assert f(*a(**kw)) == ERANGE, kw
    for kw in [dict(x=P + 1), dict(x=P + 2, dt=F32), dict(scores=P + 2), dict(o=P + 1), dict(tok=P + 4), dict(par=P + 4),
               dict(ws=P + 8)]:
        assert f(*a(**kw)) == EALIGN, kw
    need = qmm.beam_select_workspace_bytes(2, 4, 1000, 4)
    assert need == 8 * (16 + 4 * 8) and qmm.beam_select_workspace_bytes(2, 4, 8193, 4) == 2 * need
    assert f(*a(ws=None)) == EWS and f(*a(wsb=need - 1)) == EWS
    for bad in [(0, 4, 1000, 4), (2, 0, 1000, 4), (2, 65, 1000, 4), (2, 4, 0, 4), (2, 4, 1000, 65), (2, 4, 1 << 30, 4),
                (1 << 24, 4, 1000, 4)]:
        assert qmm.beam_select_workspace_bytes(*bad) == 0, bad


def test_select_checks():
    f, x, s = qmm.beam_select, t((8, 100), bf16), t((2, 4), f32)
    raises(lambda: f(x, s.half()), "scores has dtype")
    raises(lambda: f(x, s.view(-1)), "scores must have 2")
    raises(lambda: f(x.int(), s), "logits has dtype")
    raises(lambda: f(x[:7], s), "7 rows for 2 sequences")
    raises(lambda: f(x.t().contiguous().t(), s), "consecutive")
    raises(lambda: f(x, s, 0), "1 to 64")
    raises(lambda: f(x, s, 65), "1 to 64")
    raises(lambda: f(t((130, 100), bf16), t((2, 65), f32)), "1 to 64")
    raises(lambda: f(x, s, 4, t((2, 4), u8)), "finished has dtype")
    raises(lambda: f(x, s, 4, t((4, 2), torch.bool)), "finished has shape")
    raises(lambda: f(x, s, 4, pad=100), "pad")
    raises(lambda: f(x, s, 4), "device tensors")


def reorder_args(**k):
    g = k.get
    return [g("cache", P), g("layers", 2), g("pages", 100), g("heads", 8), g("D", 128), g("page", 64), g("group", 64),
            g("table", P), g("width", 20), g("context", P), g("tails", P), g("parents", P), g("seqs", 2), g("beams", 4),
            g("to", P + 4096), g("co", P + 4096), None]


def test_reorder_errors():
    f, a = qmm.lib().kv4_beam_reorder, reorder_args
    assert f(*a(seqs=0, cache=None)) == OK
    for kw in [dict(cache=None), dict(table=None), dict(context=None), dict(tails=None), dict(parents=None), dict(to=None),
               dict(co=None), dict(layers=0), dict(width=0), dict(seqs=-1), dict(beams=0), dict(to=P), dict(co=P),
               dict(pages=0), dict(heads=0)]:
        assert f(*a(**kw)) == EINVAL, kw
    for kw in [dict(D=96), dict(page=48), dict(group=16)]:
        assert f(*a(**kw)) == EUNSUP, kw
    for kw in [dict(layers=70000), dict(width=1 << 31), dict(width=1 << 25), dict(seqs=1 << 22), dict(beams=1 << 40),
               dict(seqs=1 << 20, layers=32), dict(heads=5000)]:
        assert f(*a(**kw)) == ERANGE, kw
    for kw in [dict(cache=P + 8), dict(table=P + 2), dict(context=P + 1), dict(tails=P + 2), dict(parents=P + 4),
               dict(to=P + 2), dict(co=P + 2)]:
        assert f(*a(**kw)) == EALIGN, kw


def test_reorder_checks():
    cache, table, ctx = t((3, 9, 2, 64, 144), u8), t((8, 5), i32), t(8, i32)
    tails, parents, f = t((8, 2), i32), t((2, 4), i64), qmm.kv4_beam_reorder
    raises(lambda: f(cache[0, 0], 128, table, ctx, tails, parents), "4 dimensions")
    raises(lambda: f(cache[:0], 128, table, ctx, tails, parents), "no layers")
    raises(lambda: f(cache, 64, table, ctx, tails, parents), "token of head_dim")
    raises(lambda: f(cache, 128, table, ctx, tails, parents.int()), "parents has dtype")
    raises(lambda: f(cache, 128, table[:7], ctx, tails, parents), "page_table has shape")
    raises(lambda: f(cache, 128, table, ctx[:7], tails, parents), "context has shape")
    raises(lambda: f(cache, 128, table, ctx, tails.view(-1), parents), "tails has shape")
    raises(lambda: f(cache, 128, table, ctx, tails, parents, table_out=table), "other memory")
    raises(lambda: f(cache, 128, table, ctx, tails, parents, context_out=ctx), "other memory")
    raises(lambda: f(cache, 128, table, ctx, tails, parents, table_out=t((8, 4), i32)), "table_out has shape")
    raises(lambda: f(cache, 128, table, ctx, tails, parents), "device tensors")


# ---------------------------------------------------------------------------
# Attention over shared prefixes.
# ---------------------------------------------------------------------------
def prefix_args(**k):
    g = k.get
    return [g("q", P), g("qts", 4096), g("qhs", 128), g("dt", BF16), g("T", 4), g("hq", 32), g("cu", None), g("seqs", 4),
            g("max_q", 1), g("context", P), g("table", P), g("width", 20), g("stride", 20), g("groups", P), g("prefix", P),
            g("n", 2), g("mg", 3), g("mp", 1000), g("mt", 100), g("cache", P), g("pages", 100), g("hk", 8), g("D", 128),
            g("page", 64), g("group", 64), ctypes.c_float(g("scale", 0.1)), g("out", P), None, g("ws", P),
            g("wsb", 10 ** 12), None]


def test_prefix_attention_errors():
    f, a = qmm.lib().kv4_prefix_attention, prefix_args
    assert f(*a(T=0, q=None)) == OK
    for kw in [dict(q=None), dict(context=None), dict(table=None), dict(groups=None), dict(prefix=None), dict(cache=None),
               dict(out=None), dict(T=-1), dict(seqs=0), dict(T=5), dict(max_q=0), dict(n=0), dict(n=-1), dict(mg=0),
               dict(mp=0), dict(mt=-2), dict(width=0), dict(stride=19), dict(scale=float("nan")), dict(hq=33), dict(hq=0),
               dict(hk=0), dict(dt=8), dict(pages=0)]:
        assert f(*a(**kw)) == EINVAL, kw
    for kw in [dict(dt=F32), dict(D=96), dict(page=8), dict(group=16)]:
        assert f(*a(**kw)) == EUNSUP, kw
    for kw in [dict(T=1 << 31, cu=P), dict(seqs=70000, T=70000), dict(n=70000), dict(width=1 << 25, stride=1 << 25),
               dict(hq=80000, hk=8), dict(T=1 << 27, cu=P), dict(hk=4096, hq=4096, n=65535)]:
        assert f(*a(**kw)) == ERANGE, kw
    for kw in [dict(q=MIS), dict(out=MIS), dict(cache=P + 8), dict(qts=4100), dict(qhs=4), dict(table=P + 2),
               dict(context=P + 1), dict(cu=P + 2), dict(groups=P + 2), dict(prefix=P + 3), dict(ws=MIS)]:
        assert f(*a(**kw)) == EALIGN, kw
    need = qmm.kv4_prefix_attention_workspace_bytes(4, 4, 1, 2, 3, 1000, 100, 32, 8, 128, 64, 20 * 64)
    assert need >= 2 * 4 * 32 * (128 + 2) * 4 and need % (4 * 32 * 4) == 0
    assert f(*a(ws=None)) == EWS and f(*a(wsb=need - 1)) == EWS
    w = lambda **k: qmm.lib().kv4_prefix_attention_workspace_bytes(*[k.get(x, d) for x, d in dict(
        T=4, seqs=4, max_q=1, n=2, mg=3, mp=1000, mt=100, hq=32, hk=8, D=128, group=64, tokens=1280).items()])
    assert w() == need
    for kw in [dict(T=0), dict(seqs=0), dict(max_q=0), dict(n=0), dict(mg=0), dict(mp=0), dict(mt=0), dict(hq=33), dict(hk=0),
               dict(D=0), dict(group=0), dict(tokens=0), dict(tokens=1 << 31), dict(seqs=1 << 17), dict(n=1 << 17)]:
        assert w(**kw) == 0, kw


def test_prefix_attention_checks():
    q, cache, table, ctx = t((4, 8, 128), bf16), t((3, 2, 64, 144), u8), t((4, 5), i32), t(4, i32)
    groups, prefix, f = t(3, i32), t(2, i32), qmm.kv4_prefix_attention
    raises(lambda: f(q.float(), cache, table, ctx, groups, prefix), "q has dtype")
    raises(lambda: f(q[:, :7], cache, table, ctx, groups, prefix), "multiple")
    raises(lambda: f(q, cache, table.long(), ctx, groups, prefix), "page_table has dtype")
    raises(lambda: f(q, cache, table, ctx[:3], groups, prefix), "context has shape")
    raises(lambda: f(q, cache, table, ctx, groups[:2], prefix), "groups has shape")
    raises(lambda: f(q, cache, table, ctx, groups.long(), prefix), "groups has dtype")
    raises(lambda: f(q, cache, table, ctx, groups, prefix.long()), "prefix has dtype")
    raises(lambda: f(q, cache, table, ctx, groups[:1], prefix[:0]), "at least one group")
    raises(lambda: f(q[:3], cache, table, ctx, groups, prefix), "3 rows for 4")
    raises(lambda: f(q, cache, table, ctx, groups, prefix, cu_q=t(4, i32)), "cu_q has shape")
    raises(lambda: f(q, cache, table, ctx, groups, prefix, out=t((4, 8, 64), bf16)), "out has shape")
    raises(lambda: f(q, cache, table, ctx, groups, prefix), "device tensors")
