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
               dict(hq=80000, hk=8), dict(T=1 << 27, cu=P), dict(hk=4096, hq=4096, n=65535),
               dict(hk=200, hq=5000, n=65535, mg=4)]:        # (blocks of 512 threads)
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


# ---------------------------------------------------------------------------
# Which pages hold which beam's tokens.
# ---------------------------------------------------------------------------
class Store:
    """A cache of one integer a slot, moved as kv4_copy_pages and kv4_beam_reorder move theirs."""

    def __init__(self, pages, page):
        self.k, self.page, self.cells = qmm.KvPages(pages, page), page, torch.full((pages, page), -7)

    def prompt(self, n, g):
        s = self.k.add()
        slots, _, _ = self.k.extend([s], [n])
        tokens = torch.randint(0, 10 ** 6, (n,), generator=g)
        self.cells.view(-1)[slots] = tokens
        return s, tokens.tolist()

    def reorder(self, table, context, tails, parents):
        new, cells = table.clone(), self.cells.clone()
        for slot in range(len(table)):
            src = slot // parents.shape[1] * parents.shape[1] + int(parents.view(-1)[slot])
            new[slot] = table[src]
            column, filled = divmod(int(context[src]), self.page)
            if filled and src != slot:
                spare = tails[slot, 1] if table[slot, column] == tails[slot, 0] else tails[slot, 0]
                cells[spare, :filled] = self.cells[table[src, column], :filled]
                new[slot, column] = spare
        self.cells = cells
        return new

    def read(self, table, slot, n):
        j = torch.arange(n)
        return self.cells[table[slot, j // self.page].long(), j % self.page].tolist()


@pytest.mark.parametrize("page", [1, 4, 16])
@pytest.mark.parametrize("beams", [1, 2, 5])
def test_beams_hold_their_tokens(page, beams):
    g = torch.Generator().manual_seed(100 * page + beams)
    m = Store(600, page)
    prompts = [m.prompt(n, g) for n in (3 * page + 1, 2 * page, 7, 0)]
    free = m.k.free_pages
    b = qmm.KvBeams(m.k, [s for s, _ in prompts], beams, 40)
    assert b.groups.tolist() == list(range(0, 4 * beams + 1, beams)) and b.prefix.tolist() == [len(t) for _, t in prompts]
    m.cells[b.dst] = m.cells[b.src]
    table, context, tails = b.table, b.context, b.tails
    want = [list(t) for _, t in prompts for _ in range(beams)]
    for step in range(40):
        if step == 5:
            m.k.free(prompts[0][0])                          # the beams hold what they need
        if step == 7:
            slots, src, dst = m.k.extend([prompts[2][0]], [3])
            m.cells[dst] = m.cells[src]
            m.cells.view(-1)[slots] = -9                     # a prompt goes on by itself
        grown = b.room(table)
        assert (grown is not None) == bool((context % page == 0).any())
        if grown is not None:
            table, tails = grown
        at = torch.arange(len(table))
        slots = table[at, (context // page).long()].long() * page + context % page
        assert len(set(slots.tolist())) == len(slots)
        new = torch.randint(0, 10 ** 6, slots.shape, generator=g)
        m.cells.view(-1)[slots] = new
        want = [w + [int(x)] for w, x in zip(want, new)]
        context = context + 1
        parents = torch.randint(0, beams, (4, beams), generator=g)
        table = m.reorder(table, context, tails, parents)
        want = [want[i // beams * beams + int(parents.view(-1)[i])] for i in range(len(want))]
        want = [list(w) for w in want]
        for slot, w in enumerate(want):
            assert m.read(table, slot, len(w)) == w
    assert m.read(m.k.table([prompts[2][0]])[0], 0, 10) == prompts[2][1] + [-9] * 3
    with pytest.raises(ValueError, match="no room"):
        b.room(table)
    with pytest.raises(ValueError, match="cannot be moved"):
        m.k.compact()
    kept = [(b.keep(table, slot), want[slot]) for slot in (0, len(table) - 1)]
    b.free()
    for seq, w in kept:
        row, n = m.k.table([seq])
        assert m.read(row, 0, int(n)) == w
        m.k.free(seq)
    for s, _ in prompts[1:]:
        m.k.free(s)
    assert m.k.free_pages == 600
    m.k.compact()
    for f in (lambda: b.room(table), lambda: b.keep(table, 0), b.free):
        raises(f, "were freed")


@pytest.mark.parametrize("page,beams", [(4, 2), (4, 3), (16, 3), (16, 1)])
@pytest.mark.parametrize("before", [False, True], ids=["moved", "before the move"])
def test_a_beam_that_is_kept_stays_as_it_was(page, beams, before):
    """Set aside in the middle of a page, while the search goes on and moves its slots; then read on by itself."""
    g = torch.Generator().manual_seed(page + beams)
    m = Store(900, page)
    prompts = [m.prompt(n, g) for n in (page + 1, 2 * page, 7)]
    b = qmm.KvBeams(m.k, [s for s, _ in prompts], beams, 8 * page)
    m.cells[b.dst] = m.cells[b.src]
    table, context, tails = b.table, b.context, b.tails
    want, kept = [list(t) for _, t in prompts for _ in range(beams)], []
    for step in range(8 * page):
        grown = b.room(table)
        assert grown is None or step % 3 == 1 or bool((context % page == 0).any())
        if grown is not None:
            table, tails = grown
        at = torch.arange(len(table))
        new = torch.randint(0, 10 ** 6, (len(table),), generator=g)
        m.cells[table[at, (context // page).long()].long(), (context % page).long()] = new
        want = [w + [int(x)] for w, x in zip(want, new)]
        context = context + 1
        slot = int(torch.randint(0, len(table), (), generator=g))
        if before and step % 3 == 0:
            kept.append((b.keep(table, slot), list(want[slot])))
        parents = torch.randint(0, beams, (3, beams), generator=g)
        table = m.reorder(table, context, tails, parents)
        want = [list(want[i // beams * beams + int(parents.view(-1)[i])]) for i in range(len(want))]
        if not before and step % 3 == 0:
            kept += [(b.keep(table, s), list(want[s])) for s in {slot, 0}]
        if step % 5 == 0 and kept:                           # one of them goes on by itself
            seq, w = kept.pop(int(torch.randint(0, len(kept), (), generator=g)))
            slots, src, dst = m.k.extend([seq], [2])
            m.cells[dst] = m.cells[src]
            m.cells.view(-1)[slots] = torch.tensor([-8, -9])
            kept.append((seq, w + [-8, -9]))
        if step % 11 == 0 and kept:
            m.k.free(kept.pop(0)[0])
        for seq, w in kept:
            row, n = m.k.table([seq])
            assert int(n) == len(w) and m.read(row, 0, len(w)) == w
        for s, w in enumerate(want):
            assert m.read(table, s, len(w)) == w
        used = set(tails.flatten().tolist()) - {-1}
        assert not used & set(m.k._free)
    b.free()
    for seq, w in kept:
        row, n = m.k.table([seq])
        assert m.read(row, 0, len(w)) == w
        m.k.free(seq)
    for s, _ in prompts:
        m.k.free(s)
    assert m.k.free_pages == 900


def test_a_kept_beam_takes_a_page_only_where_the_search_goes_on():
    m = Store(12, 4)
    s, _ = m.prompt(6, torch.Generator().manual_seed(0))
    b = qmm.KvBeams(m.k, [s], 2, 20)
    assert m.k.free_pages == 6
    assert b.room(b.table) is None                           # token 6: the page is not full
    kept = [b.keep(b.table, 0), b.keep(b.table, 1), b.keep(b.table, 0)]
    assert m.k.free_pages == 6
    held = [m.k.table([k])[0][0, 1].item() for k in kept]
    assert held[0] == held[2] and set(held) <= set(b.tails.flatten().tolist())
    old = b.tails
    table, tails = b.room(b.table)
    assert m.k.free_pages == 4 and torch.equal(table, b.table) and not set(held) & set(tails.flatten().tolist())
    assert torch.equal(old[:, 1], tails[:, 1]) and len(set(tails.flatten().tolist())) == 4
    b.free()
    assert m.k.free_pages == 12 - 2 - 2                      # the prompt's two and the kept ones' last
    for k in kept + [s]:
        m.k.free(k)
    assert m.k.free_pages == 12


@pytest.mark.parametrize("pages", range(6, 10))
def test_kept_pages_are_not_counted_as_free(pages):
    """A full page whose beam is gone stays in use while a sequence holds it: too few pages are found before anything has
    changed, and enough are enough."""
    m = Store(pages, 4)
    s, _ = m.prompt(6, torch.Generator().manual_seed(0))
    b = qmm.KvBeams(m.k, [s], 2, 20)
    table, context, tails = b.table, b.context, b.tails
    for _ in range(2):
        assert b.room(table) is None
        context = context + 1
    kept = [b.keep(table, slot) for slot in (0, 1)]          # with the page that is full now
    other = m.k.add()
    table = m.reorder(table, context, tails, torch.zeros((1, 2), dtype=i64))     # slot 1's page is in no row any more

    def state():
        return (list(m.k._free), list(m.k._users), {k: list(v) for k, v in m.k._held.items()}, [set(x) for x in b._own],
                b.tails.tolist(), list(b._length), list(b._tokens))

    # in use: the prompt's two, two tails a slot; the spare ones are given back, the kept ones are not
    enough = pages - 6 + 2 >= 4
    was = state()
    if enough:
        table, tails = b.room(table)
        assert len(set(tails.flatten().tolist())) == 4 and m.k.free_pages == pages - 8
    else:
        with pytest.raises(RuntimeError, match=f"4 needed, {pages - 4} of {pages} free"):
            b.room(table)
        assert state() == was
        m.k.free(kept[1])
        m.k.free(other)
        if pages - 6 + 3 >= 4:
            b.room(table)


def test_beams_need_few_pages():
    """The pages in use never exceed the prompt's, those that the beams' histories can hold and two a slot."""
    m = Store(200, 4)
    s, _ = m.prompt(20, torch.Generator().manual_seed(0))
    b = qmm.KvBeams(m.k, [s], 3, 100)
    table, context, tails = b.table, b.context, b.tails
    for step in range(100):
        grown = b.room(table)
        if grown is not None:
            table, tails = grown
        context = context + 1
        table = m.reorder(table, context, tails, torch.zeros((1, 3), dtype=i64))      # all go on from the first
        assert 200 - m.k.free_pages <= 5 + step // 4 + 3 + 6
    b.free()


def test_beams_refusals():
    m = Store(20, 4)
    s, _ = m.prompt(10, torch.Generator().manual_seed(0))
    for f, match in [(lambda: qmm.KvBeams(m.k, [], 2, 5), "needs sequences"), (lambda: qmm.KvBeams(m.k, [s], 0, 5), "needs sequences"),
                     (lambda: qmm.KvBeams(m.k, [s], 2, -1), "needs sequences"), (lambda: qmm.KvBeams(m.k, [s, s], 2, 5), "twice"),
                     (lambda: qmm.KvBeams(m.k, [s + 1], 2, 5), "no sequence")]:
        raises(f, match)
    with pytest.raises(RuntimeError, match="18 needed, 17 of 20 free"):
        qmm.KvBeams(m.k, [s], 9, 5)
    assert m.k.free_pages == 17
    b = qmm.KvBeams(m.k, [s], 5, 20)
    assert m.k.free_pages == 7
    raises(lambda: b.room(b.table[:4]), "shape")
    raises(lambda: b.keep(b.table, 5), "no slot")
    strange = b.table.clone()
    strange[0, 0] = 19
    raises(lambda: b.keep(strange, 0), "does not hold")
    assert b.room(b.table) is None and b.room(b.table) is None         # tokens 10 and 11
    raises(lambda: b.room(strange), "does not hold")
    with pytest.raises(RuntimeError, match="out of pages: 10 needed"):
        other = m.k.add()
        m.k.extend([other], [20])
        b.room(b.table)
    m.k.free(other)
    table, tails = b.room(b.table)
    assert sorted(tails.flatten().tolist()) == sorted(set(tails.flatten().tolist())) and (table[:, 3] == tails[:, 0]).all()
    w = m.k.add()
    m.k.extend([w], [8])
    m.k.forget(w, 1)
    m.k.shrink(w, 8)
    with pytest.raises(ValueError):
        qmm.KvBeams(m.k, [w, 99], 1, 1)


def test_runs_of_sequences_that_share_pages():
    k = qmm.KvPages(50, 4)
    a = k.add()
    k.extend([a], [13])
    forks = [k.fork(a) for _ in range(3)]
    k.extend([forks[0]], [5])
    b, empty = k.add(), k.add()
    k.extend([b], [9])
    c = k.fork(b)
    groups, prefix = k.shared([a, *forks, b, empty, c, b])
    assert groups.tolist() == [0, 4, 5, 6, 8] and prefix.tolist() == [12, 9, 0, 9]
    assert groups.dtype == prefix.dtype == i32
    k.shrink(forks[1], 6)                                    # in the middle of the second page
    assert k.shared([a, forks[1], forks[0]])[1].tolist() == [7]
    assert k.shared([a, a])[1].tolist() == [13]
    assert [t.tolist() for t in k.shared([])] == [[0], []]
    raises(lambda: k.shared([99]), "no sequence")


def test_runs_are_cut_where_parts_of_them_share_more():
    """Two prompts that fork from a page of the same text, with samples of each; and others, against all ways to cut."""
    k = qmm.KvPages(600, 4)
    text = k.add()
    k.extend([text], [4])
    samples = []
    for n in (80, 121):
        prompt = k.fork(text)
        k.extend([prompt], [n])
        samples += [k.fork(prompt) for _ in range(5)]
    groups, prefix = k.shared(samples)
    assert groups.tolist() == [0, 5, 10] and prefix.tolist() == [84, 125]
    assert [x.tolist() for x in k.shared([text] + samples)] == [[0, 1, 6, 11], [4, 84, 125]]
    k.extend(samples, range(1, 11))
    assert [x.tolist() for x in k.shared(samples)] == [[0, 5, 10], [84, 124]]
    assert [x.tolist() for x in k.shared(samples[4:6])] == [[0, 2], [4]]

    g = torch.Generator().manual_seed(0)
    draw = lambda n: int(torch.randint(0, n, (), generator=g))
    for _ in range(60):
        k, seqs = qmm.KvPages(900, 4), []
        for _ in range(9):                                   # a random family: roots, forks of any, shortened or extended
            s = k.fork(seqs[draw(len(seqs))]) if seqs and draw(4) else k.add()
            if k.length(s) and draw(2):
                k.shrink(s, draw(k.length(s) + 1))
            k.extend([s], [draw(30)])
            seqs.append(s)
        seqs = [seqs[draw(9)] for _ in range(8)]
        held = [k._held[s] for s in seqs]

        def common(i, j):
            pages = 0
            while all(pages < len(h) and h[pages] == held[i][pages] for h in held[i:j]):
                pages += 1
            return min([pages * 4] + [k.length(s) for s in seqs[i:j]])

        groups, prefix = (x.tolist() for x in k.shared(seqs))
        assert groups[0] == 0 and groups[-1] == 8 and all(a < b for a, b in zip(groups, groups[1:]))
        assert prefix == [common(a, b) for a, b in zip(groups, groups[1:])]
        got = sum((b - a - 1) * n for a, b, n in zip(groups, groups[1:], prefix))
        every = []
        for cuts in range(128):
            at = [0] + [c for c in range(1, 8) if cuts >> (c - 1) & 1] + [8]
            every.append(sum((b - a - 1) * common(a, b) for a, b in zip(at, at[1:])))
        assert got == max(every)
