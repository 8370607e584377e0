"""Attention of groups of sequences that share a prefix, against fp64 of each
sequence by itself.

Bounds: kv4_bounds.py's, of one pass over a row's keys.  Here a row has up to
60 parts, each within that (its statistics are relative to its own largest),
joined in fp32: a factor (2 u), a product and a sum a part, (60 + 4) u of the
mass and of the sum of probabilities.  The kernel for prefixes of many rows
rounds each value to binary16, (c - z) / 16 times its scale: 2^-11 of it, so
twice the rounding of the probabilities, or half a step of 2^-24 below 2^-14,
2^-21 of the value."""
import math

import numpy as np
import pytest
import torch

import kv4_bounds as bounds
import kv4_reference as ref
import quantized_matmul_quantize_amd as qmm
from gpu_util import OUT_HALF_ULP, note

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16
FORMATS = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)]
U = 2.0 ** -24


def half(x, dtype):
    return torch.from_numpy(np.asarray(x, np.float32)).to(dtype)


class Groups:
    """plan: per group (tokens of the prefix, tokens of each sequence behind it).  A number of tokens below 0 is a sequence
    that holds only so many less than the prefix; None an unused slot.  The page in which a prefix ends is a copy of each
    sequence's own; the cache's other bytes are all ones.  before, after: sequences in no group."""

    def __init__(self, seed, dtype, D, group, page, hq, hkv, plan, queries=None, before=(), after=(), edit=None):
        g = np.random.Generator(np.random.PCG64(seed))
        self.dtype, self.D, self.hq, self.hkv = dtype, D, hq, hkv
        plan_all = [(0, [n]) for n in before] + list(plan) + [(0, [n]) for n in after]
        rows, self.lens, k_of, v_of, free = [], [], [], [], 0
        draw = lambda n: [half(g.standard_normal((n, hkv, D)) * np.exp(0.5 * g.standard_normal((hkv, D))), dtype),
                          half(g.standard_normal((n, hkv, D)), dtype)]
        for p, tails in plan_all:
            k0, v0 = draw(p)
            whole = p // page
            shared = list(range(free, free + whole))
            free += whole
            for t in tails:
                n = 0 if t is None else p + t
                mine = max(0, -(-n // page) - whole)
                rows.append((shared + list(range(free, free + mine)))[:-(-n // page)])
                free += mine
                kt, vt = draw(max(0, t or 0))
                k_of.append(torch.cat((k0, kt))[:n])
                v_of.append(torch.cat((v0, vt))[:n])
                self.lens.append(n)
        if edit:
            edit(k_of, v_of)
        order = g.permutation(free + 1)
        self.cache = qmm.kv4_cache(free + 1, hkv, D, page, group).fill_(255)
        table = np.full((len(rows), max(1, max(len(r) for r in rows)) + 1), -1, np.int32)
        self.k, self.v, self.sk, self.sv = [], [], [], []
        for b, r in enumerate(rows):
            table[b, :len(r)] = order[r]
            k, v, j = k_of[b], v_of[b], np.arange(self.lens[b])
            if len(j):
                slots = table[b, j // page].astype(np.int64) * page + j % page
                qmm.kv4_append(k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), self.cache)
            for x, val, sc in ((k, self.k, self.sk), (v, self.v, self.sv)):
                c, z, s = ref.quantize(x.float().numpy(), group)
                val.append(ref.values(c, z, s))
                sc.append(s.astype(np.float64))
        self.queries = [1] * len(rows) if queries is None else list(queries)
        i32 = lambda x: torch.from_numpy(np.asarray(x, np.int32)).cuda()
        self.table, self.context = i32(table), i32(self.lens)
        self.groups = i32(np.cumsum([len(before)] + [len(t) for _, t in plan]))
        self.prefix = i32([p for p, _ in plan])
        self.starts = np.concatenate([[0], np.cumsum(self.queries)]).astype(np.int32)
        self.q = half(g.standard_normal((int(self.starts[-1]), hq, D)), dtype)
        most, at = 0, len(before)
        for _, t in plan:
            most = max(most, sum(self.queries[at:at + len(t)]))
            at += len(t)
        # more rows than the kernel for few takes: values (of a sequence's own keys, bf16 probabilities) rounded as well
        self.many = most * (hq // hkv) > 96
        self.roundings = 2 if self.many or dtype == BF16 and max(self.queries) * (hq // hkv) > 96 else 1
        self.hints = dict(max_group=max(len(t) for _, t in plan), max_prefix=max(1, max(p for p, _ in plan)),
                          max_tail=max([1] + self.lens[:len(before)] + [x or 1 for _, t in plan for x in t]))

    def run(self, q=None, **kw):
        if max(self.queries) != 1 or min(self.queries) != 1:
            kw.setdefault("cu_q", torch.from_numpy(self.starts).cuda())
            kw.setdefault("max_q", max(self.queries))
        kw = {**self.hints, **kw}
        return qmm.kv4_prefix_attention((self.q if q is None else q).cuda(), self.cache, kw.pop("table", self.table),
                                        self.context, kw.pop("groups", self.groups), kw.pop("prefix", self.prefix),
                                        return_lse=True, **kw)

    def check(self, got, scale=None, q=None, rows=None):
        out, lse = got
        q = (self.q if q is None else q).float().numpy()
        T, hq, D = q.shape
        o, l, b_out, b_lse, count = bounds.attention(q, self.k, self.v, self.sk, self.sv, self.lens, self.queries,
                                                     D ** -0.5 if scale is None else scale, roundings=self.roundings)
        rows = np.ones((T, hq), bool) if rows is None else rows
        none = np.repeat((count == 0)[:, None], hq, 1)
        assert (out.cpu().float()[torch.from_numpy(none & rows)] == 0).all()
        mass = np.abs(np.concatenate([v.reshape(-1) for v in self.v])).max()
        bound = b_out + 64 * U * mass + self.many * 2.0 ** -21 + OUT_HALF_ULP[self.dtype] * np.abs(o) + (2.0 ** -25 if self.dtype == F16 else 0.0)
        err = np.abs(out.float().cpu().numpy() - o)
        bad = ~(err <= bound) & (rows & ~none)[..., None]
        assert not bad.any(), f"out: {bad.sum()} past their bounds, at {np.argwhere(bad)[:3]}"
        got_l = lse.cpu().numpy().astype(np.float64)
        assert np.isneginf(got_l[none & rows]).all()
        bad = ~(np.abs(got_l - l) <= b_lse + 64 * U) & rows & ~none
        assert not bad.any(), f"lse: {bad.sum()} past their bounds, at {np.argwhere(bad)[:3]}"


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("D,group", FORMATS)
@pytest.mark.parametrize("page", [16, 64])
def test_formats(dtype, D, group, page):
    note(f"kv4_prefix_attention D={D} group={group} page={page} {dtype}")
    b = Groups(D + group + page, dtype, D, group, page, 4, 2, [(70, [1, 30, 65]), (0, [40]), (128, []), (131, [5, 1, 17, None]),
                                                              (31, [9, 9])], before=[33], after=[1, 50])
    b.check(b.run())


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (5, 5), (16, 1), (14, 2), (40, 2), (32, 8)])
@pytest.mark.parametrize("page", [16, 32, 128, 256])
def test_heads(hq, hkv, page):
    note(f"kv4_prefix_attention heads {hq}/{hkv} page={page}")
    b = Groups(hq * 10 + page, BF16, 128, 64, page, hq, hkv, [(300, [1, 200, 7]), (64, [10])])
    b.check(b.run())


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("D,group", FORMATS)
def test_groups_of_many_rows(dtype, D, group):
    """Past 96 rows a prefix goes to the kernel for chunks; several chunks of its keys."""
    note(f"kv4_prefix_attention, many rows, D={D} group={group} {dtype}")
    b = Groups(D - group, dtype, D, group, 32, 4, 1, [(1000, [1 + 3 * i for i in range(37)]), (333, [20] * 2), (95, [1] * 26)])
    b.check(b.run())


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("D,group", [(64, 32), (128, 64), (128, 128), (256, 32)])
@pytest.mark.parametrize("many", [False, True], ids=["few", "many"])
def test_several_queries_of_a_sequence(dtype, D, group, many):
    """Drafts to verify, and questions on a document; sequences without queries, and with so many that the first of them
    stand inside the prefix."""
    note(f"kv4_prefix_attention, several queries, D={D} group={group} many={many} {dtype}")
    plan = [(200, [3, 40, 12, 5, None]), (97, [60, 1])]
    b = Groups(D + group, dtype, D, group, 32, 6, 2, plan, queries=[3, 5, 0, 9, 0, 60 if many else 4, 2])
    b.check(b.run())


def test_sequences_shorter_than_their_prefix_are_attended_to_by_themselves():
    """Among them the group's first, so that the prefix is read through another's pages; and a group of such ones alone."""
    b = Groups(5, BF16, 128, 64, 16, 8, 2, [(160, [None, -50, 20, -1, -160, 3]), (80, [-40, -80, None]), (40, [None]), (64, [2, -32])])
    b.check(b.run())


@pytest.mark.parametrize("hints", [dict(max_group=1, max_prefix=1, max_tail=1), dict(max_group=65, max_prefix=10 ** 9, max_tail=10 ** 9),
                                   dict(max_group=None, max_prefix=None, max_tail=None), dict(max_group=30, max_prefix=3000, max_tail=1)])
def test_hints_change_no_result(hints):
    b = Groups(6, F16, 64, 32, 32, 4, 2, [(700, [40] * 5), (64, [300, 2]), (1000, [1] * 30)])
    b.check(b.run(**hints))


def test_prefixes_beyond_what_is_held_and_groups_that_overrun():
    """A prefix longer than the table or negative shares nothing; bounds of groups past the batch are held to it."""
    b = Groups(7, BF16, 64, 64, 16, 4, 4, [(48, [5, 6]), (48, [7, 8, 9]), (32, [10])])
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    b.check(b.run(prefix=i32(10 ** 9, -5, 32)))
    b.check(b.run(prefix=i32(48, 2 ** 31 - 1, -2 ** 31)))
    b.check(b.run(groups=i32(0, 2, 5, 1000)))
    b.check(b.run(groups=i32(-3, 2, 5, 6)))
    b.check(b.run(groups=i32(6, 6, 6, 6)))


def test_more_groups_than_lanes_and_a_group_of_more_sequences():
    b = Groups(8, F16, 64, 64, 16, 2, 1, [(32 + i % 40, [1 + i % 5] * (i % 3)) for i in range(150)] + [(70, [None] * 70 + [3] * 60)])
    b.check(b.run())


@pytest.mark.parametrize("many", [False, True], ids=["few", "many"])
def test_a_query_that_is_not_finite_stays_in_its_row(many):
    for dtype in (BF16, F16):
        b = Groups(9, dtype, 128, 64, 32, 4, 1, [(256, [5] * (40 if many else 4)), (64, [9])])
        q = b.q.clone()
        q[1, 2, 7], q[2, 0, 100], q[3, 1, 3] = math.inf, math.nan, -math.inf
        rows = np.ones(q.shape[:2], bool)
        rows[1, 2] = rows[2, 0] = rows[3, 1] = False
        out, lse = b.run(q=q)
        b.check((out, lse), q=torch.where(q.isfinite(), q, 0), rows=rows)
        assert out[2, 0].isnan().all() and lse[2, 0].isnan()


def test_values_of_very_different_sizes():
    """Scales of the prefix far above and far below those of the sequences' own tokens."""
    for rise in (2.0 ** 8, 2.0 ** -8):
        def edit(ks, vs):
            for v in vs:
                v[:64] *= rise
        b = Groups(10, F16, 128, 64, 32, 8, 2, [(64, [30, 40, 1])], edit=edit)
        b.check(b.run())


def test_table_rows_apart_strided_queries_given_outputs_and_scale():
    b = Groups(11, BF16, 128, 128, 64, 6, 2, [(200, [3, 70]), (64, [1, 1, 5])])
    T = b.q.shape[0]
    wide = torch.full((T, 10, 128), math.nan, dtype=BF16, device="cuda")
    wide[:, 2:8] = b.q.cuda()
    table = torch.full((b.table.shape[0], b.table.shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    table[:, 1:1 + b.table.shape[1]] = b.table
    out = torch.empty((T, 6, 128), dtype=BF16, device="cuda")
    need = qmm.kv4_prefix_attention_workspace_bytes(T, 5, 1, 2, 3, 200, 70, 6, 2, 128, 128, b.table.shape[1] * 64)
    work = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    got = qmm.kv4_prefix_attention(wide[:, 2:8], b.cache, table[:, 1:1 + b.table.shape[1]], b.context, b.groups, b.prefix,
                                   max_group=3, max_prefix=200, max_tail=70, scale=0.3, return_lse=True, out=out, workspace=work)
    assert got[0] is out
    b.check(got, scale=0.3)


def test_rows_of_no_sequence_are_left_as_they_were():
    b = Groups(12, F16, 64, 32, 16, 4, 2, [(64, [3, 7]), (32, [1])], queries=[2, 1, 1])
    q = torch.cat((b.q, b.q[:3]))
    out = torch.full((7, 4, 64), 7.0, dtype=F16, device="cuda")
    got = qmm.kv4_prefix_attention(q.cuda(), b.cache, b.table, b.context, b.groups, b.prefix,
                                   cu_q=torch.from_numpy(b.starts).cuda(), max_q=2, return_lse=True, out=out)
    b.check((got[0][:4], got[1][:4]))
    assert (out[4:] == 7.0).all()


def test_long_prefix_of_high_pages():
    """A prefix of 20000 tokens in the last pages of a cache past 2^32 bytes: against kv4_attention, whose results differ by
    roundings alone (twice the bound of each)."""
    D, hkv, hq, page, group, pages, P, S = 128, 8, 16, 64, 64, 60000, 20000, 5
    cache = qmm.kv4_cache(pages, hkv, D, page, group)
    assert cache.numel() > 2 ** 32
    gen = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda").to(BF16)
    own = 100
    whole = P // page
    shared = torch.arange(pages - whole, pages, device="cuda")
    mine = torch.arange(pages - whole - 3 * S, pages - whole, device="cuda").view(S, 3)
    table = torch.cat((shared.expand(S, -1), mine), 1).int()
    j = torch.arange(P + own, device="cuda")
    for s in range(S):
        start = 0 if s == 0 else whole * page
        slots = table[s].long()[j[start:] // page] * page + j[start:] % page
        if s == 0:
            k, v = rand(P + own, hkv, D), rand(P + own, hkv, D)
        else:
            k[P:], v[P:] = rand(own, hkv, D), rand(own, hkv, D)
        qmm.kv4_append(k[start:], v[start:], slots, cache)
    q = rand(S, hq, D) * 2
    context = torch.full((S,), P + own, dtype=torch.int32, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    got = qmm.kv4_prefix_attention(q, cache, table, context, i32(0, S), i32(P), return_lse=True)
    want = qmm.kv4_attention(q, cache, table, context, return_lse=True)
    # each is within 2^-11 mass and an output rounding of fp64 (mass <= 1: values of variance 1 under weights that sum to 1)
    assert (got[0].float() - want[0].float()).abs().max() <= 2 * (2.0 ** -11 + 2.0 ** -12) + 2 * 2.0 ** -8 * want[0].float().abs().max()
    assert (got[1] - want[1]).abs().max() <= 2e-5


def test_no_queries_another_stream_and_a_replayed_graph():
    b = Groups(13, BF16, 64, 64, 16, 4, 2, [(100, [5, 6, 7]), (40, [50, 1])])
    none = qmm.kv4_prefix_attention(b.q[:0].cuda(), b.cache, b.table[:0], b.context[:0], torch.zeros(2, dtype=torch.int32, device="cuda"),
                                    b.prefix[:1])
    assert none.shape == (0, 4, 64)
    want = b.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q = b.q.cuda()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = b.run(q=q)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = b.run(q=q)
    for turn in range(3):
        q.copy_(torch.roll(q, 1, 0))
        b.context[turn] -= 1                                # lengths change between replays
        b.lens[turn] -= 1
        b.k[turn], b.v[turn] = b.k[turn][:-1], b.v[turn][:-1]
        b.sk[turn], b.sv[turn] = b.sk[turn][:-1], b.sv[turn][:-1]
        graph.replay()
        want = b.run(q=q)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        b.check(got, q=q.cpu())


def long_table(b):
    """A table and a hint by which prefixes could be long: the kernel for many rows is chosen by what they allow."""
    return dict(table=torch.nn.functional.pad(b.table, (0, 200000 // (b.cache.shape[2])), value=-1), max_prefix=10 ** 9)


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("D,group", FORMATS)
def test_many_rows_of_prefixes_that_may_be_long(dtype, D, group):
    """Chunks of few rounds, one round and half a round, of one row tile and of several."""
    note(f"kv4_prefix_attention, many rows of long prefixes, D={D} group={group} {dtype}")
    b = Groups(D - group, dtype, D, group, 32, 4, 1, [(1000, [1 + 3 * i for i in range(37)]), (333, [20] * 2), (95, [1] * 26),
                                                      (170, [2] * 90), (0, [5]), (40, [])], after=[9])
    b.check(b.run(**long_table(b)))


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("D,group", FORMATS)
@pytest.mark.parametrize("page", [16, 256])
def test_many_rows_of_long_chunks(dtype, D, group, page):
    """So many groups, all but one empty, that a prefix is one chunk: its pages are read in several batches."""
    note(f"kv4_prefix_attention, long chunks, D={D} group={group} page={page} {dtype}")
    b = Groups(D + group, dtype, D, group, page, 4, 1, [(2700, [3] * 25)] + [(16, [])] * 300)
    b.check(b.run())


@pytest.mark.parametrize("D,group", [(64, 32), (128, 64), (128, 128), (256, 32)])
def test_several_queries_of_a_sequence_after_a_prefix_that_may_be_long(D, group):
    note(f"kv4_prefix_attention, several queries, long, D={D} group={group}")
    plan = [(200, [3, 40, 12, 5, None]), (97, [60, 1])]
    b = Groups(D + group, F16, D, group, 32, 6, 2, plan, queries=[3, 5, 0, 9, 0, 60, 2])
    b.check(b.run(**long_table(b)))


def test_a_query_that_is_not_finite_among_many():
    for dtype in (BF16, F16):
        b = Groups(9, dtype, 128, 64, 32, 4, 1, [(256, [5] * 40), (64, [9])])
        q = b.q.clone()
        q[1, 2, 7], q[2, 0, 100], q[3, 1, 3] = math.inf, math.nan, -math.inf
        rows = np.ones(q.shape[:2], bool)
        rows[1, 2] = rows[2, 0] = rows[3, 1] = False
        out, lse = b.run(q=q, **long_table(b))
        b.check((out, lse), q=torch.where(q.isfinite(), q, 0), rows=rows)
        assert out[2, 0].isnan().all() and lse[2, 0].isnan()


@pytest.mark.parametrize("D,group", [(64, 64), (128, 64), (256, 128)])
@pytest.mark.parametrize("many", [False, True], ids=["few", "many"])
def test_pages_that_the_table_does_not_name(D, group, many):
    """Keys of a page outside of the cache are left out, in the prefix for the whole group."""
    b = Groups(14, F16, D, group, 32, 4, 1, [(400, [7] * (40 if many else 3)), (64, [9])])
    members = 40 if many else 3
    kept = np.ones(407, bool)
    for column, name in ((0, -1), (5, b.cache.shape[0]), (6, 2 ** 31 - 1), (11, -2 ** 31)):
        b.table[:members, column] = name
        kept[32 * column:32 * column + 32] = False
    for s in range(members):
        b.k[s], b.v[s], b.sk[s], b.sv[s] = (x[s][kept] for x in (b.k, b.v, b.sk, b.sv))
        b.lens[s] = int(kept.sum())
    b.check(b.run(**(long_table(b) if many else {})))


@pytest.mark.parametrize("D,group", [(64, 32), (128, 64), (256, 64)])
def test_rows_enough_for_a_wavefront_each(D, group):
    """In the join: heads that do not fill its blocks, sequences without and with a prefix, of one chunk and of several."""
    b = Groups(15, BF16, D, group, 16, 15, 5, [(100, [3] * 40), (64, [400, 1]), (600, [2] * 60), (48, [None, -5])] + [(16, [1])] * 70, before=[1, 300])
    assert b.q.shape[0] * 15 >= 8 * torch.cuda.get_device_properties(0).multi_processor_count
    b.check(b.run())


def test_more_rows_of_a_prefix_than_products_of_their_tiles_hold():
    """8.4 million rows of one kv head: against kv4_attention, whose results differ by roundings alone (twice the bound of
    each)."""
    D, hkv, hq, page, group, P, S = 64, 1, 128, 16, 32, 64, 65535
    gen = torch.Generator(device="cuda").manual_seed(7)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda").to(BF16)
    cache = qmm.kv4_cache(P // page + S, hkv, D, page, group).zero_()
    i32 = lambda x: torch.as_tensor(x, dtype=torch.int32, device="cuda")
    table = torch.empty((S, P // page + 1), dtype=torch.int32, device="cuda")
    table[:, :-1] = torch.arange(P // page)
    table[:, -1] = torch.arange(P // page, P // page + S)
    v = rand(P + S, hkv, D)
    slots = torch.cat((torch.arange(P), (P // page + torch.arange(S)) * page)).cuda()
    qmm.kv4_append(rand(P + S, hkv, D), v, slots, cache)
    q = rand(S, hq, D)
    context = i32([P + 1]).expand(S).contiguous()
    got = qmm.kv4_prefix_attention(q, cache, table, context, i32([0, S]), i32([P]), max_group=S, max_prefix=P, max_tail=1)
    want = qmm.kv4_attention(q, cache, table, context).float()
    # of fp64 each is within 2^-11 of the mass a rounding (two each), 2^-21, 64 roundings of the join, 2 dx and an output
    # rounding; dx = 16 u 31 S sk |scale| with S <= 64 |q| and sk a fifteenth of a key's range, at most 12
    mass, most_q = float(v.float().abs().max()), float(q.float().abs().max())
    dx = 16 * U * 31 * 64 * most_q * 12 / 15 * D ** -0.5
    bound = (4 * 2.0 ** -11 + 128 * U + 4 * dx) * mass + 2.0 ** -21
    for at in range(0, S, 8192):
        part = want[at:at + 8192]
        assert ((got[at:at + 8192].float() - part).abs() <= bound + 2 * OUT_HALF_ULP[BF16] * (part.abs() + bound)).all()


@pytest.mark.parametrize("scale", [1e9, 1e20, -1e30])
@pytest.mark.parametrize("kind", ["few", "many", "long", "chunks"])
@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("D,group", [(64, 64), (128, 64), (128, 128), (256, 32)])
def test_scores_past_the_range_in_which_ones_differ(scale, kind, dtype, D, group):
    """Where scores are known no better than to 16 and more the largest has the weight: results are finite, mean values of
    the keys', and their log-sum-exp is a score."""
    note(f"kv4_prefix_attention scale={scale} {kind} D={D} group={group} {dtype}")
    queries = [1 + 40 * (i % 3) for i in range(12)] if kind == "chunks" else None
    b = Groups(18, dtype, D, group, 32, 4, 1, [(320, [90 + i for i in range(10 if queries else 5 if kind == "few" else 40)]), (64, [70, 99])],
               queries=queries)
    out, lse = b.run(scale=scale, **(long_table(b) if kind == "long" else {}))
    _, l, _, b_lse, _ = bounds.attention(b.q.float().numpy(), b.k, b.v, b.sk, b.sv, b.lens, b.queries, scale)
    assert (np.abs(lse.cpu().numpy() - l) <= b_lse).all()
    row = 0
    for n, ctx, v in zip(b.queries, b.lens, b.v):
        got = out[row:row + n].double().cpu().numpy()
        most = np.abs(v[:, 0]).max()
        # (a probability of 2^7 .. 2^15, its product with a scale and sums of codes with 64 added, as in kv4_bounds.py)
        slack = (b.roundings * 2.0 ** -11 + 2 * OUT_HALF_ULP[dtype]) * most + (ctx / 16 + 96) * U * 158 * most + 2.0 ** -20
        assert (got <= v[:, 0].max(0) + slack).all() and (got >= v[:, 0].min(0) - slack).all()
        row += n


@pytest.mark.parametrize("kind", ["few", "many", "long"])
@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("D,group", [(64, 64), (128, 64), (256, 32)])
def test_queries_of_very_different_sizes_keep_to_their_rows(kind, dtype, D, group):
    """Unused slots, sequences shorter than the prefix and sequences that share it, whose queries are far larger or smaller
    than the others': whatever they are, the others have their bounds."""
    note(f"kv4_prefix_attention, queries of other sizes, {kind} D={D} group={group} {dtype}")
    own = [3, 9, None, 20, -40, 1, 6] * (6 if kind != "few" else 1)
    b = Groups(16, dtype, D, group, 32, 4, 1, [(160, own), (64, [9, None, 2])])
    q, rows, T = b.q.clone(), np.ones(b.q.shape[:2], bool), b.q.shape[0]
    far = {BF16: (1e12, 1e30, 1e-30, 1e-12, 3e4, 1e-4), F16: (3e4, 1e-4)}[dtype]
    for i, t in enumerate(range(2, T - 3, 3)):               # every third sequence; the unused and the short ones
        q[t] = (q[t].float() * far[i % len(far)]).clamp(-6e4 if dtype == F16 else -1e38, 6e4 if dtype == F16 else 1e38).to(dtype)
        rows[t] = far[i % len(far)] < 1
    for t, n in enumerate(own):
        if n is None or n < 0:
            q[t], rows[t] = (q[t].float().sign() * (6e4 if dtype == F16 else 1e35)).to(dtype), False
    q[T - 2], rows[T - 2] = q[T - 2].sign() * 5e4, False
    b.check(b.run(q=q, **(long_table(b) if kind == "long" else {})), q=q, rows=rows)


def test_rows_without_a_finite_query_but_zero_among_others_of_other_sizes():
    b = Groups(17, BF16, 128, 64, 32, 4, 1, [(256, [5] * 70)])
    q, rows = b.q.clone(), np.ones(b.q.shape[:2], bool)
    q[3] = 0
    q[4], q[5, 1] = math.nan, math.inf
    q[6] = (q[6].float() * 1e20).to(BF16)
    q[7:] = (q[7:].float() * 1e-20).to(BF16)
    rows[4], rows[5, 1], rows[6] = False, False, False
    out, lse = b.run(q=q, **long_table(b))
    b.check((out, lse), q=torch.where(q.isfinite(), q, 0), rows=rows)
    assert out[4].isnan().all() and lse[4].isnan().all() and out[6].isfinite().all()


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("D,group", FORMATS)
@pytest.mark.parametrize("queries,back", [([21, 12, 24, 9, 5, 17], 1), ([21, 12, 24, 9, 5, 17], 7), ([130, 60, 300, 1, 200, 150], 1),
                                          ([130, 60, 300, 1, 200, 150], 90)], ids=["few", "few, before", "chunks", "chunks, before"])
def test_what_later_tokens_hold_changes_nothing(queries, back, dtype, D, group):
    """The values of a token near the end of each sequence have scales of NaN, infinity or the largest there is: whether it
    is in the last round of keys of a row that stands before it or rounds behind.  (Scales that are not finite, which no
    append writes: where many rows share the operands of a block, that has to hold for the rows of other blocks, of up to
    128 rows each, as in kv4_attention: 0 times the block's scale is not 0.)"""
    note(f"kv4_prefix_attention, later tokens, D={D} group={group} {queries[0]} {back} {dtype}")
    page = 32
    b = Groups(19, dtype, D, group, page, 4, 1, [(100, [300, 77]), (64, [301, 20]), (0, [200])], queries=queries, after=[170])
    G, finite, others = D // group, np.ones(b.q.shape[:2], bool), np.ones(b.q.shape[:2], bool)
    for at, n in zip(b.starts, queries):
        first = max(0, n - back)                             # that sees the token
        finite[at + first:at + n] = False
        others[at + (first * 4 // 128 * 32 if max(queries) > 24 else first):at + n] = False
    for word in (-1, 0x7C00, 0xFC00, 0x000F7BFF):
        rec = b.cache.cpu().view(torch.int32).view(b.cache.shape[0], 1, -1)
        for s, (n, ctx) in enumerate(zip(queries, b.lens)):
            if n >= back:
                place, params = (ctx - back) % page, page * D // 4 + G * page
                rec[int(b.table[s, (ctx - back) // page]), :, params + place:params + G * page:page] = word
        b.cache.copy_(rec.view(torch.uint8).view(b.cache.shape))
        b.check(b.run(), rows=finite if word == 0x000F7BFF else others)


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("D,group", FORMATS)
def test_many_rows_by_the_kernel_for_few_have_its_bounds(dtype, D, group):
    """Prefixes of few steps run by it whatever their rows: no rounding of the values."""
    note(f"kv4_prefix_attention, many rows by the kernel for few, D={D} group={group} {dtype}")
    for plan, queries in (([(1000, [1 + 3 * i for i in range(37)]), (333, [20] * 2), (95, [1] * 26)], None),
                          ([(200, [30, 40, 25, 5, None]), (97, [60, 1])], [20, 24, 3, 0, 0, 24, 1])):
        b = Groups(20 + D - group, dtype, D, group, 32, 4, 1, plan, queries=queries)
        assert b.many
        b.many, b.roundings = False, 1
        b.check(b.run())
