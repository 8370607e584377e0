"""Attention over the 4-bit cache where a mask hides keys inside the context:
whatever their memory holds, it changes nothing; and the results against
bounds derived from the kernels' own arithmetic (kv4_bounds.py)."""
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


def half(x, dtype):
    return torch.from_numpy(np.asarray(x, np.float32)).to(dtype)


class Case:
    """Sequences in a cache whose other bytes are all ones; edit(b, k, v) may change a sequence's keys and values."""

    def __init__(self, seed, dtype, D, group, page, hq, hkv, lens, queries, edit=None):
        g = np.random.Generator(np.random.PCG64(seed))
        self.dtype, self.D, self.group, self.page, self.lens, self.queries = dtype, D, group, page, lens, queries
        pages = sum(-(-n // page) for n in lens) + 1
        order, at = g.permutation(pages), 0
        self.cache = qmm.kv4_cache(pages, hkv, D, page, group).fill_(255)
        table = np.full((len(lens), max(1, -(-max(lens) // page))), -1, np.int32)
        self.k, self.v, self.sk, self.sv, self.slots = [], [], [], [], []
        for b, n in enumerate(lens):
            need = -(-n // page)
            table[b, :need] = order[at:at + need]
            at += need
            k = half(g.standard_normal((n, hkv, D)) * np.exp(0.5 * g.standard_normal((hkv, D))), dtype)
            v = half(g.standard_normal((n, hkv, D)), dtype)
            if edit and n:
                edit(b, k, v)
            j = np.arange(n)
            self.slots.append(table[b, j // page].astype(np.int64) * page + j % page)
            if n:
                qmm.kv4_append(k.cuda(), v.cuda(), torch.from_numpy(self.slots[b]).cuda(), self.cache)
            for x, val, sc in ((k, self.k, self.sk), (v, self.v, self.sv)):
                c, z, s = ref.quantize(x.float().numpy(), group)
                val.append(ref.values(c, z, s))
                sc.append(s.astype(np.float64))
        self.table = torch.from_numpy(table).cuda()
        self.context = torch.tensor(lens, dtype=torch.int32).cuda()
        self.starts = np.concatenate([[0], np.cumsum(queries)]).astype(np.int32)
        self.q = half(g.standard_normal((int(self.starts[-1]), hq, D)), dtype)
        # the kernel for chunks takes bf16 probabilities through two roundings
        self.written, self.fp64 = self.cache.clone(), {}
        self.roundings = 2 if dtype == BF16 and max(queries) * (hq // hkv) > 96 else 1

    def fill_hidden(self, window, sinks, word):
        """Of the cache as it was written: every word of the keys and values that no query sees becomes `word` (their
        scales its low half)."""
        pages, heads, page, token = self.cache.shape
        D, G = self.D, self.D // self.group
        rec = torch.from_numpy(self.written.cpu().numpy().view(np.uint32).reshape(pages, heads, -1).view(np.int32)).clone()
        word, words, hidden = int(np.uint32(word).view(np.int32)), page * D // 8, 0
        for b, (n, ctx) in enumerate(zip(self.queries, self.lens)):
            for slot in self.slots[b][bounds.hidden(ctx, n, window, sinks)]:
                p, t = divmod(int(slot), page)
                hidden += 1
                rec[p, :, t * (D // 8):(t + 1) * (D // 8)] = word
                rec[p, :, words + t // 4 * (D // 2) + t % 4:words + (t // 4 + 1) * (D // 2):4] = word
                rec[p, :, 2 * words + t:2 * words + 2 * G * page:page] = word
        self.cache.copy_(rec.view(torch.uint8).reshape(self.cache.shape))
        return hidden

    def run(self, q=None, **kw):
        if set(self.queries) != {1}:
            kw.update(cu_q=torch.from_numpy(self.starts).cuda(), max_q=max(self.queries))
        q = self.q if q is None else q
        return [x.cpu() for x in qmm.kv4_attention(q.cuda(), self.cache, self.table, self.context, return_lse=True, **kw)]

    def check(self, got, window=0, sinks=0, rows=None):
        """Of the tokens where `rows` is true (all by default)."""
        if (window, sinks) not in self.fp64:
            self.fp64[window, sinks] = bounds.attention(
                self.q.float().numpy(), self.k, self.v, self.sk, self.sv, self.lens, self.queries, self.D ** -0.5, window,
                sinks, roundings=self.roundings)
        o, l, b_out, b_lse, count = self.fp64[window, sinks]
        rows = np.ones(len(o), bool) if rows is None else rows
        seen = rows & (count > 0)
        out, lse = (x.double().numpy() for x in got)
        bound = b_out + OUT_HALF_ULP[self.dtype] * np.abs(o) + (2.0 ** -25 if self.dtype == F16 else 0.0)
        worst = (np.abs(out - o) / np.maximum(bound, 1e-300))[seen]
        assert (worst <= 1).all(), f"out: {np.nanmax(worst)} of its bound, {np.isnan(worst).sum()} are NaN"
        worst = np.abs(lse[seen] - l[seen]) / b_lse[seen]
        assert (worst <= 1).all(), f"lse: {np.nanmax(worst)} of its bound, {np.isnan(worst).sum()} are NaN"
        none = rows & (count == 0)
        assert (out[none] == 0).all() and np.isneginf(lse[none]).all()


def several(n):
    return 16, 4, [(7 * i) % 61 + 5 * (i % 3 == 0) + 40 for i in range(n)], [5, 1, 4, 0, 5, 3, 2, 5] * (n // 8)


# one query; few (tiles of 8 rows); enough sequences for tiles of 16 rows, and of 32; chunks
SHAPES = {"one": (4, 2, [3, 40, 333, 150, 0], [1] * 5), "few": (4, 2, [290, 150], [6, 20]), "some": several(40),
          "many": several(80), "chunk": (4, 2, [500, 170], [90, 61])}


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("D,group", FORMATS)
@pytest.mark.parametrize("shape", list(SHAPES))
def test_against_the_arithmetic(dtype, D, group, shape):
    note(f"kv4 bounds D={D} group={group} {shape} {dtype}")
    hq, hkv, lens, queries = SHAPES[shape]
    c = Case(D + group, dtype, D, group, 16, hq, hkv, lens, queries)
    c.check(c.run())


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("D,group", FORMATS)
@pytest.mark.parametrize("shape", list(SHAPES))
def test_what_hidden_keys_hold_changes_nothing(dtype, D, group, shape):
    """Only the sinks and the window are written: the other tokens of their pages hold NaN, infinities or the largest
    scale, and the table still names their pages."""
    note(f"kv4 hidden keys D={D} group={group} {shape} {dtype}")
    hq, hkv, lens, queries = SHAPES[shape]
    c = Case(1 + D + group, dtype, D, group, 16 if D == 128 else 64, hq, hkv, lens, queries)
    for window, sinks in ((20, 4), (33, 0)):
        for word in (0xFFFFFFFF, 0x7C00, 0xFC00, 0x000F7BFF):
            assert c.fill_hidden(window, sinks, word) > 0
            got = c.run(window=window, sinks=sinks)
            c.check(got, window, sinks)


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("D,group", FORMATS)
@pytest.mark.parametrize("shape", ["few", "some", "many", "chunk"])
def test_later_tokens_change_nothing(dtype, D, group, shape):
    """The last token's values are infinite (stored with the largest scale): the rows before it do not see it."""
    note(f"kv4 later tokens D={D} group={group} {shape} {dtype}")
    hq, hkv, lens, queries = SHAPES[shape]

    def edit(b, k, v):
        v[-1, :, ::group] = math.inf
    c = Case(2 + D + group, dtype, D, group, 16, hq, hkv, lens, queries, edit)
    rows = np.ones(int(c.starts[-1]), bool)
    rows[c.starts[1:][np.array(queries) > 0] - 1] = False
    c.check(c.run(), rows=rows)


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("hq,hkv,lens,queries", [(4, 2, [200, 70], [1, 1]), (4, 2, [200, 70], [3, 2]), (4, 2, [200, 70], [90, 5]),
                                                 (4, 2, [3000, 700], [1, 1]), (6, 2, [3000, 700], [9, 3]),
                                                 (6, 2, [3000, 700], [70, 25])])
def test_a_query_that_is_not_finite_has_no_log_sum(dtype, hq, hkv, lens, queries):
    """NaN, not the -inf of a row that sees no key: a merge by log-sum-exp would drop it without a word."""
    note(f"kv4 not finite {lens} {queries} {dtype}")
    c = Case(3, dtype, 128, 64, 16, hq, hkv, lens, queries)
    q = c.q.clone()
    q[0, 0, 5], q[1, 1, 7], q[1, 3, 100] = math.inf, math.nan, -math.inf
    bad = torch.zeros(q.shape[:2], dtype=torch.bool)
    bad[0, 0] = bad[1, 1] = bad[1, 3] = True
    out, lse = c.run(q=q)
    assert lse[bad].isnan().all() and out[bad].isnan().all()
    assert lse[~bad].isfinite().all() and out[~bad].isfinite().all()
