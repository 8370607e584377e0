"""The 4-bit paged key/value cache on the GPU: appended bytes bit for bit and
values read back, page copies, and the attention against fp64.

Bounds of the attention (set from the arithmetic, with u = 2^-24):
  scores   an fp32 sum of at most D products q c with c <= 143 (a code and its
           offset), scaled: dx = 8 u 143 sum|q| max(s) |scale|;
  out      the probabilities are rounded once to bf16 (2^-9 of each, and of
           their sum): 2^-8 mass, mass = sum p |v|; the scores' error: 2 dx mass;
           fp32 accumulation of n keys with codes offset by 128:
           (n / 16 + 32) u 143 max(s); the output's own rounding;
  lse      dx + 8 u (1 + |lse|)."""
import math

import numpy as np
import pytest
import torch

import kv4_reference as ref
import quantized_matmul_quantize_amd as qmm
from gpu_util import OUT_HALF_ULP, note

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -24


def rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def half(x, dtype):
    return torch.from_numpy(np.asarray(x, np.float32)).to(dtype)


def dirty(pages, heads, D, page, group):
    """A cache whose bytes are all ones: every scale a NaN."""
    c = qmm.kv4_cache(pages, heads, D, page, group)
    return c.fill_(255)


# ---------------------------------------------------------------------------
# Append, read.
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("D,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 128)])
@pytest.mark.parametrize("T,page,heads", [(1, 16, 1), (37, 16, 3), (70, 64, 2), (5, 256, 7)])
def test_append_bytes_and_read_values(dtype, D, group, T, page, heads):
    note(f"kv4 append D={D} group={group} T={T} page={page} heads={heads} {dtype}")
    g = rng(T * 1000 + D + group)
    pages = -(-T // page) + 3
    k = half(g.standard_normal((T, heads, D)) * np.exp(g.standard_normal((heads, D))), dtype)
    v = half(g.standard_normal((T, heads, D)) + 0.7, dtype)
    if T > 20:   # groups of one sign, of zeros, of one large entry, of the type's smallest numbers
        k[1] = k[1].abs() + 1
        k[2] = -k[2].abs() - 1
        v[3] = 0
        v[4, :, 5] = 3e4
        k[5] = k[5] * 1e-7
        v[6] = torch.finfo(dtype).smallest_normal
        k[7, :, 3], k[7, :, 4] = torch.finfo(dtype).max, torch.finfo(dtype).min
    slots = torch.from_numpy(g.permutation(pages * page)[:T].astype(np.int64))
    if T > 4:
        slots[2], slots[4] = -1, pages * page
    cache = dirty(pages, heads, D, page, group)
    want = cache.cpu().numpy().copy()
    qmm.kv4_append(k.cuda(), v.cuda(), slots.cuda(), cache)
    ref.store(want, k.float().numpy(), v.float().numpy(), slots.tolist())
    got = cache.cpu().numpy()
    assert np.array_equal(got, want), f"{(got != want).sum()} bytes differ"

    ok = ((slots >= 0) & (slots < pages * page)).numpy()
    for out_dtype in (F32, dtype):
        kr, vr = qmm.kv4_read(cache, slots.cuda(), D, dtype=out_dtype)
        for x, y in ((k, kr), (v, vr)):
            val = ref.values(*ref.quantize(x.float().numpy(), group))
            val[~ok] = 0
            assert torch.equal(y.cpu(), torch.from_numpy(val).float().to(out_dtype))


@pytest.mark.parametrize("D,group,heads,T", [(64, 32, 8, 4099), (128, 64, 5, 2050), (256, 128, 3, 2049)])
def test_append_of_many_tokens(D, group, heads, T):
    """Enough tokens for the form that takes several a thread, their count no multiple of what a thread takes."""
    note(f"kv4 append of many tokens D={D} group={group} heads={heads} T={T}")
    g, page = rng(T), 64
    pages = -(-T // page)
    k, v = (half(g.standard_normal((T, heads, D)), F16) for _ in range(2))
    slots = torch.from_numpy(g.permutation(pages * page)[:T].astype(np.int64))
    slots[7] = -1
    cache = dirty(pages, heads, D, page, group)
    want = cache.cpu().numpy().copy()
    qmm.kv4_append(k.cuda(), v.cuda(), slots.cuda(), cache)
    ref.store(want, k.float().numpy(), v.float().numpy(), slots.tolist())
    assert np.array_equal(cache.cpu().numpy(), want)
    kr, vr = qmm.kv4_read(cache, slots.cuda(), D, dtype=F32)
    for x, y in ((k, kr), (v, vr)):
        val = ref.values(*ref.quantize(x.float().numpy(), group))
        val[7] = 0
        assert np.array_equal(y.cpu().numpy(), val.astype(np.float32))


def test_append_infinities_and_nan_stay_in_their_group():
    D, group, page = 128, 32, 16
    k = half(rng(3).standard_normal((4, 2, D)), BF16)
    v = k.clone()
    k[0, 0, 3], k[1, 0, 40], v[2, 1, 70], v[3, 1, 127] = math.inf, -math.inf, math.nan, math.inf
    cache = dirty(2, 2, D, page, group)
    slots = torch.arange(4)
    qmm.kv4_append(k.cuda(), v.cuda(), slots.cuda(), cache)
    want = torch.full_like(cache.cpu(), 255).numpy()
    ref.store(want, k.float().numpy(), v.float().numpy(), slots.tolist())
    assert np.array_equal(cache.cpu().numpy(), want)
    kr, vr = qmm.kv4_read(cache, slots.cuda(), D, dtype=F32)
    assert kr.isfinite().all() and vr.isfinite().all()


def test_append_takes_views_of_a_projection_and_offsets():
    """k and v as slices of one projection's output; the last slots of a cache past 2^32 bytes."""
    D, heads, page, group, T = 128, 8, 64, 64, 21
    pages = 61000
    cache = qmm.kv4_cache(pages, heads, D, page, group)
    assert cache.numel() > 2 ** 32
    qkv = half(rng(4).standard_normal((T, 4 * heads * D)), BF16).cuda()
    k = qkv[:, 2 * heads * D:3 * heads * D].view(T, heads, D)
    v = qkv[:, 3 * heads * D:].view(T, heads, D)
    slots = torch.arange(pages * page - T, pages * page, device="cuda")
    qmm.kv4_append(k, v, slots, cache)
    kr, vr = qmm.kv4_read(cache, slots, D, dtype=F32)
    for x, y in ((k, kr), (v, vr)):
        val = ref.values(*ref.quantize(x.float().cpu().numpy(), group))
        assert np.array_equal(y.cpu().numpy(), val.astype(np.float32))


# ---------------------------------------------------------------------------
# Page copies.
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("layers,pages,shape,n", [(1, 9, (1, 16, 80), 4), (3, 40, (2, 64, 144), 17), (2, 5, (8, 256, 320), 2),
                                                  (1, 4, (1, 16, 96), 1)])
def test_copy_pages(layers, pages, shape, n):
    note(f"kv4 copy layers={layers} pages={pages} shape={shape} n={n}")
    g = rng(pages)
    cache = torch.from_numpy(g.integers(0, 256, (layers, pages, *shape), dtype=np.uint8)).cuda()
    order = torch.from_numpy(g.permutation(pages).astype(np.int64)).cuda()
    src, dst = order[:n], order[pages - n:]
    want = cache.clone()
    want[:, dst] = cache[:, src]
    qmm.kv4_copy_pages(cache, src, dst)
    assert torch.equal(cache, want)
    # pairs with an id outside the cache copy nothing; one source may have several destinations
    s2 = torch.tensor([-1, pages, int(src[0]), int(src[0])], device="cuda")
    d2 = torch.tensor([int(dst[0]), int(dst[0]), -1, pages], device="cuda")
    qmm.kv4_copy_pages(cache, s2, d2)
    assert torch.equal(cache, want)
    if pages > 8:
        one = src[:1].expand(2).contiguous()
        want[0, dst[:2]] = want[0, one]
        qmm.kv4_copy_pages(cache[0], one, dst[:2])
        assert torch.equal(cache, want)


def test_calls_on_nothing():
    cache = dirty(2, 2, 64, 16, 32)
    before = cache.clone()
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    x = torch.empty((0, 2, 64), dtype=BF16, device="cuda")
    qmm.kv4_append(x, x, none, cache)
    qmm.kv4_copy_pages(cache, none, none)
    k, v = qmm.kv4_read(cache, none, 64)
    assert k.shape == v.shape == (0, 2, 64) and torch.equal(cache, before)
    i32 = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")
    assert qmm.kv4_attention(x, cache, i32(0, 1), i32(0)).shape == (0, 2, 64)


# ---------------------------------------------------------------------------
# Attention.
# ---------------------------------------------------------------------------
class Batch:
    """Sequences in a dirty cache, in pages of a random order."""

    def __init__(self, seed, dtype, D, group, page, hq, hkv, lens, queries, gone=(), spread=1.0):
        g = rng(seed)
        self.dtype, self.lens, self.queries = dtype, lens, queries
        self.width = max(1, -(-max(lens) // page)) + 1
        pages = sum(-(-n // page) for n in lens) + 2
        order = g.permutation(pages)
        self.cache = dirty(pages, hkv, D, page, group)
        table = np.full((len(lens), self.width), -1, np.int32)
        self.k, self.v, self.here, at, top = [], [], [], 0, 0.0
        for b, n in enumerate(lens):
            need = -(-n // page)
            table[b, :need] = order[at:at + need]
            at += need
            k = half(g.standard_normal((n, hkv, D)) * np.exp(0.5 * g.standard_normal((hkv, D))) * spread, dtype)
            v = half(g.standard_normal((n, hkv, D)) + 0.3, dtype)
            j = np.arange(n)
            slots = table[b, j // page].astype(np.int64) * page + j % page
            if n:
                qmm.kv4_append(k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), self.cache)
            kq, vq = (ref.quantize(x.float().numpy(), group) for x in (k, v))
            if n:
                top = max(top, float(kq[2].max()))
            self.k.append(ref.values(*kq))
            self.v.append(ref.values(*vq))
            self.sv = max(getattr(self, "sv", 0.0), float(vq[2].max()) if n else 0.0)
            self.here.append(np.array([(b, int(x)) not in gone for x in j // page], bool).reshape(n))
        for b, p in gone:
            table[b, p] = -1 if (b + p) % 2 else pages + 7     # gone from the table: no page, or none of this cache
        self.sk = top
        self.table = torch.from_numpy(table).cuda()
        self.context = torch.tensor(lens, dtype=torch.int32).cuda()
        self.starts = np.concatenate([[0], np.cumsum(queries)]).astype(np.int32)
        self.q = half(g.standard_normal((int(self.starts[-1]), hq, D)), dtype)

    def check(self, got, window=0, sinks=0, scale=None, q=None, rows=None):
        """The results (of the tokens and heads where `rows` is true) against fp64."""
        out, lse = got
        q = (self.q if q is None else q).float().numpy()
        T, hq, D = q.shape
        scale = D ** -0.5 if scale is None else scale
        o, l, mass, count = ref.attention(q, self.k, self.v, self.lens, self.queries, scale, window, sinks, self.here)
        dx = 8 * U * 143 * np.abs(q).sum(-1) * self.sk * abs(scale)
        bound = (2.0 ** -8 + 2 * dx[..., None]) * mass + (count[:, None, None] / 16 + 32) * U * 143 * self.sv
        bound = bound + OUT_HALF_ULP[self.dtype] * np.abs(o) + (2.0 ** -24 if self.dtype == F16 else 0.0)
        err = np.abs(out.float().cpu().numpy() - o)
        none = np.repeat((count == 0)[:, None], hq, 1)
        rows = np.ones((T, hq), bool) if rows is None else rows
        assert (out.cpu()[torch.from_numpy(none)] == 0).all()
        assert (err <= bound)[~none & rows].all(), f"out: worst {np.nanmax(err / bound)} of its bound at {np.argmax(err / bound)}"
        got_l = lse.cpu().numpy().astype(np.float64)
        assert np.isneginf(got_l[none]).all()
        seen = ~none & rows
        worst = np.abs(got_l[seen] - l[seen]) - (dx + 8 * U * (1 + np.abs(l)))[seen]
        assert (worst <= 0).all(), f"lse: {worst.max()} past its bound"

    def run(self, **kw):
        q = kw.pop("q", self.q.cuda())
        if max(self.queries) != 1 or min(self.queries) != 1:
            kw.setdefault("cu_q", torch.from_numpy(self.starts).cuda())
            kw.setdefault("max_q", max(self.queries))
        return qmm.kv4_attention(q, self.cache, self.table, self.context, return_lse=True, **kw)


FORMATS = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)]


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("D,group", FORMATS)
@pytest.mark.parametrize("page", [16, 64])
def test_decode_formats(dtype, D, group, page):
    lens = [1, 15, 16, 17, 33, 0, 100, 131, 260]
    note(f"kv4 decode D={D} group={group} page={page} {dtype}")
    b = Batch(D + group + page, dtype, D, group, page, 4, 2, lens, [1] * len(lens))
    b.check(b.run())


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (5, 5), (16, 1), (14, 2), (17, 1), (40, 2), (32, 8)])
@pytest.mark.parametrize("page", [16, 32, 128, 256])
def test_decode_heads(hq, hkv, page):
    lens = [70, 5, 300]
    note(f"kv4 decode heads {hq}/{hkv} page={page}")
    b = Batch(hq * 10 + page, BF16, 128, 64, page, hq, hkv, lens, [1, 1, 1])
    b.check(b.run())


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("D,group", [(64, 64), (128, 32), (128, 128), (256, 64)])
@pytest.mark.parametrize("queries,lens", [([2, 5, 3], [2, 64, 131]), ([17, 1, 40, 0], [17, 90, 41, 30]),
                                          ([70, 33], [200, 33]), ([4], [2]), ([129], [300]), ([0, 260], [7, 261])])
def test_chunks(dtype, D, group, queries, lens):
    """Ragged queries, all of a sequence's tokens among them, and more than it has (whose first see nothing)."""
    note(f"kv4 chunks D={D} group={group} queries={queries} lens={lens} {dtype}")
    b = Batch(sum(queries) + D, dtype, D, group, 32, 6, 2, lens, queries)
    b.check(b.run())
    b.check(b.run(max_q=None))           # the hint only shapes the launch
    b.check(b.run(max_q=1))


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 3), (16, 4), (33, 40), (64, 0), (100, 64), (1000, 4)])
@pytest.mark.parametrize("queries,lens", [([1, 1, 1, 1], [3, 40, 333, 0]), ([6, 20], [290, 150]), ([90], [500])])
def test_window_and_sinks(dtype, D, window, sinks, queries, lens):
    note(f"kv4 window={window} sinks={sinks} D={D} queries={queries} lens={lens} {dtype}")
    b = Batch(window + D, dtype, D, 64, 16, 4, 2, lens, queries)
    b.check(b.run(window=window, sinks=sinks), window, sinks)


@pytest.mark.parametrize("queries", [[1, 1, 1], [9, 3, 20]])
def test_pages_gone_from_the_table_are_not_seen(queries):
    """Pages below a window went back; and a table with holes inside the window, a whole short sequence among them."""
    gone = [(0, 0), (0, 1), (0, 2), (1, 4), (1, 0), (2, 0), (2, 1)]
    b = Batch(5, BF16, 128, 64, 16, 4, 2, [200, 120, 20], queries, gone=gone)
    b.check(b.run(window=50), 50)
    b.check(b.run())


def test_table_rows_apart_strided_queries_and_given_outputs():
    b = Batch(6, F16, 128, 32, 32, 8, 4, [100, 31, 64], [1, 1, 1])
    wide = torch.full((3, b.width + 5), 12345, dtype=torch.int32, device="cuda")
    wide[:, :b.width] = b.table
    b.table = wide[:, :b.width]
    qkv = torch.zeros((3, 16, 128), dtype=F16, device="cuda")
    qkv[:, 4:12] = b.q.cuda()
    out = torch.full((3, 8, 128), 7.0, dtype=F16, device="cuda")
    need = qmm.kv4_attention_workspace_bytes(3, 3, 1, 8, 4, 128, 32, b.width * 32)
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")     # bytes of NaN
    got = b.run(q=qkv[:, 4:12], out=out, workspace=ws)
    assert got[0].data_ptr() == out.data_ptr()
    b.check(got)
    # a transposed view: heads outermost
    qt = b.q.cuda().transpose(0, 1).contiguous().transpose(0, 1)
    assert not qt.is_contiguous()
    b.check(b.run(q=qt))


@pytest.mark.parametrize("scale", [0.0, 0.05, 3.0, -0.4])
def test_scales(scale):
    b = Batch(7, BF16, 64, 32, 16, 4, 2, [90, 200], [1, 1])
    b.check(b.run(scale=scale), scale=scale)


def test_large_scores_and_a_context_beyond_the_table():
    b = Batch(8, BF16, 128, 64, 16, 4, 2, [150, 64], [1, 1], spread=30.0)
    b.check(b.run())
    # a context longer than the table counts as the table's tokens
    got = qmm.kv4_attention(b.q[1:].cuda(), b.cache, b.table[1:, :4], torch.tensor([10 ** 6], dtype=torch.int32).cuda())
    same = qmm.kv4_attention(b.q[1:].cuda(), b.cache, b.table[1:, :4], b.context[1:])
    assert torch.equal(got, same)


@pytest.mark.parametrize("queries", [[1, 1], [3, 2], [90, 5]])
def test_a_query_that_is_not_finite_stays_in_its_row(queries):
    b = Batch(12, BF16, 128, 64, 16, 4, 2, [200, 70], queries)
    q = b.q.clone()
    q[0, 0, 5], q[1, 2, 7] = math.inf, math.nan
    out, lse = (x.cpu() for x in b.run(q=q.cuda()))
    rest = np.ones(q.shape[:2], bool)
    rest[0, 0] = rest[1, 2] = False
    safe = q.clone()
    safe[0, 0], safe[1, 2] = 0, 0
    b.check((out, lse), q=safe, rows=rest)
    assert not out[~torch.from_numpy(rest)].isfinite().all()


@pytest.mark.parametrize("queries", [[1, 1], [90, 5]])
@pytest.mark.parametrize("size", [2.0 ** -30, 2.0 ** 40])
def test_queries_of_any_size(queries, size):
    """bf16 queries far from the middle of the binary16 range, with a scale to match."""
    b = Batch(13, BF16, 128, 64, 16, 4, 2, [200, 70], queries)
    b.q = (b.q.float() * size).to(BF16)
    b.check(b.run(scale=128 ** -0.5 / size), scale=128 ** -0.5 / size)


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("D,group", FORMATS)
@pytest.mark.parametrize("queries,lens", [([1, 1, 1], [2, 5, 20]), ([4, 2], [4, 9]), ([20], [20]), ([60, 25], [60, 25])])
def test_log_sums_of_few_keys(dtype, D, group, queries, lens):
    """Small queries, so that the scores' own bound is small beside any rounding of a row's few probabilities."""
    b = Batch(19 + D + group, dtype, D, group, 16, 16, 2, lens, queries)
    b.q = (b.q.float() * 2.0 ** -6).to(dtype)
    b.check(b.run())


@pytest.mark.parametrize("queries", [[1, 1], [90, 5]])
@pytest.mark.parametrize("rise", [True, False])
def test_values_of_very_different_sizes(queries, rise):
    """Values that grow (or fall) a hundredfold along the sequence: the power of two that binary16 weights carry moves."""
    D, group, page, n = 128, 32, 16, 300
    b = Batch(14, F16, D, group, page, 4, 2, [n, 70], queries)
    g = rng(15)
    ramp = np.exp(np.linspace(0, np.log(100.0), n) * (1 if rise else -1))[:, None, None]
    v = half(g.standard_normal((n, 2, D)) * ramp * np.repeat([1.0, 30.0, 0.05, 1.0], 32), F16)
    j = np.arange(n)
    k = half(g.standard_normal((n, 2, D)), F16)
    slots = b.table[0].cpu().numpy()[j // page].astype(np.int64) * page + j % page
    qmm.kv4_append(k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), b.cache)
    kq, vq = (ref.quantize(x.float().numpy(), group) for x in (k, v))
    b.k[0], b.v[0], b.sk, b.sv = ref.values(*kq), ref.values(*vq), max(b.sk, float(kq[2].max())), float(vq[2].max())
    b.check(b.run())


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("D,group", FORMATS)
def test_a_few_queries_of_many_sequences(dtype, D, group):
    """Enough sequences to fill the chip with blocks of 32 rows each."""
    note(f"kv4 many sequences D={D} group={group} {dtype}")
    queries = [5, 1, 4, 0, 5, 3, 2, 5] * 10
    b = Batch(18 + D + group, dtype, D, group, 16, 16, 4, [(7 * i) % 61 + 5 * (i % 3 == 0) for i in range(80)], queries)
    b.check(b.run())
    b.check(b.run(window=9, sinks=2), window=9, sinks=2)


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("D,group", FORMATS)
def test_chunks_over_split_keys(dtype, D, group):
    """Few rows and heads over a long context: blocks share the keys, for chunks and for a few queries alike."""
    note(f"kv4 split chunks D={D} group={group} {dtype}")
    b = Batch(16 + D + group, dtype, D, group, 64, 6, 2, [3000, 700], [70, 25])
    b.check(b.run())
    b.check(b.run(window=900, sinks=5), window=900, sinks=5)
    few = Batch(17 + D + group, dtype, D, group, 64, 6, 2, [2600, 90], [9, 3])
    few.check(few.run())


def test_long_context_splits_and_high_pages():
    """A long sequence (the work is split over it) in the last pages of a cache past 2^32 bytes, against fp64."""
    D, group, page, heads, n = 128, 64, 64, 8, 9000
    pages = 61000
    g = rng(9)
    cache = qmm.kv4_cache(pages, heads, D, page, group)
    assert cache.numel() > 2 ** 32
    need = -(-n // page)
    table = torch.arange(pages - 1, pages - 1 - need, -1, dtype=torch.int32, device="cuda")[None]
    k, v = (half(g.standard_normal((n, heads, D)), BF16) for _ in range(2))
    j = torch.arange(n, device="cuda")
    qmm.kv4_append(k.cuda(), v.cuda(), table[0].long()[j // page] * page + j % page, cache)
    b = Batch.__new__(Batch)
    kq, vq = (ref.quantize(x.float().numpy(), group) for x in (k, v))
    b.dtype, b.lens, b.queries, b.cache, b.table, b.here = BF16, [n], [1], cache, table, [np.ones(n, bool)]
    b.k, b.v, b.sk, b.sv = [ref.values(*kq)], [ref.values(*vq)], float(kq[2].max()), float(vq[2].max())
    b.context = torch.tensor([n], dtype=torch.int32, device="cuda")
    b.q = half(g.standard_normal((1, 16, D)) * 2, BF16)
    b.check(b.run())
    again = b.run()
    assert torch.equal(again[0], b.run()[0]) and torch.equal(again[1], b.run()[1])


def test_another_stream_and_replayed_graph():
    """A decode step (append, attend) on a stream of its own, and captured and replayed with new inputs."""
    b = Batch(10, BF16, 128, 64, 16, 8, 2, [100, 37], [1, 1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = b.run()
    torch.cuda.current_stream().wait_stream(side)
    b.check(got)

    page, hkv, D = 16, 2, 128
    k, v = (torch.zeros((2, hkv, D), dtype=BF16, device="cuda") for _ in range(2))
    slots = torch.zeros(2, dtype=torch.int64, device="cuda")
    q = b.q.cuda()
    with torch.cuda.stream(side):
        for _ in range(2):
            qmm.kv4_append(k, v, slots.fill_(-1), b.cache)
            qmm.kv4_attention(q, b.cache, b.table, b.context, return_lse=True)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        qmm.kv4_append(k, v, slots, b.cache)
        out, lse = qmm.kv4_attention(q, b.cache, b.table, b.context, return_lse=True)
    g = rng(11)
    for step in range(3):
        b.context += 1
        at = b.context.long() - 1
        row = b.table.long()
        slots.copy_(row[torch.arange(2, device="cuda"), at // page] * page + at % page)
        for x in (k, v, q):
            x.copy_(half(g.standard_normal(x.shape), BF16))
        graph.replay()
        torch.cuda.synchronize()
        want = qmm.kv4_attention(q, b.cache, b.table, b.context, return_lse=True)
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        for i in range(2):
            for x, y in ((b.k, k), (b.v, v)):
                new = ref.values(*ref.quantize(y[i].float().cpu().numpy(), 64))
                x[i] = np.concatenate([x[i], new[None]])
            b.here[i] = np.ones(len(b.k[i]), bool)
        b.lens = [n + 1 for n in b.lens]
        b.sk = max(b.sk, float(ref.quantize(k.float().cpu().numpy(), 64)[2].max()))
        b.check((out, lse), q=q.cpu())
