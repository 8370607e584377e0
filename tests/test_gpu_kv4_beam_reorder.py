"""The reordering of the beams' pages: tables and cache bytes against a plain
loop over slots, layers, heads and tokens."""
import numpy as np
import pytest
import torch

import quantized_matmul_quantize_amd as qmm
from gpu_util import note

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def plain(cache, D, table, context, tails, parents):
    """numpy: cache [layers, pages, heads, page, token] (changed), the new table and context."""
    layers, pages, heads, page, token = cache.shape
    G = (token - D) // 8
    record = cache.reshape(layers, pages, heads, page * token)
    new, ctx = table.copy(), context.copy()
    seqs, beams = parents.shape
    width = table.shape[1]
    before = record.copy()
    for r in range(seqs * beams):
        b = parents[r // beams, r % beams]
        p = r // beams * beams + b if 0 <= b < beams else r
        n = min(max(int(context[p]), 0), width * page)
        new[r], ctx[r] = table[p], n
        if p == r or n % page == 0:
            continue
        at = min(max(int(context[r]), 0), width * page) // page
        mine = table[r, at] if at < width else -1
        spare = tails[r, 1] if mine == tails[r, 0] else tails[r, 0]
        src = table[p, n // page]
        new[r, n // page] = spare
        if not (0 <= src < pages and 0 <= spare < pages and src != spare):
            continue
        n = -(-(n % page) // 4) * 4
        at = np.concatenate([np.arange(n * D // 2), page * D // 2 + np.arange(n * D // 2)] +
                            [page * D + 4 * page * row + np.arange(4 * n) for row in range(2 * G)])
        record[:, spare, :, at] = before[:, src, :, at]
    return new, ctx


def state(g, seqs, beams, D, group, page, heads, layers, prompt, generated):
    """Beams of sequences with their own lengths; tail pages with the filled one first or second."""
    rows, tails, context, free = [], [], [], 0
    for s in range(seqs):
        total = int(prompt[s % len(prompt)]) + int(generated[s % len(generated)])
        whole = int(prompt[s % len(prompt)]) // page
        shared = list(range(free, free + whole))
        free += whole
        for _ in range(beams):
            own = list(range(free, free + total // page - whole))
            pair = [free + len(own), free + len(own) + 1]
            free += len(own) + 2
            rows.append(shared + own + ([pair[g.integers(0, 2)]] if total % page else []))
            tails.append(pair)
            context.append(total)
    width = max(len(r) for r in rows) + 1
    order = g.permutation(free)
    table = np.full((len(rows), width), -1, np.int32)
    for i, r in enumerate(rows):
        table[i, :len(r)] = order[r]
    token = D + 8 * D // group
    cache = g.integers(0, 256, (layers, free, heads, page, token)).astype(np.uint8)
    return cache, table, np.array(context, np.int32), order[np.array(tails)].astype(np.int32)


def run(cache, D, table, context, tails, parents, four=False):
    c = torch.from_numpy(cache).cuda()
    put = lambda x: torch.from_numpy(x).cuda()
    got_t, got_c = qmm.kv4_beam_reorder(c[0] if four else c, D, put(table), put(context), put(tails), put(parents))
    want = cache.copy()
    want_t, want_c = plain(want, D, table, context, tails, parents)
    assert np.array_equal(got_t.cpu().numpy(), want_t) and np.array_equal(got_c.cpu().numpy(), want_c)
    got = c.cpu().numpy()
    assert np.array_equal(got, want), f"{(got != want).sum()} bytes differ"
    return got_t, got_c, c


@pytest.mark.parametrize("D,group,page,heads,layers", [(64, 32, 16, 3, 2), (64, 64, 256, 1, 1), (128, 32, 64, 8, 3),
                                                       (128, 64, 32, 2, 5), (128, 128, 128, 5, 1), (256, 64, 16, 4, 2)])
@pytest.mark.parametrize("seqs,beams", [(1, 1), (1, 4), (5, 3), (2, 16)])
def test_formats(D, group, page, heads, layers, seqs, beams):
    note(f"kv4_beam_reorder D={D} group={group} page={page} heads={heads} layers={layers} {seqs} x {beams}")
    g = rng(D + page + beams)
    st = state(g, seqs, beams, D, group, page, heads, layers, [3 * page, 1, page + 5], [1, page - 1, page, 2 * page + 3, 6])
    parents = g.integers(0, beams, (seqs, beams))
    run(st[0], D, *st[1:], parents, four=layers == 1)


def test_parents_outside_lengths_that_differ_and_pages_outside():
    g = rng(3)
    D, group, page, beams = 128, 64, 32, 6
    cache, table, context, tails = state(g, 2, beams, D, group, page, 2, 2, [40], [30])
    parents = np.array([[-1, 6, 2, 0, 0, 5], [1, 1, 1, 1, 1, 2 ** 40]])
    run(cache, D, table, context, tails, parents)
    context[3], context[4], context[7] = 0, 64, 33          # beams of other lengths, one at a page's end
    run(cache, D, table, context, tails, parents)
    context[1], context[7] = -5, 10 ** 6                    # beyond the table
    parents = np.array([[1, 0, 1, 1, 0, 5], [1, 0, 1, 1, 1, 1]])
    run(cache, D, table, context, tails, parents)
    context[:] = 70
    table[0, 2], tails[8] = -1, 10 ** 6                     # pages that are none are not copied
    run(cache, D, table, context, tails, np.array([[0, 0, 0, 3, 4, 5], [0, 1, 1, 1, 1, 1]]))


def test_given_outputs_nothing_to_do_and_a_replayed_graph():
    g = rng(4)
    D, group, page, beams = 64, 32, 16, 4
    cache, table, context, tails = state(g, 3, beams, D, group, page, 2, 3, [20], [11])
    c, t0, n0, tl = (torch.from_numpy(x).cuda() for x in (cache, table, context, tails))
    none = torch.empty((0, beams), dtype=torch.int64, device="cuda")
    out = qmm.kv4_beam_reorder(c, D, t0[:0], n0[:0], tl[:0], none)
    assert out[0].shape == (0, table.shape[1]) and out[1].shape == (0,)
    t1, n1 = torch.empty_like(t0), torch.empty_like(n0)
    parents = torch.empty((3, beams), dtype=torch.int64, device="cuda").copy_(torch.from_numpy(g.integers(0, beams, (3, beams))))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        a, b = qmm.kv4_beam_reorder(c, D, t0, n0, tl, parents, table_out=t1, context_out=n1)
        qmm.kv4_beam_reorder(c, D, t1, n1, tl, parents, table_out=t0, context_out=n0)
    assert a is t1 and b is n1
    for _ in range(3):
        parents.copy_(torch.from_numpy(g.integers(0, beams, (3, beams))))
        p = parents.cpu().numpy()
        t, n = plain(cache, D, *plain(cache, D, table, context, tails, p), tails, p)
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(t0.cpu().numpy(), t) and np.array_equal(n0.cpu().numpy(), n)
        assert np.array_equal(c.cpu().numpy(), cache)
        table, context = t, n


def test_pages_past_4_gib():
    D, group, page, heads, beams = 128, 64, 64, 8, 2
    pages = 60000
    cache = qmm.kv4_cache(pages, heads, D, page, group)
    assert cache.numel() > 2 ** 32
    cache[-4:] = torch.randint(0, 256, cache[-4:].shape, dtype=torch.uint8, device="cuda")
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    old = cache[-4:].clone()
    table, context = qmm.kv4_beam_reorder(cache, D, i([pages - 1], [pages - 3]), i(64 - 4, 64 - 4),
                                          i([pages - 1, pages - 2], [pages - 3, pages - 4]),
                                          torch.tensor([[1, 1]], device="cuda"))
    assert table.tolist() == [[pages - 2], [pages - 3]]
    assert torch.equal(cache[-1], old[3]) and torch.equal(cache[-3:-1][0], old[1]) and torch.equal(cache[-4], old[0])
    k, v = qmm.kv4_read(cache, torch.arange(60, device="cuda") + (pages - 2) * page, D)
    k1, v1 = qmm.kv4_read(cache, torch.arange(60, device="cuda") + (pages - 3) * page, D)
    assert torch.equal(k.view(torch.int16), k1.view(torch.int16)) and torch.equal(v.view(torch.int16), v1.view(torch.int16))
