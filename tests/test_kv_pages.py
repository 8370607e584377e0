"""The host bookkeeping of cache pages, against a model that stores each token's value in a plain array of slots."""
import numpy as np
import pytest
import torch

from quantized_matmul_quantize_amd import KvPages


class Model:
    """A cache of one integer per slot, and what each sequence should read back (None: forgotten)."""

    def __init__(self, pages, page):
        self.k, self.store, self.want, self.page = KvPages(pages, page), np.full(pages * page, -7), {}, page

    def copy(self, src, dst):
        assert not set(src.tolist()) & set(dst.tolist()) and len(set(dst.tolist())) == len(dst)
        rows = self.store.reshape(-1, self.page)
        rows[dst.numpy()] = rows[src.numpy()]

    def extend(self, seqs, counts, g):
        slots, src, dst = self.k.extend(seqs, counts)
        assert slots.dtype == src.dtype == dst.dtype == torch.int64 and len(slots) == sum(counts)
        assert len(set(slots.tolist())) == len(slots)
        self.copy(src, dst)
        new = g.integers(0, 10 ** 6, sum(counts))
        self.store[slots.numpy()] = new
        at = 0
        for s, n in zip(seqs, counts):
            self.want[s] = self.want[s] + new[at:at + n].tolist()
            at += n

    def check(self):
        seqs = list(self.want)
        table, context = self.k.table(seqs)
        assert table.dtype == context.dtype == torch.int32
        held = set()
        for row, n, s in zip(table.tolist(), context.tolist(), seqs):
            assert n == self.k.length(s) == len(self.want[s])
            held |= {p for p in row if p >= 0}
            for j, w in enumerate(self.want[s]):
                if w is not None:
                    assert row[j // self.page] >= 0 and self.store[row[j // self.page] * self.page + j % self.page] == w
        assert self.k.free_pages == self.k.pages - len(held)


@pytest.mark.parametrize("seed", range(8))
@pytest.mark.parametrize("page", [1, 4, 16])
def test_random_operations(seed, page):
    g = np.random.Generator(np.random.PCG64(seed))
    m = Model(200, page)
    for step in range(200):
        seqs = list(m.want)
        what = g.integers(0, 10)
        if what == 0 or not seqs:
            m.want[m.k.add()] = []
        elif what <= 4:
            some = [s for s in seqs if g.random() < 0.6]
            counts = g.integers(0, 2 * page + 3, len(some)).tolist()
            before = m.k.table(seqs)
            try:
                m.extend(some, counts, g)
            except RuntimeError:
                after = m.k.table(seqs)
                assert torch.equal(before[0], after[0]) and torch.equal(before[1], after[1])
                s = seqs[g.integers(len(seqs))]
                m.k.free(s)
                del m.want[s]
        elif what <= 6:
            s = seqs[g.integers(len(seqs))]
            m.want[m.k.fork(s)] = list(m.want[s])
        elif what == 7:
            s = seqs[g.integers(len(seqs))]
            n = int(g.integers(0, min(len(m.want[s]), 2 * page) + 1))
            if all(w is not None for w in m.want[s]):
                m.k.shrink(s, n)
                m.want[s] = m.want[s][:len(m.want[s]) - n]
        elif what == 8:
            s = seqs[g.integers(len(seqs))]
            window, sinks = int(g.integers(1, 5 * page)), int(g.integers(0, page + 2))
            m.k.forget(s, window, sinks)
            n = len(m.want[s])
            m.want[s] = [w if j < sinks or j > n - window else None for j, w in enumerate(m.want[s])]
        else:
            src, dst = m.k.compact()
            m.copy(src, dst)
            used = m.k.pages - m.k.free_pages
            assert all(p < used for row in m.k.table(list(m.want))[0].tolist() for p in row)
            if g.random() < 0.5 and seqs:
                m.k.free(seqs[0])
                del m.want[seqs[0]]
        m.check()


def test_a_fork_copies_only_the_page_it_writes():
    m, g = Model(10, 4), np.random.Generator(np.random.PCG64(1))
    a = m.k.add()
    m.want[a] = []
    m.extend([a], [6], g)
    b = m.k.fork(a)
    c = m.k.fork(a)
    m.want[b], m.want[c] = list(m.want[a]), list(m.want[a])
    assert m.k.free_pages == 8
    slots, src, dst = m.k.extend([a, b, c], [1, 1, 1])
    assert src.tolist() == [1, 1] and dst.tolist() == [2, 3]          # the last of the three keeps the page
    assert slots.tolist() == [2 * 4 + 2, 3 * 4 + 2, 1 * 4 + 2] and m.k.free_pages == 6
    d = m.k.fork(a)
    m.k.shrink(d, 7)
    assert m.k.extend([d], [1])[1].numel() == 0                       # nothing left of the shared pages
    e = KvPages(4, 4)
    s = e.add()
    e.extend([s], [8])
    t = e.fork(s)
    slots, src, dst = e.extend([t], [1])                              # full pages are never copied
    assert src.numel() == 0 and slots.tolist() == [8]


def test_errors_change_nothing():
    k = KvPages(3, 4)
    a = k.add()
    k.extend([a], [9])
    for call, error in [(lambda: k.extend([a], [4]), RuntimeError), (lambda: k.extend([a, a], [0, 0]), ValueError),
                        (lambda: k.extend([a], [-1]), ValueError), (lambda: k.extend([a], []), ValueError),
                        (lambda: k.extend([99], [1]), ValueError), (lambda: k.shrink(a, 10), ValueError),
                        (lambda: k.forget(a, 0), ValueError), (lambda: k.free(99), ValueError),
                        (lambda: k.fork(99), ValueError), (lambda: k.table([a], 2), ValueError),
                        (lambda: k.length(99), ValueError), (lambda: KvPages(0, 4), ValueError)]:
        with pytest.raises(error):
            call()
        assert k.table([a])[0].tolist() == [[0, 1, 2]] and k.length(a) == 9 and k.free_pages == 0
    k.forget(a, 2)
    assert k.table([a], 5)[0].tolist() == [[-1, -1, 2, -1, -1]] and k.free_pages == 2
    with pytest.raises(ValueError):
        k.shrink(a, 2)
    assert k.length(a) == 9
    k.shrink(a, 1)
    assert k.table([a])[0].tolist() == [[-1, -1]] and k.length(a) == 8
    assert k.table([])[0].shape == (0, 1)


def test_drafts_dropped_after_a_window_was_forgotten():
    """A shorter sequence's next query sees further back: what it would see must not have been given back."""
    for tokens, drafts, window, drop in [(106, 5, 64, 5), (200, 0, 64, 20)]:
        k = KvPages(40, 16)
        s = k.add()
        k.extend([s], [tokens + drafts])
        k.forget(s, window)
        before = k.table([s])[0]
        with pytest.raises(ValueError, match="forgotten"):
            k.shrink(s, drop)
        assert k.length(s) == tokens + drafts and torch.equal(k.table([s])[0], before)
        k.extend([s], [1])                                            # as long as it is not shortened it goes on
    # with room for the drafts they may be dropped, and every key that the next query sees is held
    k = KvPages(40, 16)
    s = k.add()
    k.extend([s], [111])
    k.forget(s, 64, drafts=5)
    k.shrink(s, 5)
    assert k.table([s])[0][0, 43 // 16:].min() >= 0 and k.table([s])[0][0, 1] == -1
    k.extend([s], [1])
    t = k.fork(s)
    with pytest.raises(ValueError, match="forgotten"):                # a fork has forgotten the same
        k.shrink(t, 20)
    with pytest.raises(ValueError):
        k.forget(s, 64, drafts=-1)
    # back to before anything forgotten, among the first tokens kept
    k = KvPages(40, 16)
    s = k.add()
    k.extend([s], [200])
    k.forget(s, 32, 20)
    k.shrink(s, 200 - 32)
    k.extend([s], [100])
    assert k.table([s])[0].min() >= 0
    # a sequence that holds no page any more has nothing to go on from
    k = KvPages(4, 4)
    s = k.add()
    k.extend([s], [9])
    k.forget(s, 2)
    k.shrink(s, 1)
    with pytest.raises(ValueError, match="forgotten"):
        k.extend([s], [1])
    assert k.length(s) == 8 and k.free_pages == 4
    k.shrink(s, 8)
    assert k.extend([s], [1])[0].tolist() == [2 * 4]


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("page", [1, 4, 16])
def test_a_window_never_loses_a_key(seed, page):
    """Each sequence with a window of its own, shortened at random: a shrink is refused exactly where the next query
    would see a forgotten token, and every new query's keys are in the table with what was written."""
    g = np.random.Generator(np.random.PCG64(100 + seed))
    m, sees = Model(120, page), {}
    shrunk = 0

    def missing(s, length):
        row = m.k.table([s])[0][0].tolist()
        window, sinks = sees[s]
        return [j for j in range(length) if (j > length - window or j < sinks) and row[j // page] < 0]
    for step in range(300):
        seqs = list(m.want)
        what = g.integers(0, 8)
        if not seqs or (what == 0 and len(seqs) < 6):
            s = m.k.add()
            m.want[s], sees[s] = [], (int(g.integers(1, 4 * page + 2)), int(g.integers(0, page + 2)))
            continue
        s = seqs[g.integers(len(seqs))]
        if what <= 2:
            n = int(g.integers(1, 2 * page + 3))
            try:
                lost = missing(s, len(m.want[s]))
                m.extend([s], [n], g)
                assert not lost
            except RuntimeError:
                m.k.free(s)
                del m.want[s], sees[s]
            except ValueError:
                assert lost and all(p < 0 for p in m.k.table([s])[0][0].tolist())
                m.k.free(s)
                del m.want[s], sees[s]
        elif what == 3:
            t = m.k.fork(s)
            m.want[t], sees[t] = list(m.want[s]), sees[s]
        elif what <= 5:
            window, sinks = sees[s]
            drafts = int(g.integers(0, page + 1))
            m.k.forget(s, window, sinks, drafts)
            n = len(m.want[s]) - drafts
            m.want[s] = [w if j < sinks or j > n - window else None for j, w in enumerate(m.want[s])]
        else:
            n = int(g.integers(0, min(len(m.want[s]), 2 * page) + 1))
            length = len(m.want[s]) - n
            lost, row = missing(s, length), m.k.table([s])[0][0].tolist()
            into = length % page and row[length // page] < 0
            try:
                m.k.shrink(s, n)
                shrunk += 1
                assert not into and (not lost or all(p < 0 for p in row[:-(-length // page)]))
                m.want[s] = m.want[s][:length]
            except ValueError:
                assert into or lost
        m.check()
    assert shrunk > 5
