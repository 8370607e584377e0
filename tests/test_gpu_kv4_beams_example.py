"""The beam search example: append, attention over shared prompts, selection and reordering together, each call of a run
against its plain form on the very inputs it got."""
import importlib.util
import os
import sys

import pytest
import torch

import quantized_matmul_quantize_amd as qmm

pytestmark = pytest.mark.gpu
folder = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples")


def load(name):
    spec = importlib.util.spec_from_file_location(name, os.path.join(folder, name + ".py"))
    module = importlib.util.module_from_spec(spec)
    sys.path.insert(0, folder)
    try:
        spec.loader.exec_module(module)
    finally:
        sys.path.remove(folder)
    return module


example = load("kv4_beams")
VOCABULARY = 1504


def search(beams, steps, lengths, D=64, group=32, page=16, end=-1, **kw):
    model = example.Decoder(**{**dict(layers=2, hidden=512, q_heads=8, kv_heads=2, head_dim=D, pages=300, page=page, group=group,
                                      rows=512, seed=3), **kw})
    g = torch.Generator(device="cuda").manual_seed(4)
    normal = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    embed, head = normal(VOCABULARY, 512), qmm.quantize_groupwise(normal(VOCABULARY, 512) / 8)
    seqs = [model.pages.add() for _ in lengths]
    last = torch.cat([model.step([s], normal(n, 512), [n])[-1:] for s, n in zip(seqs, lengths)])
    return example.BeamSearch(model, seqs, beams, steps, embed, head, last, end=end), model


class Checked:
    """In place of the library's calls: each is made, then held against plain ones."""

    def __init__(self, monkeypatch, page):
        self.page, self.calls, self.chosen = page, {}, []
        for name in ("kv4_rope_append", "kv4_prefix_attention", "beam_select", "kv4_beam_reorder"):
            monkeypatch.setattr(qmm, name, lambda *a, _own=getattr(qmm, name), _name=name, **kw: self.call(_name, _own, a, kw))

    def call(self, name, own, a, kw):
        self.calls[name] = self.calls.get(name, 0) + 1
        return getattr(self, name)(own, *a, **kw)

    def read(self, cache, table, context, D):
        """Keys and values of each row of the table, as they would be read."""
        out = []
        for row, n in zip(table.tolist(), context.tolist()):
            slots = [row[j // self.page] * self.page + j % self.page for j in range(n)]
            out.append(qmm.kv4_read(cache, torch.tensor(slots, device="cuda"), D, torch.float32))
        return out

    def kv4_rope_append(self, own, q, k, v, slots, cache, positions, table, qw, kw):
        got = own(q, k, v, slots, cache, positions, table, qw, kw)
        q_want, k_want = qmm.qk_norm_rope(q.clone(), k.clone(), positions, table, qw, kw)
        assert torch.equal(got, q_want)
        keys, values = qmm.kv4_read(cache, slots, k.shape[2], torch.float32)
        # half a step of a group's 15, the scale's own rounding (2^-11 of 15 steps) and the key's rounding to bf16
        for x, y, extra in ((keys, k_want.float(), 2.0 ** -8), (values, v.float(), 0.0)):
            x, y = x.unflatten(2, (-1, self.group)), y.unflatten(2, (-1, self.group))
            span = y.amax(3, keepdim=True).clamp(min=0) - y.amin(3, keepdim=True).clamp(max=0)
            most = y.abs().amax(3, keepdim=True)
            assert ((x - y).abs() <= span * (1 + 2.0 ** -7) / 15 + (2.0 ** -10 + 2 * extra) * most).all()
        return got

    def kv4_prefix_attention(self, own, q, cache, table, context, groups, prefix, **hints):
        got = own(q, cache, table, context, groups, prefix, **hints)
        want = qmm.kv4_attention(q, cache, table, context)
        mass = max(float(v.abs().max()) for _, v in self.read(cache, table, context, q.shape[2]))
        # each is within 2^-11 of the mass (and 64 roundings where parts are joined) and an output rounding of fp64
        bound = 2 * (2.0 ** -11 + 64 * 2.0 ** -24) * mass + 2 * 2.0 ** -9 * (want.float().abs() + 2.0 ** -8)
        assert ((got.float() - want.float()).abs() <= bound).all()
        return got

    def beam_select(self, own, logits, scores, finished=None, pad=0):
        best, tokens, parents = got = own(logits, scores, finished=finished, pad=pad)
        seqs, beams = scores.shape
        every = logits.double().log_softmax(1).view(seqs, beams, -1)
        done = torch.full_like(every, -torch.inf)
        done[:, :, pad] = 0.0
        every = (torch.where(finished[:, :, None], done, every) + scores.double()[:, :, None]).flatten(1)
        want = every.topk(beams, 1)[0]
        tolerance = 2.0 ** -18 + 2.0 ** -22 * want.abs().clamp(max=1e30)
        assert ((best - want).abs() <= tolerance).all()
        flat = parents * logits.shape[1] + tokens
        assert ((every.gather(1, flat) - want).abs() <= tolerance).all()
        assert all(len(set(row)) == beams for row in flat.tolist())
        self.chosen.append((tokens.cpu(), parents.cpu()))
        return got

    def kv4_beam_reorder(self, own, cache, D, table, context, tails, parents):
        before = [self.read(layer, table, context, D) for layer in cache]
        new, lengths = own(cache, D, table, context, tails, parents)
        after = [self.read(layer, new, lengths, D) for layer in cache]
        source = (torch.arange(parents.shape[0], device="cuda")[:, None] * parents.shape[1] + parents).flatten().tolist()
        assert lengths.tolist() == [context.tolist()[s] for s in source]
        for was, now in zip(before, after):
            for slot, s in enumerate(source):
                assert torch.equal(was[s][0], now[slot][0]) and torch.equal(was[s][1], now[slot][1])
        return new, lengths


@pytest.mark.parametrize("beams,lengths,D,group,page", [(4, [45, 32, 7], 64, 32, 16), (3, [130], 128, 64, 64), (1, [5, 16], 64, 64, 16)])
def test_every_call_of_a_search(beams, lengths, D, group, page, monkeypatch):
    checked = Checked(monkeypatch, page)
    checked.group = group
    run, model = search(beams, 36, lengths, D, group, page)
    for _ in range(36):
        run.step(graph=False)
    assert checked.calls == {"kv4_rope_append": 72, "kv4_prefix_attention": 72, "beam_select": 37, "kv4_beam_reorder": 37}
    want = [[[] for _ in range(beams)] for _ in lengths]
    for tokens, parents in checked.chosen:
        want = [[want[s][p] + [t] for t, p in zip(tokens[s].tolist(), parents[s].tolist())] for s in range(len(lengths))]
    scores, tokens = run.best()
    assert tokens.tolist() == want and (scores[:, :-1] >= scores[:, 1:]).all()
    assert run.context.view(-1, beams).tolist() == [[n + 36] * beams for n in lengths]
    kept = run.host.keep(run.table, 0)
    run.host.free()
    assert model.pages.length(kept) == lengths[0] + 36


@pytest.mark.parametrize("beams,lengths", [(4, [45, 32, 7]), (8, [100])])
def test_replayed_steps_are_the_eager_ones(beams, lengths):
    runs = [search(beams, 40, lengths)[0] for _ in range(2)]
    for _ in range(40):
        for run, graph in zip(runs, (True, False)):
            run.step(graph=graph)
    (a, x), (b, y) = (run.best() for run in runs)
    assert torch.equal(a, b) and torch.equal(x, y) and torch.equal(runs[0].context, runs[1].context)


def test_finished_beams_stay_as_they_are():
    plain = search(3, 1, [45])[0]
    end = int(plain.tokens[0, 1])                            # a first choice ends at once
    run = search(3, 20, [45], end=end)[0]
    score = float(run.scores[0, 1])
    for _ in range(20):
        run.step(graph=False)
    scores, tokens = run.best()
    ended = [row for row in tokens[0].tolist() if row[0] == end]
    assert ended and ended[0] == [end] * 21 and score in scores[0].tolist()


def test_the_example_runs():
    scores, tokens = example.main(["--layers", "2", "--hidden", "512", "--q-heads", "8", "--kv-heads", "2", "--head-dim", "64",
                                   "--page", "16", "--group", "32", "--sequences", "3", "--beams", "4", "--prompt", "100",
                                   "--chunk", "64", "--steps", "40", "--vocabulary", "1000"])
    assert tokens.shape == (3, 4, 41) and scores.isfinite().all()


@pytest.mark.parametrize("graph", [False, True], ids=["eager", "replayed"])
@pytest.mark.parametrize("beams,lengths,page", [(4, [45, 32, 7], 16), (3, [100], 64)])
def test_kept_beams_outlive_the_moves_of_their_slots(beams, lengths, page, graph):
    """Set aside after some steps, in the middle of a page, and read again when the search is over."""
    run, model = search(beams, 40, lengths, page=page)

    def read(seq):
        row, n = model.pages.table([seq])
        at = torch.arange(int(n))
        slots = (row[0, at // page].long() * page + at % page).cuda()
        return [x for cache in model.cache for x in qmm.kv4_read(cache, slots, 64, torch.float32)]

    kept = []
    for step in range(40):
        run.step(graph=graph)
        if step in (2, 3, 9, 17, 30):
            kept += [(seq, read(seq)) for seq in (run.host.keep(run.table, slot) for slot in (0, beams - 1))]
    for seq, was in kept:
        assert all(torch.equal(x, y) for x, y in zip(read(seq), was))
    run.host.free()
