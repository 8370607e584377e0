"""Beam search over a 4-bit key/value cache, end to end on one GPU.

Prompts are read in chunks; then the beams of each of them decode together,
with the prompt's keys and values taken for all of its beams. Every step
of a layer, and every step of the search, is one library call:

    q, k, v   w4a16_gemv / w4a16_gemm
    q, cache  kv4_rope_append (norms, rotation by position, keys and values)
    o         kv4_prefix_attention
    y         w4a16_gemv / w4a16_gemm

    beams     beam_select on the logits
    cache     kv4_beam_reorder; KvBeams hands out pages as they fill up

A step is captured once and replayed: nothing in it depends on the host.
Weights are random, so the figures are times and not text:

    python examples/kv4_beams.py --sequences 8 --beams 4 --prompt 4000 --steps 64
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from kv4_decode import Decoder, project, qmm  # noqa: E402


class BeamSearch:
    """beams continuations of each of the sequences seqs of a Decoder, by `embed` [vocabulary, hidden] and a 4-bit head."""

    def __init__(self, model: Decoder, seqs, beams, steps, embed, head, last, end=-1):
        """last [sequences, hidden]: each prompt's last row, from which the first tokens are chosen."""
        self.model, self.embed, self.head, self.end = model, embed, head, end
        self.seqs, self.beams = len(seqs), beams
        self.host = qmm.KvBeams(model.pages, seqs, beams, steps)
        model.copy(self.host.src, self.host.dst)
        self.table, self.context, self.tails, self.groups, self.prefix = (
            t.cuda() for t in (self.host.table, self.host.context, self.host.tails, self.host.groups, self.host.prefix))
        self.hints = dict(max_group=beams, max_prefix=max(1, int(self.host.prefix.max())), max_tail=max(1, steps))
        self.scores = torch.full((self.seqs, beams), -torch.inf, device="cuda")
        self.scores[:, 0] = 0.0                              # one beam until the first choice
        self.finished = torch.zeros((self.seqs, beams), dtype=torch.bool, device="cuda")
        self.history, self.graph = [], None
        self.choose(last.repeat_interleave(beams, 0))
        self.last = self.tokens.clone()
        self.record()

    def choose(self, x):
        """The next tokens from rows x; beams go on from their parents."""
        scores, tokens, parents = qmm.beam_select(project(self.head, x), self.scores, finished=self.finished, pad=max(0, self.end))
        table, context = qmm.kv4_beam_reorder(self.model.cache, self.model.D, self.table, self.context, self.tails, parents)
        for mine, new in ((self.table, table), (self.context, context), (self.scores, scores),
                          (self.finished, self.finished.gather(1, parents) | (tokens == self.end))):
            mine.copy_(new)
        self.tokens, self.parents = tokens, parents

    def rows(self, x):
        """Rows x of the slots through every layer; their keys and values are appended."""
        m, T = self.model, x.shape[0]
        page = self.model.pages.page
        at = self.context.long()
        slots = self.table.gather(1, (at // page)[:, None])[:, 0] * page + at % page
        self.context += 1
        for layer, cache in zip(m.layers, m.cache):
            h = x * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6).to(x.dtype)
            q, k, v = project(layer["qkv"], h).view(T, -1, m.D).split([m.hq, m.hk, m.hk], 1)
            q = qmm.kv4_rope_append(q, k, v, slots, cache, at, m.table, layer["qw"], layer["kw"])
            o = qmm.kv4_prefix_attention(q, cache, self.table, self.context, self.groups, self.prefix, **self.hints)
            x = x + project(layer["out"], o.view(T, -1))
        return x

    def body(self):
        self.choose(self.rows(self.embed[self.last.view(-1)]))
        self.last.copy_(self.tokens)

    def record(self):
        self.history.append((self.tokens.clone(), self.parents.clone()))

    def step(self, graph=True):
        """One more token of every beam."""
        grown = self.host.room(self.table)
        if grown is not None:
            self.table.copy_(grown[0])
            self.tails.copy_(grown[1])
        if not graph or len(self.history) == 1:              # (the first step runs by itself)
            self.body()
        else:
            if self.graph is None:
                self.graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(self.graph):
                    self.body()
            self.graph.replay()
        self.record()

    def best(self):
        """(scores [sequences, beams], tokens [sequences, beams, steps]) of the beams, the best first."""
        at = torch.arange(self.beams, device="cuda").expand(self.seqs, -1)
        out = []
        for tokens, parents in reversed(self.history):
            out.append(tokens.gather(1, at))
            at = parents.gather(1, at)
        return self.scores, torch.stack(out[::-1], 2)


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in dict(layers=4, hidden=4096, q_heads=32, kv_heads=8, head_dim=128, page=64, group=64, sequences=8,
                            beams=4, prompt=4000, chunk=1024, steps=64, vocabulary=32000, seed=0).items():
        p.add_argument("--" + name.replace("_", "-"), type=int, default=value)
    a = p.parse_args(argv)
    whole, tail = -(-a.prompt // a.page), -(-a.steps // a.page) + 1
    model = Decoder(a.layers, a.hidden, a.q_heads, a.kv_heads, a.head_dim, a.sequences * (whole + a.beams * 3 * tail) + 8,
                    a.page, a.group, rows=a.prompt + a.steps + 1, seed=a.seed)
    g = torch.Generator(device="cuda").manual_seed(a.seed + 1)
    normal = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    embed = normal(a.vocabulary, a.hidden)
    head = qmm.quantize_groupwise(normal(a.vocabulary, a.hidden) * a.hidden ** -0.5)
    seqs, last = [model.pages.add() for _ in range(a.sequences)], []
    for s in seqs:
        for at in range(0, a.prompt, a.chunk):
            x = model.step([s], normal(min(a.chunk, a.prompt - at), a.hidden), [min(a.chunk, a.prompt - at)])
        last.append(x[-1:])
    search = BeamSearch(model, seqs, a.beams, a.steps, embed, head, torch.cat(last))
    for _ in range(min(2, a.steps)):
        search.step()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps - 2):
        search.step()
    torch.cuda.synchronize()
    t = (time.perf_counter() - t) / max(1, a.steps - 2)
    print(f"search: {a.sequences} x {a.beams} beams after {a.prompt} tokens on {model.pages.pages - model.pages.free_pages} pages, "
          f"{a.layers} layers, {t * 1e3:.2f} ms a step", flush=True)
    return search.best()


if __name__ == "__main__":
    main()
