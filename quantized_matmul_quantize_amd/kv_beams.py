"""Which pages of a 4-bit key/value cache hold which beam's tokens.

Host bookkeeping only, as ``KvPages`` is: several continuations (beams) of each
of some sequences, which ``kv4_beam_reorder`` moves from slot to slot on the
device.  Slot s * beams + b is beam b of sequence s; all beams of a sequence
have the same number of tokens.  A slot shares every page that is full and has
two tail pages of its own, one that it fills and a spare one that a parent's
tokens are copied to.  The host hears of the moves only when a page is full:
then it reads the table, gives back what no beam of the sequence names any more
and hands out two pages a slot.  (And when a beam was kept: a page that a kept
sequence ends in is no longer a slot's to copy to, which gets another one.)
"""
from __future__ import annotations

from typing import List, Optional, Sequence, Set, Tuple

import torch

from .kv_pages import KvPages, _ids

__all__ = ["KvBeams"]


class KvBeams:
    """beams continuations of each of the sequences seqs of a KvPages, up to `tokens` more tokens each.

    table (int32 [slots, width]), context (int32 [slots]) and tails (int32 [slots, 2]) are those at the start, on the
    CPU; src and dst (int64) the pages to copy before the first step (``kv4_copy_pages``: the page that a sequence ends
    in, once a slot).  groups and prefix (int32) are ``kv4_prefix_attention``'s.  The sequences stay as they are and may
    be freed meanwhile.  RuntimeError if there are not enough free pages; then nothing has changed."""

    def __init__(self, pages: KvPages, seqs: Sequence[int], beams: int, tokens: int):
        seqs = list(seqs)
        pages._check(seqs)
        if not seqs or beams < 1 or tokens < 0:
            raise ValueError(f"needs sequences, beams >= 1 and tokens >= 0, not {seqs}, {beams} and {tokens}")
        lengths = [pages.length(s) for s in seqs]
        for s, n in zip(seqs, lengths):
            if pages._sees_gone(s, n):
                raise ValueError(f"tokens that the next ones of sequence {s} see were forgotten")
        partial = [s for s, n in zip(seqs, lengths) if n % pages.page]
        if 2 * beams * len(partial) > len(pages._free):
            raise RuntimeError(f"out of pages: {2 * beams * len(partial)} needed, {len(pages._free)} of {pages.pages} free")
        self.pages, self.beams, self._length, self._tokens = pages, beams, lengths, [tokens] * len(seqs)
        self._prompts: Optional[List[int]] = [pages.fork(s) for s in seqs]      # hold the pages that are full
        self._own: List[Set[int]] = [set() for _ in seqs]
        self._kept: Set[int] = set()                    # tail pages that sequences which were kept end in
        width = max(1, max(-(-(n + tokens) // pages.page) for n in lengths))
        slots = len(seqs) * beams
        table = pages.table(self._prompts, width)[0].repeat_interleave(beams, 0)
        self.tails = torch.full((slots, 2), -1, dtype=torch.int32)
        src, dst = [], []
        for i, (s, n) in enumerate(zip(seqs, lengths)):
            if n % pages.page:
                last = pages._held[s][n // pages.page]
                self._hand_out(i)
                for slot in range(i * beams, i * beams + beams):
                    src.append(last)
                    dst.append(int(self.tails[slot, 0]))
                    table[slot, n // pages.page] = dst[-1]
        self.table, self.src, self.dst = table, _ids(src), _ids(dst)
        self.context = torch.tensor(lengths, dtype=torch.int32).repeat_interleave(beams)
        self.groups = torch.arange(0, slots + 1, beams, dtype=torch.int32)
        self.prefix = torch.tensor(lengths, dtype=torch.int32)
        pages._beams += 1

    def room(self, table: torch.Tensor) -> Optional[Tuple[torch.Tensor, torch.Tensor]]:
        """Before the append of each step: room for one more token of every beam, in the place table[slot, context //
        page] * page + context % page.  None where the slots have it; else the (table, tails) to go on with, on the CPU,
        made from the table as the beams were last moved (on any device: only then is it read).  So also where a beam was
        kept since the last call.  RuntimeError if there are not enough free pages; then nothing has changed."""
        self._alive()
        page, beams = self.pages.page, self.beams
        if table.shape != self.table.shape:
            raise ValueError(f"table has shape {tuple(table.shape)}, the beams' is {tuple(self.table.shape)}")
        if any(t <= 0 for t in self._tokens):
            raise ValueError("the beams have no room for more tokens")
        full = [i for i, n in enumerate(self._length) if n % page == 0]
        # (a full sequence's slots get two other pages in any case)
        taken = [(slot, t) for slot, pair in enumerate(self.tails.tolist() if self._kept else []) for t in range(2)
                 if pair[t] in self._kept and self._length[slot // beams] % page]
        out = None
        if full or taken:
            new, left, free = table.detach().to("cpu", copy=True), [], len(self.pages._free)
            for i in full:
                named = set(new[i * beams:i * beams + beams, :self._length[i] // page].flatten().tolist())
                strange = named - self._own[i] - set(self.pages._held[self._prompts[i]])
                if strange:
                    raise ValueError(f"the table names pages that sequence {i} does not hold: {sorted(strange)}")
                left.append(self._own[i] - named)
                free += sum(self.pages._users[p] == 1 for p in left[-1])       # (others may be kept)
            need = 2 * beams * len(full) + len(taken)
            if need > free:
                raise RuntimeError(f"out of pages: {need} needed, {free} of {self.pages.pages} free")
            for i, pages in zip(full, left):
                for p in sorted(pages, reverse=True):
                    self.pages._drop(p)
                self._own[i] -= pages
            self.tails = self.tails.clone()
            for i in full:
                self._hand_out(i)
                new[i * beams:i * beams + beams, self._length[i] // page] = self.tails[i * beams:i * beams + beams, 0]
            for slot, t in taken:
                self._tail(slot, t)
            out = new, self.tails
        self._kept.clear()
        self._length = [n + 1 for n in self._length]
        self._tokens = [t - 1 for t in self._tokens]
        return out

    def keep(self, table: torch.Tensor, slot: int) -> int:
        """A beam, with the tokens that the row table[slot] holds now, as a sequence of its own of the KvPages; returns its
        id.  The search may go on: the page that the sequence ends in is nobody's to copy to from the next `room` on."""
        self._alive()
        if not 0 <= slot < self.table.shape[0]:
            raise ValueError(f"no slot {slot} of {self.table.shape[0]}")
        i, pages = slot // self.beams, self.pages
        row = table[slot, :-(-self._length[i] // pages.page)].tolist()
        strange = set(row) - self._own[i] - set(pages._held[self._prompts[i]])
        if strange:
            raise ValueError(f"the table names pages that sequence {i} does not hold: {sorted(strange)}")
        seq = pages.add()
        pages._held[seq], pages._length[seq], pages._gone[seq] = row, self._length[i], dict(pages._gone[self._prompts[i]])
        for p in row:
            if p >= 0:
                pages._users[p] += 1
        if self._length[i] % pages.page and row[-1] in self._own[i]:
            self._kept.add(row[-1])
        return seq

    def free(self) -> None:
        """Give back the pages of all beams, but for those that were kept."""
        self._alive()
        for i, seq in enumerate(self._prompts):
            self.pages.free(seq)
            for p in sorted(self._own[i], reverse=True):
                self.pages._drop(p)
        self._prompts = None
        self.pages._beams -= 1

    def _alive(self) -> None:
        if self._prompts is None:
            raise ValueError("the beams were freed")

    def _hand_out(self, i: int) -> None:
        """Two pages to each slot of sequence i."""
        for slot in range(i * self.beams, i * self.beams + self.beams):
            for t in range(2):
                self._tail(slot, t)

    def _tail(self, slot: int, t: int) -> None:
        self.tails[slot, t] = page = self.pages._take()
        self._own[slot // self.beams].add(page)
