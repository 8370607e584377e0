"""Which pages of a 4-bit key/value cache hold which sequence's tokens.

Host bookkeeping only, in plain integers: it allocates nothing on a device and
launches nothing.  Its tensors are the operands of ``kv4_append`` (slots),
``kv4_attention`` (page table and contexts) and ``kv4_copy_pages`` (pairs of
pages), on the CPU; the caller copies them to the cache's device.

Sequences share pages after a fork.  A shared page is only read: a sequence
that extends into one gets a copy of its own first, so ``extend`` returns pairs
of pages to copy before the append.
"""
from __future__ import annotations

from typing import Dict, List, Optional, Sequence, Tuple

import torch

__all__ = ["KvPages"]


def _ids(values) -> torch.Tensor:
    return torch.tensor(values, dtype=torch.int64)


class KvPages:
    def __init__(self, pages: int, page: int = 64):
        if pages < 1 or page < 1:
            raise ValueError(f"pages and page must be positive, not {pages} and {page}")
        self.pages, self.page = pages, page
        self._free: List[int] = list(range(pages - 1, -1, -1))     # the lowest id is taken first
        self._users = [0] * pages                                  # sequences that hold the page
        self._held: Dict[int, List[int]] = {}                      # pages of a sequence, -1 where forgotten
        self._length: Dict[int, int] = {}
        self._gone: Dict[int, Dict[int, Tuple[int, int]]] = {}     # by window: the tokens that it let go, first and end
        self._next = 0
        self._beams = 0                                            # KvBeams that hold pages too

    @property
    def free_pages(self) -> int:
        return len(self._free)

    def length(self, seq: int) -> int:
        """Tokens of a sequence."""
        self._check([seq])
        return self._length[seq]

    def add(self) -> int:
        """A new sequence of no tokens; returns its id."""
        seq, self._next = self._next, self._next + 1
        self._held[seq], self._length[seq], self._gone[seq] = [], 0, {}
        return seq

    def extend(self, seqs: Sequence[int], counts: Sequence[int]) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
        """Room for counts[i] more tokens of sequence seqs[i].  Returns (slots, src, dst), int64: the slots of the new
        tokens in the order of seqs, and the pages to copy (src to dst) before anything is appended to the slots.
        RuntimeError if there are not enough free pages, ValueError if a sequence has been shortened to where its new
        tokens would see forgotten ones; then nothing has changed."""
        seqs, counts = list(seqs), list(counts)
        self._check(seqs)
        if len(counts) != len(seqs) or any(n < 0 for n in counts):
            raise ValueError(f"needs a count >= 0 for each of {len(seqs)} sequences, not {counts}")
        for seq, n in zip(seqs, counts):
            if n and self._sees_gone(seq, self._length[seq]):
                raise ValueError(f"tokens that the next ones of sequence {seq} see were forgotten")
        need, left = 0, {}                                         # users left of a page, as copies are made
        for seq, n in zip(seqs, counts):
            need += -(-(self._length[seq] + n) // self.page) - len(self._held[seq])
            shared = self._shared(seq, n, left)
            if shared is not None:
                need += 1
                left[shared] = left.get(shared, self._users[shared]) - 1
        if need > len(self._free):
            raise RuntimeError(f"out of pages: {need} needed, {len(self._free)} of {self.pages} free")
        slots, src, dst = [], [], []
        for seq, n in zip(seqs, counts):
            held, start = self._held[seq], self._length[seq]
            shared = self._shared(seq, n, {})
            if shared is not None:
                own = self._take()
                src.append(shared)
                dst.append(own)
                self._users[shared] -= 1
                held[start // self.page] = own
            while len(held) * self.page < start + n:
                held.append(self._take())
            at = torch.arange(start, start + n)
            if n:
                first = start // self.page
                slots.append(_ids(held[first:])[at // self.page - first] * self.page + at % self.page)
            self._length[seq] = start + n
        return torch.cat(slots) if slots else _ids([]), _ids(src), _ids(dst)

    def shrink(self, seq: int, n: int) -> None:
        """Drop the last n tokens (such as drafts that were not accepted).  ValueError, and nothing has changed, where
        the next token would then see forgotten ones (`forget` with `drafts` keeps them); only a sequence that is left
        without any page may be shortened that far, to be freed or shortened on."""
        self._check([seq])
        if not 0 <= n <= self._length[seq]:
            raise ValueError(f"cannot drop {n} of {self._length[seq]} tokens")
        length = self._length[seq] - n
        held, keep = self._held[seq], -(-length // self.page)
        if length % self.page and held[keep - 1] < 0:
            raise ValueError("cannot shrink into a page that was forgotten")
        if self._sees_gone(seq, length) and any(page >= 0 for page in held[:keep]):
            raise ValueError(f"cannot drop {n} tokens: the window would reach tokens that were forgotten")
        self._length[seq] = length
        self._gone[seq] = {w: (a, min(b, length)) for w, (a, b) in self._gone[seq].items() if a < length}
        for page in held[keep:]:
            self._drop(page)
        del held[keep:]

    def forget(self, seq: int, window: int, sinks: int = 0, drafts: int = 0) -> None:
        """Give back the pages that no later query sees: whole pages before the last `window` tokens and after the
        first `sinks`.  They stay in the table as -1.  The last `drafts` tokens may still be dropped (`shrink`): what
        the query in the place of the first of them sees is kept too."""
        self._check([seq])
        if window < 1 or sinks < 0 or drafts < 0:
            raise ValueError(f"needs window >= 1, sinks >= 0 and drafts >= 0, not {window}, {sinks} and {drafts}")
        held = self._held[seq]
        # the next query stands at position length and sees keys from length - window + 1 on
        last = max(0, self._length[seq] - drafts - window + 1) // self.page
        gone = [i for i in range(-(-sinks // self.page), last) if held[i] >= 0]
        for i in gone:
            self._drop(held[i])
            held[i] = -1
        if gone:
            first, end = self._gone[seq].get(window, (gone[0] * self.page, 0))
            self._gone[seq][window] = min(first, gone[0] * self.page), max(end, (gone[-1] + 1) * self.page)

    def fork(self, seq: int) -> int:
        """A new sequence of the same tokens, in the same pages; returns its id."""
        self._check([seq])
        new = self.add()
        self._held[new], self._length[new], self._gone[new] = list(self._held[seq]), self._length[seq], dict(self._gone[seq])
        for page in self._held[new]:
            if page >= 0:
                self._users[page] += 1
        return new

    def free(self, seq: int) -> None:
        """Forget a sequence; pages that no other one holds are free again."""
        self._check([seq])
        for page in self._held.pop(seq):
            self._drop(page)
        del self._length[seq], self._gone[seq]

    def compact(self) -> Tuple[torch.Tensor, torch.Tensor]:
        """Move the pages in use to the lowest ids.  Returns (src, dst), int64, to copy before the next append or
        attention; no page is both.  ValueError while there are KvBeams, whose tables are on the device."""
        if self._beams:
            raise ValueError("beams hold pages that cannot be moved")
        used = self.pages - len(self._free)
        to = sorted(page for page in self._free if page < used)
        move = dict(zip((page for page in range(used, self.pages) if self._users[page]), to))
        for held in self._held.values():
            held[:] = [move.get(page, page) for page in held]
        for a, b in move.items():
            self._users[b], self._users[a] = self._users[a], 0
        self._free = list(range(self.pages - 1, used - 1, -1))
        return _ids(list(move.keys())), _ids(list(move.values()))

    def table(self, seqs: Sequence[int], width: Optional[int] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """(page_table int32 [len(seqs), width], context int32 [len(seqs)]) of sequences, the table as wide as the
        longest needs (at least 1), or `width`."""
        seqs = list(seqs)
        self._check(seqs, distinct=False)
        longest = max([1] + [len(self._held[s]) for s in seqs])
        if width is not None and width < longest:
            raise ValueError(f"a table of {longest} pages does not fit a width of {width}")
        width = longest if width is None else width
        rows = [self._held[s] + [-1] * (width - len(self._held[s])) for s in seqs]
        return (torch.tensor(rows, dtype=torch.int32).reshape(len(seqs), width),
                torch.tensor([self._length[s] for s in seqs], dtype=torch.int32))

    def shared(self, seqs: Sequence[int]) -> Tuple[torch.Tensor, torch.Tensor]:
        """(groups int32 [n + 1], prefix int32 [n]) of ``kv4_prefix_attention``: of the sequences in their order, runs
        with pages in common, and the tokens in the pages that all of a run have in common; cut so that the most tokens
        need not be read again (two prompts that begin with the same page of text, with samples of each, are two runs)."""
        seqs = list(seqs)
        self._check(seqs, distinct=False)
        count = len(seqs)
        common = [0] * count                                       # tokens that a sequence shares with the one before
        for i in range(1, count):
            a, b = seqs[i - 1], seqs[i]
            mine, theirs = self._held[b], self._held[a]
            if mine and theirs and mine[0] == theirs[0] >= 0:
                same = next((k for k, (x, y) in enumerate(zip(mine, theirs)) if x != y), min(len(mine), len(theirs)))
                common[i] = min(same * self.page, self._length[a], self._length[b])
        # Of the first j sequences: the most that is saved, and where the last run starts.  That is, of all starts i,
        # saved[i] + (j - 1 - i) n with n the least in common from i on.  Starts are kept by n, which rises; of those with
        # the same only the ones that no later start beats (as n falls, the later ones gain).
        saved, begin = [0] * (count + 1), [0] * (count + 1)
        starts: List[Tuple[int, List[int]]] = []
        for j in range(1, count + 1):
            saved[j], begin[j] = saved[j - 1], j - 1               # a run of one
            n = common[j - 1]
            if n == 0:
                starts = []
                continue
            merged = [j - 2]
            while starts and starts[-1][0] >= n:
                merged = starts.pop()[1] + merged
            kept: List[int] = []
            for i in reversed(merged):
                if not kept or saved[i] - i * n >= saved[kept[-1]] - kept[-1] * n:
                    kept.append(i)
            starts.append((n, kept[::-1]))
            for least, (i, *_) in reversed(starts):
                now = saved[i] + (j - 1 - i) * least
                if now >= saved[j]:
                    saved[j], begin[j] = now, i
        groups, j = [], count
        while j:
            i = begin[j]
            groups.append((i, self._length[seqs[i]] if j - i == 1 else min(common[i + 1:j])))
            j = i
        groups.reverse()
        return (torch.tensor([i for i, _ in groups] + [count], dtype=torch.int32),
                torch.tensor([n for _, n in groups], dtype=torch.int32))

    def _check(self, seqs, distinct: bool = True) -> None:
        for seq in seqs:
            if seq not in self._held:
                raise ValueError(f"no sequence {seq}")
        if distinct and len(set(seqs)) != len(seqs):
            raise ValueError(f"a sequence twice in {seqs}")

    def _sees_gone(self, seq: int, position: int) -> bool:
        """Whether a query at `position` sees tokens before it that were forgotten, by the windows that let them go."""
        return any(first < position and min(end, position) - 1 > position - window
                   for window, (first, end) in self._gone[seq].items())

    def _shared(self, seq: int, n: int, left: Dict[int, int]) -> Optional[int]:
        """The page that the next of n tokens falls into, if others hold it too."""
        if n == 0 or self._length[seq] % self.page == 0:
            return None
        page = self._held[seq][self._length[seq] // self.page]
        return page if left.get(page, self._users[page]) > 1 else None

    def _take(self) -> int:
        page = self._free.pop()
        self._users[page] = 1
        return page

    def _drop(self, page: int) -> None:
        if page >= 0:
            self._users[page] -= 1
            if self._users[page] == 0:
                self._free.append(page)
