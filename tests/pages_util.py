"""Plain model of the page tables for the tests: lists and loops, straight from
include/kvq.h ("Page tables")."""
from __future__ import annotations

import numpy as np
import torch

from bit_kv_cache_14_gb300 import kvq


class Model:
    """What the device tables have to be after each call."""

    def __init__(self, n_pages, page, n_seqs, width):
        self.n_pages, self.page, self.width = n_pages, page, width
        self.rows = [[] for _ in range(n_seqs)]
        self.lens = [0] * n_seqs

    def entries(self, n):
        return -(-n // self.page)

    @property
    def refs(self):
        refs = np.zeros(self.n_pages, np.int32)
        for r in self.rows:
            for i in r:
                refs[i] += 1
        return refs

    def reserve(self, n):
        """The copies, or None where the call fails and nothing changes."""
        refs = self.refs
        free = list(np.flatnonzero(refs == 0))
        begun = {}
        for b, m in enumerate(n):
            if m and self.lens[b] % self.page and refs[self.rows[b][-1]] > 1:
                begun.setdefault(self.rows[b][-1], []).append(b)
        copying = set()
        for i, who in begun.items():
            copying.update(who[1:] if len(who) == refs[i] else who)
        need = [(self.entries(k + m) - self.entries(k) if m else 0) + (b in copying)
                for b, (k, m) in enumerate(zip(self.lens, n))]
        if sum(need) > len(free) or any(m and k + m > self.width * self.page
                                        for k, m in zip(self.lens, n)):
            return None
        copies = []
        for b, m in enumerate(n):
            if not m:
                continue
            if b in copying:
                i = int(free.pop(0))
                copies.append((self.rows[b][-1], i))
                self.rows[b][-1] = i
            self.lens[b] += m
            while len(self.rows[b]) < self.entries(self.lens[b]):
                self.rows[b].append(int(free.pop(0)))
        return copies

    def drop(self, tokens):
        for b, m in enumerate(tokens):
            self.lens[b] -= min(max(m, 0), self.lens[b])
            del self.rows[b][self.entries(self.lens[b]):]

    def select(self, parents):
        rows, lens = [list(r) for r in self.rows], list(self.lens)
        for b, a in enumerate(parents):
            if -1 <= a < len(rows):
                self.rows[b] = list(rows[a]) if a >= 0 else []
                self.lens[b] = lens[a] if a >= 0 else 0

    def compact(self):
        refs = self.refs
        front = int((refs > 0).sum())
        src = [i for i in range(front, self.n_pages) if refs[i]]
        dst = [i for i in range(front) if not refs[i]]
        to = dict(zip(src, dst))
        self.rows = [[to.get(i, i) for i in r] for r in self.rows]
        return list(zip(src, dst))

    # ---- against the device
    def table(self):
        t = np.full((len(self.rows), self.width), -1, np.int32)
        for b, r in enumerate(self.rows):
            t[b, :len(r)] = r
        return t

    def check(self, tab):
        refs = self.refs
        assert np.array_equal(tab.seq_lens.cpu().numpy(), np.array(self.lens, np.int32))
        assert np.array_equal(tab.block_table.cpu().numpy(), self.table())
        assert np.array_equal(tab.page_refs.cpu().numpy(), refs)
        assert int(tab.free_pages) == int((refs == 0).sum())
        # the free map (behind the 16-byte head of the state), and where it begins
        words = -(-self.n_pages // 32)
        bits = np.unpackbits(tab.state[16:16 + 4 * words].cpu().numpy(), bitorder="little")
        assert np.array_equal(bits[:self.n_pages], (refs == 0).astype(np.uint8))
        assert not bits[self.n_pages:].any()
        hint = int(tab.state[4:8].view(torch.int32))
        free = np.flatnonzero(refs == 0)
        assert len(free) == 0 or hint <= free[0] // 32


def i32(x, device="cuda"):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=device)


def cu_of(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


def pairs_of(copies, rows):
    out = np.full((rows, 2), -1, np.int32)
    out[:len(copies)] = np.array(copies, np.int32).reshape(-1, 2)
    return out


def both(n_pages, page, n_seqs, width):
    return (Model(n_pages, page, n_seqs, width),
            kvq.PageTable(n_pages, page, n_seqs=n_seqs, width=width))
