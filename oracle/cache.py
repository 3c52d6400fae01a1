"""CPU oracle for the 8-bit latent cache and the pages of a paged cache.

TEST INFRASTRUCTURE ONLY.  It shares no code with the CUDA library.

The 8-bit cache (float64 numpy): cache row r has the value
scale[r // g] * e4m3(codes[r]); ``quantize_append`` is the append as the header
defines it.  Attention over the cache is ``dsa_ref.sparse_mla`` on the values.

The pages (Python ints, one entry after the other): ``resize``, ``fork`` and
``compact`` on a page table, sequence lengths and reference counts.

Pins (tests/test_oracle_cache.py): exact rational arithmetic, PyTorch's casts,
and invariants of a pool (every page's count equals the number of sequences
that hold it; what a sequence reads is what was written to it).
"""
from __future__ import annotations

import math

import numpy as np

from .dsa_ref import e4m3_decode, e4m3_encode_rne

E4M3_MAX = 448.0
MIN_EXP, MAX_EXP = -100, 100


def need_exponent(amax: float) -> int:
    """Smallest e in [-100, 100] with 448 * 2^e >= amax (100 if there is none)."""
    for e in range(MIN_EXP, MAX_EXP + 1):
        if E4M3_MAX * math.ldexp(1.0, e) >= amax:
            return e
    return MAX_EXP


def values(codes: np.ndarray, scale: np.ndarray, g: int) -> np.ndarray:
    """float64 values of every cache row."""
    return e4m3_decode(codes) * np.repeat(scale.astype(np.float64), g)[:codes.shape[0], None]


def _encode(x: np.ndarray) -> np.ndarray:
    """float64 -> E4M3 codes: nearest even, saturating, NaN kept."""
    return np.where(np.isnan(x), 0x7F, e4m3_encode_rne(np.where(np.isnan(x), 0.0, np.clip(x, -E4M3_MAX, E4M3_MAX))))


def quantize_append(codes, scale, g, kv, q_seq, q_pos, row_of):
    """codes uint8 [rows, 576], scale [rows / g], kv float64 [T, 576]; row_of(seq, pos)
    is the cache row.  Returns new (codes, scale)."""
    codes, scale = codes.copy(), scale.astype(np.float64).copy()
    blocks = {}
    for t in range(len(q_pos)):
        blocks.setdefault((int(q_seq[t]), int(q_pos[t]) // g), []).append(t)
    for (seq, blk), ts in blocks.items():
        new = kv[ts]
        finite = np.abs(new[np.isfinite(new)])
        s = math.ldexp(1.0, need_exponent(float(finite.max()) if finite.size else 0.0))
        p0 = min(int(q_pos[t]) for t in ts)
        b = row_of(seq, blk * g) // g
        if p0 > blk * g:
            old = scale[b]
            if 2.0 ** MIN_EXP <= old <= 2.0 ** MAX_EXP:
                if s > old:
                    rows = [row_of(seq, x) for x in range(blk * g, p0)]
                    codes[rows] = _encode(e4m3_decode(codes[rows]) * (old / s))
                else:
                    s = float(old)
        for t in ts:
            codes[row_of(seq, int(q_pos[t]))] = _encode(kv[t] / s)
        scale[b] = s
    return codes, scale


# ------------------------------------------------------------------- pages
class Pool:
    """A page state on the host; calls change it in place and return the page copies
    (from, to) that go with them."""

    def __init__(self, table, lens, refs, page_size):
        self.table, self.lens, self.refs = np.array(table), np.array(lens), np.array(refs)
        self.P = page_size
        self.bad = False          # an entry was skipped
        self.no_pages = False

    def pages(self, n: int) -> int:
        return -(-int(n) // self.P)

    def resize(self, seqs, new_len):
        S, pps = self.table.shape
        seen, entries, copies = set(), [], []
        for s, n in zip(map(int, seqs), map(int, new_len)):
            if s in seen or not 0 <= s < S or not 0 <= n <= pps * self.P:
                self.bad = True
                if 0 <= s < S:
                    seen.add(s)
                continue
            seen.add(s)
            entries.append((s, n, int(self.lens[s])))
        for s, n, old in entries:
            if n <= old:
                for j in range(self.pages(n), self.pages(old)):
                    self.refs[self.table[s, j]] -= 1
                    self.table[s, j] = -1
                self.lens[s] = n
        grow = [(s, n, old) for s, n, old in entries if n > old]
        after = self.refs.copy()
        plan = []
        for s, n, old in grow:                            # copies in the order of the list
            last = int(self.table[s, old // self.P]) if old % self.P else -1
            copy = last >= 0 and after[last] > 1
            if copy:
                after[last] -= 1
            plan.append((s, n, old, last if copy else -1))
        free = [p for p in range(len(self.refs)) if self.refs[p] == 0]
        need = sum(self.pages(n) - self.pages(old) + (c >= 0) for _, n, old, c in plan)
        if need > len(free):
            self.no_pages = True
            return []
        for s, n, old, c in plan:
            if c >= 0:
                to = free.pop(0)
                copies.append((c, to))
                self.table[s, old // self.P] = to
                self.refs[to] = 1
                self.refs[c] -= 1
            for j in range(self.pages(old), self.pages(n)):
                self.table[s, j] = free.pop(0)
                self.refs[self.table[s, j]] = 1
            self.lens[s] = n
        return copies

    def fork(self, src, dst):
        S, _ = self.table.shape
        was = self.lens.copy()
        named = set()
        for i, (a, b) in enumerate(zip(map(int, src), map(int, dst))):
            ok = 0 <= a < S and 0 <= b < S and was[b] == 0 and b not in named and a not in list(map(int, dst))
            named.add(b)
            if not ok:
                self.bad = True
                continue
            n = self.pages(was[a])
            self.table[b] = -1
            self.table[b, :n] = self.table[a, :n]
            self.refs[self.table[a, :n]] += 1
            self.lens[b] = was[a]

    def compact(self):
        """Returns (page_map, copies)."""
        live = [p for p in range(len(self.refs)) if self.refs[p] > 0]
        count = len(live)
        holes = [p for p in range(count) if self.refs[p] <= 0]
        new = np.full(len(self.refs), -1)
        copies = []
        for p in live:
            new[p] = p if p < count else holes[len(copies)]
            if p >= count:
                copies.append((p, int(new[p])))
        for a, b in copies:
            self.refs[b], self.refs[a] = self.refs[a], 0
        for s in range(self.table.shape[0]):
            n = self.pages(self.lens[s])
            self.table[s, :n] = new[self.table[s, :n]]
        return new, copies
