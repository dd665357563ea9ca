"""CPU oracle for the decoding operators: rotary positions, the paged cache's
bookkeeping, and attention of drafted trees.

TEST INFRASTRUCTURE, like ``pbs_oracle``: plain numpy in fp64 and Python
lists, one definition after the other, sharing no code with the CUDA library.
"""
from __future__ import annotations

import math

import numpy as np


def rope(x, pos, inv_freq, gain=1.0, layout="half", transpose=False):
    """x [b, h, n, d], pos [b, n]: pair (x0, x1) times gain * exp(+-i pos f)."""
    y = np.array(x, dtype=np.float64)
    r = 2 * len(inv_freq)
    a = pos.astype(np.float64)[:, None, :, None] * np.asarray(inv_freq, dtype=np.float64)
    turn = gain * np.exp((-1j if transpose else 1j) * a)
    if layout == "half":
        lo, hi = np.s_[..., :r // 2], np.s_[..., r // 2:r]
    else:
        lo, hi = np.s_[..., 0:r:2], np.s_[..., 1:r:2]
    z = (y[lo] + 1j * y[hi]) * turn
    y[lo], y[hi] = z.real, z.imag
    return y


def visible(parents, count):
    """[tree, tree] bool: draft i sees draft j."""
    t = len(parents)
    see = np.zeros((t, t), dtype=bool)
    for i in range(t):
        j = i
        while j >= 0:
            see[i, j] = True
            j = parents[j]
    see[:, count:] = False
    return see


def attend(q, k, v, start, see, sigma):
    """One sequence and KV head: q [rows, d], k, v [n, d], see [rows, n -
    start]. Returns (o, lse, spread): spread = sum_j p_j |v_j|, for bounds. A
    row that sees nothing gives 0 and -inf; what a row does not see has no
    part in it."""
    rows, n = q.shape[0], k.shape[0]
    o, spread = np.zeros((rows, v.shape[1])), np.zeros((rows, v.shape[1]))
    lse = np.full(rows, -np.inf)
    for r in range(rows):
        idx = np.concatenate([np.arange(start), start + np.nonzero(see[r])[0]])
        if not len(idx):
            continue
        a = sigma * (k[idx] @ q[r])
        m = a.max()
        with np.errstate(invalid="ignore"):
            p = np.exp(a - m)
            lse[r] = m + math.log(p.sum()) if np.isfinite(m) else np.nan
            p = p / p.sum()
            o[r], spread[r] = p @ v[idx], p @ np.abs(v[idx])
    return o, lse, spread


class Books:
    """The page bookkeeping on lists, by its definition."""

    def __init__(self, seqs, width, pages, page):
        self.page, self.width = page, width
        self.table = [[-1] * width for _ in range(seqs)]
        self.refs, self.lens = [0] * pages, [0] * seqs

    def held(self, s):
        return [p for p in self.table[s] if p >= 0]

    def reserve(self, want):
        """Copy pairs per sequence, or None when the pages do not suffice."""
        table, refs = [list(r) for r in self.table], list(self.refs)
        free = [p for p, r in enumerate(refs) if r == 0]
        pairs = []
        for s, w in enumerate(want):
            pair = (-1, -1)
            if w > self.lens[s]:
                for j in range(self.lens[s] // self.page, -(-w // self.page)):
                    old = table[s][j]
                    if old >= 0 and refs[old] == 1:
                        continue
                    if not free:
                        return None
                    new = free.pop(0)
                    table[s][j], refs[new] = new, 1
                    if old >= 0:
                        refs[old] -= 1
                        if j * self.page < self.lens[s]:
                            pair = (old, new)
            pairs.append(pair)
        self.table, self.refs = table, refs
        return pairs

    def fork(self, src, dst):
        for s, t in zip(src, dst):
            n = -(-self.lens[s] // self.page)
            self.table[t][:n] = self.table[s][:n]
            self.lens[t] = self.lens[s]
            for p in self.table[s][:n]:
                self.refs[p] += 1

    def trim(self, keep):
        for s, k in enumerate(keep):
            if k < 0:
                continue
            self.lens[s] = min(self.lens[s], k)
            for j in range(-(-self.lens[s] // self.page), self.width):
                if self.table[s][j] >= 0:
                    self.refs[self.table[s][j]] -= 1
                    self.table[s][j] = -1

    def compact(self):
        n = sum(r > 0 for r in self.refs)
        src = [p for p in range(n, len(self.refs)) if self.refs[p]]
        dst = [p for p in range(n) if not self.refs[p]]
        for a, b in zip(src, dst):
            self.refs[b], self.refs[a] = self.refs[a], 0
        to = dict(zip(src, dst))
        self.table = [[to.get(p, p) for p in row] for row in self.table]
        return list(zip(src, dst))
