"""Paged cache in plain loops and float64: page bookkeeping, rotary append, chunk attention.

Test infrastructure (see ``oracle/__init__``).  The definitions are the paged-cache section of
``include/qe.h``; rotary pairs and angles as in ``oracle/rope.py``, with an axis per channel pair.
"""
from __future__ import annotations

import math

import numpy as np


class Pages:
    """Page table, lengths and reference counts (lists) over a pool [L][P][H][S][D] of keys and values."""

    def __init__(self, n_rows, max_pages, n_pages, page_size):
        self.table = [[-1] * max_pages for _ in range(n_rows)]
        self.kv_len = [0] * n_rows
        self.refs = [0] * n_pages
        self.S = page_size

    def _free(self):
        return [p for p, r in enumerate(self.refs) if r == 0]

    def resize(self, rows, new_len):
        """Returns the (src, dst, used rows) page copies; pages given back are free from the next call on.  A call
        short of pages changes nothing and returns None."""
        free, plan = self._free(), []
        for r, n in zip(rows, new_len):
            old, edge = self.kv_len[r], min(self.kv_len[r], n)
            own = edge % self.S and old != n and self.refs[self.table[r][edge // self.S]] > 1
            plan.append((r, n, bool(own), max(0, -(-n // self.S) - -(-old // self.S))))
        if sum(o + w for _, _, o, w in plan) > len(free):
            return None
        copies = []
        for r, n, own, want in plan:
            old, edge = self.kv_len[r], min(self.kv_len[r], n)
            if own:
                p, was = free.pop(0), self.table[r][edge // self.S]
                copies.append((was, p, edge % self.S))
                self.refs[was] -= 1
                self.refs[p] = 1
                self.table[r][edge // self.S] = p
            for j in range(-(-old // self.S), -(-n // self.S)):
                p = free.pop(0)
                self.table[r][j], self.refs[p] = p, 1
            for j in range(-(-n // self.S), -(-old // self.S)):
                self.refs[self.table[r][j]] -= 1
                self.table[r][j] = -1
            self.kv_len[r] = n
        return copies

    def fork(self, src, dst):
        free = self._free()
        lens = list(self.kv_len)
        if sum(lens[s] % self.S > 0 for s in src) > len(free):
            return None
        copies = []
        for s, d in zip(src, dst):
            full = lens[s] // self.S
            for j in range(full):
                p = self.table[s][j]
                self.table[d][j] = p
                self.refs[p] += 1
            if lens[s] % self.S:
                p = free.pop(0)
                copies.append((self.table[s][full], p, lens[s] % self.S))
                self.table[d][full], self.refs[p] = p, 1
            self.kv_len[d] = lens[s]
        return copies

    def compact(self):
        n = sum(r > 0 for r in self.refs)
        src = [p for p in range(n, len(self.refs)) if self.refs[p] > 0]
        dst = [p for p in range(n) if self.refs[p] == 0]
        to = dict(zip(src, dst))
        for a, b in to.items():
            self.refs[a], self.refs[b] = 0, self.refs[a]
        self.table = [[to.get(p, p) for p in row] for row in self.table]
        return [(a, b, self.S) for a, b in to.items()], n


def rotate(x, positions, axis, inv_freq, rot_dim, halves):
    """Rows x [tokens][heads][D] rotated (float64); positions [axes][tokens]."""
    out = np.array(x, np.float64)
    for i in range(rot_dim // 2):
        a, b = (i, i + rot_dim // 2) if halves else (2 * i, 2 * i + 1)
        ang = np.asarray(positions[axis[i]], np.float64) * inv_freq[i]
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        out[..., a], out[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    return out


def attend(q, k, v, n_kv_heads, scale, causal):
    """One sequence: q [m][Hq][D] (its last m tokens), k, v [kv_len][Hkv][D] -> (out, lse, spread, sum of exps).

    spread is sum_i w_i |v_i| and the last the softmax's denominator relative to its maximum: what a rounding
    of the probabilities is measured against."""
    m, hq, d = q.shape
    n = k.shape[0]
    out, spread = np.zeros((m, hq, d)), np.zeros((m, hq, d))
    lse, den = np.full((m, hq), -np.inf), np.ones((m, hq))
    for h in range(hq):
        g = h // (hq // n_kv_heads)
        for j in range(m):
            vis = max(0, n - m + j + 1) if causal else n
            if vis == 0:
                continue
            s = scale * (k[:vis, g].astype(np.float64) @ q[j, h].astype(np.float64))
            w = np.exp(s - s.max())
            den[j, h] = w.sum()
            lse[j, h] = s.max() + math.log(w.sum())
            w /= w.sum()
            out[j, h] = w @ v[:vis, g]
            spread[j, h] = w @ np.abs(v[:vis, g])
    return out, lse, spread, den
