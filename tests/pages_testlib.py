"""Helpers of the paged-cache tests: seeded pools, the oracle's answer, and derived tolerances."""
from __future__ import annotations

import numpy as np

from oracle import pages as op


def cdiv(a, b):
    return -(-a // b)


def bits(t):
    return t.float().cpu().numpy().astype(np.float64)


class Case:
    """A pool with rows of the given lengths on shuffled pages; what no row holds is NaN."""

    def __init__(self, torch, lens, *, hkv, d, ps, dtype="bf16", layers=1, layout="plain", seed=0, spare=2, garbage=float("nan"),
                 n_rows=None, max_pages=None):
        self.torch, self.dev = torch, torch.device("cuda:0")
        self.dt = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
        self.rng = np.random.default_rng(seed)
        self.lens, self.hkv, self.d, self.ps, self.layers = list(lens), hkv, d, ps, layers
        rows = n_rows or len(self.lens)
        need = [cdiv(x, ps) for x in self.lens]
        self.n_pages = sum(need) + spare
        cols = max_pages or max(max(need), 1)
        perm = self.rng.permutation(self.n_pages)
        self.table = np.full((rows, cols), -1, np.int32)
        self.refs = np.zeros(self.n_pages, np.int32)
        at = 0
        for r, n in enumerate(need):
            self.table[r, :n] = perm[at:at + n]
            self.refs[perm[at:at + n]] = 1
            at += n
        self.kv_len = np.array(self.lens + [0] * (rows - len(self.lens)), np.int32)
        # keys [row][layer][len][H][D], in the pool's type
        self.kh = [self.draw(layers, n, hkv, d, outliers=True) for n in self.lens]
        self.vh = [self.draw(layers, n, hkv, d) for n in self.lens]
        self.k, self.v = self.pool(layout, garbage)
        for r, n in enumerate(self.lens):
            pos = torch.arange(n)
            page = torch.from_numpy(self.table[r].astype(np.int64))[pos // ps].to(self.dev)
            tok = (pos % ps).to(self.dev)
            for l in range(layers):
                self.k[l][page, :, tok] = self.kh[r][l].to(self.dev)
                self.v[l][page, :, tok] = self.vh[r][l].to(self.dev)

    def draw(self, *shape, outliers=False):
        x = self.rng.standard_normal(shape, dtype=np.float32)
        if outliers:
            x[..., :2] *= 8
        return self.torch.from_numpy(x).to(self.dt)

    def pool(self, layout, garbage):
        """[L][P][H][S][D] views of the layouts that pools come in."""
        torch, L, P, H, S, D = self.torch, self.layers, self.n_pages, self.hkv, self.ps, self.d
        full = lambda *s: torch.full(s, garbage, dtype=self.dt, device=self.dev)  # noqa: E731
        if layout == "plain":
            return full(L, P, H, S, D), full(L, P, H, S, D)
        if layout == "token_major":          # tokens before heads
            return full(L, P, S, H, D).transpose(2, 3), full(L, P, S, H, D).transpose(2, 3)
        if layout == "kv_together":          # one tensor, keys and values side by side, layers inside pages
            kv = full(P, L, 2, H, S, D + 8)
            return kv[:, :, 0, ..., :D].transpose(0, 1), kv[:, :, 1, ..., :D].transpose(0, 1)
        raise ValueError(layout)

    def objects(self, qe, refs=False):
        t = self.torch
        self.pool_obj = qe.PagePool(self.k, self.v)
        self.seqs = qe.PageTable(t.from_numpy(self.table).to(self.dev), t.from_numpy(self.kv_len).to(self.dev),
                                 t.from_numpy(self.refs).to(self.dev) if refs else None)
        return self.pool_obj, self.seqs

    def ints(self, x):
        return self.torch.tensor(np.asarray(x, np.int32)).to(self.dev)


def attend_bounds(torch, c, q, m, row, hq, scale, causal, layer=0):
    """(out, tolerance, lse, lse tolerance) of one sequence, float64.

    With u the half step of the type (bf16 2^-8, fp16 2^-11):
      * the result is rounded once: u |out|;
      * each probability is rounded once before it meets the values: u sum w |v|; fp16 below 2^-14 loses up to 2^-25
        absolutely, against a denominator of at least `den`: 2^-25 sum |v| / den;
      * logits: products are exact in float32, their sum of D terms and the scaling are off by at most
        (D + 4) 2^-24 sum_c |q_c k_c| scale, which moves a weight by that much relatively, numerator and
        denominator alike (2 x); exp2 and the running sums add 2^-20 relatively (n 2^-24 at these lengths)."""
    k, v = bits(c.kh[row][layer]), bits(c.vh[row][layer])
    out, lse, spread, den = op.attend(q, k, v, c.hkv, scale, causal)
    u = float(torch.finfo(c.dt).eps) / 2
    d = c.d
    grp = hq // c.hkv
    mag = np.zeros((m, hq))
    if k.shape[0]:
        for h in range(hq):
            mag[:, h] = scale * (np.abs(q[:, h]) @ np.abs(k[:, h // grp]).T).max(-1)
    dl = (d + 4) * 2.0 ** -24 * mag
    rel = u + 2 * dl + 2.0 ** -20 + k.shape[0] * 2.0 ** -24
    tol = u * np.abs(out) + rel[..., None] * spread
    if c.dt == torch.float16 and k.shape[0]:
        tol += 2.0 ** -25 * np.repeat(np.abs(v).sum(0), grp, 0)[None] / den[..., None]
        tol += 2.0 ** -25    # a result below 2^-14
    return out, tol * 1.01, lse, dl + 2.0 ** -20 + 2.0 ** -23 * np.where(np.isfinite(lse), np.abs(lse), 0)
