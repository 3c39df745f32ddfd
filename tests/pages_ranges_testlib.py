"""Helpers for attention over two ranges of keys: the oracle's answer with tolerances, checks, poisoned pools."""
from __future__ import annotations

import numpy as np

from oracle import pages as op
from pages_testlib import bits


def seen_bounds(torch, dt, q, k, v, hkv, scale, seen):
    """(out, tolerance, lse, lse tolerance) of one sequence's queries, float64; query j sees the keys seen[j].

    With u the half step of the type (bf16 2^-8, fp16 2^-11):
      * the result is rounded once: u |out|;
      * each probability is rounded once before it meets the values: u sum w |v|; in fp16 it is off by 2^-32 of the row's
        reference weight where that is more, against a denominator of at least `den`: 2^-32 sum |v| / den;
      * logits: products are exact in float32, their sum of D terms and the scaling are off by at most
        (D + 4) 2^-24 sum_c |q_c k_c| scale, which moves a weight by that much relatively, numerator and
        denominator alike (2 x); exp2 and the running sums add 2^-20 relatively and n 2^-24."""
    out, lse, spread, den = op.attend_seen(q, k, v, hkv, scale, seen)
    u = float(torch.finfo(dt).eps) / 2
    m, hq, d = q.shape
    grp = hq // hkv
    mag, most, total = np.zeros((m, hq)), np.zeros(m), np.zeros((m, hkv, d))
    for j in range(m):
        vis = np.fromiter(seen[j], np.int64)
        most[j] = vis.size
        if vis.size:
            total[j] = np.abs(v[vis]).sum(0)
            for h in range(hq):
                mag[j, h] = scale * (np.abs(k[vis, h // grp]) @ np.abs(q[j, h])).max()
    dl = (d + 4) * 2.0 ** -24 * mag
    rel = u + 2 * dl + 2.0 ** -20 + most[:, None] * 2.0 ** -24
    tol = u * np.abs(out) + rel[..., None] * spread
    if dt == torch.float16:
        tol += 2.0 ** -32 * np.repeat(total, grp, 1) / den[..., None]
        tol += 2.0 ** -25    # a result below 2^-14
    return out, tol * 1.01, lse, dl + 2.0 ** -20 + 2.0 ** -23 * np.where(np.isfinite(lse), np.abs(lse), 0)


def check(got, lse, want, what):
    ref, tol, lref, ltol = want
    err = np.abs(got - ref)
    assert np.isfinite(got).all(), f"{what}: not finite"
    assert (err <= tol).all(), f"{what}: error {err.max():.3e}, {np.max(err / np.maximum(tol, 1e-30)):.2f} of the bound"
    if lse is not None:
        assert np.array_equal(np.isinf(lse), np.isinf(lref)) and not np.isnan(lse).any(), what
        fin = np.isfinite(lref)
        off = np.abs(lse[fin] - lref[fin])
        assert (off <= ltol[fin]).all(), f"{what}: lse off by {off.max():.3e}"


def poison(c, row, keys):
    """NaN in the keys and values of a row's tokens, in the pool (not in what the oracle is given)."""
    if len(keys):
        pos = c.torch.tensor(sorted(keys))
        page, tok = c.torch.from_numpy(c.table[row].astype(np.int64))[pos // c.ps].to(c.dev), (pos % c.ps).to(c.dev)
        for x in (c.k, c.v):
            x[:, page, :, tok] = float("nan")


def queries(c, total, hq, layout="plain"):
    """(host values, device tensor, output filled with NaN)"""
    torch = c.torch
    qh = c.draw(total, hq, c.d)
    nan = float("nan")
    if layout == "plain":
        return qh, qh.to(c.dev), torch.full((total, hq, c.d), nan, dtype=c.dt, device=c.dev)
    if layout == "heads_first":
        return qh, qh.transpose(0, 1).contiguous().to(c.dev).transpose(0, 1), torch.full((hq, total, c.d), nan, dtype=c.dt, device=c.dev).transpose(0, 1)
    q = torch.zeros(total, hq + 2, c.d + 8, dtype=c.dt, device=c.dev)[:, 1:-1, :c.d]     # a slice of a fused projection
    q.copy_(qh)
    return qh, q, torch.full((total, hq + 1, c.d), nan, dtype=c.dt, device=c.dev)[:, :hq]


__all__ = ["bits", "check", "poison", "queries", "seen_bounds"]
