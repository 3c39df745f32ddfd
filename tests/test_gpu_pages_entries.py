"""Attention over a table whose entries are no pages of the pool: all of them are reported, whatever the number."""
import pytest

from pages_ranges_testlib import bits, check, seen_bounds
from pages_testlib import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return pytest.importorskip("torch")


@pytest.mark.parametrize("entry", [-1, -3, -2 ** 31, -2 ** 31 + 1, 2 ** 31 - 1])
@pytest.mark.parametrize("hint", [0, 1, 20])
@pytest.mark.parametrize("kind", ["all", "window", "shared"])
def test_entries(torch, kind, hint, entry):
    """Such a page counts as zeros."""
    import tiered_quantize_evict_gb300 as qe
    c = Case(torch, [150, 90], hkv=1, d=64, ps=16)
    c.table[1, 3] = entry
    c.kh[1][0, 48:64], c.vh[1][0, 48:64] = 0, 0
    pool, seqs = c.objects(qe)
    qh = c.draw(2, 4, 64)
    q, starts = qh.to(c.dev), c.ints([0, 1, 2])
    if kind == "shared":
        out = pool.attend_shared(0, q, starts, seqs, c.ints([0, 1, 2]), c.ints([64, 32]), max_group_len=hint)
    else:
        out = pool.attend(0, q, starts, seqs, max_q_len=hint, window=80 if kind == "window" else None)
    with pytest.raises(qe.QEError, match="page index"):
        pool.check()
    for r, n in ((0, 150), (1, 90)):
        want = seen_bounds(torch, c.dt, bits(qh[r:r + 1]), bits(c.kh[r][0]), bits(c.vh[r][0]), 1, 0.125, [range(max(0, n - 80) if kind == "window" else 0, n)])
        check(bits(out[r:r + 1]), None, want, f"row {r}")
