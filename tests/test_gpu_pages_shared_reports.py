"""Attention of sequences that share prefixes: what it gives for groups it reports, and values that are not finite."""
import numpy as np
import pytest

from pages_ranges_testlib import bits, check, seen_bounds
from test_gpu_pages_shared import shared_case

pytestmark = pytest.mark.gpu

HINTS = (0, 4, 20)     # two halves, few rows, one half (4 heads to a KV head)


@pytest.fixture(scope="module")
def torch():
    return pytest.importorskip("torch")


def against(torch, c, out, qh, rows, starts, seen, kv=None):
    """out of the sequences named in `seen` (keys of (row, token) pairs seen by each of its tokens)."""
    for i, vis in seen.items():
        a, b = starts[i], starts[i + 1]
        k, v = kv[i] if kv else (bits(c.kh[rows[i]][0]), bits(c.vh[rows[i]][0]))
        want = seen_bounds(torch, c.dt, bits(qh[a:b]), k, v, c.hkv, c.d ** -0.5, vis)
        check(bits(out[a:b]), None, want, f"sequence {i}")


@pytest.mark.parametrize("hint", HINTS)
@pytest.mark.parametrize("gs,prefix,alone", [([0, 2], 64, [2]), ([1, 3], 64, [0]), ([0, 3], 80, []), ([0, 3], 2 ** 31 - 1, []), ([0, 2 ** 31 - 1], 64, [])])
def test_what_bad_groups_come_to(torch, hint, gs, prefix, alone):
    """Sequences of no group are left alone; a prefix is cut to the first sequence's length; the others are as if nothing was wrong."""
    import tiered_quantize_evict_gb300 as qe
    c, flat, order, lens = shared_case(torch, [(64, [(1, 9), (2, 20), (1, 14)])], ps=16, hkv=1, d=64, garbage_entries=False)
    pool, seqs = c.objects(qe)
    qh, starts = c.draw(4, 4, 64), [0, 1, 3, 4]
    out = torch.full((4, 4, 64), 3.0, dtype=c.dt, device=c.dev)
    pool.attend_shared(0, qh.to(c.dev), c.ints(starts), seqs, c.ints(gs), c.ints([prefix]), max_group_len=hint, out=out)
    with pytest.raises(qe.QEError, match="row"):
        pool.check()
    for i in alone:
        assert (out[starts[i]:starts[i + 1]] == 3).all()
    seen = {i: [range(lens[i] - m + j + 1) for j in range(m)] for i, m in ((0, 1), (1, 2), (2, 1)) if i not in alone}
    against(torch, c, out, qh, order, starts, seen)


@pytest.mark.parametrize("hint", HINTS)
def test_a_chunk_that_begins_inside_its_prefix(torch, hint):
    """It sees all of the prefix, and behind that what its positions allow."""
    import tiered_quantize_evict_gb300 as qe
    c, flat, order, lens = shared_case(torch, [(96, [(1, 104), (2, 0), (10, 4)])], ps=16, hkv=1, d=64, garbage_entries=False)
    c.kv_len[1] = lens[1] = 70                       # its last two tokens are inside of the prefix of 96
    pool, seqs = c.objects(qe)
    qh, starts = c.draw(13, 4, 64), [0, 1, 3, 13]
    out = pool.attend_shared(0, qh.to(c.dev), c.ints(starts), seqs, c.ints([0, 3]), c.ints([96]), max_group_len=hint)
    with pytest.raises(qe.QEError, match="row"):
        pool.check()
    kv = {r: (bits(c.kh[r][0]), bits(c.vh[r][0])) for r in range(3)}
    kv[1] = kv[0]
    seen = {0: [range(200)], 1: [range(96)] * 2, 2: [range(max(96, 100 - 10 + j + 1)) for j in range(10)]}
    against(torch, c, out, qh, order, starts, seen, kv)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("hint", HINTS)
@pytest.mark.parametrize("prefix", [64, 2000])     # tiles that a CTA finishes, and such that are joined
def test_values_that_are_not_finite(torch, bad, dtype, hint, prefix):
    """A value of one sequence's own tokens may reach its group, which is then reported, and no other group."""
    import tiered_quantize_evict_gb300 as qe
    c, flat, order, lens = shared_case(torch, [(prefix, [(1, 9), (2, 20), (1, 14)]), (48, [(1, 30), (1, 5)]), (0, [(2, 40)])], ps=16, hkv=2, d=64, dtype=dtype)
    starts = np.cumsum([0] + [x[3] for x in flat])
    qh, gs, pre = c.draw(int(starts[-1]), 8, 64), [0, 3, 5, 6], [prefix, 48, 0]
    pool, seqs = c.objects(qe)
    call = lambda: pool.attend_shared(0, qh.to(c.dev), c.ints(starts), seqs, c.ints(gs), c.ints(pre), max_group_len=hint)  # noqa: E731
    call()
    pool.check()
    for row, tok in ((1, prefix + 3), (5, 7)):
        page = int(c.table[row, tok // 16])
        was = c.v[0, page, 1, tok % 16, 5].clone()
        c.v[0, page, 1, tok % 16, 5] = bad
        out = call()
        with pytest.raises(qe.QEError, match="not finite"):
            pool.check()
        own = [i for g in range(3) if not gs[g] <= row < gs[g + 1] for i in range(gs[g], gs[g + 1])]
        seen = {i: [range(lens[i] - flat[i][3] + j + 1) for j in range(flat[i][3])] for i in own}
        against(torch, c, out, qh, order, starts, seen)
        assert not torch.isfinite(out[starts[row]:starts[row + 1]]).all()
        c.v[0, page, 1, tok % 16, 5] = was
    call()
    pool.check()
