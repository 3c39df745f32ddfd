"""Attention of sequences that share prefixes: how many bits the probabilities have, in all of its kernels."""
import numpy as np
import pytest

from pages_ranges_testlib import bits, check, seen_bounds
from test_gpu_pages_extremes import plain_probabilities, put_keys, remainder_bounds
from test_gpu_pages_shared import shared_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return pytest.importorskip("torch")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,m,hq,hkv", [(3, 1, 4, 1), (14, 2, 4, 1), (40, 1, 4, 1), (9, 4, 8, 2), (5, 16, 4, 1), (70, 1, 8, 2), (150, 1, 1, 1)])
@pytest.mark.parametrize("hint", ["unknown", "right"])
def test_remainders_of_the_probabilities(torch, d, n, m, hq, hkv, hint):
    """Chunks that are known to have up to 128 rows of a KV head, in groups of any size: the bound that attend keeps for the same rows,
    which holds only if the remainders of the probabilities meet their values too."""
    import tiered_quantize_evict_gb300 as qe
    rng = np.random.default_rng(n + d)
    c, flat, order, lens = shared_case(torch, [(96, [(m, m + int(x)) for x in rng.integers(0, 60, n)])], ps=32, hkv=hkv, d=d, seed=n)
    for row in range(n):
        c.kh[row][0].mul_(0.25)
    c.table[1:, :3] = c.table[0, :3]      # (what put_keys writes there for the others is the first's own)
    for row in range(n):
        put_keys(torch, c, row)
    pool, seqs = c.objects(qe)
    qh = c.draw(n * m, hq, d)
    out = pool.attend_shared(0, qh.to(c.dev), c.ints(range(0, n * m + 1, m)), seqs, c.ints([0, n]), c.ints([96]), max_q_len=m,
                             max_group_len=n * m if hint == "right" else 0)
    pool.check()
    worst = 0
    for row in range(n):
        q = bits(qh[row * m:(row + 1) * m])
        ref, tol = remainder_bounds(torch, c, q, row, hq, d ** -0.5)
        if row < 3:
            k, v = bits(c.kh[row][0]), bits(c.vh[row][0])
            assert (np.abs(plain_probabilities(q, k, v, hkv, d ** -0.5, True) - ref) <= tol).all()
            worst = max(worst, (np.abs(plain_probabilities(q, k, v, hkv, d ** -0.5, False) - ref) / tol).max())
        err = np.abs(bits(out[row * m:(row + 1) * m]) - ref)
        assert (err <= tol).all(), f"row {row}: {(err / tol).max():.2f} of the bound"
    assert worst > 2


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
def test_any_longest_chunk(torch, d, dtype):
    """max_q_len is a hint: right results whatever it says, over cut tiles and such with nothing of a block for some rows."""
    import tiered_quantize_evict_gb300 as qe
    c, flat, order, lens = shared_case(torch, [(1500, [(1 + i % 3, 10 + 37 * i) for i in range(30)]), (0, [(70, 70), (1, 400)])], ps=16, hkv=2, d=d,
                                       dtype=dtype, garbage_entries=False)
    pool, seqs = c.objects(qe)
    ms = [x[3] for x in flat]
    starts = np.cumsum([0] + ms)
    qh = c.draw(int(starts[-1]), 8, d)
    for hint in (0, 1, 32, 33, 2 ** 31 - 1):
        out, lse = pool.attend_shared(0, qh.to(c.dev), c.ints(starts), seqs, c.ints([0, 30, 32]), c.ints([1500, 0]), max_q_len=hint, return_lse=True)
        pool.check()
        for i, (a, m) in enumerate(zip(starts, ms)):
            want = seen_bounds(torch, c.dt, bits(qh[a:a + m]), bits(c.kh[i][0]), bits(c.vh[i][0]), 2, d ** -0.5, [range(lens[i] - m + j + 1) for j in range(m)])
            check(bits(out[a:a + m]), lse[a:a + m].cpu().numpy(), want, f"hint {hint}, row {i}")
    for bad in (-1, 2 ** 31):
        with pytest.raises(qe.QEError, match="max_q_len"):
            pool.attend_shared(0, qh.to(c.dev), c.ints(starts), seqs, c.ints([0, 30, 32]), c.ints([1500, 0]), max_q_len=bad)
