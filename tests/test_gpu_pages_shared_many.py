"""Attention of sequences that share prefixes, for calls of many sequences: the checks of their arrays."""
import numpy as np
import pytest

from pages_testlib import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return pytest.importorskip("torch")


def many(torch, n, per):
    """n sequences of a token, in groups of `per`, over two rows that share 32 tokens."""
    c = Case(torch, [40, 37], hkv=1, d=64, ps=16)
    c.kh[1][:, :32], c.vh[1][:, :32] = c.kh[0][:, :32], c.vh[0][:, :32]
    c.table[1, :2] = c.table[0, :2]
    return c, np.arange(n + 1), np.arange(n) % 2, np.arange(0, n + 1, per), np.full(n // per, 32)


@pytest.mark.parametrize("hint", [0, 1, 8])
def test_mistakes_anywhere_are_reported(torch, hint):
    """One wrong number among 20000 sequences or 2500 groups, wherever it stands."""
    import tiered_quantize_evict_gb300 as qe
    n, per = 20000, 8
    c, starts, rows, gs, pre = many(torch, n, per)
    pool, seqs = c.objects(qe)
    q = c.draw(n, 8, 64).to(c.dev)

    def call(starts=starts, rows=rows, gs=gs, pre=pre):
        pool.attend_shared(0, q, c.ints(starts), seqs, c.ints(gs), c.ints(pre), rows=c.ints(rows), max_group_len=hint)

    call()
    pool.check()
    for at in (0, 31, 32, 4863, 4864, 4865, 12000, n - 1):
        g = at // per
        wrong = [dict(rows=np.where(np.arange(n) == at, 2, rows)), dict(pre=np.where(np.arange(n // per) == g, 48, pre)),
                 dict(pre=np.where(np.arange(n // per) == g, -16, pre)), dict(starts=np.where(np.arange(n + 1) == at, n + 1, starts))]
        if g:
            wrong.append(dict(gs=np.where(np.arange(n // per + 1) == g, gs[g + 1] + 1, gs)))
        for kw in wrong:
            call(**kw)
            with pytest.raises(qe.QEError, match="row"):
                pool.check()
    call()
    pool.check()


def test_the_checks_do_not_bound_the_call(torch):
    """65536 sequences in groups of 16: less than twice as long as attend over the same rows (1.2 ms and 1.25; with the checks one after the
    other 3.7)."""
    import tiered_quantize_evict_gb300 as qe
    n = 65536
    c, starts, rows, gs, pre = many(torch, n, 16)
    pool, seqs = c.objects(qe)
    q, starts, rows, gs, pre = c.draw(n, 4, 64).to(c.dev), *map(c.ints, (starts, rows, gs, pre))
    calls = {"shared": lambda: pool.attend_shared(0, q, starts, seqs, gs, pre, rows=rows), "all": lambda: pool.attend(0, q, starts, seqs, rows=rows, max_q_len=1)}
    best = dict.fromkeys(calls, float("inf"))
    for _ in range(4):       # (in turn; the first round is the warm-up)
        for k, f in calls.items():
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            f()
            a.record()
            for _ in range(3):
                f()
            b.record()
            torch.cuda.synchronize()
            best[k] = min(best[k], a.elapsed_time(b) / 3)
    pool.check()
    assert best["shared"] < 2 * best["all"], best
