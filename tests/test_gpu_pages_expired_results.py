"""An attention with a window or with shared prefixes that is told to take a wait as expired either says so or gives what it always does."""
import numpy as np
import pytest

from pages_testlib import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return pytest.importorskip("torch")


def either(torch, pool, call):
    import tiered_quantize_evict_gb300 as qe
    want = call()
    pool.check()
    said = 0
    for role in range(3):            # copies of keys and values, products, copies of queries
        for k in (1, 2, 3, 4, 9):
            assert qe.debug_inject(qe.QE_DEBUG_EXPIRE_PAGES_WAIT, 4 * k + role) == qe.QE_OK
            got = call()
            bits = int(pool.err.item())
            pool.err.zero_()
            assert not bits or bits & 8, bits     # (what it leaves may be no numbers)
            assert bits or torch.equal(got, want), f"role {role}, wait {k}: nothing said, another result"
            said += bits != 0
            assert torch.equal(call(), want)
            pool.check()
    assert said >= 3


@pytest.mark.parametrize("lens", [[3000], [900, 40, 700, 1500] * 100], ids=["cut", "many"])
@pytest.mark.parametrize("m,hint", [(2, 2), (20, 20), (300, 0)], ids=["few", "one_half", "two_halves"])
@pytest.mark.parametrize("d", [64, 128])
def test_window(torch, lens, m, hint, d):
    import tiered_quantize_evict_gb300 as qe
    c = Case(torch, lens, hkv=1, d=d, ps=32, seed=d)
    pool, seqs = c.objects(qe)
    chunks = [min(m, n) for n in lens]
    q, starts = c.draw(sum(chunks), 2, d).to(c.dev), c.ints(np.cumsum([0] + chunks))
    either(torch, pool, lambda: pool.attend(0, q, starts, seqs, max_q_len=hint, window=2000 if len(lens) == 1 else 600, sinks=40))


@pytest.mark.parametrize("groups", [1, 100], ids=["cut", "many"])
@pytest.mark.parametrize("rows", [12, 60, 200], ids=["few", "one_half", "two_halves"])
@pytest.mark.parametrize("d", [64, 128])
def test_shared(torch, groups, rows, d):
    import tiered_quantize_evict_gb300 as qe
    n = rows // 4
    lens = [(3000 if groups == 1 else 320) + 7 * i + 1 for i in range(n)] * groups
    c = Case(torch, lens, hkv=1, d=d, ps=32, seed=d)
    pool, seqs = c.objects(qe)
    q, starts = c.draw(len(lens), 4, d).to(c.dev), c.ints(range(len(lens) + 1))
    gs, pre = c.ints([n * g for g in range(groups + 1)]), c.ints([2976 if groups == 1 else 320] * groups)
    either(torch, pool, lambda: pool.attend_shared(0, q, starts, seqs, gs, pre, max_group_len=n))
