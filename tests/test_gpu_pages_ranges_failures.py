"""An attention with a window or with shared prefixes whose wait expires (qe_debug_inject: a wait taken as expired, nothing is broken for
it) ends by itself after what it issued has landed, reports it, and leaves the GPU and the next call as they were."""
import time

import numpy as np
import pytest

from pages_testlib import Case

pytestmark = pytest.mark.gpu

# (chunk, hint, query heads) of one KV head
KERNELS = {"few": (2, 2, 2), "one_half": (20, 20, 2), "two_halves": (300, 0, 2)}


@pytest.fixture(scope="module")
def torch():
    return pytest.importorskip("torch")


def expire(torch, pool, call, sure):
    """sure(role, k): whether a CTA has that wait for certain."""
    import tiered_quantize_evict_gb300 as qe
    want = call()
    pool.check()
    for role in range(3):            # copies of keys and values, products, copies of queries
        for k in (1, 2, 3, 10 ** 6):
            assert qe.debug_inject(qe.QE_DEBUG_EXPIRE_PAGES_WAIT, 4 * k + role) == qe.QE_OK
            t = time.perf_counter()
            got = call()
            torch.cuda.synchronize()
            t = time.perf_counter() - t
            assert t < 1.0, f"role {role}, wait {k}: {t:.2f} s"
            if k == 10 ** 6:         # no CTA has so many
                pool.check()
                assert torch.equal(got, want)
            elif sure(role, k):
                with pytest.raises(qe.QEError, match="wait expired"):
                    pool.check()
            else:
                pool.err.zero_()     # (as many waits there or not)
            assert torch.equal(call(), want)   # one-shot
            pool.check()


@pytest.mark.parametrize("lens", [[3000], [900, 40, 700, 1500] * 100], ids=["cut", "many"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kernel", KERNELS)
def test_window(torch, kernel, d, lens):
    import tiered_quantize_evict_gb300 as qe
    m, hint, hq = KERNELS[kernel]
    c = Case(torch, lens, hkv=1, d=d, ps=32, seed=d)
    pool, seqs = c.objects(qe)
    chunks = [min(m, n) for n in lens]
    q, starts = c.draw(sum(chunks), hq, d).to(c.dev), c.ints(np.cumsum([0] + chunks))
    call = lambda: pool.attend(0, q, starts, seqs, max_q_len=hint, window=2000 if len(lens) == 1 else 600, sinks=40)  # noqa: E731
    expire(torch, pool, call, lambda role, k: k < 3 and (role < 2 or len(lens) > 1) or k == 1)


@pytest.mark.parametrize("groups", [1, 100], ids=["cut", "many"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [12, 60, 200])
def test_shared(torch, rows, d, groups):
    """rows of a group: few, one half, two halves."""
    import tiered_quantize_evict_gb300 as qe
    n = rows // 4
    lens = [(3000 if groups == 1 else 320) + 7 * i + 1 for i in range(n)] * groups
    c = Case(torch, lens, hkv=1, d=d, ps=32, seed=d)
    pool, seqs = c.objects(qe)
    q, starts = c.draw(len(lens), 4, d).to(c.dev), c.ints(range(len(lens) + 1))
    gs, pre = c.ints([n * g for g in range(groups + 1)]), c.ints([2976 if groups == 1 else 320] * groups)
    call = lambda: pool.attend_shared(0, q, starts, seqs, gs, pre, max_group_len=n)  # noqa: E731
    expire(torch, pool, call, lambda role, k: k == 1 or k < 3 and role < 2)
