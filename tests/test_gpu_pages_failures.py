"""An attention whose wait expires (qe_debug_inject: a wait taken as expired, nothing is broken for it) ends by itself after what it
issued has landed, reports it, and leaves the GPU and the next call as they were."""
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


@pytest.mark.parametrize("lens", [[3000], [700, 20, 300, 1500] * 100], ids=["cut", "many"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kernel", KERNELS)
def test_expired_waits(torch, kernel, d, lens):
    import tiered_quantize_evict_gb300 as qe
    m, hint, hq = KERNELS[kernel]
    c = Case(torch, lens, hkv=1, d=d, ps=32, seed=d)
    pool, seqs = c.objects(qe)
    chunks = [min(m, n) for n in lens]
    q, starts = c.draw(sum(chunks), hq, d).to(c.dev), c.ints(np.cumsum([0] + chunks))
    want = pool.attend(0, q, starts, seqs, max_q_len=hint)
    pool.check()
    for role in range(3):            # copies of keys and values, products, copies of queries
        for k in (1, 2, 3, 10 ** 6):
            if role == 2 and len(lens) == 1 and k == 2 and kernel != "two_halves":
                continue             # (a CTA has one tile there)
            assert qe.debug_inject(qe.QE_DEBUG_EXPIRE_PAGES_WAIT, 4 * k + role) == qe.QE_OK
            t = time.perf_counter()
            got = pool.attend(0, q, starts, seqs, max_q_len=hint)
            torch.cuda.synchronize()
            t = time.perf_counter() - t
            assert t < 1.0, f"role {role}, wait {k}: {t:.2f} s"
            if k == 10 ** 6:         # no CTA has so many
                pool.check()
                assert torch.equal(got, want)
            elif k < 3 or len(lens) > 1 and role < 2:
                with pytest.raises(qe.QEError, match="wait expired"):
                    pool.check()
            else:
                pool.err.zero_()     # (as many waits there or not)
            assert torch.equal(pool.attend(0, q, starts, seqs, max_q_len=hint), want)   # one-shot
            pool.check()


def test_a_call_without_work_keeps_the_injection(torch):
    import tiered_quantize_evict_gb300 as qe
    c = Case(torch, [40], hkv=1, d=64, ps=16)
    pool, seqs = c.objects(qe)
    assert qe.debug_inject(qe.QE_DEBUG_EXPIRE_PAGES_WAIT, 4) == qe.QE_OK
    pool.attend(0, torch.zeros(0, 1, 64, dtype=c.dt, device=c.dev), c.ints([0, 0]), seqs)
    pool.check()
    assert qe.debug_inject(qe.QE_DEBUG_EXPIRE_PAGES_WAIT, 0) == qe.QE_OK
    pool.attend(0, c.draw(1, 1, 64).to(c.dev), c.ints([0, 1]), seqs)
    pool.check()
