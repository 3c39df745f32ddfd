"""Calls of the paged cache from other threads, with numbers outside of what a C int holds, and the hand-over of
fp16 to the tiered cache."""
import threading

import numpy as np
import pytest

from pages_testlib import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return pytest.importorskip("torch")


def in_thread(fn):
    """fn's result on a thread of its own."""
    got = []

    def body():
        try:
            got.append((True, fn()))
        except BaseException as e:  # noqa: BLE001
            got.append((False, e))
    t = threading.Thread(target=body)
    t.start()
    t.join()
    ok, x = got[0]
    if not ok:
        raise x
    return x


@pytest.mark.parametrize("n", [40, 3000])
def test_first_call_of_a_thread(torch, n):
    """A thread that has made no CUDA call before; all it needs is there, so the binding allocates nothing either."""
    import tiered_quantize_evict_gb300 as qe
    c = Case(torch, [n], hkv=2, d=64, ps=16)
    pool, seqs = c.objects(qe)
    q, starts = c.draw(1, 4, 64).to(c.dev), c.ints([0, 1])
    want = pool.attend(0, q, starts, seqs, max_q_len=1)
    out = torch.zeros_like(q)
    torch.cuda.synchronize()
    in_thread(lambda: pool.attend(0, q, starts, seqs, max_q_len=1, out=out))
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    pool.check()


def test_every_call_from_a_thread_of_its_own(torch):
    import tiered_quantize_evict_gb300 as qe

    def state():
        k = torch.zeros(2, 24, 2, 16, 64, device="cuda", dtype=torch.bfloat16)
        return qe.PagePool(k, torch.zeros_like(k)), qe.PageTable.empty(4, 8, 24, k.device)

    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    k, q = torch.randn(30, 2, 64, device="cuda").bfloat16(), torch.randn(30, 4, 64, device="cuda").bfloat16()
    rows, lens, starts, page = ints(0, 1), ints(20, 10), ints(0, 20, 30), ints(23)
    rope = qe.Rope(64)

    def steps(pool, seqs):
        return [lambda: pool.resize(seqs, rows, lens), lambda: pool.append(1, k, k, starts, seqs, rows=rows, q=q, rope=rope),
                lambda: pool.attend(1, q, starts, seqs, rows=rows), lambda: pool.fork(seqs, ints(0), ints(2)), lambda: pool.free(seqs, ints(1)),
                lambda: pool.compact(seqs), lambda: pool.copy(ints(0), page), lambda: pool.gather(1, seqs, 0, 20), lambda: pool.check()]

    here, there = state(), state()
    want = [f() for f in steps(*here)]
    got = [in_thread(f) for f in steps(*there)]
    for a, b in zip(want, got):
        for x, y in zip(*((t if isinstance(t, tuple) else (t,)) for t in (a, b))):
            assert x is y is None or torch.equal(x, y)
    for a, b in ((here[0].k, there[0].k), (here[1].table, there[1].table), (here[1].refs, there[1].refs)):
        assert torch.equal(a, b)


def test_threads_that_share_a_pool(torch):
    """Each on a stream of its own, over rows that are cut (so that each needs scratch)."""
    import tiered_quantize_evict_gb300 as qe
    c = Case(torch, [5000, 1500, 900], hkv=2, d=128, ps=32)
    pool, seqs = c.objects(qe)
    q, starts = c.draw(6, 8, 128).to(c.dev), c.ints([0, 3, 4, 6])
    want = {hint: pool.attend(0, q, starts, seqs, max_q_len=hint) for hint in (0, 1, 3, 16)}
    torch.cuda.synchronize()
    outs = {}

    def work(hint):
        with torch.cuda.stream(torch.cuda.Stream()):
            outs[hint] = [pool.attend(0, q, starts, seqs, max_q_len=hint) for _ in range(50)]
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(hint,)) for hint in want]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for hint, x in want.items():
        assert all(torch.equal(x, y) for y in outs[hint])
    pool.check()


def test_numbers_outside_of_a_c_int(torch):
    import tiered_quantize_evict_gb300 as qe
    c = Case(torch, [40], hkv=1, d=64, ps=16, layers=2)
    pool, seqs = c.objects(qe)
    q, k, starts = c.draw(1, 1, 64).to(c.dev), c.draw(1, 1, 64).to(c.dev), c.ints([0, 1])
    for bad in (2 ** 32, 2 ** 32 + 1, -2 ** 32, 2 ** 63, 2, -1):
        with pytest.raises(qe.QEError, match="layer"):
            pool.attend(bad, q, starts, seqs)
        with pytest.raises(qe.QEError, match="layer"):
            pool.append(bad, k, k, starts, seqs)
        with pytest.raises(qe.QEError, match="layer"):
            pool.gather(bad, seqs, 0, 8)
    for start, n in ((2 ** 32, 8), (-2 ** 32, 8), (0, 2 ** 40), (2 ** 31 - 1, 8), (-1, 8), (0, -1)):
        with pytest.raises(qe.QEError, match="start"):
            pool.gather(0, seqs, start, n)
    for bad in (2 ** 31, 2 ** 40, -1, -2 ** 40):
        with pytest.raises(qe.QEError, match="max_q_len"):
            pool.attend(0, q, starts, seqs, max_q_len=bad)


def test_the_tiered_cache_takes_no_fp16(torch):
    """Its keys, values and queries are bf16: fp16 bits are not read as if they were."""
    import tiered_quantize_evict_gb300 as qe
    c = Case(torch, [40], hkv=1, d=64, ps=16, dtype="fp16")
    pool, seqs = c.objects(qe)
    k, v = pool.gather(0, seqs, 0, 32)
    cfg = qe.QEConfig(batch=1, n_layers=1, n_q_heads=4, n_kv_heads=1, head_dim=64, window=16, route_period=16, n_sink=4, n_recent=16,
                      max_context=512, cap_mode=0, kf=8, kq=8, out_fp32=0)
    cache = qe.QECache(cfg, torch.cuda.current_stream().cuda_stream)
    for a, b in ((k, v), (k.bfloat16(), v), (k, v.bfloat16()), (k.cpu().numpy(), v.cpu().numpy())):
        with pytest.raises(qe.QEError, match="bf16"):
            cache.qe_append(0, a, b, 32)
    cache.qe_append(0, k.bfloat16(), v.bfloat16(), 32)
    cache.qe_synchronize()
    cache.close()


def test_calls_of_no_token(torch):
    """Empty chunks, as empty tensors come: with strides of 0 from numpy."""
    import tiered_quantize_evict_gb300 as qe
    c = Case(torch, [40], hkv=2, d=64, ps=16)
    pool, seqs = c.objects(qe)
    before = c.k.clone()
    for x, q in ((torch.zeros(0, 2, 64), torch.zeros(0, 4, 64)), (torch.from_numpy(np.zeros((0, 2, 64), np.float32)), torch.from_numpy(np.zeros((0, 4, 64), np.float32)))):
        x, q = x.to(c.dt).to(c.dev), q.to(c.dt).to(c.dev)
        assert pool.append(0, x, x, c.ints([0, 0]), seqs, q=q, rope=qe.Rope(64)).shape == (0, 4, 64)
        out, lse = pool.attend(0, q, c.ints([0, 0]), seqs, return_lse=True)
        assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    none = c.ints(np.zeros(0))
    pool, seqs = c.objects(qe, refs=True)
    pool.resize(seqs, none, none)
    pool.fork(seqs, none, none)
    pool.copy(none, none)
    assert pool.gather(0, seqs, 5, 0)[0].shape == (1, 2, 0, 64) and pool.gather(0, seqs, 0, 8, rows=none)[1].shape == (0, 2, 8, 64)
    pool.check()
    assert torch.equal(c.k.view(torch.int16), before.view(torch.int16))
