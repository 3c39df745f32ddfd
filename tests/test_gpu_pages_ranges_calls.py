"""Windows, shared prefixes and dropped pages: as many sequences as a call takes, other threads, odd strides, rows and groups of all kinds."""
import threading

import numpy as np
import pytest

from oracle import pages as op
from pages_ranges_testlib import bits, check, seen_bounds
from pages_testlib import Case
from test_gpu_pages_shared import run as run_shared

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return pytest.importorskip("torch")


@pytest.mark.parametrize("hint", [0, 3])
@pytest.mark.parametrize("kind", ["window", "shared"])
def test_as_many_sequences_as_a_call_takes(torch, kind, hint):
    """65536 sequences of up to 3 tokens over three rows; sampled against float64."""
    import tiered_quantize_evict_gb300 as qe
    n, d, hq = 65536, 64, 2
    c = Case(torch, [300, 35, 37], hkv=1, d=d, ps=16)
    c.kh[2][:, :32], c.vh[2][:, :32] = c.kh[1][:, :32], c.vh[1][:, :32]
    c.table[2, :2] = c.table[1, :2]
    pool, seqs = c.objects(qe)
    rng = np.random.default_rng(2)
    m, rows = rng.integers(0, 4, n), rng.integers(1, 3, n) if kind == "shared" else rng.integers(0, 3, n)
    starts = np.cumsum([0, *m])
    q = c.draw(int(starts[-1]), hq, d)
    if kind == "window":
        out = pool.attend(0, q.to(c.dev), c.ints(starts), seqs, rows=c.ints(rows), max_q_len=hint, window=20, sinks=3).cpu()
    else:
        size = rng.integers(0, 5, n)
        gs = np.minimum(np.cumsum([0, *size]), n)
        gs[-1] = n
        out = pool.attend_shared(0, q.to(c.dev), c.ints(starts), seqs, c.ints(gs), c.ints(rng.integers(0, 2, n) * 32), rows=c.ints(rows),
                                 max_group_len=hint).cpu()
    pool.check()
    assert torch.isfinite(out).all()
    for i in [0, 1, n - 2, n - 1, *rng.integers(0, n, 300)]:
        a, b, r = starts[i], starts[i + 1], rows[i]
        if b > a:
            k = c.lens[r]
            seen = op.window_seen(b - a, k, 20, 3) if kind == "window" else [range(k - (b - a) + j + 1) for j in range(b - a)]
            want = seen_bounds(torch, c.dt, bits(q[a:b]), bits(c.kh[r][0]), bits(c.vh[r][0]), 1, d ** -0.5, seen)
            check(bits(out[a:b]), None, want, i)


def test_groups_of_all_kinds(torch):
    """Chunks longer than the cache that fill both halves, a first sequence that only holds the prefix, prefixes of part of a page."""
    run_shared(torch, [(0, [(300, 40), (1, 5)]), (0, [(140, 0)]), (160, [(0, 0), (40, 60), (60, 60)]), (15, [(1, 1), (70, 70)])], hq=4, hkv=1, d=64, ps=16)
    run_shared(torch, [(0, [(300, 40), (1, 5)]), (0, [(140, 0)]), (160, [(0, 0), (40, 60), (60, 60)])], hq=2, hkv=2, d=128, ps=32, dtype="fp16")


def test_one_row_many_times(torch):
    """Sequences of one call that are the same row: samples that have not parted yet."""
    import tiered_quantize_evict_gb300 as qe
    c = Case(torch, [10, 200], hkv=2, d=64, ps=16)
    pool, seqs = c.objects(qe)
    q = c.draw(40, 8, 64)
    for hint in (0, 40):
        got = pool.attend_shared(0, q.to(c.dev), c.ints(range(41)), seqs, c.ints([0, 40]), c.ints([199]), rows=c.ints([1] * 40), max_group_len=hint)
        pool.check()
        for i in range(40):
            want = seen_bounds(torch, c.dt, bits(q[i:i + 1]), bits(c.kh[1][0]), bits(c.vh[1][0]), 2, 0.125, [range(200)])
            check(bits(got[i:i + 1]), None, want, i)


@pytest.mark.parametrize("pad", [8, 24, 64])
def test_padded_pages(torch, pad):
    """Pages a few elements further apart than their heads take: heads and pages have but 8 elements in common."""
    import tiered_quantize_evict_gb300 as qe
    c = Case(torch, [500, 260], hkv=2, d=128, ps=16)
    room = 2 * 16 * 128 + pad
    flat = torch.full((2, c.n_pages * room), float("nan"), dtype=c.dt, device=c.dev)
    k, v = (x.as_strided((1, c.n_pages, 2, 16, 128), (room, room, 16 * 128, 128, 1), x.storage_offset()) for x in (flat[0], flat[1]))
    k.copy_(c.k)
    v.copy_(c.v)
    pool, seqs = qe.PagePool(k, v), qe.PageTable(c.ints(c.table), c.ints(c.kv_len))
    for m, hint in ((2, 2), (20, 20), (150, 0)):
        q = c.draw(2 * m, 8, 128)
        for window in (None, 100):
            got = pool.attend(0, q.to(c.dev), c.ints([0, m, 2 * m]), seqs, max_q_len=hint, window=window)
            pool.check()
            for r in range(2):
                n = c.lens[r]
                want = seen_bounds(torch, c.dt, bits(q[r * m:(r + 1) * m]), bits(c.kh[r][0]), bits(c.vh[r][0]), 2, 128 ** -0.5,
                                   op.window_seen(m, n, window or n, 0))
                check(bits(got[r * m:(r + 1) * m]), None, want, f"{m} tokens, window {window}, row {r}")


def test_threads_that_share_a_pool(torch):
    """Each on a stream of its own, over rows that are cut (so that each needs scratch)."""
    import tiered_quantize_evict_gb300 as qe
    c = Case(torch, [5000, 1500, 900], hkv=2, d=128, ps=32)
    pool, seqs = c.objects(qe)
    q, starts, gs, pre = c.draw(6, 8, 128).to(c.dev), c.ints([0, 3, 4, 6]), c.ints([0, 1, 3]), c.ints([0, 640])
    calls = {"w0": lambda: pool.attend(0, q, starts, seqs, window=1400, sinks=70), "w3": lambda: pool.attend(0, q, starts, seqs, window=700, max_q_len=3),
             "s0": lambda: pool.attend_shared(0, q, starts, seqs, gs, pre), "s3": lambda: pool.attend_shared(0, q, starts, seqs, gs, pre, max_group_len=3)}
    want = {k: f() for k, f in calls.items()}
    torch.cuda.synchronize()
    outs = {}

    def work(k):
        with torch.cuda.stream(torch.cuda.Stream()):
            outs[k] = [calls[k]() for _ in range(50)]
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(k,)) for k in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for k, x in want.items():
        assert all(torch.equal(x, y) for y in outs[k]), k
    pool.check()


def test_what_sees_dropped_pages_reports_them(torch):
    import tiered_quantize_evict_gb300 as qe
    c = Case(torch, [300, 300], hkv=1, d=64, ps=16, spare=8)
    pool, seqs = c.objects(qe, refs=True)
    pool.drop(seqs, c.ints([0]), 100, sinks=16)
    q, starts = c.draw(2, 4, 64).to(c.dev), c.ints([0, 1, 2])
    pool.attend(0, q, starts, seqs, window=100, sinks=16, max_q_len=1)
    pool.check()
    for call in (lambda: pool.attend(0, q, starts, seqs, max_q_len=1), lambda: pool.attend(0, q, starts, seqs, window=200, sinks=16),
                 lambda: pool.attend_shared(0, q, starts, seqs, c.ints([0, 1, 2]), c.ints([0, 0])), lambda: pool.gather(0, seqs, 0, 300)):
        call()
        with pytest.raises(qe.QEError, match="page index"):
            pool.check()
    pool.gather(0, seqs, 208, 92)
    pool.check()


def test_refusals_of_the_binding(torch):
    import tiered_quantize_evict_gb300 as qe
    c = Case(torch, [40, 30], hkv=1, d=64, ps=16)
    pool, seqs = c.objects(qe, refs=True)
    q, starts = c.draw(2, 1, 64).to(c.dev), c.ints([0, 1, 2])
    for w, s in ((0, 0), (-1, 0), (2 ** 31, 0), (2 ** 40, 0), (5, -1), (5, 2 ** 31)):
        with pytest.raises(qe.QEError, match="window"):
            pool.attend(0, q, starts, seqs, window=w, sinks=s)
        with pytest.raises(qe.QEError, match="window"):
            pool.drop(seqs, c.ints([0]), w, sinks=s)
    with pytest.raises(qe.QEError, match="sinks"):
        pool.attend(0, q, starts, seqs, sinks=3)
    with pytest.raises(qe.QEError, match="causal"):
        pool.attend(0, q, starts, seqs, window=3, causal=False)
    gs, pre = c.ints([0, 2]), c.ints([16])
    for bad in (dict(group_start=c.ints([0, 1, 2])), dict(group_start=gs.long()), dict(group_start=gs.cpu()), dict(prefix_len=pre.float()),
                dict(prefix_len=pre.cpu()), dict(prefix_len=c.ints([[16]])), dict(max_group_len=-1), dict(max_group_len=2 ** 31)):
        with pytest.raises(qe.QEError):
            pool.attend_shared(0, q, starts, seqs, **{**dict(group_start=gs, prefix_len=pre), **bad})
    with pytest.raises(qe.QEError, match="layer"):
        pool.attend_shared(1, q, starts, seqs, gs, pre)
    with pytest.raises(qe.QEError, match="refs"):
        pool.drop(qe.PageTable(seqs.table, seqs.kv_len), c.ints([0]), 4)
    with pytest.raises(qe.QEError, match="rows"):
        pool.drop(seqs, torch.zeros(1, dtype=torch.int64, device=c.dev), 4)
    none = torch.zeros(0, 1, 64, dtype=c.dt, device=c.dev)
    assert pool.attend(0, none, c.ints([0]), seqs, window=3).shape == none.shape
    assert pool.attend_shared(0, none, c.ints([0]), seqs, c.ints([0]), c.ints([])).shape == none.shape
    pool.check()
