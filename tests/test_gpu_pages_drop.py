"""Giving back pages that a window has left, alone and together with the other calls on pages."""
import numpy as np
import pytest

from oracle import pages as op
from pages_ranges_testlib import bits, check, seen_bounds
from pages_testlib import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return pytest.importorskip("torch")


def same_books(seqs, o):
    assert seqs.table.cpu().tolist() == o.table and seqs.kv_len.cpu().tolist() == o.kv_len and seqs.refs.cpu().tolist() == o.refs


def setup(torch, lens, ps, n_pages, cols, rows, **kw):
    import tiered_quantize_evict_gb300 as qe
    k = torch.zeros(1, n_pages, 1, ps, 64, dtype=torch.bfloat16, device="cuda")
    pool, seqs, o = qe.PagePool(k, torch.zeros_like(k)), qe.PageTable.empty(rows, cols, n_pages, k.device), op.Pages(rows, cols, n_pages, ps)
    ints = lambda x: torch.tensor(np.asarray(x, np.int32)).cuda()  # noqa: E731
    pool.resize(seqs, ints(range(len(lens))), ints(lens))
    o.resize(range(len(lens)), lens)
    return qe, pool, seqs, o, ints


@pytest.mark.parametrize("ps", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 0), (16, 16), (17, 4), (100, 65), (300, 0), (2 ** 31 - 1, 0), (1, 2 ** 31 - 1)])
def test_books_follow_the_oracle(torch, ps, window, sinks):
    lens = [0, 1, 15, 16, 17, 255, 256, 257, 1000, 5000]
    qe, pool, seqs, o, ints = setup(torch, lens, ps, 2 * sum(-(-x // ps) for x in lens), 400, 12)
    rows = [9, 0, 1, 2, 3, 4, 5, 6, 8, 11]
    for w, s in ((window, sinks), (window, sinks), (max(1, window // 2), sinks), (window, 0)):
        pool.drop(seqs, ints(rows), w, sinks=s)
        o.drop(rows, w, s)
        same_books(seqs, o)
    pool.check()


def test_with_the_other_calls(torch):
    """A random run of drops between resizes, forks, frees and compactions: books and contents."""
    qe, pool, seqs, o, ints = setup(torch, [0], 16, 80, 12, 10)
    tag = torch.arange(80 * 16, device="cuda").view(80, 1, 16, 1).remainder(251).bfloat16()
    pool.k[0].copy_(tag)
    pool.v[0].copy_(-tag)
    hk = pool.k.cpu().clone()
    rng = np.random.default_rng(3)
    dropped = 0
    for step in range(120):
        kind = rng.choice(["resize", "fork", "free", "compact", "drop"], p=[0.3, 0.2, 0.1, 0.1, 0.3])
        pairs = []
        if kind == "fork":
            dst = [r for r in rng.permutation(10).tolist() if o.kv_len[r] == 0][:2]
            src = rng.choice([r for r in range(10) if r not in dst], len(dst)).tolist()
            pool.fork(seqs, ints(src), ints(dst))
            pairs = o.fork(src, dst)
        elif kind == "compact":
            pool.compact(seqs)
            pairs, _ = o.compact()
        elif kind == "drop":
            rows, window, sinks = rng.permutation(10)[:4].tolist(), int(rng.integers(1, 60)), int(rng.integers(0, 40))
            pool.drop(seqs, ints(rows), window, sinks=sinks)
            o.drop(rows, window, sinks)
        else:
            rows = rng.permutation(10)[: rng.integers(1, 4)].tolist()
            lens = [0 if kind == "free" else int(rng.integers(0, 193)) for _ in rows]
            # (not back to inside of a dropped page)
            lens = [n if n >= o.kv_len[r] or n % 16 == 0 or o.table[r][n // 16] != op.DROPPED else n // 16 * 16 for r, n in zip(rows, lens)]
            pool.resize(seqs, ints(rows), ints(lens))
            pairs = o.resize(rows, lens)
        if pairs is None:
            with pytest.raises(qe.QEError, match="free pages"):
                pool.check()
            pairs = []
        pool.check()
        for a, b, n in pairs:
            hk[:, b, :, :n] = hk[:, a, :, :n].clone()
        same_books(seqs, o)
        assert torch.equal(pool.k.cpu(), hk) and torch.equal(pool.v.cpu(), -hk), f"step {step} ({kind}): contents"
        dropped += sum(p == op.DROPPED for row in o.table for p in row)
        live = {p for row in o.table for p in row if p >= 0}
        assert live == {p for p, r in enumerate(o.refs) if r > 0}
    assert dropped > 0


def test_rows_named_twice_and_wrongly(torch):
    qe, pool, seqs, o, ints = setup(torch, [300, 200], 16, 64, 20, 3)
    pool.drop(seqs, ints([0] * 40 + [1, 0]), 50, sinks=20)
    o.drop([0, 1], 50, 20)
    same_books(seqs, o)
    pool.check()
    for bad in ([-1], [3], [2 ** 31 - 1, 1]):
        pool.drop(seqs, ints(bad), 50, sinks=20)
        with pytest.raises(qe.QEError, match="row"):
            pool.check()
    same_books(seqs, o)


def test_entries_of_no_page_are_reported(torch):
    qe, pool, seqs, o, ints = setup(torch, [300], 16, 64, 20, 1)
    seqs.table[0, 3], seqs.table[0, 5] = -1, 64
    refs = seqs.refs.clone()
    pool.drop(seqs, ints([0]), 100)
    with pytest.raises(qe.QEError, match="page index"):
        pool.check()
    assert (refs - seqs.refs).sum() == 10 and (seqs.table[0, :12] == -2).all()      # 12 pages before token 201, two of them bad


def test_cutting_back_into_a_dropped_page_is_reported(torch):
    qe, pool, seqs, o, ints = setup(torch, [300], 16, 64, 20, 1)
    pool.drop(seqs, ints([0]), 50)
    pool.resize(seqs, ints([0]), ints([100]))
    with pytest.raises(qe.QEError, match="page index"):
        pool.check()
    assert seqs.refs.sum() == 0 and int(seqs.kv_len) == 100
    pool.free(seqs, ints([0]))
    pool.check()
    assert (seqs.table == -1).all()


def test_many_rows_and_long_tables(torch):
    """A sliced table, more rows and entries than the kernel has warps at once."""
    import tiered_quantize_evict_gb300 as qe
    P, R, cols = 300_000, 5000, 80
    k = torch.zeros(1, P, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    pool = qe.PagePool(k, torch.zeros_like(k))
    table = torch.full((R, cols + 5), -9, dtype=torch.int32, device="cuda")[:, 2:-3]
    lens = torch.randint(0, 60 * 16, (R,), device="cuda", dtype=torch.int32)
    need = (lens + 15) // 16
    col = torch.arange(cols, device="cuda", dtype=torch.int32)
    first = need.cumsum(0).to(torch.int32) - need
    table.copy_(torch.where(col[None] < need[:, None], first[:, None] + col[None], -1))
    refs = torch.zeros(P, dtype=torch.int32, device="cuda")
    refs[: int(need.sum())] = 1
    seqs = qe.PageTable(table, lens, refs)
    rows = torch.randperm(R, device="cuda").to(torch.int32)
    pool.drop(seqs, rows, 200, sinks=7)
    pool.check()
    end = ((lens - 199).clamp_min(0) // 16)[:, None]
    gone = (col[None] >= 1) & (col[None] < end)
    want = torch.where(gone, -2, torch.where(col[None] < need[:, None], first[:, None] + col[None], -1))
    assert torch.equal(table, want.to(torch.int32)) and int(refs.sum()) == int(need.sum()) - int(gone.sum())
    one = qe.PageTable(torch.arange(200_000, dtype=torch.int32, device="cuda")[None], torch.tensor([3_200_000], dtype=torch.int32, device="cuda"),
                       torch.ones(P, dtype=torch.int32, device="cuda"))
    pool.drop(one, torch.zeros(1, dtype=torch.int32, device="cuda"), 160, sinks=16)
    pool.check()
    assert (one.table[0, 1:199_990] == -2).all() and one.table[0, 0] == 0 and int(one.table[0, 199_990]) == 199_990 and int(one.refs.sum()) == P - 199_989


def test_generation_under_a_window(torch):
    """Prefill in chunks, then tokens one by one, windows dropped after each step, a fork on the way; against attention over all keys."""
    import tiered_quantize_evict_gb300 as qe
    window, sinks, ps, hq, hkv, d, L = 40, 5, 16, 4, 2, 64, 2
    P = 34
    k = torch.zeros(L, P, hkv, ps, d, dtype=torch.bfloat16, device="cuda")
    pool, seqs = qe.PagePool(k, torch.zeros_like(k)), qe.PageTable.empty(3, 40, P, k.device)
    g = torch.Generator().manual_seed(0)
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    all_k = [[torch.zeros(0, hkv, d).bfloat16() for _ in range(L)] for _ in range(3)]
    all_v = [[torch.zeros(0, hkv, d).bfloat16() for _ in range(L)] for _ in range(3)]
    steps = [([0, 1], [60, 33]), ([0, 1], [50, 70])] + [([0, 1], [1, 1])] * 20 + [("fork",)] + [([0, 1, 2], [1, 3, 2])] * 25
    for step in steps:
        if step[0] == "fork":
            pool.fork(seqs, ints(0), ints(2))
            for x in (all_k, all_v):
                x[2] = [t.clone() for t in x[0]]
            continue
        rows, new = step
        lens = [all_k[r][0].shape[0] + m for r, m in zip(rows, new)]
        pool.resize(seqs, ints(*rows), ints(*lens))
        starts = np.cumsum([0] + new)
        for layer in range(L):
            kn, vn, q = (torch.randn(int(starts[-1]), h, d, generator=g).bfloat16() for h in (hkv, hkv, hq))
            pool.append(layer, kn.cuda(), vn.cuda(), ints(*starts), seqs, rows=ints(*rows))
            got = pool.attend(layer, q.cuda(), ints(*starts), seqs, rows=ints(*rows), max_q_len=max(new), window=window, sinks=sinks)
            for r, m, n, a in zip(rows, new, lens, starts):
                all_k[r][layer] = torch.cat([all_k[r][layer], kn[a:a + m]])
                all_v[r][layer] = torch.cat([all_v[r][layer], vn[a:a + m]])
                want = seen_bounds(torch, torch.bfloat16, bits(q[a:a + m]), bits(all_k[r][layer]), bits(all_v[r][layer]), hkv, d ** -0.5,
                                   op.window_seen(m, n, window, sinks))
                check(bits(got[a:a + m]), None, want, f"row {r} at {n}")
        pool.drop(seqs, ints(*rows), window, sinks=sinks)
    pool.check()
    assert sum(-(-x[0].shape[0] // ps) for x in all_k) > P     # more than the pool could hold
    pool.compact(seqs)
    pool.check()
    held = int((seqs.refs > 0).sum())
    assert held <= 3 * 5     # a page of sinks and the window's four at most, of each row


def test_captured_and_replayed(torch):
    """Resize, window attention and drop in one graph, replayed on a fresh state and then on and on."""
    import tiered_quantize_evict_gb300 as qe
    c = Case(torch, [200, 90], hkv=1, d=64, ps=16, spare=8, garbage=0.0, max_pages=16)
    pool, seqs = c.objects(qe, refs=True)
    state = [seqs.table, seqs.kv_len, seqs.refs]
    saved = [x.clone() for x in state]
    rows, lens, starts, q = c.ints([0, 1]), c.ints([201, 91]), c.ints([0, 1, 2]), c.draw(2, 4, 64).to(c.dev)

    def step():
        pool.resize(seqs, rows, lens)
        out = pool.attend(0, q, starts, seqs, window=30, sinks=2, max_q_len=1)
        pool.drop(seqs, rows, 30, sinks=2)
        lens.add_(1)
        return out

    def eager(n):
        for x, y in zip(state, saved):
            x.copy_(y)
        lens.copy_(c.ints([201, 91]))
        out = [step().clone() for _ in range(n)]
        return out, [x.clone() for x in state]

    want = eager(20)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for x, y in zip(state, saved):
        x.copy_(y)
    lens.copy_(c.ints([201, 91]))
    for i in range(20):
        g.replay()
        assert torch.equal(out, want[0][i])
    for x, y in zip(state, want[1]):
        assert torch.equal(x, y)
    pool.check()
