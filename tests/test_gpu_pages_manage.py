"""Appending with rotary positions, resizing, forking, compacting, copying and gathering pages, against the oracle."""
import numpy as np
import pytest

from oracle import pages as op
from pages_testlib import Case, bits, cdiv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return pytest.importorskip("torch")


def make_axis(kind, n):
    if kind == "one":
        return [0] * n, 1
    if kind == "sections":
        return [0] * (n // 4) + [1] * (n // 2 - n // 4) + [2] * (n - n // 2), 3
    return [i % 3 for i in range(n)], 3   # interleaved


def check_rotated(torch, dt, got, want, x):
    """One rounding of the result, float32 products and sums, and the sine and cosine off by at most 2^-21 (the angle
    as a signed 32-bit fraction of a half turn, rounded to float32: 2^-25 of a half turn; sincospif itself 2^-22)."""
    u = float(torch.finfo(dt).eps) / 2
    tol = u * np.abs(want) + 2.0 ** -20 * np.abs(x).max(-1, keepdims=True) * 2 + (2.0 ** -25 if dt == torch.float16 else 0)
    err = np.abs(got - want)
    assert (err <= tol).all(), f"off by {err.max():.3e}"


@pytest.mark.parametrize("d,rot", [(64, 64), (128, 128), (128, 96), (64, 32), (128, 0)])
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("axes", ["one", "sections", "interleaved"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_append(torch, d, rot, halves, axes, dtype):
    import tiered_quantize_evict_gb300 as qe
    chunks = [(1, 1), (5, 40), (0, 9), (33, 33), (2, 66)]
    hq, hkv, ps = 6, 2, 16
    c = Case(torch, [n for _, n in chunks], hkv=hkv, d=d, ps=ps, dtype=dtype, layers=2, layout="kv_together", seed=d + rot)
    pool, seqs = c.objects(qe)
    before = [c.k.clone(), c.v.clone()]
    total = sum(m for m, _ in chunks) + 2     # two packed tokens behind the last sequence
    starts = np.cumsum([0] + [m for m, _ in chunks])
    k, v, q = (c.draw(total, h, d) for h in (hkv, hkv, hq))
    axis, n_axes = make_axis(axes, rot // 2)
    pos = c.rng.integers(-5, 2 ** 20, (n_axes, total)).astype(np.int32)
    pos[:, 0] = 2 ** 31 - 1
    pos[:, 1] = -2 ** 31
    f = [1e4 ** (-2 * i / max(rot, 1)) for i in range(rot // 2)]
    rope = qe.Rope(d, rot_dim=rot, axis=axis, inv_freq=f, halves=halves)
    qo = torch.full_like(q, 3.0).to(c.dev)
    got = pool.append(1, k.to(c.dev), v.to(c.dev), c.ints(starts), seqs, q=q.to(c.dev), rope=rope,
                      positions=c.ints(pos[: rope.n_axes]), q_out=qo)
    pool.check()
    assert got is qo
    end = starts[-1]
    want = op.rotate(bits(q), pos, axis, f, rot, halves)
    check_rotated(torch, c.dt, bits(got)[:end], want[:end], bits(q)[:end])
    assert (got[end:] == 3).all()
    kw = op.rotate(bits(k), pos, axis, f, rot, halves)
    same = torch.zeros(c.n_pages, ps, dtype=torch.bool, device=c.dev)
    for r, ((m, n), a) in enumerate(zip(chunks, starts)):
        for j in range(m):
            p, t = c.table[r][(n - m + j) // ps], (n - m + j) % ps
            same[p, t] = True
            check_rotated(torch, c.dt, bits(c.k[1, p, :, t]), kw[a + j], bits(k[a + j]))
            assert torch.equal(c.v[1, p, :, t].cpu(), v[a + j])
    keep = (~same)[None, :, None, :, None].expand_as(c.k[1:])
    bit16 = lambda x: x.contiguous().view(torch.int16)  # noqa: E731
    for now, was in zip((c.k, c.v), before):
        assert torch.equal(bit16(now[0]), bit16(was[0]))
        assert torch.equal(bit16(now[1:])[keep], bit16(was[1:])[keep])


def test_append_without_queries_positions_or_rope(torch):
    import tiered_quantize_evict_gb300 as qe
    c = Case(torch, [20, 7], hkv=1, d=64, ps=16)
    pool, seqs = c.objects(qe)
    k, v, q = (c.draw(5, h, 64) for h in (1, 1, 2))
    starts = c.ints([0, 3, 5])
    rope = qe.Rope(64, theta=500.0)
    assert pool.append(0, k.to(c.dev), v.to(c.dev), starts, seqs, rope=rope) is None
    pos = np.array([[17, 18, 19, 5, 6]])
    f = [500.0 ** (-2 * i / 64) for i in range(32)]
    want = op.rotate(bits(k), pos, [0] * 32, f, 64, False)
    for i, (r, p) in enumerate([(0, 17), (0, 18), (0, 19), (1, 5), (1, 6)]):
        check_rotated(torch, c.dt, bits(c.k[0, c.table[r][p // 16], :, p % 16]), want[i], bits(k[i]))
    # in place queries, row order, no rotation: everything is copied bit for bit
    qd = q.to(c.dev)
    out = pool.append(0, k.to(c.dev), v.to(c.dev), c.ints([0, 2, 5]), seqs, rows=c.ints([1, 0]), q=qd, q_out=qd)
    assert out is qd and torch.equal(qd.cpu(), q)
    for i, (r, p) in enumerate([(1, 5), (1, 6), (0, 17), (0, 18), (0, 19)]):
        assert torch.equal(c.k[0, c.table[r][p // 16], :, p % 16].cpu(), k[i])


@pytest.mark.parametrize("n,most,hq,hkv,d,rot,halves", [(1100, 3, 5, 3, 64, 64, True), (40, 130, 16, 1, 128, 32, False), (3, 900, 1, 1, 128, 128, True)])
def test_append_many_tokens(torch, n, most, hq, hkv, d, rot, halves):
    """More sequences than two steps of the search tell apart, more tokens than blocks; chunks of no token among them."""
    import tiered_quantize_evict_gb300 as qe
    rng = np.random.default_rng(n)
    m = rng.integers(0, most + 1, n)
    lens = m + rng.integers(0, 20, n)
    ps = 16
    c = Case(torch, lens.tolist(), hkv=hkv, d=d, ps=ps)
    pool, seqs = c.objects(qe)
    starts = np.cumsum([0, *m])
    total = int(starts[-1])
    k, v, q = (c.draw(total, h, d) for h in (hkv, hkv, hq))
    f = [1e4 ** (-2 * i / rot) for i in range(rot // 2)]
    got = pool.append(0, k.to(c.dev), v.to(c.dev), c.ints(starts), seqs, q=q.to(c.dev), rope=qe.Rope(d, rot_dim=rot, halves=halves))
    pool.check()
    seq = np.repeat(np.arange(n), m)
    pos = lens[seq] - m[seq] + np.arange(total) - starts[seq]
    axis = [0] * (rot // 2)
    check_rotated(torch, c.dt, bits(got), op.rotate(bits(q), pos[None].astype(np.int32), axis, f, rot, halves), bits(q))
    page, row = torch.from_numpy(c.table[seq, pos // ps].astype(np.int64)).to(c.dev), torch.from_numpy(pos % ps).to(c.dev)
    check_rotated(torch, c.dt, bits(c.k[0][page, :, row]), op.rotate(bits(k), pos[None].astype(np.int32), axis, f, rot, halves), bits(k))
    assert torch.equal(c.v[0][page, :, row].cpu(), v)


def test_append_longer_than_the_cache_drops_keys(torch):
    import tiered_quantize_evict_gb300 as qe
    c = Case(torch, [3, 0], hkv=1, d=64, ps=16, garbage=0.0)
    pool, seqs = c.objects(qe)
    before = c.k.clone()
    k, v = c.draw(7, 1, 64), c.draw(7, 1, 64)
    pool.append(0, k.to(c.dev), v.to(c.dev), c.ints([0, 5, 7]), seqs)
    pool.check()
    page = c.table[0][0]
    assert torch.equal(c.k[0, page, :, :3].cpu(), k[2:5].transpose(0, 1))
    c.k[0, page, :, :3] = before[0, page, :, :3]
    assert torch.equal(c.k, before)


def test_append_bad_pages_and_starts(torch):
    """Tokens on pages outside the pool, of rows that do not exist and behind wrong starts are dropped and reported."""
    import tiered_quantize_evict_gb300 as qe
    c = Case(torch, [40, 20], hkv=1, d=64, ps=16, garbage=0.0)
    k, v = c.draw(6, 1, 64).to(c.dev), c.draw(6, 1, 64).to(c.dev)
    c.table[0, 2], c.table[1, 1] = -1, c.n_pages
    pool, seqs = c.objects(qe)
    before = c.k.clone(), c.v.clone()
    pool.append(0, k, v, c.ints([0, 4, 6]), seqs)
    with pytest.raises(qe.QEError, match="page index"):
        pool.check()
    for starts, rows in (([4, 2, 1], [0, 1]), ([-3, -1, -1], [0, 1]), ([0, 3, 6], [2, -1])):
        pool.append(0, k, v, c.ints(starts), seqs, rows=c.ints(rows))
        with pytest.raises(qe.QEError, match="row"):
            pool.check()
    assert torch.equal(c.k, before[0]) and torch.equal(c.v, before[1])


def as_lists(seqs):
    return seqs.table.cpu().tolist(), seqs.kv_len.cpu().tolist(), seqs.refs.cpu().tolist()


def same_books(seqs, o):
    t, n, r = as_lists(seqs)
    assert t == o.table and n == o.kv_len and r == o.refs


@pytest.mark.parametrize("ps,layout", [(16, "plain"), (64, "token_major"), (128, "kv_together")])
def test_books_follow_the_oracle(torch, ps, layout):
    """A random run of resizes, forks, frees and compactions; contents are followed by tagging every token."""
    import tiered_quantize_evict_gb300 as qe
    rng = np.random.default_rng(ps)
    L, H, D, P, R, cols = 3, 2, 64, 60, 12, 9
    c = Case(torch, [0], hkv=H, d=D, ps=ps, layers=L, layout=layout, spare=P, garbage=0.0)
    assert c.n_pages == P
    c.k.copy_(c.draw(L, P, H, ps, D))
    c.v.copy_(c.draw(L, P, H, ps, D))
    pool = qe.PagePool(c.k, c.v)
    seqs = qe.PageTable.empty(R, cols, P, c.dev)
    o = op.Pages(R, cols, P, ps)
    hk, hv = c.k.cpu().clone(), c.v.cpu().clone()

    def copied(pairs):
        for a, b, n in pairs:
            hk[:, b, :, :n] = hk[:, a, :, :n].clone()
            hv[:, b, :, :n] = hv[:, a, :, :n].clone()

    short = 0
    for step in range(60):
        kind = rng.choice(["resize", "fork", "free", "compact"], p=[0.45, 0.3, 0.15, 0.1])
        if kind == "fork":
            empty = [r for r in range(R) if o.kv_len[r] == 0]
            dst = rng.permutation(empty)[: rng.integers(1, 4)].tolist()
            if not dst:
                continue
            src = rng.choice([r for r in range(R) if r not in dst], len(dst)).tolist()
            pairs = o.fork(src, dst)
            pool.fork(seqs, c.ints(src), c.ints(dst))
        elif kind == "compact":
            pairs, n = o.compact()
            got = c.ints([0])
            pool.compact(seqs, n_live=got)
            assert got.item() == n
        else:
            rows = rng.permutation(R)[: rng.integers(1, 5)].tolist()
            lens = [0] * len(rows) if kind == "free" else rng.integers(0, cols * ps + 1, len(rows)).tolist()
            pairs = o.resize(rows, lens)
            if kind == "free":
                pool.free(seqs, c.ints(rows))
            else:
                pool.resize(seqs, c.ints(rows), c.ints(lens))
        if pairs is None:
            short += 1
            with pytest.raises(qe.QEError, match="free pages"):
                pool.check()
        else:
            pool.check()
            copied(pairs)
        same_books(seqs, o)
        assert torch.equal(c.k.cpu(), hk) and torch.equal(c.v.cpu(), hv), f"step {step} ({kind}): contents"
    assert short > 0


def test_many_pages_and_rows(torch):
    """More entries, rows and pages than one block has threads."""
    import tiered_quantize_evict_gb300 as qe
    P, R, cols, ps = 5000, 1500, 4, 16
    k = torch.zeros(1, P, 1, ps, 64, dtype=torch.bfloat16, device="cuda")
    pool = qe.PagePool(k, torch.zeros_like(k))
    seqs = qe.PageTable.empty(R, cols, P, k.device)
    o = op.Pages(R, cols, P, ps)
    rng = np.random.default_rng(1)
    ints = lambda x: torch.tensor(np.asarray(x, np.int32)).cuda()  # noqa: E731
    rows, lens = rng.permutation(R)[:1200].tolist(), rng.integers(0, cols * ps, 1200).tolist()
    o.resize(rows, lens)
    pool.resize(seqs, ints(rows), ints(lens))
    gone = rng.permutation(rows)[:600].tolist()
    o.resize(gone, [0] * 600)
    pool.free(seqs, ints(gone))
    _, n = o.compact()
    live = ints([0])
    t, r = torch.empty_like(seqs.table), torch.empty_like(seqs.refs)
    old = as_lists(seqs)
    pool.compact(seqs, table_out=t, refs_out=r, n_live=live)
    pool.check()
    assert live.item() == n and t.cpu().tolist() == o.table and r.cpu().tolist() == o.refs and as_lists(seqs) == old


def test_rows_named_wrongly(torch):
    """The first entry that names a row counts; bad entries are skipped and reported; others are done."""
    import tiered_quantize_evict_gb300 as qe
    c = Case(torch, [20, 16, 0, 0], hkv=1, d=64, ps=16, spare=6)
    pool, seqs = c.objects(qe, refs=True)
    o = op.Pages(4, c.table.shape[1], c.n_pages, 16)
    o.table, o.kv_len, o.refs = c.table.tolist(), c.kv_len.tolist(), c.refs.tolist()
    pool.fork(seqs, c.ints([0, 1, 0, 9, 0]), c.ints([2, 2, 1, 3, -1]))   # row 2 twice, row 1 not empty, no rows 9, -1
    o.fork([0], [2])
    with pytest.raises(qe.QEError, match="row"):
        pool.check()
    same_books(seqs, o)
    pool.resize(seqs, c.ints([1, 1, 4, 0, 2]), c.ints([30, 2, 5, -1, 10 ** 6]))
    o.resize([1], [30])
    with pytest.raises(qe.QEError, match="row"):
        pool.check()
    same_books(seqs, o)


def test_copy_pages(torch):
    import tiered_quantize_evict_gb300 as qe
    c = Case(torch, [160], hkv=3, d=128, ps=16, layers=4, layout="token_major", garbage=1.0)
    pool = qe.PagePool(c.k, c.v)
    k, v = c.k.clone(), c.v.clone()
    pool.copy(c.ints([3, 3, 5]), c.ints([0, 1, 5]))
    k[:, 0], k[:, 1], v[:, 0], v[:, 1] = k[:, 3], k[:, 3], v[:, 3], v[:, 3]
    assert torch.equal(c.k, k) and torch.equal(c.v, v)
    pool.check()
    pool.copy(c.ints([3, -1, 0]), c.ints([c.n_pages, 2, 0]))
    with pytest.raises(qe.QEError, match="page index"):
        pool.check()
    assert torch.equal(c.k, k)


@pytest.mark.parametrize("start,n", [(0, 40), (0, 1), (13, 50), (15, 2), (39, 30), (64, 16)])
@pytest.mark.parametrize("rows", [None, [2, 0]])
def test_gather(torch, start, n, rows):
    import tiered_quantize_evict_gb300 as qe
    c = Case(torch, [40, 17, 70], hkv=2, d=64, ps=16, layers=2, layout="kv_together")
    pool, seqs = c.objects(qe)
    k, v = pool.gather(1, seqs, start, n, rows=None if rows is None else c.ints(rows))
    pool.check()
    for i, r in enumerate(range(3) if rows is None else rows):
        for got, x in ((k, c.kh[r][1]), (v, c.vh[r][1])):
            want = torch.zeros(n, 2, 64, dtype=c.dt)
            part = x[start: start + n]
            want[: part.shape[0]] = part
            assert torch.equal(got[i].cpu(), want.transpose(0, 1))


def test_captured_and_replayed(torch):
    """Resize, append, fork, gather and compact in one graph, replayed on a fresh state."""
    import tiered_quantize_evict_gb300 as qe
    c = Case(torch, [20, 0, 0], hkv=1, d=64, ps=16, spare=8, garbage=0.0, max_pages=4)
    pool, seqs = c.objects(qe, refs=True)
    state = [seqs.table, seqs.kv_len, seqs.refs, c.k, c.v]
    saved = [x.clone() for x in state]
    rows, lens, dst, starts = c.ints([0]), c.ints([37]), c.ints([2]), c.ints([0, 17])
    k, v = (c.draw(17, 1, 64).to(c.dev) for _ in range(2))

    def step():
        pool.resize(seqs, rows, lens)
        pool.append(0, k, v, starts, seqs, rows=rows, rope=rope)
        pool.fork(seqs, rows, dst)
        pool.compact(seqs)
        return pool.gather(0, seqs, 0, 40)

    rope = qe.Rope(64)
    want = [x.clone() for x in step()] + [x.clone() for x in state]
    for x, y in zip(state, saved):
        x.copy_(y)
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        out = step()
    for x, y in zip(state, saved):
        x.copy_(y)
    g.replay()
    for x, y in zip(list(out) + state, want):
        assert torch.equal(x, y)
    pool.check()
