"""Paged cache: inputs, positions and tables that are slices of larger tensors, and as many sequences as a call takes."""
import numpy as np
import pytest

from oracle import pages as op
from pages_testlib import Case, attend_bounds, bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return pytest.importorskip("torch")


def slices(torch, c, total, heads, kind):
    """(tensor of random values as the kernels get it, the same on the host)."""
    x = c.draw(total, heads, c.d)
    if kind == "fused":      # heads of a fused projection, with channels of another width
        y = torch.full((total, heads + 3, c.d + 16), float("nan"), dtype=c.dt, device=c.dev)[:, 2:-1, 8:-8]
    else:                    # heads before tokens
        y = torch.full((heads, total + 1, c.d), float("nan"), dtype=c.dt, device=c.dev)[:, 1:].transpose(0, 1)
    y.copy_(x)
    return y, x


@pytest.mark.parametrize("kind", ["fused", "heads_first"])
@pytest.mark.parametrize("d,rot,halves", [(64, 64, False), (128, 96, True), (64, 16, True), (128, 2, False), (64, 48, True), (128, 6, False)])
@pytest.mark.parametrize("in_place", [False, True])
def test_append_from_slices(torch, kind, d, rot, halves, in_place):
    import tiered_quantize_evict_gb300 as qe
    chunks = [(3, 40), (0, 5), (30, 33), (1, 1)]
    c = Case(torch, [n for _, n in chunks], hkv=2, d=d, ps=16, layout="token_major", seed=rot)
    pool, seqs = c.objects(qe)
    total, hq = sum(m for m, _ in chunks), 6
    starts = np.cumsum([0] + [m for m, _ in chunks])
    (k, kh), (v, vh), (q, qh) = (slices(torch, c, total, h, kind) for h in (2, 2, hq))
    wide = c.ints(c.rng.integers(0, 10 ** 6, (2, total + 5)))
    pos, axis = wide[:, 3:-2], [i % 2 for i in range(rot // 2)]
    f = [1e4 ** (-2 * i / rot) for i in range(rot // 2)]
    out = q if in_place else slices(torch, c, total, hq, kind)[0]
    got = pool.append(0, k, v, c.ints(starts), seqs, q=q, rope=qe.Rope(d, rot_dim=rot, axis=axis, inv_freq=f, halves=halves) if rot > 2 else
                      qe.Rope(d, rot_dim=rot, sections=[1, 0], inv_freq=f), positions=pos, q_out=out)
    pool.check()
    assert got is out
    p = pos.cpu().numpy()
    u = 2.0 ** -8

    def near(got, x):     # one rounding, float32 products, sine and cosine off by at most 2^-21
        want = op.rotate(bits(x), p, axis, f, rot, halves)
        assert (np.abs(got - want) <= u * np.abs(want) + 2.0 ** -19 * np.abs(bits(x)).max(-1, keepdims=True)).all()

    near(bits(out), qh)
    seq = np.repeat(np.arange(len(chunks)), [m for m, _ in chunks])
    at = np.array([n - m for m, n in chunks])[seq] + np.arange(total) - starts[seq]
    page, tok = torch.from_numpy(c.table[seq, at // 16].astype(np.int64)).to(c.dev), torch.from_numpy(at % 16).to(c.dev)
    near(bits(c.k[0][page, :, tok]), kh)
    assert torch.equal(c.v[0][page, :, tok].cpu(), vh)


def test_tables_that_are_slices(torch):
    """A run of every call on a table whose rows are parts of wider ones; what lies beside them is left."""
    import tiered_quantize_evict_gb300 as qe
    P, S, H, D = 40, 16, 1, 64
    k = torch.randn(2, P, H, S, D, device="cuda").bfloat16()
    dev = k.device
    ints = lambda x: torch.tensor(np.asarray(x, np.int32)).to(dev)  # noqa: E731
    o, runs = op.Pages(5, 6, P, S), []
    for wide in (False, True):
        base = torch.full((5, 11), 77, dtype=torch.int32, device=dev)
        table = base[:, 2:8] if wide else torch.empty(5, 6, dtype=torch.int32, device=dev)
        table.fill_(-1)
        pool = qe.PagePool(k.clone(), k.clone())
        seqs = qe.PageTable(table, torch.zeros(5, dtype=torch.int32, device=dev), torch.zeros(P, dtype=torch.int32, device=dev))
        pool.resize(seqs, ints([0, 3]), ints([50, 90]))
        pool.fork(seqs, ints([3, 0]), ints([1, 4]))
        pool.resize(seqs, ints([1, 0]), ints([70, 5]))
        pool.free(seqs, ints([3]))
        q = k[0, :10, 0, :4].reshape(-1, 1, D).contiguous()
        x = pool.append(1, q, q, ints([0, 5, 40]), seqs, rows=ints([0, 1]), q=q, rope=qe.Rope(D))
        a = pool.attend(1, x, ints([0, 5, 40]), seqs, rows=ints([4, 1]))
        g = pool.gather(1, seqs, 3, 60)
        kept = seqs.table.clone()
        out = torch.full((5, 11), 78, dtype=torch.int32, device=dev)[:, 2:8] if wide else torch.empty_like(table)
        refs = torch.empty_like(seqs.refs)
        pool.compact(seqs, table_out=out, refs_out=refs)
        pool.check()
        runs.append([x, a, *g, kept, out.clone(), refs, pool.k, pool.v])
        if wide:
            assert (base[:, :2] == 77).all() and (base[:, 8:] == 77).all()
    assert all(torch.equal(x, y) for x, y in zip(*runs))
    o.resize([0, 3], [50, 90])
    o.fork([3, 0], [1, 4])
    o.resize([1, 0], [70, 5])
    o.resize([3], [0])
    assert runs[0][4].cpu().tolist() == o.table


@pytest.mark.parametrize("hint", [0, 1])
def test_most_sequences(torch, hint):
    """65536 sequences of up to 3 tokens over three rows; sampled against float64."""
    import tiered_quantize_evict_gb300 as qe
    n, d, hq = 65536, 64, 2
    c = Case(torch, [300, 17, 5], hkv=1, d=d, ps=16)
    pool, seqs = c.objects(qe)
    rng = np.random.default_rng(2)
    m, rows = rng.integers(0, 4, n), rng.integers(0, 3, n)
    starts = np.cumsum([0, *m])
    q = c.draw(int(starts[-1]), hq, d)
    out = pool.attend(0, q.to(c.dev), c.ints(starts), seqs, rows=c.ints(rows), max_q_len=hint).cpu()
    pool.check()
    assert torch.isfinite(out).all()
    for i in [0, 1, n - 2, n - 1, *rng.integers(0, n, 300)]:
        a, b = starts[i], starts[i + 1]
        if b > a:
            ref, tol, _, _ = attend_bounds(torch, c, bits(q[a:b]), int(b - a), rows[i], hq, d ** -0.5, True)
            assert (np.abs(bits(out[a:b]) - ref) <= tol).all(), i
