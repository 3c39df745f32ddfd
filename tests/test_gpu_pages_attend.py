"""qe_pages_attend against float64, over lengths, heads, page sizes, layouts and masks."""
import numpy as np
import pytest

from pages_testlib import Case, attend_bounds, bits

pytestmark = pytest.mark.gpu


def run(torch, chunks, *, hq, hkv, d, ps, dtype="bf16", layout="plain", causal=True, scale=None, q_layout="plain", hint=0, seed=0,
        rows=None, layer=0, layers=1, lse=True, **kw):
    """chunks: (new tokens, kv_len) of each sequence; rows: which table row each is (a permutation)."""
    import tiered_quantize_evict_gb300 as qe
    lens = [0] * len(chunks)
    order = list(range(len(chunks))) if rows is None else list(rows)
    for (m, n), r in zip(chunks, order):
        lens[r] = n
    c = Case(torch, lens, hkv=hkv, d=d, ps=ps, dtype=dtype, layout=layout, layers=layers, seed=seed, **kw)
    pool, seqs = c.objects(qe)
    total = sum(m for m, _ in chunks)
    qh = c.draw(total, hq, d)
    if q_layout == "plain":
        q, out = qh.to(c.dev), torch.full((total, hq, d), float("nan"), dtype=c.dt, device=c.dev)
    elif q_layout == "heads_first":
        q = qh.transpose(0, 1).contiguous().to(c.dev).transpose(0, 1)
        out = torch.full((hq, total, d), float("nan"), dtype=c.dt, device=c.dev).transpose(0, 1)
    else:   # a slice of a fused projection
        q = torch.zeros(total, hq + 2, d + 8, dtype=c.dt, device=c.dev)[:, 1:-1, :d]
        q.copy_(qh)
        out = torch.full((total, hq + 1, d), float("nan"), dtype=c.dt, device=c.dev)[:, :hq]
    starts = np.cumsum([0] + [m for m, _ in chunks])
    s = d ** -0.5 if scale is None else scale
    got = pool.attend(layer, q, c.ints(starts), seqs, rows=None if rows is None else c.ints(rows), scale=scale, causal=causal,
                      max_q_len=hint, out=out, return_lse=lse)
    pool.check()
    o, ls = (bits(got[0]), got[1].cpu().numpy()) if lse else (bits(got), None)
    for (m, n), r, a in zip(chunks, order, starts):
        if m == 0:
            continue
        ref, tol, lref, ltol = attend_bounds(torch, c, bits(qh[a:a + m]), m, r, hq, s, causal, layer)
        err = np.abs(o[a:a + m] - ref)
        assert np.isfinite(o[a:a + m]).all(), f"sequence {r}: not finite"
        assert (err <= tol).all(), f"sequence {r}: error {err.max():.3e}, {np.max(err / np.maximum(tol, 1e-30)):.2f} of the bound"
        if lse:
            x = ls[a:a + m]
            assert np.array_equal(np.isinf(x), np.isinf(lref)) and not np.isnan(x).any()
            fin = np.isfinite(lref)
            off = np.abs(x[fin] - lref[fin])
            assert (off <= ltol[fin]).all(), f"sequence {r}: lse off by {off.max():.3e}"
    return o


@pytest.fixture(scope="module")
def torch():
    return pytest.importorskip("torch")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("ps", [16, 32, 64, 128, 256])
def test_pages_and_types(torch, d, dtype, ps):
    run(torch, [(1, 1), (5, 130), (40, 40), (3, 257)], hq=8, hkv=2, d=d, ps=ps, dtype=dtype, seed=ps + d)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (4, 4), (14, 2), (8, 1), (40, 1), (128, 1)])
def test_head_groups(torch, hq, hkv):
    run(torch, [(9, 70), (1, 33), (2, 2)], hq=hq, hkv=hkv, d=64, ps=16, seed=hq)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 127, 128, 129, 255, 256, 257, 1025])
def test_one_token_lengths(torch, n):
    run(torch, [(1, n), (1, max(1, n - 1))], hq=8, hkv=2, d=128, ps=32, hint=1, seed=n)


@pytest.mark.parametrize("m", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 300])
@pytest.mark.parametrize("hint", [0, 1])
def test_prompt_lengths(torch, m, hint):
    """Whole prompts; the hint may be wrong."""
    run(torch, [(m, m)], hq=4, hkv=2, d=64, ps=16, hint=hint, seed=m)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
def test_empty_rows_and_sequences(torch, causal, d):
    """Chunks longer than the cache (queries before position 0 see nothing), empty caches, empty chunks."""
    o = run(torch, [(5, 3), (0, 17), (4, 0), (300, 40), (1, 0), (2, 129)], hq=4, hkv=2, d=d, ps=16, causal=causal)
    if causal:
        assert not o[:2].any() and not o[9:9 + 260].any()
    assert not o[5:9].any()


def test_cross_attention_lengths(torch):
    """causal = 0: an encoder's states of another length, shorter and longer than the queries."""
    run(torch, [(70, 9), (3, 500), (130, 128), (1, 1)], hq=6, hkv=2, d=128, ps=64, causal=False, dtype="fp16")


@pytest.mark.parametrize("layout", ["plain", "token_major", "kv_together"])
@pytest.mark.parametrize("q_layout", ["plain", "heads_first", "slice"])
def test_layouts(torch, layout, q_layout):
    run(torch, [(7, 100), (20, 20)], hq=6, hkv=3, d=64, ps=32, layout=layout, q_layout=q_layout, layers=3, layer=2)


def test_rows_in_another_order_and_scale(torch):
    run(torch, [(3, 50), (17, 90), (1, 5)], hq=4, hkv=1, d=128, ps=16, rows=[2, 0, 1], scale=0.31)


def test_without_lse(torch):
    run(torch, [(3, 50)], hq=4, hkv=1, d=128, ps=16, lse=False)


@pytest.mark.parametrize("m,n,hint", [(1, 6000, 1), (4, 9001, 4), (130, 2500, 0)])
def test_few_rows_over_a_long_cache(torch, m, n, hint):
    """The long axis is split over the SMs and joined."""
    run(torch, [(m, n)], hq=4, hkv=1, d=128, ps=64, hint=hint)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("m,hq,hkv", [(1, 4, 1), (4, 8, 2), (16, 1, 1), (5, 3, 1), (1, 14, 2), (3, 16, 2), (8, 8, 2), (13, 4, 1), (16, 4, 1),
                                      (9, 14, 2), (1, 128, 1)])
def test_chunks_of_a_few_tokens(torch, d, dtype, causal, m, hq, hkv):
    """The longest chunk is named, so tiles have as few rows as it needs: 1 to 16, to 64, to 128; ragged, some without keys."""
    run(torch, [(m, m), (max(1, m - 1), 300), (m, 1000 + m), (0, 40), (1, 128), (m, max(0, m - 2)), (1, 129), (2 * m + 1, 200)], hq=hq, hkv=hkv, d=d,
        ps=32, dtype=dtype, causal=causal, hint=m, seed=m + hq)


@pytest.mark.parametrize("layout", ["plain", "token_major", "kv_together"])
@pytest.mark.parametrize("q_layout", ["heads_first", "slice"])
@pytest.mark.parametrize("ps", [16, 128, 256])
def test_layouts_of_a_few_tokens(torch, layout, q_layout, ps):
    run(torch, [(2, 500), (1, 20), (2, 1300)], hq=6, hkv=3, d=64, ps=ps, layout=layout, q_layout=q_layout, layers=2, layer=1, hint=2)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("m,hint", [(1, 1), (3, 3), (16, 16), (16, 0), (4, 4), (32, 32)])
def test_long_caches_of_several_sequences(torch, d, m, hint):
    """Every SM walks many blocks, finishes rows and starts others in the middle of them."""
    rng = np.random.default_rng(d + m)
    n = 24 if m < 16 else 10
    run(torch, [(m, int(x)) for x in rng.integers(4000, 9000, n)], hq=4 if m < 16 else 2, hkv=2 if m < 16 else 1, d=d, ps=64, hint=hint, seed=m)


@pytest.mark.parametrize("lens,hq,hkv,d,hint", [
    ([(60, 15000)], 6, 2, 64, 0), ([(100, 6000), (3, 5000)], 1, 1, 128, 100), ([(300, 3000), (7, 900), (40, 700)], 4, 2, 128, 0),
    ([(1, 9000), (1, 300)], 4, 4, 64, 1), ([(5, 4000)] * 3, 9, 3, 128, 5), ([(70, 2500)] + [(1, 600)] * 5, 8, 4, 64, 70)])
def test_rows_cut_into_many_parts(torch, lens, hq, hkv, d, hint):
    """Few tiles over long caches: each is cut into many parts, joined by blocks of 4, 8 or 16 channels."""
    run(torch, lens, hq=hq, hkv=hkv, d=d, ps=32, hint=hint, seed=len(lens))


@pytest.mark.parametrize("n,hint", [(32, 0), (33, 0), (33, 9), (33, 1), (64, 40)])
def test_as_many_sequences_as_a_warp(torch, n, hint):
    """Sequences of very different lengths, some empty, around the number whose pieces a warp finds."""
    rng = np.random.default_rng(n + hint)
    m = np.minimum(rng.integers(0, 10 if hint != 1 else 2, n), hint or 100)
    run(torch, [(int(a), int(a + b)) for a, b in zip(m, rng.integers(0, 300, n) + 4000 * (np.arange(n) == n - 1))], hq=4, hkv=2, d=64, ps=16, hint=hint)


@pytest.mark.parametrize("hint", [0, 1])
def test_many_short_sequences(torch, hint):
    rng = np.random.default_rng(7)
    run(torch, [(1, int(x)) for x in rng.integers(1, 200, 700)], hq=2, hkv=1, d=64, ps=16, hint=hint)


def test_mixed_prompts_and_decode(torch):
    run(torch, [(200, 200), (1, 700), (1, 1), (65, 300), (1, 128), (0, 0), (31, 31)], hq=8, hkv=2, d=128, ps=16)


@pytest.mark.parametrize("hint", [0, 1, 3, 24])
def test_large_logits_and_growing_maximum(torch, hint):
    """Logits that climb along the keys by far more than float32's exponent takes without a running maximum (in every kernel:
    the hint and the heads make tiles of 6, 2, 6 and 96 rows)."""
    import tiered_quantize_evict_gb300 as qe
    n, d, heads = 700, 64, 4 if hint == 24 else 2
    c = Case(torch, [n], hkv=1, d=d, ps=16, dtype="bf16")
    k = torch.zeros(n, 1, d, dtype=c.dt)
    k[:, 0, 0] = torch.linspace(-120, 120, n).to(c.dt)
    c.kh[0][0].copy_(k)
    page = torch.from_numpy(c.table[0].astype(np.int64))[torch.arange(n) // 16].to(c.dev)
    c.k[0][page, :, (torch.arange(n) % 16).to(c.dev)] = k.to(c.dev)
    pool, seqs = c.objects(qe)
    q = torch.zeros(3, heads, d, dtype=c.dt)
    q[:, 0::2, 0], q[:, 1::2, 0] = 8.0, -8.0
    out, lse = pool.attend(0, q.to(c.dev), c.ints([0, 3]), seqs, scale=1.0, max_q_len=hint, return_lse=True)
    ref, tol, lref, ltol = attend_bounds(torch, c, bits(q), 3, 0, heads, 1.0, True)
    assert (np.abs(bits(out) - ref) <= tol).all()
    assert (np.abs(lse.cpu().numpy() - lref) <= ltol).all()


def test_tokens_behind_the_last_sequence_are_left(torch):
    import tiered_quantize_evict_gb300 as qe
    c = Case(torch, [20, 9], hkv=1, d=64, ps=16)
    pool, seqs = c.objects(qe)
    q = c.draw(11, 2, 64).to(c.dev)
    out = torch.full((11, 2, 64), 7.0, dtype=c.dt, device=c.dev)
    pool.attend(0, q, c.ints([0, 4, 6]), seqs, out=out)
    assert (out[6:] == 7).all() and not (out[:6] == 7).all(-1).any()


def test_bad_pages_rows_and_starts_are_reported(torch):
    """Entries outside the pool count as zero keys and set the error word; nothing is read out of range."""
    import tiered_quantize_evict_gb300 as qe
    c = Case(torch, [40, 20], hkv=1, d=64, ps=16)
    c.table[0, 1] = 10 ** 6
    pool, seqs = c.objects(qe)
    q = c.draw(3, 2, 64).to(c.dev)
    out = pool.attend(0, q, c.ints([0, 2, 3]), seqs)
    with pytest.raises(qe.QEError, match="page index"):
        pool.check()
    pool.check()   # cleared
    k, v = bits(c.kh[0][0]), bits(c.vh[0][0])
    k[16:32], v[16:32] = 0, 0
    from oracle import pages as op
    ref, _, spread, _ = op.attend(bits(q[:2]), k, v, 1, 0.125, True)
    assert (np.abs(bits(out[:2]) - ref) <= 2.0 ** -8 * (np.abs(ref) + 1.01 * spread) + 1e-4 * spread).all()
    for starts, rows, lens in (([0, 2, 9], [0, 1], None), ([2, 0, 3], [0, 1], None), ([0, 2, 3], [0, 2], None), ([0, 2, 3], [-1, 1], None),
                               ([0, 2, 3], [0, 1], [10 ** 6, 20]), ([0, 2, 3], [0, 1], [-4, 20])):
        c.table[0, 1] = 0
        c.kv_len[:] = [40, 20] if lens is None else lens
        pool, seqs = c.objects(qe)
        pool.attend(0, q, c.ints(starts), seqs, rows=c.ints(rows))
        with pytest.raises(qe.QEError):
            pool.check()


def test_offsets_past_32_bits(torch):
    """A pool of 2^31 elements and more: pages at its far end, through every operator."""
    import tiered_quantize_evict_gb300 as qe
    from oracle import pages as op
    H, S, D = 8, 256, 128
    P = 2 ** 31 // (H * S * D) + 40
    k = torch.empty(1, P, H, S, D, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    rng = np.random.default_rng(5)
    table = np.array([[P - 1, P - 3], [P - 8, -1]], np.int32)
    ints = lambda x: torch.tensor(np.asarray(x, np.int32)).cuda()  # noqa: E731
    pool, seqs = qe.PagePool(k, v), qe.PageTable(ints(table), ints([300, 20]))
    kn, vn = (torch.from_numpy(rng.standard_normal((320, H, D), dtype=np.float32)).to(torch.bfloat16) for _ in range(2))
    starts = ints([0, 300, 320])
    pool.append(0, kn.cuda(), vn.cuda(), starts, seqs)
    q = torch.from_numpy(rng.standard_normal((2, H, D), dtype=np.float32)).to(torch.bfloat16)
    out = pool.attend(0, q.cuda(), ints([0, 1, 2]), seqs)
    for r, (a, b) in enumerate(((0, 300), (300, 320))):
        ref, _, spread, _ = op.attend(bits(q[r:r + 1]), bits(kn[a:b]), bits(vn[a:b]), H, D ** -0.5, True)
        assert (np.abs(bits(out[r:r + 1]) - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -14) * spread).all()
    gk, gv = pool.gather(0, seqs, 0, 300)
    assert torch.equal(gk[0].cpu(), kn[:300].transpose(0, 1)) and torch.equal(gv[1, :, :20].cpu(), vn[300:].transpose(0, 1))
    pool.copy(ints([P - 8]), ints([P - 20]))
    assert torch.equal(k[0, P - 20, :, :20].cpu(), kn[300:].transpose(0, 1))
    pool.check()


def test_a_row_read_twice(torch):
    """Two chunks may name one row (the same prefix, two continuations' queries)."""
    import tiered_quantize_evict_gb300 as qe
    c = Case(torch, [90, 40], hkv=2, d=64, ps=16)
    pool, seqs = c.objects(qe)
    q = c.draw(5, 4, 64).to(c.dev)
    both = pool.attend(0, q, c.ints([0, 2, 5]), seqs, rows=c.ints([0, 0]))
    assert torch.equal(both[:2], pool.attend(0, q[:2], c.ints([0, 2]), seqs, rows=c.ints([0])))
    assert torch.equal(both[2:], pool.attend(0, q[2:], c.ints([0, 3]), seqs, rows=c.ints([0])))


def test_captured_and_replayed_with_new_lengths(torch):
    import tiered_quantize_evict_gb300 as qe
    c = Case(torch, [300, 260], hkv=2, d=64, ps=16)
    pool, seqs = c.objects(qe)
    q = c.draw(2, 4, 64).to(c.dev)
    starts = c.ints([0, 1, 2])
    pool.attend(0, q, starts, seqs, max_q_len=1)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = pool.attend(0, q, starts, seqs, max_q_len=1)
    for lens in ([300, 260], [7, 260], [129, 0]):
        seqs.kv_len.copy_(c.ints(lens))
        g.replay()
        eager = pool.attend(0, q, starts, seqs, max_q_len=1)
        assert torch.equal(out, eager)
    pool.check()


def test_two_streams_and_repeats_agree(torch):
    import tiered_quantize_evict_gb300 as qe
    c = Case(torch, [2000, 1500, 900], hkv=2, d=128, ps=32)
    pool, seqs = c.objects(qe)
    q = c.draw(6, 8, 128).to(c.dev)
    starts = c.ints([0, 3, 4, 6])
    want = pool.attend(0, q, starts, seqs)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            outs.append(pool.attend(0, q, starts, seqs))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
