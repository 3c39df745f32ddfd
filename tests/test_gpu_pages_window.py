"""Attention with a sliding window and sinks against float64, over lengths, windows, heads, page sizes and layouts."""
import numpy as np
import pytest

from oracle import pages as op
from pages_ranges_testlib import bits, check, poison, queries, seen_bounds
from pages_testlib import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return pytest.importorskip("torch")


def run(torch, chunks, window, sinks, *, hq, hkv, d, ps, dtype="bf16", layout="plain", q_layout="plain", scale=None, hint=0, seed=0, rows=None,
        layer=0, layers=1, lse=True, gone=True, edit=None, **kw):
    """chunks: (new tokens, kv_len) of each sequence.  What no query sees is NaN, and pages of nothing else are dropped."""
    import tiered_quantize_evict_gb300 as qe
    order = list(range(len(chunks))) if rows is None else list(rows)
    lens = [0] * len(chunks)
    for (m, n), r in zip(chunks, order):
        lens[r] = n
    c = Case(torch, lens, hkv=hkv, d=d, ps=ps, dtype=dtype, layout=layout, layers=layers, seed=seed, **kw)
    if edit:
        edit(c)
    for (m, n), r in zip(chunks, order):
        used = set().union(*op.window_seen(m, n, window, sinks)) if m else set()
        poison(c, r, [i for i in range(n) if i not in used])
        if gone:
            for j in range(-(-n // ps)):
                if not used.intersection(range(j * ps, min(n, j * ps + ps))):
                    c.table[r, j] = qe.QE_PAGES_DROPPED
    pool, seqs = c.objects(qe)
    starts = np.cumsum([0] + [m for m, _ in chunks])
    qh, q, out = queries(c, int(starts[-1]), hq, q_layout)
    if edit:
        qh = getattr(c, "queries", qh)
        q.copy_(qh)
    s = d ** -0.5 if scale is None else scale
    got = pool.attend(layer, q, c.ints(starts), seqs, rows=None if rows is None else c.ints(rows), scale=scale, max_q_len=hint, out=out,
                      return_lse=lse, window=window, sinks=sinks)
    pool.check()
    o, ls = (bits(got[0]), got[1].cpu().numpy()) if lse else (bits(got), None)
    for (m, n), r, a in zip(chunks, order, starts):
        if m:
            want = seen_bounds(torch, c.dt, bits(qh[a:a + m]), bits(c.kh[r][layer]), bits(c.vh[r][layer]), hkv, s, op.window_seen(m, n, window, sinks))
            check(o[a:a + m], None if ls is None else ls[a:a + m], want, f"sequence {r}")
    return o


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("ps", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("hint", [0, 5])
def test_pages_and_types(torch, d, dtype, ps, hint):
    run(torch, [(1, 1), (5, 700), (5, 5), (3, 1301)], 150, 9, hq=8, hkv=2, d=d, ps=ps, dtype=dtype, hint=hint, seed=ps + d)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (1, 300), (2, 5), (63, 64), (64, 0), (127, 17), (128, 128), (129, 1), (400, 3), (1000, 0), (999, 500),
                                          (2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (7, 2 ** 30)])
@pytest.mark.parametrize("m,hint", [(1, 1), (4, 4), (20, 20), (70, 0), (300, 0)])
def test_windows_and_chunks(torch, window, sinks, m, hint):
    """Every kernel, from windows of one token to those that are longer than any row."""
    run(torch, [(m, 1000), (max(1, m // 3), 333)], window, sinks, hq=4, hkv=1, d=64, ps=16, hint=hint, seed=m)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (4, 4), (14, 2), (8, 1), (40, 1), (128, 1)])
def test_head_groups(torch, hq, hkv):
    run(torch, [(9, 470), (1, 233), (2, 2)], 100, 20, hq=hq, hkv=hkv, d=64, ps=16, seed=hq)


@pytest.mark.parametrize("m", [1, 2, 31, 32, 33, 64, 65, 127, 129, 260])
@pytest.mark.parametrize("hint", [0, 1])
def test_prompts(torch, m, hint):
    """Whole prompts; the hint may be wrong."""
    run(torch, [(m, m), (m, m)], 50, 3, hq=4, hkv=2, d=128, ps=16, hint=hint, seed=m)


@pytest.mark.parametrize("offset", range(0, 130, 13))
def test_window_edges(torch, offset):
    """Where the window's first key falls: in pages, between them, between blocks."""
    run(torch, [(1, 600 + offset), (3, 641 + offset), (40, 700 + offset)], 256, 4, hq=8, hkv=2, d=64, ps=64, hint=40, seed=offset)
    run(torch, [(1, 600 + offset)], 256, 4, hq=8, hkv=2, d=128, ps=32, hint=1, seed=offset)


@pytest.mark.parametrize("d", [64, 128])
def test_empty_rows_and_sequences(torch, d):
    """Chunks longer than the cache (queries before position 0 see nothing), empty caches, empty chunks."""
    o = run(torch, [(5, 3), (0, 17), (4, 0), (300, 40), (1, 0), (2, 129)], 16, 2, hq=4, hkv=2, d=d, ps=16)
    assert not o[:2].any() and not o[9:9 + 260].any() and not o[5:9].any()


@pytest.mark.parametrize("layout", ["plain", "token_major", "kv_together"])
@pytest.mark.parametrize("q_layout", ["plain", "heads_first", "slice"])
def test_layouts(torch, layout, q_layout):
    run(torch, [(7, 400), (20, 320)], 130, 40, hq=6, hkv=3, d=64, ps=32, layout=layout, q_layout=q_layout, layers=3, layer=2)


def test_rows_in_another_order_and_scale(torch):
    run(torch, [(3, 350), (17, 290), (1, 5)], 64, 1, hq=4, hkv=1, d=128, ps=16, rows=[2, 0, 1], scale=0.31, lse=False)


@pytest.mark.parametrize("m,n,hint,window", [(1, 9000, 1, 6000), (4, 9001, 4, 7000), (40, 9001, 40, 6500), (130, 6500, 0, 5000)])
@pytest.mark.parametrize("d", [64, 128])
def test_long_windows_are_split(torch, m, n, hint, window, d):
    run(torch, [(m, n)], window, 33, hq=4, hkv=1, d=d, ps=64, hint=hint)


@pytest.mark.parametrize("m,hint", [(4, 4), (16, 16), (30, 30), (90, 0)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_rows_whose_first_block_is_hidden(torch, m, hint, dtype):
    """Later rows of a tile see nothing of its first block, and all logits are far below zero: nothing but the logits
    themselves may set a row's reference."""
    def far(c):
        for x in c.kh:
            x[..., 0] = 16
        c.k[..., 0] = 16
        c.queries = c.draw(m, 2, c.d) * 0.25
        c.queries[..., 0] = -16
    for extra in range(0, 128, 31):
        run(torch, [(m, 512 + extra)], 100, 0, hq=2, hkv=1, d=64, ps=16, dtype=dtype, hint=hint, scale=1.0, edit=far, seed=extra)


def test_equals_plain_attention_where_the_window_holds_all(torch):
    """A window as long as the rows gives bit for bit what attention without one does."""
    import tiered_quantize_evict_gb300 as qe
    c = Case(torch, [700, 129, 1], hkv=2, d=64, ps=32)
    pool, seqs = c.objects(qe)
    for chunks, hint in (([1, 1, 1], 1), ([30, 12, 1], 30), ([200, 129, 1], 0)):
        starts = c.ints(np.cumsum([0] + chunks))
        q = c.draw(sum(chunks), 8, 64).to(c.dev)
        a = pool.attend(0, q, starts, seqs, max_q_len=hint, return_lse=True)
        b = pool.attend(0, q, starts, seqs, max_q_len=hint, return_lse=True, window=700, sinks=5)
        for x, y in zip(a, b):
            assert torch.equal(x, y)
    pool.check()


def test_visible_pages_that_are_gone_are_reported(torch):
    """A dropped or bad page inside the window counts as zeros and is reported; outside of it nothing is."""
    import tiered_quantize_evict_gb300 as qe
    c = Case(torch, [300], hkv=1, d=64, ps=16)
    c.table[0, 3:8] = [-2, -1, -7, c.n_pages, 2 ** 30]
    pool, seqs = c.objects(qe)
    q = c.draw(2, 4, 64).to(c.dev)
    pool.attend(0, q, c.ints([0, 2]), seqs, window=100, sinks=48, max_q_len=2)
    pool.check()
    got = pool.attend(0, q, c.ints([0, 2]), seqs, window=176, sinks=48, max_q_len=2)   # from key 123 on: page 7
    with pytest.raises(qe.QEError, match="page index"):
        pool.check()
    c.kh[0][0, 112:128], c.vh[0][0, 112:128] = 0, 0
    want = seen_bounds(torch, c.dt, bits(q), bits(c.kh[0][0]), bits(c.vh[0][0]), 1, 0.125, op.window_seen(2, 300, 176, 48))
    check(bits(got), None, want, "zeros")


def test_bad_lengths_and_starts_are_reported(torch):
    import tiered_quantize_evict_gb300 as qe
    c = Case(torch, [40, 30], hkv=1, d=64, ps=16)
    pool, _ = c.objects(qe)
    q = c.draw(6, 4, 64).to(c.dev)
    for starts, rows, lens in (([4, 2, 1], [0, 1], None), ([0, 3, 9], [0, 1], None), ([0, 3, 6], [2, -1], None), ([0, 3, 6], [0, 1], [-1, 2 ** 31 - 1])):
        seqs = qe.PageTable(c.ints(c.table), c.ints(c.kv_len if lens is None else lens))
        for hint in (0, 3, 30):
            pool.attend(0, q, c.ints(starts), seqs, rows=c.ints(rows), window=9, max_q_len=hint)
            with pytest.raises(qe.QEError, match="row"):
                pool.check()


def test_tokens_behind_the_last_sequence_are_left_alone(torch):
    import tiered_quantize_evict_gb300 as qe
    c = Case(torch, [200], hkv=2, d=64, ps=16)
    pool, seqs = c.objects(qe)
    q = c.draw(9, 8, 64).to(c.dev)
    for hint in (0, 4, 20):
        out = torch.full_like(q, 3.0)
        pool.attend(0, q, c.ints([1, 5]), seqs, window=50, max_q_len=hint, out=out)
        assert (out[5:] == 3).all() and (out[:1] == 3).all() and not (out[1:5] == 3).any()
    pool.check()


def test_captured_and_replayed_with_other_lengths(torch):
    import tiered_quantize_evict_gb300 as qe
    c = Case(torch, [900, 500, 700], hkv=2, d=128, ps=32)
    pool, seqs = c.objects(qe)
    q, starts = c.draw(9, 8, 128).to(c.dev), c.ints([0, 3, 6, 9])
    for hint, window in ((3, 200), (0, 640)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = pool.attend(0, q, starts, seqs, window=window, sinks=4, max_q_len=hint, return_lse=True)
        for lens, at in (([900, 500, 700], [0, 3, 6, 9]), ([13, 499, 1], [0, 1, 4, 5]), ([640, 3, 300], [0, 3, 6, 9])):
            seqs.kv_len.copy_(c.ints(lens))
            starts.copy_(c.ints(at))
            g.replay()
            want = pool.attend(0, q, starts, seqs, window=window, sinks=4, max_q_len=hint, return_lse=True)
            for a, b in zip(got, want):
                assert torch.equal(a[:at[-1]], b[:at[-1]])
    pool.check()


def test_two_streams(torch):
    """Two streams at work on one pool, each with its own scratch."""
    import tiered_quantize_evict_gb300 as qe
    c = Case(torch, [3000, 2500], hkv=2, d=64, ps=16)
    pool, seqs = c.objects(qe)
    qs = [c.draw(2 * m, 8, 64).to(c.dev) for m in (1, 60)]
    starts = [c.ints([0, m, 2 * m]) for m in (1, 60)]
    call = lambda i: pool.attend(0, qs[i], starts[i], seqs, window=2200, sinks=10, max_q_len=(1, 0)[i])  # noqa: E731
    want = [call(i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got.append(call(i))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    pool.check()


def test_past_32_bit_offsets(torch):
    """Pages whose keys lie behind 2^31 elements of the pool."""
    import tiered_quantize_evict_gb300 as qe
    ps, d, hkv = 256, 128, 8
    pages = 2 ** 31 // (ps * d * hkv) + 40
    k = torch.zeros(1, pages, hkv, ps, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    rng = np.random.default_rng(0)
    n, m = 1500, 3
    cols = -(-n // ps)
    table = np.full((1, cols + 2), -2, np.int32)
    table[0, 0], table[0, cols - 3:cols] = pages - 1, rng.permutation(np.arange(pages - 30, pages - 1))[:3]
    kh, vh = (torch.from_numpy(rng.standard_normal((n, hkv, d), dtype=np.float32)).bfloat16() for _ in range(2))
    for i in list(range(ps)) + list(range((cols - 3) * ps, n)):
        k[0, int(table[0, i // ps]), :, i % ps] = kh[i].cuda()
        v[0, int(table[0, i // ps]), :, i % ps] = vh[i].cuda()
    ints = lambda x: torch.tensor(np.asarray(x, np.int32)).cuda()  # noqa: E731
    pool, seqs = qe.PagePool(k, v), qe.PageTable(ints(table), ints([n]))
    for hint in (3, 20, 0):
        q = torch.from_numpy(rng.standard_normal((m, 16, d), dtype=np.float32)).bfloat16()
        got = pool.attend(0, q.cuda(), ints([0, m]), seqs, window=600, sinks=100, max_q_len=hint)
        pool.check()
        want = seen_bounds(torch, torch.bfloat16, bits(q), bits(kh), bits(vh), hkv, d ** -0.5, op.window_seen(m, n, 600, 100))
        check(bits(got), None, want, f"hint {hint}")
