"""Attention of sequences that share prefixes against float64, over groups, lengths, heads, page sizes and layouts."""
import numpy as np
import pytest

from pages_ranges_testlib import bits, check, queries, seen_bounds
from pages_testlib import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return pytest.importorskip("torch")


def shared_case(torch, groups, *, ps, rows=None, garbage_entries=True, **kw):
    """groups: (prefix, [(new tokens, own tokens behind the prefix), ...]).  The others' entries of the prefix name no page."""
    flat = [(p // ps * ps, p, i, m, n) for p, seqs in groups for i, (m, n) in enumerate(seqs)]
    order = list(range(len(flat))) if rows is None else list(rows)
    lens = [0] * len(flat)
    for (pre, p, i, m, n), r in zip(flat, order):
        lens[r] = (p if i == 0 else pre) + n      # (the first keeps all of its prefix, in whole pages or not)
    c = Case(torch, lens, ps=ps, **kw)
    first = None
    for (pre, p, i, m, n), r in zip(flat, order):
        if i == 0:
            first = r
        else:
            c.kh[r][:, :pre], c.vh[r][:, :pre] = c.kh[first][:, :pre], c.vh[first][:, :pre]
            c.table[r, :pre // ps] = -7 if garbage_entries else c.table[first, :pre // ps]
    return c, flat, order, lens


def run(torch, groups, *, hq, hkv, d, ps, dtype="bf16", layout="plain", q_layout="plain", causal=True, scale=None, hint=0, seed=0, rows=None,
        layer=0, layers=1, lse=True, **kw):
    import tiered_quantize_evict_gb300 as qe
    c, flat, order, lens = shared_case(torch, groups, ps=ps, rows=rows, hkv=hkv, d=d, dtype=dtype, layout=layout, layers=layers, seed=seed, **kw)
    pool, seqs = c.objects(qe)
    ms = [x[3] for x in flat]
    starts = np.cumsum([0] + ms)
    gstart = np.cumsum([0] + [len(s) for _, s in groups])
    qh, q, out = queries(c, int(starts[-1]), hq, q_layout)
    s = d ** -0.5 if scale is None else scale
    got = pool.attend_shared(layer, q, c.ints(starts), seqs, c.ints(gstart), c.ints([p for p, _ in groups]), rows=None if rows is None else c.ints(rows),
                             scale=scale, causal=causal, max_group_len=hint, out=out, return_lse=lse)
    pool.check()
    o, ls = (bits(got[0]), got[1].cpu().numpy()) if lse else (bits(got), None)
    for m, a, r in zip(ms, starts, order):
        if m:
            n = lens[r]
            seen = [range(max(0, n - m + j + 1) if causal else n) for j in range(m)]
            want = seen_bounds(torch, c.dt, bits(qh[a:a + m]), bits(c.kh[r][layer]), bits(c.vh[r][layer]), hkv, s, seen)
            check(o[a:a + m], None if ls is None else ls[a:a + m], want, f"row {r}")
    return o


MIXED = [(200, [(1, 1), (3, 40), (1, 130), (2, 5)]), (64, [(1, 300)]), (0, [(5, 5), (1, 77)]), (333, [(1, 9)] * 5)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("ps", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("hint", [0, 7])
def test_pages_and_types(torch, d, dtype, ps, hint):
    run(torch, MIXED, hq=4, hkv=2, d=d, ps=ps, dtype=dtype, hint=hint, seed=ps + d)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (3, 1), (4, 4), (14, 2), (8, 1), (40, 1), (128, 1)])
@pytest.mark.parametrize("hint", [0, 8])
def test_head_groups(torch, hq, hkv, hint):
    run(torch, MIXED, hq=hq, hkv=hkv, d=64, ps=16, hint=hint, seed=hq)


@pytest.mark.parametrize("n", [2, 15, 16, 17, 31, 33, 64, 65, 130, 300])
@pytest.mark.parametrize("hint", [0, 1, "right"])
def test_many_sequences(torch, n, hint):
    """One group that fills tiles to different heights, or several; more sequences than a warp, more than a block has threads."""
    rng = np.random.default_rng(n)
    seqs = [(1, int(x)) for x in rng.integers(1, 60, n)]
    run(torch, [(130, seqs)], hq=4, hkv=1, d=64, ps=16, hint=n if hint == "right" else hint, seed=n)


def test_more_sequences_than_threads(torch):
    rng = np.random.default_rng(5)
    groups = [(int(p), [(int(m), int(m) + int(x)) for m, x in zip(rng.integers(0, 3, k), rng.integers(0, 40, k))])
              for p, k in zip(rng.integers(0, 200, 90), rng.integers(1, 20, 90))]
    run(torch, groups, hq=4, hkv=2, d=64, ps=16)
    run(torch, groups, hq=2, hkv=1, d=64, ps=16, hint=8)


def test_more_groups_and_tiles_than_threads(torch):
    """Groups of a sequence or two, more than a block has threads; one group of more tiles than that."""
    rng = np.random.default_rng(6)
    groups = [(16 * int(p), [(1, int(x)) for x in rng.integers(1, 30, k)]) for p, k in zip(rng.integers(0, 3, 1500), rng.integers(0, 3, 1500))]
    run(torch, groups, hq=1, hkv=1, d=64, ps=16)
    run(torch, groups, hq=2, hkv=1, d=64, ps=16, hint=2)
    run(torch, [(48, [(1, 3)] * 1400)], hq=2, hkv=1, d=64, ps=16, hint=2)
    run(torch, [(32, [(1, 2)] * 1400)], hq=128, hkv=1, d=64, ps=16, lse=False)


@pytest.mark.parametrize("m", [1, 2, 5, 16, 33, 100, 300])
@pytest.mark.parametrize("hint", [0, 4])
def test_chunks_of_forks(torch, m, hint):
    """Drafts and whole continuations behind a common prefix: sequences that span several tiles, tiles of several sequences."""
    run(torch, [(150, [(m, m + 3), (1, 20), (max(1, m // 2), m)]), (40, [(m, m)])], hq=4, hkv=2, d=64, ps=16, hint=hint, seed=m)


@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 17, 127, 128, 129, 1000])
def test_prefix_lengths(torch, prefix):
    """In whole pages or not (the rest is in each sequence's own pages)."""
    run(torch, [(prefix, [(1, 30), (2, 2), (1, 200)])], hq=8, hkv=2, d=128, ps=16, seed=prefix)


@pytest.mark.parametrize("hint", [0, 3, 30])
def test_long_prefixes_are_split(torch, hint):
    run(torch, [(9000, [(1, 1), (1, 700), (1, 64)])], hq=4, hkv=1, d=128, ps=64, hint=hint)
    run(torch, [(6000, [(1, 300)] * 40)], hq=4, hkv=1, d=64, ps=32, hint=hint)


def test_cross_attention(torch):
    run(torch, [(64, [(3, 90), (70, 20), (1, 1)]), (0, [(2, 0), (1, 40)])], hq=6, hkv=2, d=128, ps=64, causal=False, dtype="fp16")


def test_empty_sequences_and_groups(torch):
    """Sequences without new tokens, groups of such, empty caches."""
    o = run(torch, [(32, [(0, 0), (2, 2), (0, 9)]), (48, [(0, 3)]), (0, []), (0, [(2, 0), (4, 3)]), (16, [(1, 1)])], hq=4, hkv=2, d=64, ps=16)
    assert not o[2:4].any() and not o[4:5].any()


@pytest.mark.parametrize("layout", ["plain", "token_major", "kv_together"])
@pytest.mark.parametrize("q_layout", ["plain", "heads_first", "slice"])
def test_layouts(torch, layout, q_layout):
    run(torch, [(100, [(2, 40), (1, 3)]), (64, [(20, 20)])], hq=6, hkv=3, d=64, ps=32, layout=layout, q_layout=q_layout, layers=3, layer=2)


def test_rows_in_another_order_and_scale(torch):
    run(torch, [(90, [(3, 50), (1, 30)]), (20, [(2, 9), (1, 1)])], hq=4, hkv=1, d=128, ps=16, rows=[2, 0, 3, 1], scale=0.31, lse=False)


@pytest.mark.parametrize("hint", [0, 12, 40])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_rows_that_see_little(torch, hint, dtype):
    """Logits far below zero, and no prefix: most blocks of a tile hold nothing for most rows, the first one too."""
    import tiered_quantize_evict_gb300 as qe
    c, flat, order, lens = shared_case(torch, [(0, [(1, 40 * i + 1) for i in range(12)])], ps=16, hkv=1, d=64, dtype=dtype)
    for x in c.kh:
        x[..., 0] = 16
    c.k[..., 0] = 16
    pool, seqs = c.objects(qe)
    qh = c.draw(12, 2, 64) * 0.25
    qh[..., 0] = -16
    got, lse = pool.attend_shared(0, qh.to(c.dev), c.ints(range(13)), seqs, c.ints([0, 12]), c.ints([0]), scale=1.0, max_group_len=hint, return_lse=True)
    pool.check()
    for i in range(12):
        want = seen_bounds(torch, c.dt, bits(qh[i:i + 1]), bits(c.kh[i][0]), bits(c.vh[i][0]), 1, 1.0, [range(lens[i])])
        check(bits(got[i:i + 1]), lse[i:i + 1].cpu().numpy(), want, f"row {i}")


def test_bad_groups_are_reported(torch):
    import tiered_quantize_evict_gb300 as qe
    c, *_ = shared_case(torch, [(64, [(1, 9), (2, 20), (1, 4)])], ps=16, hkv=1, d=64)
    pool, seqs = c.objects(qe)
    q, starts = c.draw(4, 4, 64).to(c.dev), c.ints([0, 1, 3, 4])
    for hint in (0, 4, 20):
        for gs, pre in (([0, 2], [64]), ([1, 3], [64]), ([0, 4], [64]), ([0, 2, 1, 3], [16, 16, 16]), ([-1, 3], [64]), ([0, 3], [-5]), ([0, 3], [80]),
                        ([0, 3], [2 ** 31 - 1]), ([0, 2 ** 31 - 1], [64]), ([3, 0], [64])):
            out = torch.full_like(q, 3.0)
            pool.attend_shared(0, q, starts, seqs, c.ints(gs), c.ints(pre), max_group_len=hint, out=out)
            with pytest.raises(qe.QEError, match="row"):
                pool.check()
        for st in ([0, 3, 1, 4], [0, 1, 3, 9], [-2, 1, 3, 4]):
            pool.attend_shared(0, q, c.ints(st), seqs, c.ints([0, 3]), c.ints([64]), max_group_len=hint)
            with pytest.raises(qe.QEError, match="row"):
                pool.check()


def test_bad_pages_are_reported(torch):
    """A bad page of the prefix, or of a sequence's own, counts as zeros."""
    import tiered_quantize_evict_gb300 as qe
    for row, col in ((0, 1), (2, 5)):
        for hint in (0, 4, 20):
            c, flat, order, lens = shared_case(torch, [(64, [(1, 9), (2, 20), (1, 40)])], ps=16, hkv=1, d=64)
            c.table[row, col] = c.n_pages
            for r in range(3) if col < 4 else (row,):
                c.kh[r][0, col * 16:col * 16 + 16], c.vh[r][0, col * 16:col * 16 + 16] = 0, 0
            pool, seqs = c.objects(qe)
            qh = c.draw(4, 4, 64)
            got = pool.attend_shared(0, qh.to(c.dev), c.ints([0, 1, 3, 4]), seqs, c.ints([0, 3]), c.ints([64]), max_group_len=hint)
            with pytest.raises(qe.QEError, match="page index"):
                pool.check()
            for r, a, m in ((0, 0, 1), (1, 1, 2), (2, 3, 1)):
                want = seen_bounds(torch, c.dt, bits(qh[a:a + m]), bits(c.kh[r][0]), bits(c.vh[r][0]), 1, 0.125, [range(lens[r] - m + j + 1) for j in range(m)])
                check(bits(got[a:a + m]), None, want, f"row {r}")


def test_tokens_of_no_sequence_are_left_alone(torch):
    import tiered_quantize_evict_gb300 as qe
    c, *_ = shared_case(torch, [(64, [(1, 9), (2, 20)])], ps=16, hkv=1, d=64)
    pool, seqs = c.objects(qe)
    q = c.draw(9, 4, 64).to(c.dev)
    for hint in (0, 3, 20):
        out = torch.full_like(q, 3.0)
        pool.attend_shared(0, q, c.ints([2, 3, 5]), seqs, c.ints([0, 2]), c.ints([64]), max_group_len=hint, out=out)
        assert (out[5:] == 3).all() and (out[:2] == 3).all() and not (out[2:5] == 3).any()
    pool.check()


def test_captured_and_replayed_with_other_groups(torch):
    import tiered_quantize_evict_gb300 as qe
    c, *_ = shared_case(torch, [(640, [(1, 9), (2, 200), (1, 4), (3, 60)])], ps=16, hkv=2, d=128, garbage_entries=False)
    pool, seqs = c.objects(qe)
    q, starts, gs, pre = c.draw(7, 8, 128).to(c.dev), c.ints([0, 1, 3, 4, 7]), c.ints([0, 4, 4]), c.ints([640, 0])
    lens = seqs.kv_len.clone()
    for hint in (0, 7, 2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = pool.attend_shared(0, q, starts, seqs, gs, pre, max_group_len=hint, return_lse=True)
        for a, b, less in (([0, 4, 4], [640, 0], 0), ([0, 1, 4], [0, 640], 1), ([0, 3, 4], [320, 17], 3), ([0, 0, 4], [5, 600], 4)):
            gs.copy_(c.ints(a))
            pre.copy_(c.ints(b))
            seqs.kv_len.copy_(lens - less)
            g.replay()
            want = pool.attend_shared(0, q, starts, seqs, gs, pre, max_group_len=hint, return_lse=True)
            for x, y in zip(got, want):
                assert torch.equal(x, y)
        seqs.kv_len.copy_(lens)
    pool.err.zero_()      # (a row that is cut short begins inside its prefix)


def test_two_streams(torch):
    import tiered_quantize_evict_gb300 as qe
    c, *_ = shared_case(torch, [(2000, [(1, 30 * i + 1) for i in range(20)])], ps=16, hkv=2, d=64)
    pool, seqs = c.objects(qe)
    q = [c.draw(20, 8, 64).to(c.dev) for _ in range(2)]
    call = lambda i: pool.attend_shared(0, q[i], c.ints(range(21)), seqs, c.ints([0, 20]), c.ints([2000]), max_group_len=(0, 20)[i])  # noqa: E731
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
