"""qe_pages_attend where its softmax is under strain: rows that see nothing of a block whose other rows' maxima jump."""
import numpy as np
import pytest

from pages_testlib import Case, attend_bounds, bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return pytest.importorskip("torch")


def put_keys(torch, c, row):
    """Writes the row's (edited) keys and values to its pages again."""
    n = c.lens[row]
    pos = torch.arange(n)
    page, tok = torch.from_numpy(c.table[row].astype(np.int64))[pos // c.ps].to(c.dev), (pos % c.ps).to(c.dev)
    c.k[0][page, :, tok] = c.kh[row][0].to(c.dev)
    c.v[0][page, :, tok] = c.vh[row][0].to(c.dev)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("blocks", [1, 2, 41, 42, 300])
@pytest.mark.parametrize("m,hint,hq", [(2, 2, 1), (3, 3, 4), (4, 4, 2), (2, 3, 1), (2, 8, 2), (2, 40, 1), (2, 0, 1), (4, 16, 8)])
def test_rows_without_keys_of_the_last_block(torch, d, dtype, blocks, m, hint, hq):
    """The last block is one key, seen by the chunk's last token alone, whose logit there is 400 above its others; the tokens before
    see nothing of that block, and all their logits are near -150.  In every kernel (the hint and the heads make the tile), for rows
    of one piece and rows cut into parts; with hint 3, 8 and 40 behind the chunk lie the next sequence's queries."""
    import tiered_quantize_evict_gb300 as qe
    n = 128 * blocks + 1
    c = Case(torch, [n, 40], hkv=1, d=d, ps=16, dtype=dtype, seed=blocks + m)
    k = c.draw(n, 1, d) * 0.125
    k[:, 0, 0] = 1.0
    k[:, 0, 1] = 0.0
    k[n - 1, 0, 1] = 20.0
    c.kh[0][0].copy_(k)
    put_keys(torch, c, 0)
    pool, seqs = c.objects(qe)
    q = c.draw(m + 9, hq, d)
    q[:, :, 0], q[:, :, 1] = -150.0, 0.0
    q[m - 1:, :, 1] = 20.0            # the last token, and the next sequence's
    out, lse = pool.attend(0, q.to(c.dev), c.ints([0, m, m + 9]), seqs, scale=1.0, max_q_len=hint, return_lse=True)
    pool.check()
    ref, tol, lref, ltol = attend_bounds(torch, c, bits(q[:m]), m, 0, hq, 1.0, True)
    err, off = np.abs(bits(out)[:m] - ref), np.abs(lse.cpu().numpy()[:m] - lref)
    assert (off <= ltol).all(), f"lse: {lse.cpu().numpy()[:m]} and {lref}"
    assert (err <= tol).all(), f"off by {err.max():.3e}"


# The kernels by their tiles: (chunk, hint, query heads) of one KV head
KERNELS = {"few": (2, 2, 2), "one_half": (20, 20, 1), "two_halves": (140, 0, 2)}


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [500, 512, 4000])
@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("causal", [True, False])
def test_small_weights_of_fp16(torch, d, n, kernel, causal):
    """Weights of 2^-24.5 to 2^-29 beside one of 1 whose value is zero: all of the result comes from them.

    Probabilities meet the values in fp16, 2^7 times as large as the weights or more, so where they are below 2^-14 they are off by at
    most half a step of 2^-24: a weight by 2^-25 / 2^7 = 2^-32, absolutely.  A probability above is off by half a step relatively (u), as
    in attend_bounds, whose other terms stay."""
    import tiered_quantize_evict_gb300 as qe
    m, hint, hq = KERNELS[kernel]
    c = Case(torch, [n], hkv=1, d=d, ps=32, dtype="fp16", seed=n + d)
    k, v = torch.zeros(n, 1, d, dtype=c.dt), torch.from_numpy(c.rng.uniform(500, 2000, (n, 1, d))).to(c.dt)
    k[1:, 0, 0] = torch.from_numpy(c.rng.uniform(-29, -24.5, n - 1) * np.log(2)).to(c.dt)
    v[0] = 0
    c.kh[0][0].copy_(k)
    c.vh[0][0].copy_(v)
    put_keys(torch, c, 0)
    pool, seqs = c.objects(qe)
    q = torch.zeros(m, hq, d, dtype=c.dt)
    q[:, :, 0] = 1.0
    out = pool.attend(0, q.to(c.dev), c.ints([0, m]), seqs, scale=1.0, causal=causal, max_q_len=hint)
    pool.check()
    ref, tol, _, _ = attend_bounds(torch, c, bits(q), m, 0, hq, 1.0, causal)
    from oracle import pages as op
    den = op.attend(bits(q), bits(k), bits(v), 1, 1.0, causal)[3]
    tol -= 1.01 * (2.0 ** -25 - 2.0 ** -32) * np.abs(bits(v)).sum(0)[None] / den[..., None]   # (attend_bounds' share of probabilities below 2^-14)
    assert (tol > 0).all() and (tol < 0.05 * ref).all()
    err = np.abs(bits(out) - ref)
    assert (err <= tol).all(), f"off by {(err / ref).max():.3e} of the result, {(err / tol).max():.1f} of the bound"


@pytest.mark.parametrize("kernel", ["few", "one_half", "two_halves"])
def test_small_weights_of_fp16_in_a_long_cache(torch, kernel):
    """131071 keys of a weight near 2^-25.5 under one of 1, walked by single CTAs (more tiles than SMs; their rows share the pages).

    Beside the roundings of the result and of the probabilities (u each) and 2^-32 of each weight: sums of 1024 blocks, a term of each
    added in float32 (2^-24 of the sum each, and 64 terms within a block), and products accumulated over 8192 steps of 16 keys (2^-23 of
    the sum of their sizes each, were every step cut off)."""
    import tiered_quantize_evict_gb300 as qe
    n, ps, d, dt, dev = 131072, 256, 64, torch.float16, torch.device("cuda:0")
    rng = np.random.default_rng(3)
    k, v = torch.zeros(1, n // ps, 1, ps, d, dtype=dt), torch.from_numpy(64 + rng.uniform(-4, 4, (1, n // ps, 1, ps, d))).to(dt)
    k[..., 0] = float(torch.tensor(-25.5 * np.log(2)).to(dt))
    k[0, 0, 0, 0], v[0, 0, 0, 0] = 0, 1
    seqs_n, m, hint = {"few": (400, 1, 1), "one_half": (400, 20, 20), "two_halves": (1, 80000, 0)}[kernel]
    ints = lambda x: torch.tensor(np.asarray(x, np.int32)).to(dev)  # noqa: E731
    pool = qe.PagePool(k.to(dev), v.to(dev))
    seqs = qe.PageTable(ints(np.tile(np.arange(n // ps), (seqs_n, 1))), ints([n] * seqs_n))
    q = torch.zeros(seqs_n * m, 1, d, dtype=dt, device=dev)
    q[..., 0] = 1
    out = pool.attend(0, q, ints(np.arange(seqs_n + 1) * m), seqs, scale=1.0, causal=False, max_q_len=hint)
    pool.check()
    logit = bits(k)[0, :, 0, :, 0].reshape(-1)
    w = np.exp(logit)
    vv = bits(v)[0, :, 0].reshape(-1, d)
    ref, u = w @ vv / w.sum(), 2.0 ** -11
    dl = (d + 4) * 2.0 ** -24 * np.abs(logit).max()
    tol = u * ref + (u + 2 * dl + (1024 + 64) * 2.0 ** -24 + 8192 * 2.0 ** -23) * ref + 2.0 ** -32 * vv.sum(0) / w.sum() + 2.0 ** -20
    err = (out.double().cpu() - torch.from_numpy(ref)).abs().amax((0, 1)).numpy()
    assert (err <= tol).all(), f"off by {err.max():.3e} of {ref.max():.3f}, {(err / tol).max():.1f} of the bound"


@pytest.mark.parametrize("m,hint", [((77824,), 0), ((1, 200) * 152, 0), ((1,) * 456, 1), ((20,) * 456, 20)],
                         ids=["two_halves", "one_or_two_halves", "few", "one_half"])
def test_tiles_of_a_third_of_a_second(torch, m, hint):
    """2^25 keys (one page, named over and over), so that a CTA walks its second or third tile more than 0.2 s after its first: no wait expires.
    Logits are 0 and values powers of two, so all sums are whole numbers of them that float32 holds: the result is the values."""
    import tiered_quantize_evict_gb300 as qe
    n, ps, d, dev = 2 ** 25, 256, 128, torch.device("cuda:0")
    ints = lambda x: torch.tensor(np.asarray(x, np.int32)).to(dev)  # noqa: E731
    v = 2.0 ** (torch.arange(d) % 8 - 4).to(torch.bfloat16)
    pool = qe.PagePool(torch.randn(1, 1, 1, ps, d).to(torch.bfloat16).to(dev), v.expand(1, 1, 1, ps, d).contiguous().to(dev))
    seqs = qe.PageTable(torch.zeros(1, n // ps, dtype=torch.int32, device=dev), ints([n]))
    q = torch.zeros(sum(m), 1, d, dtype=torch.bfloat16, device=dev)
    out = pool.attend(0, q, ints(np.cumsum([0, *m])), seqs, rows=ints([0] * len(m)), causal=False, max_q_len=hint)
    pool.check()
    assert torch.equal(out[:, 0], v.to(dev).expand(sum(m), d))


def remainder_bounds(torch, c, q, row, hq, scale):
    """(out, tolerance) where probabilities are kept as a rounded value and its rounded remainder (bf16).

    With u the half step 2^-8: the result is rounded once, u |out|.  A probability is off by u times its remainder, which is u of it at
    most: u^2 sum w |v|.  Were every product and sum of the tensor cores cut off instead of rounded, a logit would be off by
    (D + 4) 2^-23 of the sum of its terms' sizes (which moves numerator and denominator alike: 2 x) and a result by n 2^-23 of sum w |v|;
    exponentials and running sums take 2^-20 + n 2^-24."""
    from oracle import pages as op
    k, v = bits(c.kh[row][0]), bits(c.vh[row][0])
    out, _, spread, _ = op.attend(q, k, v, c.hkv, scale, True)
    mag = np.stack([scale * (np.abs(q[:, h]) @ np.abs(k[:, h // (hq // c.hkv)]).T).max(-1) for h in range(hq)], 1)
    u, n = 2.0 ** -8, k.shape[0]
    rel = u * u + 2 * (c.d + 4) * 2.0 ** -23 * mag + 2.0 ** -20 + n * (2.0 ** -23 + 2.0 ** -24)
    return out, (u * np.abs(out) + rel[..., None] * spread) * 1.01


def rounded(x):
    """float64 to bf16 and back, to nearest."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(m * 256) / 256, e)


def plain_probabilities(q, k, v, hkv, scale, keep):
    """Attention with probabilities in bf16, and their remainders (keep), all else in 64 bits; the result in bf16."""
    m, hq, _ = q.shape
    out = np.zeros(q.shape)
    for h in range(hq):
        for j in range(m):
            vis = k.shape[0] - m + j + 1
            s = scale * (k[:vis, h // (hq // hkv)] @ q[j, h])
            p = np.exp(s - s.max())
            hi = rounded(p)
            out[j, h] = rounded((hi + (rounded(p - hi) if keep else 0)) @ v[:vis, h // (hq // hkv)] / p.sum())
    return out


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("m,hint,hq,hkv", [(1, 1, 4, 1), (4, 4, 8, 2), (16, 16, 1, 1), (6, 6, 6, 2), (20, 20, 4, 2), (32, 32, 4, 1)])
def test_remainders_of_the_probabilities(torch, d, m, hint, hq, hkv):
    """Up to 128 rows a tile (in both kernels): the bound that holds only if the remainders of the probabilities meet their values
    too -- without them, as the oracle shows, the same inputs pass it several times over."""
    import tiered_quantize_evict_gb300 as qe
    c = Case(torch, [200, 137], hkv=hkv, d=d, ps=32, seed=d + m)
    for row in (0, 1):
        c.kh[row][0].mul_(0.25)
        put_keys(torch, c, row)
    pool, seqs = c.objects(qe)
    qh = c.draw(2 * m, hq, d)
    out = pool.attend(0, qh.to(c.dev), c.ints([0, m, 2 * m]), seqs, max_q_len=hint)
    pool.check()
    worst = 0
    for row in (0, 1):
        q = bits(qh[row * m:(row + 1) * m])
        ref, tol = remainder_bounds(torch, c, q, row, hq, d ** -0.5)
        k, v = bits(c.kh[row][0]), bits(c.vh[row][0])
        assert (np.abs(plain_probabilities(q, k, v, hkv, d ** -0.5, True) - ref) <= tol).all()
        worst = max(worst, (np.abs(plain_probabilities(q, k, v, hkv, d ** -0.5, False) - ref) / tol).max())
        err = np.abs(bits(out[row * m:(row + 1) * m]) - ref)
        assert (err <= tol).all(), f"row {row}: {(err / tol).max():.2f} of the bound"
    assert worst > 2
