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
