"""Attention over pools whose strides fit no axis of all pages' heads: keys and values are copied 8 tokens x 64 channels at a time."""
import numpy as np
import pytest

from oracle import pages as op
from pages_ranges_testlib import bits, check, seen_bounds

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return pytest.importorskip("torch")


@pytest.mark.parametrize("d,ps", [(64, 16), (128, 16), (128, 64), (128, 256)])
def test_odd_page_strides(torch, d, ps):
    """Pages 2^31 + 8 elements apart: as an axis in steps that heads and pages have in common (8 elements) they would pass 2^31 places."""
    import tiered_quantize_evict_gb300 as qe
    P, H, far = 10, 2, 2 ** 31 + 8
    room = H * ps * d
    base = torch.empty((P - 1) * far + 2 * room, dtype=torch.bfloat16, device="cuda")
    k, v = (base.as_strided((1, P, H, ps, d), (far, far, ps * d, d, 1), o) for o in (0, room))
    rng = np.random.default_rng(d + ps)
    draw = lambda *s: torch.from_numpy(rng.standard_normal(s, dtype=np.float32)).bfloat16()  # noqa: E731
    k.fill_(float("nan"))
    v.fill_(float("nan"))
    n, m = 7 * ps - 5, min(40, 3 * ps)
    order = rng.permutation(P)[:8]
    table = np.full((2, 7), -1, np.int32)
    table[0] = order[:7]
    table[1, :6], table[1, 6] = order[:6], order[7]             # shares all but its last page
    kh, vh = draw(2, n, H, d), draw(2, n, H, d)
    kh[1, :6 * ps], vh[1, :6 * ps] = kh[0, :6 * ps], vh[0, :6 * ps]
    for r in range(2):
        for i in range(0, n, ps):
            e = min(n, i + ps)
            k[0, int(table[r, i // ps]), :, :e - i] = kh[r, i:e].transpose(0, 1).cuda()
            v[0, int(table[r, i // ps]), :, :e - i] = vh[r, i:e].transpose(0, 1).cuda()
    ints = lambda x: torch.tensor(np.asarray(x, np.int32)).cuda()  # noqa: E731
    pool, seqs = qe.PagePool(k, v), qe.PageTable(ints(table), ints([n, n]))
    for m, hint in ((2, 2), (20, 20), (40, 0)):
        m = min(m, ps - 5)
        hint = min(hint, m)
        q, starts = draw(2 * m, 4, d), ints([0, m, 2 * m])
        for kind in ("all", "window", "shared"):
            if kind == "all":
                got = pool.attend(0, q.cuda(), starts, seqs, max_q_len=hint)
            elif kind == "window":
                got = pool.attend(0, q.cuda(), starts, seqs, max_q_len=hint, window=3 * ps, sinks=9)
            else:
                got = pool.attend_shared(0, q.cuda(), starts, seqs, ints([0, 2]), ints([6 * ps]), max_group_len=2 * hint)
            pool.check()
            for r in range(2):
                seen = op.window_seen(m, n, 3 * ps, 9) if kind == "window" else [range(n - m + j + 1) for j in range(m)]
                want = seen_bounds(torch, torch.bfloat16, bits(q[r * m:(r + 1) * m]), bits(kh[r]), bits(vh[r]), H, d ** -0.5, seen)
                check(bits(got[r * m:(r + 1) * m]), None, want, f"{kind}, {m} tokens, row {r}")
