"""Managing pages with a table as wide as one may be: n_rows * (max_pages + 1) just below 2^31."""
import pytest

pytestmark = pytest.mark.gpu

COLS = 2 ** 31 - 2


@pytest.fixture(scope="module")
def torch():
    return pytest.importorskip("torch")


@pytest.fixture()
def env(torch):
    """(pool, a row of COLS columns, ints)"""
    import tiered_quantize_evict_gb300 as qe
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("the table takes 8.6 GB")
    dev = torch.device("cuda:0")
    k = torch.zeros(1, 30, 1, 16, 64, dtype=torch.bfloat16, device=dev)
    return qe.PagePool(k, k.clone()), qe.PageTable.empty(1, COLS, 30), lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)


def test_drop(torch, env):
    import tiered_quantize_evict_gb300 as qe
    pool, seqs, ints = env
    last = ints(5, 7, 9)
    seqs.table[0, -3:] = last
    pool.resize(seqs, ints(0), ints(400))
    pool.drop(seqs, ints(0, 0), 100, sinks=20)         # the next token sees keys from 301 on: pages 2 .. 17 go
    pool.check()
    assert seqs.table[0, :26].tolist() == [0, 1] + [qe.QE_PAGES_DROPPED] * 16 + list(range(18, 25)) + [-1]
    assert seqs.refs.tolist() == [1, 1] + [0] * 16 + [1] * 7 + [0] * 5
    assert torch.equal(seqs.table[0, -3:], last)       # (not the row's)


def test_fork(torch, env):
    """An empty row's copy: -1 in all columns."""
    pool, seqs, ints = env
    for a in (0, 2 ** 30, COLS - 3):
        seqs.table[0, a:a + 3] = 5
    pool.fork(seqs, ints(0), ints(0))
    pool.check()
    assert not seqs.refs.any() and seqs.kv_len.tolist() == [0]
    for a in range(0, COLS, 2 ** 28):
        assert (seqs.table[0, a:a + 2 ** 28] == -1).all()
