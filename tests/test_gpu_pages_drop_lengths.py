"""Dropping pages of rows whose lengths are out of range: reported, and nothing is given back by them."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return pytest.importorskip("torch")


@pytest.mark.parametrize("bad", [20 * 16 + 1, 2 ** 31 - 1, -1, -2 ** 31])
def test_lengths(torch, bad):
    import tiered_quantize_evict_gb300 as qe
    dev = torch.device("cuda:0")
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    k = torch.zeros(1, 60, 1, 16, 64, dtype=torch.bfloat16, device=dev)
    pool, seqs = qe.PagePool(k, k.clone()), qe.PageTable.empty(3, 20, 60)
    pool.resize(seqs, ints(0, 1, 2), ints(200, 320, 200))
    pool.check()
    table, refs = seqs.table.clone(), seqs.refs.clone()
    seqs.kv_len[0] = bad
    pool.drop(seqs, ints(0), 20)
    with pytest.raises(qe.QEError, match="row"):
        pool.check()
    assert torch.equal(seqs.table, table) and torch.equal(seqs.refs, refs)
    pool.drop(seqs, ints(0, 1, 3, -1), 20)             # (the others of the call as ever: the next token of row 1 sees keys from 301 on)
    with pytest.raises(qe.QEError, match="row"):
        pool.check()
    table[1, :18] = qe.QE_PAGES_DROPPED
    assert torch.equal(seqs.table, table) and int(seqs.refs.sum()) == int(refs.sum()) - 18
