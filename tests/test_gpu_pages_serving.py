"""The paged cache's operators together, as a server uses them, and handed on to the tiered cache."""
import numpy as np
import pytest

from oracle import pages as op
from pages_testlib import bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return pytest.importorskip("torch")


def test_chunked_prefill_fork_decode_compact_hand_on(torch):
    import tiered_quantize_evict_gb300 as qe
    L, HQ, H, D, S, P, R = 2, 4, 1, 64, 16, 40, 4
    rng = np.random.default_rng(3)
    dev = torch.device("cuda:0")
    k = torch.full((L, P, H, S, D), float("nan"), dtype=torch.bfloat16, device=dev)
    v = torch.full_like(k, float("nan"))
    pool, seqs = qe.PagePool(k, v), qe.PageTable.empty(R, 16, P, dev)
    rope = qe.Rope(D, sections=[8, 12, 12])
    f = [1e4 ** (-2 * i / D) for i in range(D // 2)]
    axis = [0] * 8 + [1] * 12 + [2] * 12
    ints = lambda x: torch.tensor(np.asarray(x, np.int32)).to(dev)  # noqa: E731
    hist = {r: [[] for _ in range(L)] for r in range(R)}   # per row and layer: stored (k, v), as the pool holds them
    lens = {r: 0 for r in range(R)}

    def step(rows, counts):
        """New tokens on some rows, through every layer; each layer's outputs against float64."""
        for r, m in zip(rows, counts):
            lens[r] += m
        pool.resize(seqs, ints(rows), ints([lens[r] for r in rows]))
        starts = np.cumsum([0] + list(counts))
        total = int(starts[-1])
        pos = rng.integers(0, 4000, (3, total)).astype(np.int32)
        for layer in range(L):
            x = {n: torch.from_numpy(rng.standard_normal((total, h, D), dtype=np.float32)).to(torch.bfloat16)
                 for n, h in (("q", HQ), ("k", H), ("v", H))}
            q = pool.append(layer, x["k"].to(dev), x["v"].to(dev), ints(starts), seqs, rows=ints(rows), q=x["q"].to(dev), rope=rope,
                            positions=ints(pos))
            out = pool.attend(layer, q, ints(starts), seqs, rows=ints(rows), max_q_len=max(counts))
            kr = torch.from_numpy(op.rotate(bits(x["k"]), pos, axis, f, D, False)).to(torch.bfloat16)
            qr, o = bits(q), bits(out)
            for r, a, m in zip(rows, starts, counts):
                hist[r][layer] += [(bits(kr[a + j]), bits(x["v"][a + j])) for j in range(m)]
                hk, hv = (np.stack([t[i] for t in hist[r][layer]]) for i in range(2))
                ref, _, spread, _ = op.attend(qr[a:a + m], hk, hv, H, D ** -0.5, True)
                # the stored keys may differ from these by one rounding (2^-8 of each, moving a logit by 2^-8 of
                # its terms' size, here below 2^-8 * 64 * 0.125 * |q||k| < 0.4 at the far tail) -- in practice a few flip,
                # so the comparison of this test is by norm: 2^-8 for each of the output, the probabilities and the keys
                err = np.linalg.norm(o[a:a + m] - ref) / np.linalg.norm(spread)
                assert err < 3 * 2.0 ** -8, f"row {r}, layer {layer}: {err:.2e}"
        pool.check()

    step([0, 1], [70, 33])          # prompts in chunks
    step([1, 0], [15, 64])
    pool.fork(seqs, ints([0, 0]), ints([2, 3]))
    for r in (2, 3):
        hist[r], lens[r] = [list(h) for h in hist[0]], lens[0]
    for _ in range(3):
        step([0, 1, 2, 3], [1, 1, 1, 1])       # decode, forks included
    step([2, 0, 3], [5, 1, 2])                 # drafts on one row
    lens[2] -= 3                               # two of them accepted
    pool.resize(seqs, ints([2]), ints([lens[2]]))
    hist[2] = [h[: lens[2]] for h in hist[2]]
    pool.free(seqs, ints([0]))
    hist[0], lens[0] = [[] for _ in range(L)], 0
    live = ints([0])
    pool.compact(seqs, n_live=live)
    pool.check()
    assert int((seqs.refs > 0).sum()) == live.item() and (seqs.refs[: live.item()] > 0).all()
    step([3, 1, 2], [1, 1, 1])

    # rows 3 and 1 go on in the tiered cache: one decode step there equals the paged attention
    n = min(lens[3], lens[1])
    cfg = qe.QEConfig(batch=2, n_layers=L, n_q_heads=HQ, n_kv_heads=H, head_dim=D, window=16, route_period=16, n_sink=4, n_recent=16,
                      max_context=512, cap_mode=0, kf=8, kq=8, out_fp32=0)
    cache = qe.QECache(cfg, torch.cuda.current_stream().cuda_stream)
    rows = ints([3, 1])
    pool.resize(seqs, rows, ints([n, n]))
    for layer in range(L):
        gk, gv = pool.gather(layer, seqs, 0, n, rows=rows)
        cache.qe_append(layer, gk, gv, n)
        q = torch.from_numpy(rng.standard_normal((2, HQ, D), dtype=np.float32)).to(torch.bfloat16).to(dev)
        tiered = torch.empty_like(q)
        cache.qe_decode_step(layer, q, tiered)
        paged = pool.attend(layer, q, ints([0, 1, 2]), seqs, rows=rows)
        err = (tiered.float() - paged.float()).norm() / paged.float().norm()
        assert err < 2 * 2.0 ** -8, f"layer {layer}: {err:.2e}"
    cache.qe_synchronize()
    pool.check()
    cache.close()


def test_two_pools_and_a_side_stream(torch):
    """Calls on a side stream use that stream, and calls of two pools do not disturb each other."""
    import tiered_quantize_evict_gb300 as qe
    pools = []
    for i, dt in enumerate((torch.bfloat16, torch.float16)):
        k = torch.randn(1, 20, 2, 32, 128, device="cuda").to(dt)
        pool, seqs = qe.PagePool(k, torch.randn_like(k)), qe.PageTable.empty(2, 8, 20, k.device)
        pools.append((pool, seqs, torch.randn(5, 4, 128, device="cuda").to(dt)))
    rows = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda")
    lens = torch.tensor([100, 180], dtype=torch.int32, device="cuda")
    want = []
    for pool, seqs, q in pools:
        pool.resize(seqs, rows, lens)
        want.append(pool.attend(0, q, starts, seqs))
        pool.free(seqs, rows)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for (pool, seqs, q), st in zip(pools, streams):
        with torch.cuda.stream(st):
            pool.resize(seqs, rows, lens)
            got.append(pool.attend(0, q, starts, seqs))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_captured_step_with_copies_between(torch):
    """A whole step in one graph, every call right behind a copy of its inputs (not a kernel of ours), replayed with other inputs."""
    import tiered_quantize_evict_gb300 as qe

    def state():
        k = torch.zeros(2, 24, 2, 16, 64, device="cuda", dtype=torch.bfloat16)
        pool, seqs = qe.PagePool(k, torch.zeros_like(k)), qe.PageTable.empty(4, 8, 24, k.device)
        ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        return {"pool": pool, "seqs": seqs, "rows": ints(0, 1), "lens": ints(0, 0), "starts": ints(0, 0, 0), "src": ints(0), "dst": ints(2),
                "k": torch.zeros(9, 2, 64, device="cuda", dtype=torch.bfloat16), "v": torch.zeros(9, 2, 64, device="cuda", dtype=torch.bfloat16),
                "q": torch.zeros(9, 4, 64, device="cuda", dtype=torch.bfloat16)}

    rope = qe.Rope(64, halves=True)

    def step(s, new):
        pool, seqs = s["pool"], s["seqs"]
        s["lens"].copy_(new["lens"])
        pool.resize(seqs, s["rows"], s["lens"])
        out = []
        for layer in range(2):
            s["starts"].copy_(new["starts"])
            s["k"].copy_(new["k"])
            s["v"].copy_(new["v"])
            s["q"].copy_(new["q"])
            q = pool.append(layer, s["k"], s["v"], s["starts"], seqs, rows=s["rows"], q=s["q"], rope=rope)
            s["starts"].copy_(new["starts"])
            out.append(pool.attend(layer, q, s["starts"], seqs, rows=s["rows"]))
        s["src"].copy_(new["src"])
        pool.fork(seqs, s["src"], s["dst"])
        s["src"].copy_(new["src"])
        out += pool.gather(1, seqs, 0, 40)
        out += [seqs.table.clone(), seqs.refs.clone()]
        pool.free(seqs, s["dst"])
        s["src"].copy_(new["src"])
        pool.compact(seqs)
        return out

    def inputs(seed, lens, starts, src):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda h: torch.randn(9, h, 64, device="cuda", generator=g).bfloat16()  # noqa: E731
        ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        return {"lens": ints(lens), "starts": ints(starts), "src": ints(src), "k": rnd(2), "v": rnd(2), "q": rnd(4)}

    steps = [inputs(1, [5, 4], [0, 5, 9], [1]), inputs(2, [6, 12], [0, 1, 9], [0]), inputs(3, [40, 13], [0, 8, 9], [1]), inputs(4, [3, 17], [0, 1, 5], [0])]
    eager, replayed = state(), state()
    step(eager, steps[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(replayed, steps[0])          # the same first step, outside of the graph
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    new = {n: x.clone() for n, x in steps[1].items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(replayed, new)
    for x in steps[1:]:
        for n in new:
            new[n].copy_(x[n])
        graph.replay()
        torch.cuda.synchronize()
        want = step(eager, x)
        live = int(x["starts"][-1])       # packed tokens behind the last sequence are left alone
        for a, b in zip(got[:2], want[:2]):
            assert torch.equal(a[:live], b[:live])
        for a, b in zip(got[2:], want[2:]):
            assert torch.equal(a, b)
        for a in ("k", "v"):
            assert torch.equal(getattr(replayed["pool"], a), getattr(eager["pool"], a))
    eager["pool"].check()
    replayed["pool"].check()
