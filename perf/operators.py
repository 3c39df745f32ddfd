"""Timed cases of the paged cache's operators: appending a chunk with rotary positions of several
axes, attention of a chunk over the cached pages, and forking, compacting and gathering pages.

With ``own`` false every operator runs in its plain form (elementary torch operations in 32 bits);
with ``own`` true through the library's entry points.  ``exact`` gives the same results from the
operators' definitions in 64 bits.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
_GOLD = 0.6180339887498949


def listed():
    return [
        # one new token of one short sequence, the shape of the smallest decode workload: launch latency
        _attend("attend_one_token", n=1, q=1, kv=320, ragged=0.0, prompt=False, hq=4, hkv=1, d=64, ps=16, dtype="bf16"),
        # a decode step of 16 sequences of up to 32K tokens: reads the whole cache once
        _attend("attend_decode_32k", n=16, q=1, kv=32768, ragged=0.25, prompt=False, hq=32, hkv=8, d=128, ps=32, dtype="bf16"),
        # up to 16 drafts of each of 16 sequences (speculative decoding), ragged, with the log-sum-exp
        _attend("attend_drafts_16k", n=16, q=16, kv=16384, ragged=0.5, prompt=False, hq=32, hkv=8, d=128, ps=64, dtype="fp16", lse=True),
        # several prompts of odd lengths prefilled in one call
        _attend("attend_prompts", n=7, q=2047, kv=2047, ragged=0.6, prompt=True, hq=32, hkv=8, d=128, ps=16, dtype="bf16"),
        # a 2048-token piece of a long prompt over the 30K tokens before it
        _attend("attend_chunk_32k", n=1, q=2048, kv=32768, ragged=0.0, prompt=False, hq=32, hkv=8, d=128, ps=64, dtype="bf16"),
        # one token of one sequence, one axis, neighbouring channels paired: launch latency
        _append("append_one_token", n=1, q=1, kv=320, ragged=0.0, hq=4, hkv=1, d=64, ps=16, axes=1, halves=False, dtype="bf16"),
        # a decode step's tokens of 256 sequences
        _append("append_decode_256", n=256, q=1, kv=2048, ragged=0.5, hq=32, hkv=8, d=128, ps=32, axes=3, halves=True, dtype="bf16"),
        # video prompts: time, height and width positions
        _append("append_video_16k", n=4, q=4096, kv=4500, ragged=0.1, hq=32, hkv=8, d=128, ps=64, axes=3, halves=True, dtype="bf16"),
        # four continuations of one short prompt, dropped again
        _fork("fork_small", parents=1, children=4, kv=300, layers=1, hkv=1, d=64, ps=16, spare=32, dtype="bf16"),
        # 64 continuations of 8 prompts in a 32-layer cache, dropped again
        _fork("fork_branches", parents=8, children=64, kv=3000, layers=32, hkv=8, d=128, ps=32, spare=128, dtype="bf16"),
        # half of a 32-layer cache's pages have been freed at random: move the others together
        _compact("compact_half", pages=1024, live=0.5, rows=32, layers=32, hkv=8, d=128, ps=32, dtype="bf16"),
        # prefilled prompts handed on in the layout the tiered cache appends
        _gather("gather_prompts", n=16, kv=8192, hkv=8, d=128, ps=32, dtype="bf16"),
    ]


def _case(op, name, **kw):
    return {"op": op, **({"name": name} if name else {}), **kw}


def _attend(name, lse=False, **kw):
    return _case("attend", name, lse=lse, **kw)


def _append(name, **kw):
    return _case("append", name, **kw)


def _fork(name, **kw):
    return _case("fork", name, **kw)


def _compact(name, **kw):
    return _case("compact", name, **kw)


def _gather(name, **kw):
    return _case("gather", name, **kw)


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    d, hkv = rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
    hq, ps, dtype = hkv * rng.choice([1, 2, 3, 4, 8]), rng.choice([16, 32, 64, 128]), rng.choice(["bf16", "fp16"])
    op = rng.choice(["attend", "attend", "attend", "append", "append", "fork", "compact", "gather"])
    if op == "attend":
        prompt = rng.random() < 0.4
        n = log(1, 24)
        if prompt:
            q = kv = log(1, 3000)
        else:
            q, kv = log(1, 512), log(16, 32768)
            q = min(q, kv)
        # no more than the listed chunk's products, nor the listed decode step's cache
        n = max(1, min(n, int(2.0e9 // max(1, hq * q * kv)), int(5.0e8 // (kv * hkv))))
        return _attend("", n=n, q=q, kv=kv, ragged=round(rng.uniform(0, 0.9), 2), prompt=prompt, hq=hq, hkv=hkv, d=d, ps=ps,
                       dtype=dtype, lse=rng.random() < 0.5)
    if op == "append":
        q = log(1, 4096)
        n = max(1, min(log(1, 256), 16384 // q))
        return _append("", n=n, q=q, kv=q + log(1, 4096), ragged=round(rng.uniform(0, 0.9), 2), hq=hq, hkv=hkv, d=d, ps=ps,
                       axes=rng.choice([1, 2, 3]), halves=rng.random() < 0.5, dtype=dtype)
    layers = rng.choice([1, 4, 16, 32])
    if op == "fork":
        parents = log(1, 8)
        return _fork("", parents=parents, children=parents * log(1, 8), kv=log(1, 3000), layers=layers, hkv=hkv, d=d, ps=ps,
                     spare=64 + log(1, 64), dtype=dtype)
    if op == "compact":
        return _compact("", pages=log(16, min(1024, 32768 // ps)), live=round(rng.uniform(0.05, 0.95), 2), rows=log(1, 32),
                        layers=layers, hkv=hkv, d=d, ps=ps, dtype=dtype)
    return _gather("", n=log(1, 16), kv=log(1, 8192), hkv=hkv, d=d, ps=ps, dtype=dtype)


# ------------------------------------------------------------------------------ lengths and inputs

def _frac(i):
    """A fixed number in [0, 1) for sequence i (low-discrepancy: multiples of the golden ratio)."""
    return ((i + 1) * _GOLD) % 1.0


def _lens(c):
    """(q_lens, kv_lens) of a case: fixed by the case, the same for every seed."""
    ql, kl = [], []
    for i in range(c["n"]):
        if c.get("prompt"):
            q = kv = max(1, int(c["kv"] * (1 - c["ragged"] * _frac(i))))
        else:
            q = max(1, int(c["q"] * (1 - c["ragged"] * _frac(i + 7))))
            kv = max(q, int(c["kv"] * (1 - c["ragged"] * _frac(i))))
        ql.append(q)
        kl.append(kv)
    return ql, kl


def _cdiv(a, b):
    return -(-a // b)


def _pages_of(lens, ps, n_pages, gen):
    """A page table [n][widest] (-1 behind each sequence) over a random choice of pages, on the host."""
    perm = torch.randperm(n_pages, generator=gen, dtype=torch.int64)
    need = torch.tensor([_cdiv(x, ps) for x in lens])
    first = torch.cumsum(need, 0) - need
    col = torch.arange(max(1, int(need.max())))
    at = (first[:, None] + col[None, :]).clamp_max(n_pages - 1)
    return torch.where(col[None, :] < need[:, None], perm[at], torch.full_like(at, -1)).to(torch.int32)


def _randn(shape, dtype, g, outliers=0):
    x = torch.randn(shape, generator=g, device="cuda", dtype=_DT[dtype])
    if outliers:
        x[..., :outliers] *= 10   # keys have a few large channels
    return x


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.Generator().manual_seed(seed)
    s = {"c": c}
    ps, d, hkv, dt = c["ps"], c["d"], c["hkv"], c["dtype"]
    if c["op"] in ("attend", "append", "gather"):
        ql, kl = _lens(c) if c["op"] != "gather" else ([0] * c["n"], [c["kv"]] * c["n"])
        n_pages = sum(_cdiv(x, ps) for x in kl) + 3
        s["table"] = _pages_of(kl, ps, n_pages, h).cuda()
        s["kv_len"] = torch.tensor(kl, dtype=torch.int32).cuda()
        s["q_start"] = torch.tensor([0] + ql).cumsum(0).to(torch.int32).cuda()
        s["k"] = _randn((1, n_pages, hkv, ps, d), dt, g, outliers=2)
        s["v"] = _randn((1, n_pages, hkv, ps, d), dt, g)
        s["max_q"], s["max_kv"], total = max(ql), max(kl), sum(ql)
        if c["op"] != "gather":
            s["q"] = _randn((total, c["hq"], d), dt, g)
        if c["op"] == "append":
            s["k_new"] = _randn((total, hkv, d), dt, g, outliers=2)
            s["v_new"] = _randn((total, hkv, d), dt, g)
            s["positions"] = torch.randint(0, 131072, (c["axes"], total), generator=g, device="cuda", dtype=torch.int32)
            s["sections"] = _sections(c)
    elif c["op"] == "fork":
        lens = [max(1, int(c["kv"] * (1 - 0.5 * _frac(i)))) for i in range(c["parents"])]
        used = sum(_cdiv(x, ps) for x in lens)
        n_pages = used + c["children"] + c["spare"]
        rows = c["parents"] + c["children"]
        table = torch.full((rows, _cdiv(max(lens), ps)), -1, dtype=torch.int32)
        table[: c["parents"]] = _pages_of(lens, ps, n_pages, h)
        refs = torch.zeros(n_pages, dtype=torch.int32)
        refs[table[table >= 0].long()] = 1
        s["src"] = (torch.arange(c["children"]) % c["parents"]).to(torch.int32).cuda()
        s["dst"] = (c["parents"] + torch.randperm(c["children"], generator=h)).to(torch.int32).cuda()
        s["table"], s["refs"] = table.cuda(), refs.cuda()
        s["kv_len"] = torch.tensor(lens + [0] * c["children"], dtype=torch.int32).cuda()
        s["k"] = _randn((c["layers"], n_pages, hkv, ps, d), dt, g)
        s["v"] = _randn((c["layers"], n_pages, hkv, ps, d), dt, g)
    else:  # compact
        n_live = max(1, int(c["pages"] * c["live"]))
        rows = min(c["rows"], n_live)
        each = [n_live // rows + (i < n_live % rows) for i in range(rows)]
        s["table"] = _pages_of([x * ps for x in each], ps, c["pages"], h).cuda()
        refs = torch.zeros(c["pages"], dtype=torch.int32, device="cuda")
        refs[s["table"][s["table"] >= 0].long()] = 1
        s["refs"] = refs
        s["kv_len"] = torch.tensor([x * ps - i % ps for i, x in enumerate(each)], dtype=torch.int32).cuda()
        s["table_out"], s["refs_out"] = torch.empty_like(s["table"]), torch.empty_like(refs)
        s["n_live"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        s["k"] = _randn((c["layers"], c["pages"], hkv, ps, d), dt, g)
        s["v"] = _randn((c["layers"], c["pages"], hkv, ps, d), dt, g)
    if own:   # the handles a serving program keeps
        import tiered_quantize_evict_gb300 as qe
        s["pool"] = qe.PagePool(s["k"], s["v"])
        s["seqs"] = qe.PageTable(s["table"], s["kv_len"], s.get("refs"))
        if c["op"] == "append":
            s["rope"] = qe.Rope(d, theta=10000.0, sections=s["sections"], halves=c["halves"])
    return s


def _sections(c):
    """Channel pairs of each axis: the first axis a quarter of the pairs, the others the rest evenly."""
    pairs = c["d"] // 2
    if c["axes"] == 1:
        return [pairs]
    first = pairs // 4
    rest = pairs - first
    each = rest // (c["axes"] - 1)
    return [first] + [each] * (c["axes"] - 2) + [rest - each * (c["axes"] - 2)]


# ------------------------------------------------------------------------------ one pass

def run(s):
    c = s["c"]
    return {"attend": _run_attend, "append": _run_append, "fork": _run_fork, "compact": _run_compact,
            "gather": _run_gather}[c["op"]](s, c)


def _run_attend(s, c):
    if own:
        out = s["pool"].attend(0, s["q"], s["q_start"], s["seqs"], max_q_len=s["max_q"], return_lse=c["lse"])
        return list(out) if c["lse"] else [out]
    out, lse = _plain_attend(s["q"], s["q_start"], s["table"], s["kv_len"], s["k"][0], s["v"][0], s["max_q"])
    return [out, lse] if c["lse"] else [out]


def _token_rows(q_start, kv_len, total):
    """Sequence, index in its chunk and cache position of every packed token."""
    t = torch.arange(total, device=q_start.device)
    seq = torch.searchsorted(q_start[1:].long(), t, right=True)
    i = t - q_start.long()[seq]
    q_len = (q_start[1:] - q_start[:-1]).long()
    return seq, i, kv_len.long()[seq] - q_len[seq] + i


def _plain_attend(q, q_start, table, kv_len, k, v, max_q):
    total, hq, d = q.shape
    n, cols = table.shape
    hkv, ps = k.shape[1], k.shape[2]
    seq, i, pos = _token_rows(q_start, kv_len, total)
    at = table.clamp_min(0).long()
    inside = torch.arange(cols * ps, device=q.device)[None, :] < kv_len[:, None]            # [n][kv]
    kk = k[at].float().permute(0, 2, 1, 3, 4).reshape(n, hkv, cols * ps, d)
    vv = v[at].float().permute(0, 2, 1, 3, 4).reshape(n, hkv, cols * ps, d)
    vv = torch.where(inside[:, None, :, None], vv, torch.zeros((), device=q.device))
    qq = torch.zeros(n, max_q, hq, d, device=q.device)
    qq[seq, i] = q.float()
    see = torch.full((n, max_q), 0, device=q.device, dtype=torch.long)                      # keys each query sees
    see[seq, i] = pos + 1
    qq = qq.reshape(n, max_q, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, d)
    sc = torch.matmul(qq, kk.transpose(-1, -2)).mul_(1.0 / math.sqrt(d)).view(n, hkv, hq // hkv, max_q, cols * ps)
    off = torch.arange(cols * ps, device=q.device)[None, None, :] >= see[:, :, None]
    sc.masked_fill_(off[:, None, None], float("-inf"))
    m = sc.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    p = sc.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(n, hkv, -1, cols * ps), vv).view(n, hkv, hq // hkv, max_q, d) / l.clamp_min(1e-30)
    lse = (m + torch.log(l)).squeeze(-1)
    o = o.permute(0, 3, 1, 2, 4).reshape(n, max_q, hq, d)[seq, i]
    lse = lse.permute(0, 3, 1, 2).reshape(n, max_q, hq)[seq, i]
    return o.to(q.dtype), lse


def _run_append(s, c):
    if own:
        q = s["pool"].append(0, s["k_new"], s["v_new"], s["q_start"], s["seqs"], q=s["q"], rope=s["rope"],
                             positions=s["positions"])
        return [q, s["k"], s["v"]]
    dev = s["q"].device
    pairs = c["d"] // 2
    axis = torch.repeat_interleave(torch.arange(c["axes"], device=dev), torch.tensor(s["sections"], device=dev), output_size=pairs)
    freq = 10000.0 ** (-torch.arange(pairs, device=dev, dtype=torch.float64) * 2 / c["d"])
    ang = s["positions"].double()[axis].t() * freq                                            # [total][pairs], 64 bits
    cos, sin = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]
    seq, _, pos = _token_rows(s["q_start"], s["kv_len"], s["q"].shape[0])
    page, row = s["table"].long()[seq, pos // c["ps"]], pos % c["ps"]
    s["k"][0][page, :, row] = _plain_rotate(s["k_new"], cos, sin, c["halves"])
    s["v"][0][page, :, row] = s["v_new"]
    return [_plain_rotate(s["q"], cos, sin, c["halves"]), s["k"], s["v"]]


def _plain_rotate(x, cos, sin, halves):
    y = x.float()
    a, b = (y[..., : y.shape[-1] // 2], y[..., y.shape[-1] // 2:]) if halves else (y[..., 0::2], y[..., 1::2])
    ra, rb = a * cos - b * sin, a * sin + b * cos
    return (torch.cat([ra, rb], -1) if halves else torch.stack([ra, rb], -1).flatten(-2)).to(x.dtype)


def _run_fork(s, c):
    if own:
        s["pool"].fork(s["seqs"], s["src"], s["dst"])
        table, kv_len, refs = s["table"].clone(), s["kv_len"].clone(), s["refs"].clone()
        s["pool"].free(s["seqs"], s["dst"])
        return [s["k"], s["v"], table, kv_len, refs, s["table"], s["kv_len"], s["refs"]]
    t, ln, refs, ps = s["table"], s["kv_len"], s["refs"], c["ps"]
    src, dst = s["src"].long(), s["dst"].long()
    part = ln[src] % ps                                                     # rows of the last page that is not full
    full = (ln[src] // ps).long()
    rank = torch.cumsum((part > 0).long(), 0) - 1
    order = torch.argsort((refs > 0).to(torch.int32), stable=True)          # free pages first, the lowest before the others
    old = t[src].gather(1, full.clamp_max(t.shape[1] - 1)[:, None])[:, 0].clamp_min(0).long()
    new = torch.where(part > 0, order[rank.clamp_min(0)], old)
    copied = torch.arange(ps, device=t.device)[None, :] < part[:, None]
    where = copied[None, :, None, :, None]
    s["k"][:, new] = torch.where(where, s["k"][:, old], s["k"][:, new])
    s["v"][:, new] = torch.where(where, s["v"][:, old], s["v"][:, new])
    col = torch.arange(t.shape[1], device=t.device)[None, :]
    child = torch.where(col < full[:, None], t[src], torch.full_like(t[src], -1))
    child = torch.where((col == full[:, None]) & (part > 0)[:, None], new[:, None].to(t.dtype), child)
    t[dst] = child
    ln[dst] = ln[src]
    got = child.reshape(-1)
    refs.index_add_(0, got.clamp_min(0).long(), (got >= 0).to(refs.dtype))
    table, kv_len, held = t.clone(), ln.clone(), refs.clone()
    got = t[dst].reshape(-1)
    refs.index_add_(0, got.clamp_min(0).long(), -(got >= 0).to(refs.dtype))
    t[dst] = -1
    ln[dst] = 0
    return [s["k"], s["v"], table, kv_len, held, t, ln, refs]


def _run_compact(s, c):
    if own:
        s["pool"].compact(s["seqs"], table_out=s["table_out"], refs_out=s["refs_out"], n_live=s["n_live"])
        return [s["k"], s["v"], s["table_out"], s["refs_out"], s["n_live"]]
    live = s["refs"] > 0
    idx = torch.arange(live.numel(), device=live.device)
    n_live = live.sum()
    src, dst = torch.nonzero(live & (idx >= n_live))[:, 0], torch.nonzero(~live & (idx < n_live))[:, 0]
    s["k"][:, dst] = s["k"][:, src]
    s["v"][:, dst] = s["v"][:, src]
    to = idx.clone()
    to[src] = dst
    s["table_out"].copy_(torch.where(s["table"] >= 0, to[s["table"].clamp_min(0).long()], torch.full_like(idx[:1], -1)))
    s["refs_out"].zero_()
    s["refs_out"][to[live]] = s["refs"][live]
    s["n_live"].copy_(n_live)
    return [s["k"], s["v"], s["table_out"], s["refs_out"], s["n_live"]]


def _run_gather(s, c):
    if own:
        return list(s["pool"].gather(0, s["seqs"], 0, c["kv"]))
    pos = torch.arange(c["kv"], device=s["table"].device)
    page, row = s["table"].long()[:, pos // c["ps"]], (pos % c["ps"])[None, :]                # [n][kv]
    return [x[0][page, :, row.expand_as(page)].permute(0, 2, 1, 3).contiguous() for x in (s["k"], s["v"])]


# ------------------------------------------------------------------------------ cost and exact values

def work(case):
    c, e = case, 2
    if c["op"] == "attend":
        ql, kl = _lens(c)
        seen = sum(q * kv - q * (q - 1) // 2 for q, kv in zip(ql, kl))
        return {"bytes": e * (2 * sum(kl) * c["hkv"] * c["d"] + 2 * sum(ql) * c["hq"] * c["d"]) + (4 * sum(ql) * c["hq"] if c["lse"] else 0),
                "flops": 4 * c["d"] * c["hq"] * seen}
    if c["op"] == "append":
        t = sum(_lens(c)[0])
        return {"bytes": e * 2 * t * (c["hq"] + 2 * c["hkv"]) * c["d"] + 4 * t * c["axes"], "flops": 3 * t * (c["hq"] + c["hkv"]) * c["d"]}
    row = e * 2 * c["layers"] * c["hkv"] * c["d"] if "layers" in c else e * 2 * c["hkv"] * c["d"]   # K and V of one token
    if c["op"] == "fork":
        lens = [max(1, int(c["kv"] * (1 - 0.5 * _frac(i)))) for i in range(c["parents"])]
        copied = sum(lens[i % c["parents"]] % c["ps"] for i in range(c["children"]))
        table = sum(_cdiv(lens[i % c["parents"]], c["ps"]) for i in range(c["children"]))
        return {"bytes": 2 * copied * row + 8 * 4 * table, "flops": 0}
    if c["op"] == "compact":
        n_live = max(1, int(c["pages"] * c["live"]))
        moved = n_live * (1 - n_live / c["pages"])       # pages of index >= n_live, on average over the seeds
        return {"bytes": 2 * moved * c["ps"] * row + 16 * c["pages"], "flops": 0}
    return {"bytes": 2 * c["n"] * c["kv"] * row, "flops": 0}


def exact(case, seed):
    c = dict(case)
    s = prepare(case, seed)
    ps = c["ps"]
    if c["op"] == "attend":
        qs, kl, table = s["q_start"].tolist(), s["kv_len"].tolist(), s["table"].long()
        grp = c["hq"] // c["hkv"]
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
        for b in range(c["n"]):
            q0, q1, n = qs[b], qs[b + 1], kl[b]
            pages = table[b, : _cdiv(n, ps)]
            mask = torch.arange(n, device="cuda")[None, :] > (torch.arange(q1 - q0, device="cuda") + n - (q1 - q0))[:, None]
            for h in range(c["hq"]):
                kk = s["k"][0, pages, h // grp].reshape(-1, c["d"])[:n].double()
                vv = s["v"][0, pages, h // grp].reshape(-1, c["d"])[:n].double()
                logit = (s["q"][q0:q1, h].double() @ kk.T / c["d"] ** 0.5).masked_fill(mask, -math.inf)
                out[q0:q1, h] = torch.softmax(logit, -1) @ vv
                lse[q0:q1, h] = torch.logsumexp(logit, -1)
        return [out, lse] if c["lse"] else [out]
    if c["op"] == "append":
        k, v = s["k"].double(), s["v"].double()
        half = c["d"] // 2
        q = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        kn = torch.zeros(s["k_new"].shape, dtype=torch.float64, device="cuda")
        first = [sum(s["sections"][:a]) for a in range(c["axes"] + 1)]
        for i in range(half):
            a = max(x for x in range(c["axes"]) if first[x] <= i)
            ang = s["positions"][a].double() * math.exp(-2 * i / c["d"] * math.log(10000.0))
            z = torch.polar(torch.ones_like(ang), ang)[:, None]
            x, y = (i, i + half) if c["halves"] else (2 * i, 2 * i + 1)
            for src, to in ((s["q"], q), (s["k_new"], kn)):
                w = torch.complex(src[..., x].double(), src[..., y].double()) * z
                to[..., x], to[..., y] = w.real, w.imag
        qs, kl, table = s["q_start"].tolist(), s["kv_len"].tolist(), s["table"].long()
        for b in range(c["n"]):
            pos = torch.arange(kl[b] - (qs[b + 1] - qs[b]), kl[b], device="cuda")
            k[0][table[b, pos // ps], :, pos % ps] = kn[qs[b]: qs[b + 1]]
            v[0][table[b, pos // ps], :, pos % ps] = s["v_new"][qs[b]: qs[b + 1]].double()
        return [q, k, v]
    if c["op"] == "gather":
        t = s["table"].long()
        out = [torch.zeros(c["n"], c["hkv"], c["kv"], c["d"], dtype=torch.float64, device="cuda") for _ in range(2)]
        for b in range(c["n"]):
            for o, x in zip(out, (s["k"], s["v"])):
                o[b] = x[0, t[b, : _cdiv(c["kv"], ps)]].transpose(0, 1).reshape(c["hkv"], -1, c["d"])[:, : c["kv"]].double()
        return out
    table, refs, kl = s["table"].tolist(), s["refs"].tolist(), s["kv_len"].tolist()
    k, v = s["k"].clone(), s["v"].clone()
    if c["op"] == "fork":
        free = [i for i, r in enumerate(refs) if r == 0]
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            for j in range(kl[a] // ps):
                table[b][j] = table[a][j]
                refs[table[a][j]] += 1
            rows = kl[a] % ps
            if rows:
                p, old = free.pop(0), table[a][kl[a] // ps]
                table[b][kl[a] // ps], refs[p] = p, 1
                k[:, p, :, :rows], v[:, p, :, :rows] = k[:, old, :, :rows].clone(), v[:, old, :, :rows].clone()
            kl[b] = kl[a]
        held = [torch.tensor(x, dtype=torch.int32) for x in (table, kl, refs)]
        return [k.double(), v.double()] + held + [s["table"], s["kv_len"], s["refs"]]
    n_live = sum(r > 0 for r in refs)
    src = [i for i in range(n_live, len(refs)) if refs[i] > 0]
    dst = [i for i in range(n_live) if refs[i] == 0]
    to = dict(zip(src, dst))
    new = [refs[i] for i in range(len(refs))]
    for a, b in to.items():
        k[:, b], v[:, b] = s["k"][:, a], s["v"][:, a]
        new[a], new[b] = 0, refs[a]
    table = [[to.get(p, p) for p in row] for row in table]
    return [k.double(), v.double(), torch.tensor(table, dtype=torch.int32), torch.tensor(new, dtype=torch.int32),
            torch.tensor([n_live], dtype=torch.int32)]
