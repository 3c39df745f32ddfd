"""Timed cases of the paged cache's operators for long and for common contexts: attention with a sliding window and a few
first tokens that stay visible (``window``), giving back the pages that the window has left (``drop``), and attention for
sequences that share a long prefix, which is read once for all of them (``shared``).

With ``own`` false every operator runs in its plain form (elementary torch operations in 32 bits);
with ``own`` true through the library's entry points.  ``exact`` gives the same results from the
operators' definitions in 64 bits.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
_GOLD = 0.6180339887498949
DROPPED = -2        # what stands in the page table for a page that was given back


def listed():
    return [
        # one new token of one short sequence, the shape of the smallest decode workload: launch latency
        _window("window_one_token", n=1, q=1, kv=320, ragged=0.0, prompt=False, window=128, sinks=4, hq=4, hkv=1, d=64, ps=16, dtype="bf16"),
        # a decode step of 64 conversations of up to 32K tokens, of which the cache holds the window and the sinks
        _window("window_decode_64", n=64, q=1, kv=32768, ragged=0.7, prompt=False, window=4096, sinks=4, hq=32, hkv=8, d=128, ps=32, dtype="bf16"),
        # up to 12 drafts of each of 16 sequences, ragged, with the log-sum-exp
        _window("window_drafts_16", n=16, q=12, kv=16384, ragged=0.5, prompt=False, window=2048, sinks=64, hq=32, hkv=8, d=128, ps=64, dtype="fp16",
                lse=True),
        # several prompts of odd lengths prefilled in one call, a short window
        _window("window_prompts", n=5, q=5003, kv=5003, ragged=0.6, prompt=True, window=1024, sinks=4, hq=32, hkv=8, d=128, ps=16, dtype="bf16"),
        # a 2048-token piece of a long prompt under a long window, the largest window call
        _window("window_chunk_32k", n=1, q=2048, kv=32768, ragged=0.0, prompt=False, window=8192, sinks=128, hq=32, hkv=8, d=128, ps=64, dtype="bf16"),
        # four continuations of one short prompt: launch latency
        _shared("shared_four", groups=1, n=4, q=1, prefix=256, mine=64, ragged=0.5, hq=4, hkv=1, d=64, ps=16, dtype="bf16"),
        # a decode step of 64 conversations over one 32K document
        _shared("shared_decode_64", groups=1, n=64, q=1, prefix=32768, mine=1024, ragged=0.8, hq=32, hkv=8, d=128, ps=32, dtype="bf16"),
        # up to 4 drafts of 48 sequences in 8 groups of different sizes, some of one sequence, with the log-sum-exp
        _shared("shared_drafts_8x6", groups=8, n=48, q=4, prefix=8192, mine=400, ragged=0.6, hq=32, hkv=8, d=128, ps=64, dtype="fp16", lse=True),
        # 256 samples of one instruction prompt, short answers so far
        _shared("shared_samples_256", groups=1, n=256, q=1, prefix=4100, mine=300, ragged=0.9, hq=32, hkv=8, d=128, ps=16, dtype="bf16"),
        # the bookkeeping of one short sequence
        _drop("drop_one", n=1, kv=320, ragged=0.0, window=128, sinks=4, hkv=1, d=64, ps=16, dtype="bf16"),
        # and of 256 conversations of up to 32K tokens
        _drop("drop_256", n=256, kv=32768, ragged=0.7, window=4096, sinks=4, hkv=1, d=64, ps=16, dtype="bf16"),
    ]


def _case(op, name, **kw):
    return {"op": op, **({"name": name} if name else {}), **kw}


def _window(name, lse=False, **kw):
    return _case("window", name, lse=lse, **kw)


def _shared(name, lse=False, **kw):
    return _case("shared", name, lse=lse, **kw)


def _drop(name, **kw):
    return _case("drop", name, **kw)


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    d, hkv = rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
    hq, ps, dtype = hkv * rng.choice([1, 2, 3, 4, 8]), rng.choice([16, 32, 64, 128]), rng.choice(["bf16", "fp16"])
    op = rng.choice(["window", "window", "window", "shared", "shared", "shared", "drop"])
    ragged = round(rng.uniform(0, 0.9), 2)
    if op == "window":
        prompt = rng.random() < 0.4
        window, sinks = log(1, 8192), rng.choice([0, 1, 4, log(1, 300)])
        n = log(1, 64)
        if prompt:
            q = kv = min(log(1, 5000), int(math.sqrt(5.0e8 / hq)))
        else:
            q, kv = log(1, 512), log(16, 32768)
            q = min(q, kv)
        seen = min(kv, window + sinks)
        # no more than the listed chunk's products, nor the listed decode step's cache
        n = max(1, min(n, int(5.0e8 // max(1, hq * q * seen)), int(2.2e6 // (min(kv, seen + q) * hkv))))
        return _window("", n=n, q=q, kv=kv, ragged=ragged, prompt=prompt, window=window, sinks=sinks, hq=hq, hkv=hkv, d=d, ps=ps,
                       dtype=dtype, lse=rng.random() < 0.5)
    if op == "shared":
        groups = log(1, 16)
        n = groups * log(1, 64)
        q, prefix, mine = log(1, 16), log(16, 32768), log(1, 1024)
        # no more than the listed decode step's products and cache
        n = max(1, min(n, int(1.4e8 // (hq * q * (prefix + mine)))))
        groups = max(1, min(groups, n, int(32768 * 8 // (prefix * hkv))))
        return _shared("", groups=groups, n=n, q=q, prefix=prefix, mine=mine, ragged=ragged, hq=hq, hkv=hkv, d=d, ps=ps, dtype=dtype,
                       lse=rng.random() < 0.5)
    return _drop("", n=log(1, 256), kv=log(16, 32768), ragged=ragged, window=log(1, 8192), sinks=rng.choice([0, 1, 4, log(1, 300)]),
                 hkv=1, d=64, ps=ps, dtype=dtype)


# ------------------------------------------------------------------------------ lengths and inputs

def _frac(i):
    """A fixed number in [0, 1) for sequence i (low-discrepancy: multiples of the golden ratio)."""
    return ((i + 1) * _GOLD) % 1.0


def _cdiv(a, b):
    return -(-a // b)


def _lens(c):
    """(q_lens, kv_lens) of a case: fixed by the case, the same for every seed."""
    if c["op"] == "shared":
        ql, kl = [], []
        for g, (first, end, prefix) in enumerate(_groups(c)):
            for i in range(first, end):
                q = max(1, int(c["q"] * (1 - c["ragged"] * _frac(i + 7))))
                ql.append(q)
                kl.append(prefix + max(q, int(c["mine"] * (1 - c["ragged"] * _frac(i)))))
        return ql, kl
    ql, kl = [], []
    for i in range(c["n"]):
        if c.get("prompt"):
            q = kv = max(1, int(c["kv"] * (1 - c["ragged"] * _frac(i))))
        else:
            q = max(1, int(c.get("q", 1) * (1 - c["ragged"] * _frac(i + 7))))
            kv = max(q, int(c["kv"] * (1 - c["ragged"] * _frac(i))))
        ql.append(q)
        kl.append(kv)
    return ql, kl


def _groups(c):
    """(first sequence, end, prefix length in whole pages) of every group; sizes differ, some are 1."""
    n, k, ps = c["n"], c["groups"], c["ps"]
    weight = [1 + 2 * _frac(g) if g % 3 != 1 else 0.1 for g in range(k)]
    out, first = [], 0
    for g in range(k):
        size = n - first if g == k - 1 else max(1, min(n - first - (k - 1 - g), int(n * weight[g] / sum(weight))))
        out.append((first, first + size, int(c["prefix"] * (1 - (c["ragged"] * _frac(g + 3) if g else 0))) // ps * ps))
        first += size
    return out


def _gone(c, kv, q):
    """Pages [first, end) of a row that the window has left when its last q of kv tokens are attended."""
    return _cdiv(c["sinks"], c["ps"]), max(0, kv - q - c["window"] + 1) // c["ps"]


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
    ql, kl = _lens(c)
    need = [_cdiv(x, ps) for x in kl]
    table = torch.full((c["n"], max(need)), -1, dtype=torch.int32)
    holds = []                        # (row, column) of the entries that hold a page of their own, or their row's first
    if c["op"] == "shared":
        for first, end, prefix in _groups(c):
            for i in range(first, end):
                holds += [(i, j) for j in range(prefix // ps if i > first else 0, need[i])]
    else:
        for i, n in enumerate(need):
            lo, hi = _gone(c, kl[i], ql[i]) if c["op"] == "window" else (0, 0)
            holds += [(i, j) for j in range(n) if not lo <= j < hi]
            if lo < hi:
                table[i, lo:hi] = DROPPED
    n_pages = len(holds) + 3
    perm = torch.randperm(n_pages, generator=h, dtype=torch.int64).to(torch.int32)
    at = torch.tensor(holds)
    table[at[:, 0], at[:, 1]] = perm[: len(holds)]
    if c["op"] == "shared":
        for first, end, prefix in _groups(c):
            table[first:end, : prefix // ps] = table[first, : prefix // ps].clone()
    refs = torch.bincount(table[table >= 0].long(), minlength=n_pages).to(torch.int32)
    s["table"], s["refs"] = table.cuda(), refs.cuda()
    s["kv_len"] = torch.tensor(kl, dtype=torch.int32).cuda()
    s["lens"] = (ql, kl)              # a serving loop knows them
    s["k"] = _randn((1, n_pages, hkv, ps, d), dt, g, outliers=2)
    s["v"] = _randn((1, n_pages, hkv, ps, d), dt, g)
    if c["op"] == "drop":
        s["rows"] = torch.randperm(c["n"], generator=h).to(torch.int32).cuda()
    else:
        s["q_start"] = torch.tensor([0] + ql).cumsum(0).to(torch.int32).cuda()
        s["q"] = _randn((sum(ql), c["hq"], d), dt, g)
    if c["op"] == "shared":
        gr = _groups(c)
        s["group_start"] = torch.tensor([x[0] for x in gr] + [c["n"]], dtype=torch.int32).cuda()
        s["prefix_len"] = torch.tensor([x[2] for x in gr], dtype=torch.int32).cuda()
        s["max_group"] = max(sum(ql[a:b]) for a, b, _ in gr)
    if own:   # the handles a serving program keeps
        import tiered_quantize_evict_gb300 as qe
        s["pool"] = qe.PagePool(s["k"], s["v"])
        s["seqs"] = qe.PageTable(s["table"], s["kv_len"], s["refs"])
    return s


# ------------------------------------------------------------------------------ one pass

def run(s):
    c = s["c"]
    return {"window": _run_window, "shared": _run_shared, "drop": _run_drop}[c["op"]](s, c)


def _keys(s, row, idx):
    """Keys and values of a row's tokens idx, [hkv][n][d] in 32 bits."""
    ps = s["c"]["ps"]
    page, at = s["table"][row].long()[idx // ps], idx % ps
    return [x[0][page, :, at].float().transpose(0, 1) for x in (s["k"], s["v"])]


def _logits(q, k, scale):
    """[hkv][grp][m][n] of q [m][hq][d] and k [hkv][n][d]."""
    m, hq, d = q.shape
    hkv = k.shape[0]
    qq = q.float().view(m, hkv, hq // hkv, d).permute(1, 2, 0, 3).reshape(hkv, -1, d)
    return torch.matmul(qq, k.transpose(-1, -2)).mul_(scale).view(hkv, hq // hkv, m, -1)


def _rows_out(o):
    """[hkv][grp][m][...] -> [m][hq][...]"""
    return o.permute(2, 0, 1, *range(3, o.dim())).flatten(1, 2)


def _run_window(s, c):
    if own:
        out = s["pool"].attend(0, s["q"], s["q_start"], s["seqs"], max_q_len=max(s["lens"][0]), window=c["window"], sinks=c["sinks"],
                               return_lse=c["lse"])
        return list(out) if c["lse"] else [out]
    dev, scale = s["q"].device, 1.0 / math.sqrt(c["d"])
    out = torch.empty_like(s["q"])
    lse = torch.empty(s["q"].shape[:2], device=dev)
    t0 = 0
    for row, (m, kv) in enumerate(zip(*s["lens"])):
        for a in range(0, m, 512):                          # pieces of the chunk, so that long prompts fit
            b = min(m, a + 512)
            pos = torch.arange(kv - m + a, kv - m + b, device=dev)
            first, end = max(0, kv - m + a - c["window"] + 1), kv - m + b
            idx = torch.cat([torch.arange(min(c["sinks"], first), device=dev), torch.arange(first, end, device=dev)])
            k, v = _keys(s, row, idx)
            sc = _logits(s["q"][t0 + a: t0 + b], k, scale)
            off = (idx[None, :] > pos[:, None]) | ((idx[None, :] <= pos[:, None] - c["window"]) & (idx[None, :] >= c["sinks"]))
            sc.masked_fill_(off, float("-inf"))
            top = sc.amax(-1, keepdim=True)
            p = sc.sub_(top).exp_()
            total = p.sum(-1, keepdim=True)
            o = torch.matmul(p.flatten(1, 2), v).view(*p.shape[:3], -1) / total
            out[t0 + a: t0 + b] = _rows_out(o).to(out.dtype)
            lse[t0 + a: t0 + b] = _rows_out((top + torch.log(total)).squeeze(-1))
        t0 += m
    return [out, lse] if c["lse"] else [out]


def _run_shared(s, c):
    if own:
        out = s["pool"].attend_shared(0, s["q"], s["q_start"], s["seqs"], s["group_start"], s["prefix_len"], max_group_len=s["max_group"],
                                      return_lse=c["lse"])
        return list(out) if c["lse"] else [out]
    dev, scale = s["q"].device, 1.0 / math.sqrt(c["d"])
    out = torch.empty_like(s["q"])
    lse = torch.empty(s["q"].shape[:2], device=dev)
    ql, kl = s["lens"]
    t0 = 0
    for first, end, prefix in _groups(c):
        rows = sum(ql[first:end])
        k, v = _keys(s, first, torch.arange(prefix, device=dev))
        sc = _logits(s["q"][t0: t0 + rows], k, scale)       # every row of the group over the prefix
        top = sc.amax(-1) if prefix else torch.full(sc.shape[:3], float("-inf"), device=dev)
        parts, a = [], 0
        for i in range(first, end):
            m, kv = ql[i], kl[i]
            idx = torch.arange(prefix, kv, device=dev)
            mk, mv = _keys(s, i, idx)
            mine = _logits(s["q"][t0 + a: t0 + a + m], mk, scale)
            mine.masked_fill_(idx[None, :] > torch.arange(kv - m, kv, device=dev)[:, None], float("-inf"))
            top[:, :, a: a + m] = torch.maximum(top[:, :, a: a + m], mine.amax(-1))
            parts.append((a, m, mine, mv))
            a += m
        p = sc.sub_(top[..., None]).exp_()
        total = p.sum(-1)
        o = torch.matmul(p.flatten(1, 2), v).view(*p.shape[:3], -1)
        for a, m, mine, mv in parts:
            p = mine.sub_(top[:, :, a: a + m, None]).exp_()
            total[:, :, a: a + m] += p.sum(-1)
            o[:, :, a: a + m] += torch.matmul(p.flatten(1, 2), mv).view(*p.shape[:3], -1)
        out[t0: t0 + rows] = _rows_out(o / total[..., None]).to(out.dtype)
        lse[t0: t0 + rows] = _rows_out(top + torch.log(total))
        t0 += rows
    return [out, lse] if c["lse"] else [out]


def _run_drop(s, c):
    if own:
        s["pool"].drop(s["seqs"], s["rows"], c["window"], sinks=c["sinks"])
        return [s["table"], s["refs"]]
    rows, t = s["rows"].long(), s["table"]
    col = torch.arange(t.shape[1], device=t.device)
    end = torch.div((s["kv_len"][rows] - c["window"] + 1).clamp_min(0), c["ps"], rounding_mode="floor")
    gone = (col[None, :] >= _cdiv(c["sinks"], c["ps"])) & (col[None, :] < end[:, None])
    old = t[rows]
    held = gone & (old >= 0)
    s["refs"].index_add_(0, old.clamp_min(0).flatten().long(), -held.flatten().to(s["refs"].dtype))
    t[rows] = torch.where(gone, torch.full_like(old, DROPPED), old)
    return [t, s["refs"]]


# ------------------------------------------------------------------------------ cost and exact values

def work(case):
    c, e = case, 2
    ql, kl = _lens(c)
    if c["op"] == "drop":
        n = 0
        for kv in kl:
            lo, hi = _gone(c, kv, 0)
            n += max(0, hi - lo)
        return {"bytes": 16 * n + 8 * c["n"], "flops": 0}    # entries and counts, read and written
    io = e * 2 * sum(ql) * c["hq"] * c["d"] + (4 * sum(ql) * c["hq"] if c["lse"] else 0)
    row = e * 2 * c["hkv"] * c["d"]                          # K and V of one token
    if c["op"] == "shared":
        seen = sum(q * kv - q * (q - 1) // 2 for q, kv in zip(ql, kl))
        held = sum(p + sum(kl[a:b]) - p * (b - a) for a, b, p in _groups(c))
        return {"bytes": io + row * held, "flops": 4 * c["d"] * c["hq"] * seen}
    seen = held = 0
    for m, kv in zip(ql, kl):
        first = max(0, kv - m - c["window"] + 1)
        held += min(c["sinks"], first) + kv - first
        for pos in range(kv - m, kv):
            lo = max(0, pos - c["window"] + 1)
            seen += min(c["sinks"], lo) + pos + 1 - lo
    return {"bytes": io + row * held, "flops": 4 * c["d"] * c["hq"] * seen}


def exact(case, seed):
    c = dict(case)
    s = prepare(case, seed)
    ps = c["ps"]
    ql, kl = _lens(c)
    if c["op"] == "drop":
        table, refs = s["table"].tolist(), s["refs"].tolist()
        for i in range(c["n"]):
            for j in range(len(table[i])):
                # no token of the page is a sink, and the next token's window begins behind the last
                if table[i][j] >= 0 and j * ps >= c["sinks"] and (j + 1) * ps <= kl[i] - c["window"] + 1:
                    refs[table[i][j]] -= 1
                    table[i][j] = DROPPED
        return [torch.tensor(table, dtype=torch.int32), torch.tensor(refs, dtype=torch.int32)]
    grp = c["hq"] // c["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    q0 = 0
    for b, (m, n) in enumerate(zip(ql, kl)):
        at = torch.arange(n, device="cuda")
        pos = at[n - m:, None]
        hide = at[None, :] > pos
        if c["op"] == "window":
            hide = hide | ((pos - at[None, :] >= c["window"]) & (at[None, :] >= c["sinks"]))
            some = (~hide).any(0)               # what nobody sees is left out
            at, hide = at[some], hide[:, some]
        page, tok = s["table"][b].long()[at // ps], at % ps
        for h in range(c["hkv"]):
            kk, vv = s["k"][0, page, h, tok].double(), s["v"][0, page, h, tok].double()
            for j in range(h * grp, (h + 1) * grp):
                logit = (s["q"][q0: q0 + m, j].double() @ kk.T / c["d"] ** 0.5).masked_fill(hide, -math.inf)
                out[q0: q0 + m, j] = torch.softmax(logit, -1) @ vv
                lse[q0: q0 + m, j] = torch.logsumexp(logit, -1)
        q0 += m
    return [out, lse] if c["lse"] else [out]
