"""The packed and paged attention operators, as measured: cases, inputs, plain forms and exact values.

Five operators, the packed (sequences of different lengths, one after another) and paged (key/value
cache in fixed-size pages) forms of the dense attention forward and backward:

  packed_fwd    O, LSE of attention inside each of N packed sequences
  packed_bwd    dQ, dK, dV of it from dO, O and LSE
  paged_fwd     O, LSE of the newest tokens of each request over its pages of a key/value cache
  page_slots    new pages, slot and position of every new token from the requests' lengths
  paged_write   new key/value rows into the cache at their slots

Tensors are token major: Q [T, H, d], K and V [T, H_kv, d], caches [pages, page_size, H_kv, d],
LSE [H, T].  Query i of a sequence with S_q queries and S_k keys sits at key position i + S_k - S_q.
"""
import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------------------ cases
def _ints(text):
    return [int(x) for x in text.split(",")]


def _packed(name, op, dtype, H, H_kv, d, lens_q, lens_k=None, causal=True, window=0):
    return {"name": name, "op": op, "dtype": dtype, "H": H, "H_kv": H_kv, "d": d, "lens_q": lens_q,
            "lens_k": lens_q if lens_k is None else lens_k, "causal": causal, "window": window}


def _paged(name, dtype, H, H_kv, d, page, new, ctx, window=0):
    return {"name": name, "op": "paged_fwd", "dtype": dtype, "H": H, "H_kv": H_kv, "d": d, "page": page,
            "new": new, "ctx": ctx, "window": window}


def _spread(lo, hi, n):
    """n lengths from lo to hi, odd ones among them, the same for everybody."""
    return ",".join(str(lo + (hi - lo) * ((i * 7919 + 13) % 997) // 996) for i in range(n))


def listed():
    return [
        # a handful of short prompts, the smallest call of a packed forward: latency
        _packed("packed_fwd_small", "packed_fwd", "bf16", 8, 8, 64, "1,17,64,100,33"),
        # a batch of prompts of a grouped-head model, 1 to 4096 tokens each
        _packed("packed_fwd_prompts", "packed_fwd", "bf16", 32, 8, 128, "4096,2048,1,1733,511,2900,1024,3967"),
        # a packed training batch of the same model
        _packed("packed_bwd_batch", "packed_bwd", "bf16", 32, 8, 128, "2048,1999,7,1024,130,1777,2048,600,1500,257"),
        # fp16, two key/value heads, head dim 64, keys of another length than the queries, a window
        # to both sides, one sequence without keys
        _packed("packed_bwd_f16_cross", "packed_bwd", "f16", 16, 2, 64, "512,300,65,1,480,512", "1024,777,1024,5,0,130",
                causal=False, window=256),
        # fp32 training of a small model
        _packed("packed_bwd_f32", "packed_bwd", "f32", 8, 2, 128, "1024,333,64,700,1"),
        # one user's answer: single token of one request over a short cache, latency
        _paged("paged_decode_small", "bf16", 32, 8, 128, 16, "1", "1023"),
        # a busy server's step: one new token for each of 64 requests, 100 to 8191 tokens behind them
        _paged("paged_decode_batch", "bf16", 32, 8, 128, 16, ",".join(["1"] * 64), _spread(100, 8191, 64)),
        # chunks of prompts beside decoding requests, over up to 8000 cached tokens
        _paged("paged_chunks", "bf16", 32, 8, 128, 64, "512,512,1,1,333,512,17,1,1,200", "7680,0,5001,812,2222,4096,63,8000,1,900"),
        # tables of a decode step of 8 requests
        {"name": "page_slots_small", "op": "page_slots", "page": 16, "N": 8, "most_new": 1, "most_ctx": 2048, "max_pages": 256},
        # tables of a large mixed step
        {"name": "page_slots_large", "op": "page_slots", "page": 16, "N": 1024, "most_new": 128, "most_ctx": 8192, "max_pages": 768},
        # cache rows of a decode step of 16 requests
        {"name": "paged_write_small", "op": "paged_write", "dtype": "bf16", "T": 16, "H_kv": 8, "d": 128, "page": 16, "pages": 256},
        # cache rows of a step full of prompts
        {"name": "paged_write_prompts", "op": "paged_write", "dtype": "bf16", "T": 16384, "H_kv": 8, "d": 128, "page": 16, "pages": 4096},
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of lo..hi."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["packed_fwd", "packed_bwd", "paged_fwd", "paged_fwd", "packed_bwd", "page_slots", "paged_write"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    H_kv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 8])
    if op == "page_slots":
        N = _log(rng, 1, 1024)
        return {"op": op, "page": rng.choice([8, 16, 32, 64, 128]), "N": N, "most_new": _log(rng, 1, 128),
                "most_ctx": _log(rng, 1, 8192), "max_pages": 1048}
    if op == "paged_write":
        page = rng.choice([8, 16, 32, 64, 128])
        T = _log(rng, 1, 16384)
        return {"op": op, "dtype": rng.choice(["bf16", "f16", "f32"]), "T": T, "H_kv": H_kv, "d": rng.choice([64, 128]),
                "page": page, "pages": -(-T // page) + rng.randrange(1, 64)}
    d = rng.choice([64, 128])
    if op == "paged_fwd":
        N = _log(rng, 1, 48)
        most = rng.choice([1, 1, 64, 512])
        if most > 1:
            N = min(N, 8)
        return {"op": op, "dtype": dtype, "H": H_kv * g, "H_kv": H_kv, "d": d, "page": rng.choice([8, 16, 32, 64, 128]),
                "new": ",".join(str(_log(rng, 1, most)) for _ in range(N)),
                "ctx": ",".join(str(_log(rng, 1, 7500) - 1) for _ in range(N)), "window": rng.choice([0, 0, 0, 500])}
    if op == "packed_bwd" and rng.random() < 0.2:
        dtype = "f32"
    N = _log(rng, 1, 8)
    most = 900 if dtype == "f32" else 2048
    lens_q = [_log(rng, 1, most) for _ in range(N)]
    causal = rng.random() < 0.7
    lens_k = lens_q if rng.random() < 0.7 else [_log(rng, 1, most) for _ in range(N)]
    return {"op": op, "dtype": dtype, "H": H_kv * g, "H_kv": H_kv, "d": d, "lens_q": ",".join(map(str, lens_q)),
            "lens_k": ",".join(map(str, lens_k)), "causal": causal, "window": rng.choice([0, 0, 200])}


# ----------------------------------------------------------------------------------------- inputs
def _rand(gen, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def _cu(lens):
    return torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    op = case["op"]
    if op in ("packed_fwd", "packed_bwd"):
        lq, lk = _ints(case["lens_q"]), _ints(case["lens_k"])
        dt = _DT[case["dtype"]]
        s.update(cu_q=_cu(lq), cu_k=_cu(lk), most_q=max(lq), most_k=max(max(lk), 1))
        s["Q"] = _rand(gen, (sum(lq), case["H"], case["d"]), dt)
        s["K"] = _rand(gen, (sum(lk), case["H_kv"], case["d"]), dt)
        s["V"] = _rand(gen, (sum(lk), case["H_kv"], case["d"]), dt)
        if op == "packed_bwd":
            s["dO"] = _rand(gen, (sum(lq), case["H"], case["d"]), dt, 0.1)
            s["O"], s["LSE"] = _plain_packed_fwd(s)
    elif op == "paged_fwd":
        new, ctx = _ints(case["new"]), _ints(case["ctx"])
        dt, page = _DT[case["dtype"]], case["page"]
        total = [a + b for a, b in zip(new, ctx)]
        need = [-(-t // page) for t in total]
        pages = sum(need) + 3  # a pool with a few free pages
        order = torch.randperm(pages, generator=gen, device="cuda")
        table = torch.full((len(new), max(need)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for i, n in enumerate(need):
            table[i, :n] = order[at:at + n].to(torch.int32)
            at += n
        s.update(cu_q=_cu(new), most_q=max(new), most_k=max(total), block_table=table,
                 seq_lens=torch.tensor(total, dtype=torch.int32, device="cuda"))
        s["Q"] = _rand(gen, (sum(new), case["H"], case["d"]), dt)
        s["K_cache"] = _rand(gen, (pages, page, case["H_kv"], case["d"]), dt)
        s["V_cache"] = _rand(gen, (pages, page, case["H_kv"], case["d"]), dt)
    elif op == "page_slots":
        N, page, mp = case["N"], case["page"], case["max_pages"]
        new = torch.randint(1, case["most_new"] + 1, (N,), generator=gen, device="cuda")
        ctx = torch.randint(0, case["most_ctx"] + 1, (N,), generator=gen, device="cuda")
        have = (ctx + page - 1) // page
        pool = N * mp
        order = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
        cols = torch.arange(mp, device="cuda")
        # the pages that the requests hold already, -1 behind them; the free list holds the rest
        table = torch.where(cols[None, :] < have[:, None], order[: N * mp].view(N, mp), -1).to(torch.int32)
        free = order.view(N, mp)[cols[None, :] >= have[:, None]].contiguous()
        T = N * case["most_new"]  # rows of the step's padded token buffers
        s.update(ctx_lens=ctx.to(torch.int32), block_table=table, free_pages=free,
                 free_start=torch.tensor([3], dtype=torch.int32, device="cuda"), tokens=T,
                 cu_q=torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), new.cumsum(0)]).to(torch.int32))
    else:
        T, page, dt = case["T"], case["page"], _DT[case["dtype"]]
        s["K"] = _rand(gen, (T, case["H_kv"], case["d"]), dt)
        s["V"] = _rand(gen, (T, case["H_kv"], case["d"]), dt)
        s["K_cache"] = _rand(gen, (case["pages"], page, case["H_kv"], case["d"]), dt)
        s["V_cache"] = _rand(gen, (case["pages"], page, case["H_kv"], case["d"]), dt)
        # runs of whole pages, the pages in any order
        some = torch.randperm(case["pages"], generator=gen, device="cuda")[: -(-T // page)]
        s["slots"] = (some[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)[:T].contiguous()
    return s


# ------------------------------------------------------------------------------------ plain forms
def _rows(cu, most):
    """[N, most] row numbers of the packed tokens and whether each is one of the sequence's."""
    at = torch.arange(most, device=cu.device)
    start, n = cu[:-1].long(), (cu[1:] - cu[:-1]).long()
    return start[:, None] + at, at < n[:, None], n


def _home(cu, T):
    """Sequence and place within it of each of T packed tokens."""
    t = torch.arange(T, device=cu.device)
    n = torch.searchsorted(cu[1:].long().contiguous(), t, right=True).clamp(max=cu.numel() - 2)
    return n, t - cu[n].long()


def _take(x, rows, ok):
    """Packed rows as a padded fp32 batch [N, heads, most, d], zeros behind each sequence."""
    if x.shape[0] == 0:
        return torch.zeros((*rows.shape, *x.shape[1:]), device=x.device).permute(0, 2, 1, 3)
    y = x[rows.clamp(max=x.shape[0] - 1)].float()
    return torch.where(ok[:, :, None, None], y, 0.0).permute(0, 2, 1, 3)


def _visible(nq, nk, most_q, most_k, causal, window):
    i = torch.arange(most_q, device=nq.device)[None, :, None]
    j = torch.arange(most_k, device=nq.device)[None, None, :]
    p = i + (nk - nq)[:, None, None]
    see = (i < nq[:, None, None]) & (j < nk[:, None, None])
    if causal:
        see = see & (j <= p)
    if window > 0:
        see = see & (p - j < window)
        if not causal:
            see = see & (j - p < window)
    return see[:, None, None]  # [N, 1, 1, most_q, most_k]


def _attend(q, k, v, see, H_kv, scale):
    """Padded q [N, H, Lq, d], k and v [N, H_kv, Lk, d] in fp32 -> O [N, H, Lq, d], LSE [N, H, Lq]."""
    N, H, Lq, d = q.shape
    s = torch.matmul(q.reshape(N, H_kv, H // H_kv, Lq, d), k.transpose(-1, -2)[:, :, None]) * scale
    s = torch.where(see, s, -torch.inf)
    m = s.amax(-1, keepdim=True)
    base = torch.where(m == -torch.inf, 0.0, m)
    p = torch.exp(s - base)
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v[:, :, None]) / torch.where(l > 0, l, 1.0)
    return o.reshape(N, H, Lq, d), (base + torch.log(l)).reshape(N, H, Lq)


def _plain_packed_fwd(s):
    c = s["case"]
    rq, okq, nq = _rows(s["cu_q"], s["most_q"])
    rk, okk, nk = _rows(s["cu_k"], s["most_k"])
    see = _visible(nq, nk, s["most_q"], s["most_k"], c["causal"], c["window"])
    o, lse = _attend(_take(s["Q"], rq, okq), _take(s["K"], rk, okk), _take(s["V"], rk, okk), see, c["H_kv"], c["d"] ** -0.5)
    n, i = _home(s["cu_q"], s["Q"].shape[0])
    return o[n, :, i].to(s["Q"].dtype), lse[n, :, i].t().contiguous()


def _plain_packed_bwd(s):
    c = s["case"]
    H_kv, scale = c["H_kv"], c["d"] ** -0.5
    rq, okq, nq = _rows(s["cu_q"], s["most_q"])
    rk, okk, nk = _rows(s["cu_k"], s["most_k"])
    see = _visible(nq, nk, s["most_q"], s["most_k"], c["causal"], c["window"])
    q, do, o = (_take(s[x], rq, okq) for x in ("Q", "dO", "O"))
    k, v = (_take(s[x], rk, okk)[:, :, None] for x in ("K", "V"))
    N, H, Lq, d = q.shape
    five = (N, H_kv, H // H_kv, Lq, d)
    delta = (do * o).sum(-1).reshape(five[:4])[..., None]
    q, do = q.reshape(five), do.reshape(five)
    lse = torch.where(okq[:, None], s["LSE"].t()[rq.clamp(max=s["Q"].shape[0] - 1)].permute(0, 2, 1), 0.0)
    lse = lse.reshape(five[:4])[..., None]
    p = torch.exp(torch.where(see, torch.matmul(q, k.transpose(-1, -2)) * scale - lse, -torch.inf))
    dv = torch.matmul(p.transpose(-1, -2), do).sum(2)
    ds = p * (torch.matmul(do, v.transpose(-1, -2)) - delta)
    dq = (torch.matmul(ds, k) * scale).reshape(N, H, Lq, d)
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(2) * scale
    n, i = _home(s["cu_q"], s["Q"].shape[0])
    nk_, j = _home(s["cu_k"], s["K"].shape[0])
    return dq[n, :, i].to(s["Q"].dtype), dk[nk_, :, j].to(s["K"].dtype), dv[nk_, :, j].to(s["V"].dtype)


def _plain_paged_fwd(s):
    c = s["case"]
    rq, okq, nq = _rows(s["cu_q"], s["most_q"])
    nk = s["seq_lens"].long()
    j = torch.arange(s["most_k"], device=nk.device)
    okk = j < nk[:, None]
    page = s["block_table"].long()[:, j // c["page"]].clamp(min=0)
    at = page * c["page"] + j % c["page"]
    flat = (-1, c["H_kv"], c["d"])
    k, v = (_take(s[x].view(flat), at, okk) for x in ("K_cache", "V_cache"))
    see = _visible(nq, nk, s["most_q"], s["most_k"], True, c["window"])
    o, lse = _attend(_take(s["Q"], rq, okq), k, v, see, c["H_kv"], c["d"] ** -0.5)
    n, i = _home(s["cu_q"], s["Q"].shape[0])
    return o[n, :, i].to(s["Q"].dtype), lse[n, :, i].t().contiguous()


def _plain_page_slots(s):
    page, mp = s["case"]["page"], s["block_table"].shape[1]
    cu, ctx = s["cu_q"].long(), s["ctx_lens"].long()
    new = cu[1:] - cu[:-1]
    have, need = (ctx + page - 1) // page, (ctx + new + page - 1) // page
    taken = (need - have).cumsum(0)
    first = s["free_start"].long() + taken - (need - have)
    cols = torch.arange(mp, device=cu.device)
    fresh = (cols >= have[:, None]) & (cols < need[:, None])
    pick = (first[:, None] + cols - have[:, None]).clamp(0, s["free_pages"].numel() - 1)
    table = torch.where(fresh, s["free_pages"][pick], s["block_table"])
    n, i = _home(s["cu_q"], s["tokens"])
    pos = ctx[n] + i
    inside = torch.arange(s["tokens"], device=cu.device) < cu[-1]
    slot = table[n, (pos // page).clamp(max=mp - 1)].long() * page + pos % page
    return {"block_table": table, "slots": torch.where(inside, slot, -1),
            "positions": torch.where(inside, pos, -1).to(torch.int32), "seq_lens": (ctx + new).to(torch.int32),
            "free_next": (s["free_start"] + taken[-1]).to(torch.int32)}


def _plain_paged_write(s):
    for new, cache in ((s["K"], s["K_cache"]), (s["V"], s["V_cache"])):
        cache.view(-1, *new.shape[1:])[s["slots"]] = new
    return s["K_cache"], s["V_cache"]


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"packed_fwd": _plain_packed_fwd, "packed_bwd": _plain_packed_bwd, "paged_fwd": _plain_paged_fwd,
                "page_slots": _plain_page_slots, "paged_write": _plain_paged_write}[op](s)
    import flashattention_backward_preprocess_gb300 as fa
    if op == "packed_fwd":
        return fa.fa_varlen_fwd(s["Q"], s["K"], s["V"], s["cu_q"], s["cu_k"], causal=c["causal"], window_size=c["window"])
    if op == "packed_bwd":
        return fa.fa_varlen_bwd(s["dO"], s["Q"], s["K"], s["V"], s["O"], s["LSE"], s["cu_q"], s["cu_k"],
                                causal=c["causal"], window_size=c["window"])
    if op == "paged_fwd":
        return fa.fa_paged_fwd(s["Q"], s["K_cache"], s["V_cache"], s["block_table"], s["cu_q"], s["seq_lens"],
                               window_size=c["window"])
    if op == "page_slots":
        slots, positions, seq_lens, free_next = fa.fa_page_slots(s["ctx_lens"], s["cu_q"], s["block_table"], s["free_pages"],
                                                                 s["free_start"], c["page"], s["tokens"])
        return {"block_table": s["block_table"], "slots": slots, "positions": positions, "seq_lens": seq_lens,
                "free_next": free_next}
    return fa.fa_paged_write(s["K"], s["V"], s["slots"], s["K_cache"], s["V_cache"])


# ------------------------------------------------------------------------------------------- work
def _pairs(nq, nk, causal, window):
    """Visible (query, key) pairs of one sequence."""
    p = torch.arange(nq, dtype=torch.int64) + (nk - nq)
    lo = (p - window + 1).clamp(min=0) if window > 0 else torch.zeros_like(p)
    hi = (p + 1) if causal else ((p + window) if window > 0 else torch.full_like(p, nk))
    return int((hi.clamp(max=nk) - lo).clamp(min=0).sum())


def _keys(nq, nk, causal, window):
    """Keys of one sequence that at least one query sees."""
    if nq == 0 or nk == 0:
        return 0
    lo = max(nk - nq - window + 1, 0) if window > 0 else 0
    hi = nk if causal or window == 0 else min(nk, nk - 1 + window)
    return max(hi - lo, 0)


def work(case):
    op = case["op"]
    if op == "page_slots":
        N, T = case["N"], case["N"] * case["most_new"]
        pages = N * (case["most_new"] / 2 / case["page"] + 0.5)  # taken, about
        return {"bytes": 4 * (2 * N + 1) + 8 * pages + 12 * T + 4 * N, "flops": 0}
    es = torch.empty((), dtype=_DT[case["dtype"]]).element_size()
    row = case["H_kv"] * case["d"] * es
    if op == "paged_write":
        return {"bytes": case["T"] * (4 * row + 8), "flops": 0}
    H, d = case["H"], case["d"]
    if op == "paged_fwd":
        new, ctx = _ints(case["new"]), _ints(case["ctx"])
        pairs = sum(_pairs(a, a + b, True, case["window"]) for a, b in zip(new, ctx))
        keys = sum(_keys(a, a + b, True, case["window"]) for a, b in zip(new, ctx))
        return {"bytes": sum(new) * H * (2 * d * es + 4) + 2 * keys * row + 4 * keys // case["page"], "flops": 4 * H * d * pairs}
    lq, lk = _ints(case["lens_q"]), _ints(case["lens_k"])
    pairs = sum(_pairs(a, b, case["causal"], case["window"]) for a, b in zip(lq, lk))
    if op == "packed_fwd":
        return {"bytes": sum(lq) * H * (2 * d * es + 4) + 2 * sum(lk) * row, "flops": 4 * H * d * pairs}
    return {"bytes": sum(lq) * H * (4 * d * es + 4) + 4 * sum(lk) * row, "flops": 10 * H * d * pairs}


# ------------------------------------------------------------------------------------------ exact
def _exact_sequence(q, k, v, causal, window):
    """Softmax weights [H, S_q, S_k] and LSE [H, S_q] of one sequence in fp64; q [S_q, H, d], k, v [S_k, H, d]."""
    nq, nk = q.shape[0], k.shape[0]
    x = torch.einsum("ihc,jhc->hij", q, k) / float(q.shape[2]) ** 0.5
    dist = torch.arange(nq, device=q.device)[:, None] + (nk - nq) - torch.arange(nk, device=q.device)[None, :]
    hidden = torch.zeros_like(dist, dtype=torch.bool)
    if causal:
        hidden |= dist < 0
    if window > 0:
        hidden |= dist >= window
        if not causal:
            hidden |= dist <= -window
    x.masked_fill_(hidden, -torch.inf)
    lse = torch.logsumexp(x, -1) if nk else torch.full((q.shape[1], nq), -torch.inf, dtype=q.dtype, device=q.device)
    return x, lse


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "page_slots":
        return None
    if op == "paged_write":
        out = []
        for new, cache in ((s["K"], s["K_cache"]), (s["V"], s["V_cache"])):
            y = cache.double()
            y[s["slots"] // case["page"], s["slots"] % case["page"]] = new.double()
            out.append(y)
        return tuple(out)
    g = case["H"] // case["H_kv"]
    cu_q = s["cu_q"].tolist()
    T = cu_q[-1]
    Q = s["Q"].double()
    O = torch.zeros_like(Q)
    LSE = torch.zeros((case["H"], T), dtype=torch.float64, device="cuda")
    causal = case.get("causal", True)
    bwd = op == "packed_bwd"
    if op == "paged_fwd":
        lens, table, page = s["seq_lens"].tolist(), s["block_table"], case["page"]
    else:
        cu_k = s["cu_k"].tolist()
    if bwd:
        dO, O16, saved = s["dO"].double(), s["O"].double(), s["LSE"].double()
        dQ, dK, dV = torch.zeros_like(Q), torch.zeros_like(s["K"], dtype=torch.float64), torch.zeros_like(s["V"], dtype=torch.float64)
    for n in range(len(cu_q) - 1):
        a, b = cu_q[n], cu_q[n + 1]
        if a == b:
            continue
        if op == "paged_fwd":
            held = table[n, : -(-lens[n] // page)].long()
            k, v = (s[x][held].reshape(-1, case["H_kv"], case["d"])[: lens[n]].double() for x in ("K_cache", "V_cache"))
        else:
            k, v = (s[x][cu_k[n]:cu_k[n + 1]].double() for x in ("K", "V"))
        if k.shape[0] == 0:
            LSE[:, a:b] = -torch.inf
            continue
        for h in range(case["H_kv"]):  # one key/value head at a time, for room
            at = slice(h * g, (h + 1) * g)
            kh, vh = (y[:, h:h + 1].expand(-1, g, -1) for y in (k, v))
            x, lse = _exact_sequence(Q[a:b, at], kh, vh, causal, case["window"])
            if not bwd:
                p = torch.exp(x - torch.where(lse == -torch.inf, 0.0, lse)[..., None])
                O[a:b, at] = torch.einsum("hij,jhc->ihc", p, vh)
                LSE[at, a:b] = lse
                continue
            kept = saved[at, a:b]
            p = torch.exp(x - torch.where(kept == -torch.inf, 0.0, kept)[..., None])
            gr = dO[a:b, at]
            dV[cu_k[n]:cu_k[n + 1], h] = torch.einsum("hij,ihc->jc", p, gr)
            t = torch.einsum("ihc,jhc->hij", gr, vh) - (gr * O16[a:b, at]).sum(-1).t()[..., None]
            p *= t
            p /= float(case["d"]) ** 0.5
            dQ[a:b, at] = torch.einsum("hij,jhc->ihc", p, kh)
            dK[cu_k[n]:cu_k[n + 1], h] = torch.einsum("hij,ihc->jc", p, Q[a:b, at])
    return (dQ, dK, dV) if bwd else (O, LSE)
