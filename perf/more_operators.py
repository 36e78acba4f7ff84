"""Drafted tokens over a paged cache, and a cache held in 8 bits: cases, inputs, plain forms and exact values.

Four operators around the paged key/value cache [pages, page_size, H_kv, d]:

  store    rows of new tokens quantised into an 8-bit cache at their slots, and the cache read back
  attend   O, LSE of the newest tokens of each request over the pages of an 8-bit cache
  tree     masks and positions of a tree of drafted tokens for each request, and O, LSE of the drafted
           tokens over the cache: each sees the tokens before the tree and its own ancestors
  accept   the rows of the accepted tokens moved up behind the cached ones, the rest dropped and their
           pages given back

An 8-bit row (one token and head of K or V) is d e4m3 numbers and one exponent byte b: the values are
number * 2^(b - 127), where b - 127 is the smallest whole number (within the type's limits) with
max |x| <= 448 * 2^(b - 127).  Exponents lie beside the cache as [pages, H_kv, page_size].  Node i of a
request's tree names its parent, an earlier node of it or -1 (then it follows the cached tokens).
"""
import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# exponents an 8-bit row may have, and the largest magnitude kept, by the rows' type
_LO = {"f32": -30, "bf16": -30, "f16": -15}
_HI = {"f32": 30, "bf16": 30, "f16": 8}
_MOST = {"f32": 448.0 * 2.0 ** 30, "bf16": 448.0 * 2.0 ** 30, "f16": 61440.0}


# ------------------------------------------------------------------------------------------ cases
def _ints(text):
    return [int(x) for x in text.split(",")]


def _spread(lo, hi, n):
    """n lengths from lo to hi, odd ones among them, the same for everybody."""
    return ",".join(str(lo + (hi - lo) * ((i * 7919 + 13) % 997) // 996) for i in range(n))


def _store(name, dtype, T, H_kv, d, page):
    return {"name": name, "op": "store", "dtype": dtype, "T": T, "H_kv": H_kv, "d": d, "page": page}


def _paged(name, op, dtype, q8, H, H_kv, d, page, new, ctx, window=0):
    return {"name": name, "op": op, "dtype": dtype, "q8": q8, "H": H, "H_kv": H_kv, "d": d, "page": page,
            "new": new, "ctx": ctx, "window": window}


def _accept(name, dtype, layers, H_kv, d, page, new, ctx):
    return {"name": name, "op": "accept", "dtype": dtype, "layers": layers, "H_kv": H_kv, "d": d, "page": page,
            "new": new, "ctx": ctx}


def listed():
    return [
        # a decode step of 16 requests: 16 rows of a layer into their pages; latency
        _store("store_step", "bf16", 16, 8, 128, 16),
        # a step full of prompts
        _store("store_prompts", "bf16", 16384, 8, 128, 16),
        # fp16 rows of a small model's prompts, an odd number of them
        _store("store_f16_odd", "f16", 5001, 2, 64, 64),
        # one user's answer: single token of one request over a short cache; latency
        _paged("q8_decode_small", "attend", "bf16", True, 32, 8, 128, 16, "1", "1023"),
        # a busy server's step: one new token for each of 64 requests, 100 to 8191 tokens behind them
        _paged("q8_decode_batch", "attend", "bf16", True, 32, 8, 128, 16, ",".join(["1"] * 64), _spread(100, 8191, 64)),
        # one long document being answered about
        _paged("q8_decode_long", "attend", "f16", True, 16, 2, 128, 64, "1", "131071"),
        # chunks of prompts beside decoding requests, over up to 8000 cached tokens
        _paged("q8_chunks", "attend", "bf16", True, 32, 8, 128, 64, "512,512,1,1,333,512,17,1,1,200",
               "7680,0,5001,812,2222,4096,63,8000,1,900"),
        # the drafts of one user's answer, 12 nodes; latency
        _paged("tree_small", "tree", "bf16", False, 32, 8, 128, 16, "12", "700"),
        # drafts for 32 requests, 8 to 64 nodes each, 100 to 6000 tokens behind them
        _paged("tree_batch", "tree", "bf16", False, 32, 8, 128, 16, _spread(8, 64, 32), _spread(100, 6000, 32)),
        # the same over an 8-bit cache, fp16
        _paged("tree_q8_batch", "tree", "f16", True, 32, 8, 128, 16, _spread(8, 64, 32), _spread(100, 6000, 32)),
        # one user's accepted tokens in a model of two layers; latency
        _accept("accept_small", "bf16", 2, 8, 128, 16, "12", "700"),
        # 64 requests with 64 drafts each in a model of 16 layers
        _accept("accept_batch", "bf16", 16, 8, 128, 16, ",".join(["64"] * 64), _spread(100, 1000, 64)),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of lo..hi."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["store", "attend", "attend", "tree", "tree", "accept"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    H_kv = rng.choice([1, 2, 4, 8])
    page = rng.choice([8, 16, 32, 64, 128])
    d = rng.choice([64, 128, 128, 256])
    if op == "store":
        return {"op": op, "dtype": rng.choice(["bf16", "f16", "f32"]), "T": _log(rng, 1, 16384 * 128 // (d * 2)), "H_kv": H_kv,
                "d": d, "page": page}
    if op == "accept":
        N = _log(rng, 1, 64)
        return {"op": op, "dtype": dtype, "layers": rng.randrange(1, 9), "H_kv": H_kv, "d": d, "page": page,
                "new": ",".join(str(_log(rng, 1, 64)) for _ in range(N)),
                "ctx": ",".join(str(_log(rng, 1, 1000) - 1) for _ in range(N))}
    H = H_kv * rng.choice([1, 2, 3, 4, 8])
    if op == "tree":
        N = _log(rng, 1, 32)
        return {"op": op, "dtype": dtype, "q8": rng.random() < 0.5, "H": H, "H_kv": H_kv, "d": d, "page": page,
                "new": ",".join(str(_log(rng, 1, 100)) for _ in range(N)),
                "ctx": ",".join(str(_log(rng, 1, 4000) - 1) for _ in range(N)), "window": 0}
    N = _log(rng, 1, 48)
    most = rng.choice([1, 1, 64, 512])
    if most > 1:
        N = min(N, 8)
    return {"op": op, "dtype": dtype, "q8": True, "H": H, "H_kv": H_kv, "d": d, "page": page,
            "new": ",".join(str(_log(rng, 1, most)) for _ in range(N)),
            "ctx": ",".join(str(_log(rng, 1, 7500) - 1) for _ in range(N)), "window": rng.choice([0, 0, 0, 500])}


# ----------------------------------------------------------------------------------------- inputs
def _rows(gen, shape, dtype):
    """Rows of K or V: normal, each row with a size of its own, as heads and tokens of a model have."""
    x = torch.randn(shape, generator=gen, device="cuda")
    size = torch.randn((*shape[:-1], 1), generator=gen, device="cuda")
    return (x * torch.exp2(0.5 * size)).to(dtype)


def _cu(lens):
    return torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)


def _quantise(x, kind):
    """e4m3 numbers and exponents [...] of rows x [..., d] of type `kind`."""
    x = x.float()
    most = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)
    m, k = torch.frexp(most)  # most = m 2^k, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, k - 9, k - 8)
    e = torch.where(most == 0, _LO[kind], e).clamp(_LO[kind], _HI[kind])
    y = torch.where(torch.isfinite(x), x.clamp(-_MOST[kind], _MOST[kind]), torch.nan)
    y = y * torch.exp2(-e.float())[..., None]
    return y.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _cache(gen, pages, page, H_kv, d, kind):
    """An 8-bit cache and its exponents [pages, H_kv, page], in use already."""
    q, e = _quantise(_rows(gen, (pages, page, H_kv, d), _DT[kind]), kind)
    return q, e.transpose(1, 2).contiguous()


def _table(gen, lens, page, pages):
    """Pages of each request in any order, -1 behind its last; and the pages left over."""
    need = [-(-t // page) for t in lens]
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(max(need), 1)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return table, order, at


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    op, page, H_kv, d, kind = case["op"], case["page"], case["H_kv"], case["d"], case["dtype"]
    dt = _DT[kind]
    if op == "store":
        T = case["T"]
        pages = -(-T // page) + 3
        s["K"], s["V"] = _rows(gen, (T, H_kv, d), dt), _rows(gen, (T, H_kv, d), dt)
        s["K_cache"], s["K_exp"] = _cache(gen, pages, page, H_kv, d, kind)
        s["V_cache"], s["V_exp"] = _cache(gen, pages, page, H_kv, d, kind)
        some = torch.randperm(pages, generator=gen, device="cuda")[: -(-T // page)]
        s["slots"] = (some[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)[:T].contiguous()
        s["all"] = torch.arange(pages * page, device="cuda")
        return s
    new, ctx = _ints(case["new"]), _ints(case["ctx"])
    total = [a + b for a, b in zip(new, ctx)]
    pages = sum(-(-t // page) for t in total) + 3  # a pool with a few free pages
    s["block_table"], order, at = _table(gen, total, page, pages)
    s.update(cu_q=_cu(new), most_q=max(new), most_k=max(total),
             seq_lens=torch.tensor(total, dtype=torch.int32, device="cuda"))
    if op == "accept":
        s["K"] = [_rows(gen, (pages, page, H_kv, d), dt) for _ in range(case["layers"])]
        s["V"] = [_rows(gen, (pages, page, H_kv, d), dt) for _ in range(case["layers"])]
        s["free_pages"], s["free_start"] = order, torch.tensor([at], dtype=torch.int32, device="cuda")
        # of each request the first token and some of the far branches
        u = torch.rand((len(new), 9), generator=gen, device="cuda").tolist()
        path, count = torch.zeros(sum(new), dtype=torch.int32), []
        row = 0
        for n, r in zip(new, u):
            want = min(1 + int(r[0] * 7), 1 + (n - 1) // 2)
            far = sorted({want + int(x * (n - want)) for x in r[1:want]}) if want > 1 else []
            kept = [0] + far
            path[row:row + len(kept)] = torch.tensor(kept, dtype=torch.int32)
            count.append(len(kept))
            row += n
        s["path"], s["count"] = path.cuda(), torch.tensor(count, dtype=torch.int32, device="cuda")
        return s
    s["Q"] = torch.randn((sum(new), case["H"], d), generator=gen, device="cuda").to(dt)
    if case["q8"]:
        s["K_cache"], s["K_exp"] = _cache(gen, pages, page, H_kv, d, kind)
        s["V_cache"], s["V_exp"] = _cache(gen, pages, page, H_kv, d, kind)
    else:
        s["K_cache"], s["V_cache"] = _rows(gen, (pages, page, H_kv, d), dt), _rows(gen, (pages, page, H_kv, d), dt)
    if op == "tree":
        # node 0 is the last token of the answer so far, the others are drafted after an earlier one
        i = torch.cat([torch.arange(n, device="cuda") for n in new])
        up = (torch.rand(sum(new), generator=gen, device="cuda") * i).long()
        s["parents"] = torch.where(i == 0, -1, torch.minimum(up, i - 1)).to(torch.int32)
        s["ctx_lens"] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        s["words"] = -(-max(new) // 64)
    return s


# ------------------------------------------------------------------------------------ plain forms
def _padded(cu, most):
    """[N, most] row numbers of the packed tokens and whether each is one of the request's."""
    at = torch.arange(most, device=cu.device)
    start, n = cu[:-1].long(), (cu[1:] - cu[:-1]).long()
    return start[:, None] + at, at < n[:, None], n


def _home(cu, T):
    """Request and place within it of each of T packed tokens."""
    t = torch.arange(T, device=cu.device)
    n = torch.searchsorted(cu[1:].long().contiguous(), t, right=True).clamp(max=cu.numel() - 2)
    return n, t - cu[n].long()


def _values(cache, exp):
    """fp32 values of an 8-bit cache."""
    return cache.float() * torch.exp2(exp.transpose(1, 2).float() - 127.0)[..., None]


def _plain_store(s):
    c = s["case"]
    out = []
    for x in ("K", "V"):
        q, e = _quantise(s[x], c["dtype"])
        cache, exp = s[x + "_cache"], s[x + "_exp"]
        cache.view(torch.uint8).view(-1, c["H_kv"], c["d"])[s["slots"]] = q.view(torch.uint8)
        exp[s["slots"] // c["page"], :, s["slots"] % c["page"]] = e
        rows = _values(cache, exp).view(-1, c["H_kv"], c["d"])[s["all"]]
        out += [rows.to(s[x].dtype), exp]
    return out


def _plain_tree(s):
    """[N, most, most] whether node i sees node j, packed masks [T, words] and positions [T]."""
    cu, most = s["cu_q"], s["most_q"]
    rows, ok, n = _padded(cu, most)
    T = s["parents"].numel()
    up = torch.where(ok, s["parents"].long()[rows.clamp(max=T - 1)], -1)
    at = torch.arange(most, device=cu.device)
    see = (at[None, :, None] == at[None, None, :]) & ok[:, :, None]
    node, depth = up, torch.zeros_like(up)
    for _ in range(most):  # up the tree, all nodes at once
        see = see | ((node[:, :, None] == at) & (node >= 0)[:, :, None])
        depth = depth + (node >= 0)
        node = torch.where(node >= 0, torch.gather(up, 1, node.clamp(min=0)), -1)
    bit = torch.zeros((*see.shape[:2], s["words"] * 64), dtype=torch.int64, device=cu.device)
    bit[:, :, :most] = see.long()
    words = (bit.view(*see.shape[:2], s["words"], 64) << torch.arange(64, device=cu.device)).sum(-1)
    r, i = _home(cu, T)
    return see, words[r, i], (s["ctx_lens"][r] + depth[r, i]).to(torch.int32)


def _plain_attend(s, nodes=None):
    c = s["case"]
    H_kv, page = c["H_kv"], c["page"]
    rq, okq, nq = _padded(s["cu_q"], s["most_q"])
    nk = s["seq_lens"].long()
    q = torch.where(okq[:, :, None, None], s["Q"][rq.clamp(max=s["Q"].shape[0] - 1)].float(), 0.0)
    j = torch.arange(s["most_k"], device=nk.device)
    at = s["block_table"].long()[:, j // page].clamp(min=0) * page + j % page
    kv = []
    for x in ("K", "V"):
        rows = s[x + "_cache"]
        if c["q8"]:
            flat = rows.view(torch.uint8).view(-1, H_kv, c["d"])[at].view(torch.float8_e4m3fn).float()
            exp = s[x + "_exp"].transpose(1, 2).reshape(-1, H_kv)[at]
            rows = flat * torch.exp2(exp.float() - 127.0)[..., None]
        else:
            rows = rows.view(-1, H_kv, c["d"])[at].float()
        kv.append(torch.where((j < nk[:, None])[:, :, None, None], rows, 0.0).permute(0, 2, 1, 3))
    k, v = kv
    N, Lq = rq.shape
    i = torch.arange(Lq, device=nk.device)
    first = (nk - nq)[:, None, None]
    dist = i[None, :, None] + first - j  # of key j before query i
    see = (j < nk[:, None])[:, None, :] & okq[:, :, None]
    if nodes is None:
        see = see & (dist >= 0)
        if c["window"] > 0:
            see = see & (dist < c["window"])
    else:
        inside = torch.gather(nodes, 2, (j - first).clamp(0, Lq - 1).expand(N, Lq, j.numel()))
        see = see & ((j < first) | (inside & (j - first < Lq)))
    q = q.permute(0, 2, 1, 3).reshape(N, H_kv, c["H"] // H_kv, Lq, c["d"])
    x = torch.matmul(q, k.transpose(-1, -2)[:, :, None]) * c["d"] ** -0.5
    x = torch.where(see[:, None, None], x, -torch.inf)
    m = x.amax(-1, keepdim=True)
    base = torch.where(m == -torch.inf, 0.0, m)
    p = torch.exp(x - base)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v[:, :, None]) / torch.where(total > 0, total, 1.0)
    lse = base + torch.log(total)
    n, i = _home(s["cu_q"], s["Q"].shape[0])
    o, lse = o.reshape(N, c["H"], Lq, c["d"]), lse.reshape(N, c["H"], Lq)
    return o[n, :, i].to(s["Q"].dtype), lse[n, :, i].t().contiguous()


def _plain_accept(s):
    c = s["case"]
    page, table = c["page"], s["block_table"].long()
    cu, total, count = s["cu_q"].long(), s["seq_lens"].long(), s["count"].long()
    ctx = total - (cu[1:] - cu[:-1])
    # rows of the accepted tokens, read before any is written
    n, i = _home(s["cu_q"], s["path"].numel())
    live = i < count[n]
    n, i = n[live], i[live]
    slot = lambda pos: table[n, pos // page] * page + pos % page
    src, dst = slot(ctx[n] + s["path"].long()[live]), slot(ctx[n] + i)
    for cache in s["K"] + s["V"]:
        flat = cache.view(-1, c["H_kv"], c["d"])
        flat[dst] = flat[src]
    kept = ctx + count
    had, need = (total + page - 1) // page, (kept + page - 1) // page
    back = had - need
    start = s["free_start"].long() - back.sum()
    cols = torch.arange(table.shape[1], device=table.device)
    gone = (cols >= need[:, None]) & (cols < had[:, None])
    free = s["free_pages"].clone()
    free[start + torch.arange(int(back.sum()), device=free.device)] = s["block_table"][gone]
    return {"lens": kept.to(torch.int32), "free_next": start.to(torch.int32), "free_pages": free,
            "K": s["K"], "V": s["V"]}


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        if op == "store":
            return _plain_store(s)
        if op == "attend":
            return _plain_attend(s)
        if op == "accept":
            return _plain_accept(s)
        see, words, positions = _plain_tree(s)
        return (words, positions, *_plain_attend(s, see))
    import flashattention_backward_preprocess_gb300 as fa
    if op == "store":
        fa.fa_paged_write_q8(s["K"], s["V"], s["slots"], s["K_cache"], s["V_cache"], s["K_exp"], s["V_exp"])
        K, V = fa.fa_paged_read_q8(s["K_cache"], s["V_cache"], s["K_exp"], s["V_exp"], s["all"], s["K"].dtype)
        return [K, s["K_exp"], V, s["V_exp"]]
    if op == "accept":
        fa.fa_paged_keep(s["path"], s["count"], s["cu_q"], s["seq_lens"], s["block_table"], s["K"], s["V"])
        lens, free_next = fa.fa_page_trim(s["count"], s["cu_q"], s["seq_lens"], s["block_table"], s["free_pages"],
                                          s["free_start"], c["page"])
        return {"lens": lens, "free_next": free_next, "free_pages": s["free_pages"], "K": s["K"], "V": s["V"]}
    exps = {"K_exp": s["K_exp"], "V_exp": s["V_exp"]} if c["q8"] else {}
    if op == "attend":
        return fa.fa_paged_fwd(s["Q"], s["K_cache"], s["V_cache"], s["block_table"], s["cu_q"], s["seq_lens"],
                               window_size=c["window"], **exps)
    tree, positions = fa.fa_tree_mask(s["parents"], s["cu_q"], s["ctx_lens"], s["words"])
    O, LSE = fa.fa_paged_fwd(s["Q"], s["K_cache"], s["V_cache"], s["block_table"], s["cu_q"], s["seq_lens"], tree=tree, **exps)
    return tree, positions, O, LSE


# ------------------------------------------------------------------------------------------- work
def _pairs(nq, nk, window):
    """Visible (query, key) pairs of one request."""
    p = torch.arange(nq, dtype=torch.int64) + (nk - nq)
    lo = (p - window + 1).clamp(min=0) if window > 0 else torch.zeros_like(p)
    return int((p + 1 - lo).sum())


def work(case):
    op, H_kv, d = case["op"], case["H_kv"], case["d"]
    es = torch.empty((), dtype=_DT[case["dtype"]]).element_size()
    if op == "store":
        T, page = case["T"], case["page"]
        pool = (-(-T // page) + 3) * page
        new = 2 * T * H_kv * (d * es + d + 1) + 8 * T
        return {"bytes": new + 2 * pool * H_kv * (d + 1 + d * es) + 8 * pool, "flops": 0}
    new, ctx = _ints(case["new"]), _ints(case["ctx"])
    if op == "accept":
        # about four rows of each request, read and written in every layer
        return {"bytes": 4 * len(new) * case["layers"] * 2 * 2 * H_kv * d * es + 12 * len(new), "flops": 0}
    window, H = case["window"], case["H"]
    row = H_kv * (d + 1) if case["q8"] else H_kv * d * es
    keys = sum(a + b - (max(b - window + 1, 0) if window > 0 else 0) for a, b in zip(new, ctx))
    out = {"bytes": sum(new) * H * (2 * d * es + 4) + 2 * keys * row + 4 * keys // case["page"],
           "flops": 4 * H * d * sum(_pairs(a, a + b, window) for a, b in zip(new, ctx))}
    if op == "tree":
        out["bytes"] += sum(new) * (8 + 8 * -(-max(new) // 64))
        # the tokens before the tree and about ln n ancestors
        out["flops"] = 4 * H * d * sum(a * b + 4 * a for a, b in zip(new, ctx))
    return out


# ------------------------------------------------------------------------------------------ exact
def _exact_row(x, kind):
    """Values an 8-bit row stands for, from fp64 rows: four significant bits at most."""
    most = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(most > 0, most, 1.0) / 448.0))
    e = torch.where(most > 448.0 * torch.exp2(e), e + 1, e)  # log2 next to a power of two
    e = torch.where((most > 0) & (most <= 448.0 * torch.exp2(e - 1)), e - 1, e)
    e = torch.where(most > 0, e, float(_LO[kind])).clamp(_LO[kind], _HI[kind])
    x = x.clamp(-_MOST[kind], _MOST[kind])
    size = x.abs()
    top = torch.floor(torch.log2(torch.where(size > 0, size, 1.0)))
    top = torch.where(torch.exp2(top) > size, top - 1, top)
    top = torch.where(torch.exp2(top + 1) <= size, top + 1, top)
    step = torch.exp2(torch.maximum(top - 3, e - 9))  # between neighbours; 2^-9 at the small end
    return torch.round(x / step) * step  # halves to even


def exact(case, seed):
    s = prepare(case, seed)
    op, page, H_kv, d = case["op"], case["page"], case["H_kv"], case["d"]
    if op == "accept":
        return None
    if op == "store":
        out = []
        for x in ("K", "V"):
            old = s[x + "_cache"].double() * (2.0 ** (s[x + "_exp"].double() - 127.0)).transpose(1, 2)[..., None]
            old[s["slots"] // page, s["slots"] % page] = _exact_row(s[x].double(), case["dtype"])
            out += [old.reshape(-1, H_kv, d), None]
        return out
    H, g = case["H"], case["H"] // H_kv
    cu, lens = s["cu_q"].tolist(), s["seq_lens"].tolist()
    T = cu[-1]
    Q = s["Q"].double()
    O = torch.zeros_like(Q)
    LSE = torch.zeros((H, T), dtype=torch.float64, device="cuda")
    for n in range(len(lens)):
        a, b, nk = cu[n], cu[n + 1], lens[n]
        nq = b - a
        held = s["block_table"][n, : -(-nk // page)].long()
        kv = []
        for x in ("K", "V"):
            rows = s[x + "_cache"][held].double()
            if case["q8"]:
                rows = rows * (2.0 ** (s[x + "_exp"][held].double() - 127.0)).permute(0, 2, 1)[..., None]
            kv.append(rows.reshape(-1, H_kv, d)[:nk])
        dist = torch.arange(nq, device="cuda")[:, None] + (nk - nq) - torch.arange(nk, device="cuda")[None, :]
        if op == "tree":
            # ancestors: the closure of "is the parent of", by squaring
            up = s["parents"][a:b].long()
            reach = torch.eye(nq, dtype=torch.float64, device="cuda")
            child = torch.nonzero(up >= 0)[:, 0]
            reach[child, up[child]] = 1.0
            for _ in range(max(nq - 1, 1).bit_length()):
                reach = (reach @ reach > 0).double()
            hidden = torch.zeros((nq, nk), dtype=torch.bool, device="cuda")
            hidden[:, nk - nq:] = reach == 0
        else:
            hidden = dist < 0
            if case["window"] > 0:
                hidden |= dist >= case["window"]
        for h in range(H_kv):  # one key/value head at a time, for room
            at = slice(h * g, (h + 1) * g)
            x = torch.einsum("ihc,jc->hij", Q[a:b, at], kv[0][:, h]) / float(d) ** 0.5
            x.masked_fill_(hidden, -torch.inf)
            lse = torch.logsumexp(x, -1)
            p = torch.exp(x - torch.where(lse == -torch.inf, 0.0, lse)[..., None])
            O[a:b, at] = torch.einsum("hij,jc->ihc", p, kv[1][:, h])
            LSE[at, a:b] = lse
    return (None, None, O, LSE) if op == "tree" else (O, LSE)
