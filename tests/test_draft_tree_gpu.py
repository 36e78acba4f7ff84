"""Trees of drafted tokens over a paged cache on the GPU: masks, attention, what is kept of a step."""
import math

import pytest
import torch

import flashattention_backward_preprocess_gb300 as fa
from tests import draft_ref as dr
from tests import packed_ref as ref
from tests.test_packed_gpu import DT, _cu, _rand
from tests.test_paged_q8_gpu import F8, _errors, _setup

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")


def _parents(seed, n, kind):
    """Parents of n tokens: any earlier one or none, a chain, all of one, several short chains."""
    g = torch.Generator().manual_seed(seed)
    if kind == "chain":
        return list(range(-1, n - 1))
    if kind == "star":
        return ([-1] + [0] * n)[:n]
    if kind == "roots":
        return [-1 if i % 5 == 0 else i - 1 for i in range(n)]
    return [int(torch.randint(-1, i, (1,), generator=g)) if i else -1 for i in range(n)]


@pytest.mark.parametrize("new,words,lead,pad", [
    ([1], 1, 0, 0), ([12], 1, 0, 0), ([64, 1, 0, 63], 1, 0, 3), ([65, 3, 128, 129], 3, 2, 5), ([300, 7], 5, 0, 1), ([9] * 200, 2, 1, 0),
    ([1000], 16, 0, 0),
])
@pytest.mark.parametrize("kind", ["any", "chain", "star", "roots"])
def test_masks(new, words, lead, pad, kind):
    T = lead + sum(new) + pad
    parents = [-1] * lead + [p for i, n in enumerate(new) for p in _parents(i, n, kind)] + [7] * pad
    ctx = [(i * 37) % 500 for i in range(len(new))]
    cu = _cu([lead] + new)[1:].contiguous()
    tree, pos = fa.fa_tree_mask(torch.tensor(parents, **I32), cu, torch.tensor(ctx, **I32), words)
    assert _errors() == ""
    at = lead
    want, want_pos = torch.zeros(T, words, dtype=torch.int64), torch.full((T,), -1, dtype=torch.int32)
    for n, c in zip(new, ctx):
        see, depth = dr.ancestors(parents[at:at + n])
        want[at:at + n] = dr.pack(see, words)
        want_pos[at:at + n] = torch.tensor([c + x for x in depth], dtype=torch.int32)
        at += n
    assert torch.equal(tree.cpu(), want)
    assert torch.equal(pos.cpu(), want_pos)


def test_masks_of_wrong_trees_are_reported():
    cu, ctx = _cu([4, 3]), torch.tensor([10, 20], **I32)
    for bad in (1, 2, 100, -2, 2 ** 31 - 1):  # its own parent, a later one, none of the request's
        parents = torch.tensor([-1, bad, 1, 0, -1, 0, 1], **I32)
        tree, pos = fa.fa_tree_mask(parents, cu, ctx)
        assert "parent" in _errors()
        assert tree[:, 0].tolist() == [1, 2, 6, 9, 1, 3, 7]
        assert pos.tolist() == [10, 10, 11, 11, 20, 21, 22]
    # more tokens than bits: what there is room for
    n = 70
    tree, pos = fa.fa_tree_mask(torch.tensor(list(range(-1, n - 1)), **I32), _cu([n]), ctx[:1].contiguous())
    assert "parent" in _errors()
    assert tree[69, 0].item() == -1 and tree[3, 0].item() == 15 and pos.tolist() == list(range(10, 80))
    # lengths that do not fit
    tree, pos = fa.fa_tree_mask(parents, torch.tensor([0, 5, 4], **I32), ctx)
    assert "lengths" in _errors()
    assert (tree == 0).all() and (pos == -1).all()
    tree, pos = fa.fa_tree_mask(parents, torch.tensor([0, 4, 9], **I32), ctx)
    assert "lengths" in _errors()
    tree, pos = fa.fa_tree_mask(parents[:0], _cu([0, 0]), ctx)
    assert tree.shape == (0, 1) and pos.shape == (0,) and _errors() == ""


def _plain_setup(seed, new, ctx, H, H_kv, d, page, dtype):
    total = [a + b for a, b in zip(new, ctx)]
    need = [-(-t // page) for t in total]
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))
    table = torch.full((len(new), max(max(need), 1)), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n].int()
        at += n
    caches = [_rand(seed + i, (pages, page, H_kv, d), dtype) for i in (1, 2)]
    for c in caches:
        c[order[at:].cuda()] = math.nan
    return _rand(seed + 5, (sum(new), H, d), dtype), caches, table.cuda(), torch.tensor(total, **I32)


def _check_tree(O, LSE, Q, vals, table, new, total, sees, dtype):
    page, d = vals[0].shape[1], Q.shape[2]
    a = 0
    for i, (nq, nk) in enumerate(zip(new, total)):
        k, v = (ref.gather_pages(x, table[i].cpu(), nk, page) for x in vals)
        vis = torch.cat([torch.ones(nq, nk - nq, dtype=torch.bool), sees[i]], 1)
        o, lse, mag, e = dr.attend(Q[a:a + nq].double().cpu(), k, v, vis, 1 / math.sqrt(d))
        ref.check(f"O of request {i} ({nq} over {nk})", O[a:a + nq], o, mag, e, dtype)
        ref.check_lse(LSE[:, a:a + nq], lse, e)
        a += nq


TREES = [([1], [0]), ([12], [700]), ([8, 0, 31, 64, 1], [0, 9, 100, 127, 128]), ([33, 65, 5], [97, 250, 1]), ([130, 2], [64, 1000])]


@pytest.mark.parametrize("dtype,H,H_kv,d,page,q8", [
    ("bf16", 8, 2, 128, 16, False), ("f16", 4, 4, 64, 32, False), ("bf16", 6, 2, 256, 16, False), ("f16", 7, 1, 96, 64, False),
    ("f32", 4, 2, 64, 16, False), ("bf16", 4, 2, 128, 5, False), ("f16", 2, 1, 32, 128, False), ("bf16", 130, 1, 64, 16, False),
    ("f16", 4, 2, 256, 128, False),
    ("bf16", 8, 2, 128, 16, True), ("f16", 4, 4, 64, 32, True), ("bf16", 6, 2, 256, 16, True), ("f16", 7, 1, 96, 64, True),
    ("f32", 4, 2, 64, 16, True), ("bf16", 4, 2, 128, 5, True), ("f16", 16, 1, 128, 8, True), ("f16", 130, 1, 64, 16, True),
    ("bf16", 3, 3, 128, 16, True), ("f16", 2, 2, 64, 256, True),
])
@pytest.mark.parametrize("kind", ["any", "roots"])
def test_tree_attention(dtype, H, H_kv, d, page, q8, kind):
    dt = DT[dtype]
    for n, (new, ctx) in enumerate(TREES):
        if H > 100 and sum(new) > 40:
            continue
        if q8:
            Q, caches, exps, table, lens = _setup(10 * n, new, ctx, H, H_kv, d, page, dt)
            vals = [dr.values(c, e) for c, e in zip(caches, exps)]
            kw = dict(K_exp=exps[0], V_exp=exps[1])
        else:
            Q, caches, table, lens = _plain_setup(10 * n, new, ctx, H, H_kv, d, page, dt)
            vals, kw = [c.double().cpu() for c in caches], {}
        ups = [_parents(i + 3, m, kind) for i, m in enumerate(new)]
        words = -(-max(new) // 64)
        tree, _ = fa.fa_tree_mask(torch.tensor(sum(ups, []), **I32), _cu(new), torch.tensor(ctx, **I32), words)
        O, LSE = fa.fa_paged_fwd(Q, *caches, table, _cu(new), lens, tree=tree, **kw)
        assert _errors() == ""
        _check_tree(O, LSE, Q, vals, table, new, lens.tolist(), [dr.ancestors(u)[0] for u in ups], dt)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_that_see_nothing(dtype, q8):
    """Masks without a bit leave the cached tokens, and where there are none O = 0 and LSE = -inf; bits of
    later tokens do not count; infinities in rows that nobody sees stay there."""
    dt, new, ctx, H, H_kv, d, page = DT[dtype], [6, 5, 40], [0, 30, 0], 4, 2, 64, 16
    if q8:
        Q, caches, exps, table, lens = _setup(1, new, ctx, H, H_kv, d, page, dt)
        vals, kw = [dr.values(c, e) for c, e in zip(caches, exps)], dict(K_exp=exps[0], V_exp=exps[1])
    else:
        Q, caches, table, lens = _plain_setup(1, new, ctx, H, H_kv, d, page, dt)
        vals, kw = [c.double().cpu() for c in caches], {}
    g = torch.Generator().manual_seed(2)
    tree = torch.randint(-2 ** 62, 2 ** 62, (sum(new), 1), generator=g)
    tree[0:4] = 0          # rows 0 to 3 of the first request see nothing
    tree[6:9] = 0          # and these the cached tokens only
    tree[12:15] = -2       # every token but the first, of which only those before count
    O, LSE = fa.fa_paged_fwd(Q, *caches, table, _cu(new), lens, tree=tree.cuda(), **kw)
    assert _errors() == ""
    bits = torch.stack([(tree[:, 0] >> k) & 1 for k in range(max(new))], 1).bool()
    sees, at = [], 0
    for n in new:
        sees.append(bits[at:at + n, :n] & torch.ones(n, n, dtype=torch.bool).tril())
        at += n
    assert (O[:4] == 0).all() and (LSE[:, :4] == -math.inf).all()
    _check_tree(O, LSE, Q, vals, table, new, lens.tolist(), sees, dt)


def test_chain_is_the_causal_step():
    """A tree that is a chain gives the bits of the plain step, over both kinds of cache."""
    new, ctx, H, H_kv, d, page, dt = [30, 1, 200], [100, 40, 7], 8, 2, 128, 16, torch.bfloat16
    parents = torch.tensor([i - 1 for n in new for i in range(n)], **I32)
    tree, pos = fa.fa_tree_mask(parents, _cu(new), torch.tensor(ctx, **I32), 4)
    assert pos.tolist() == [c + i for n, c in zip(new, ctx) for i in range(n)]
    Q, caches, table, lens = _plain_setup(1, new, ctx, H, H_kv, d, page, dt)
    a, b = (fa.fa_paged_fwd(Q, *caches, table, _cu(new), lens, tree=t) for t in (None, tree))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    Q, caches, exps, table, lens = _setup(1, new, ctx, H, H_kv, d, page, dt)
    a, b = (fa.fa_paged_fwd(Q, *caches, table, _cu(new), lens, tree=t, K_exp=exps[0], V_exp=exps[1]) for t in (None, tree))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert _errors() == ""


def _paths(seed, new):
    g = torch.Generator().manual_seed(seed)
    path, count = [], []
    for n in new:
        c = int(torch.randint(0, min(n, 9) + 1, (1,), generator=g))
        p = sorted(torch.randperm(n, generator=g)[:c].tolist())
        path += p + [-7] * (n - c)  # entries behind the count are not read
        count.append(c)
    return path, count


@pytest.mark.parametrize("dtype,d,page,layers,new,ctx", [
    ("bf16", 128, 16, 1, [12], [700]), ("f16", 64, 8, 3, [5, 0, 64, 30], [0, 12, 100, 7]), ("f32", 32, 3, 2, [9, 70], [1, 30]),
    ("q8", 128, 16, 33, [12, 33], [3, 40]), ("q8", 96, 5, 2, [20, 1, 8], [14, 4, 0]), ("bf16", 256, 1, 1, [40] * 300, [5] * 300),
])
def test_keep_and_trim(dtype, d, page, layers, new, ctx):
    H_kv, N = 3, len(new)
    total = [a + b for a, b in zip(new, ctx)]
    need = [-(-t // page) for t in total]
    pages = sum(need) + 4
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).int()
    table = torch.full((N, max(need) + 1), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    q8 = dtype == "q8"
    g = torch.Generator().manual_seed(3)
    if q8:
        make = lambda: torch.randint(0, 256, (pages, page, H_kv, d), generator=g, dtype=torch.uint8).cuda().view(F8)
    else:
        make = lambda: torch.randn(pages, page, H_kv, d, generator=g).to(DT[dtype]).cuda()
    K, V = [make() for _ in range(layers)], [make() for _ in range(layers)]
    Ke, Ve = ([torch.randint(97, 158, (pages, H_kv, page), generator=g, dtype=torch.uint8).cuda() for _ in range(layers)] if q8
              else None for _ in "KV")
    raw = lambda t: t.view(torch.uint8).cpu().clone() if t.dtype == F8 else t.cpu().clone()
    before = [raw(t) for t in K + V + (Ke + Ve if q8 else [])]
    path, count = _paths(4, new)
    cu, lens = _cu(new), torch.tensor(total, **I32)
    fa.fa_paged_keep(torch.tensor(path, **I32), torch.tensor(count, **I32), cu, lens, table.cuda(), K, V, Ke, Ve)
    free, start = order.clone().cuda(), torch.tensor([at], **I32)
    for _ in range(2):  # again: the same
        out, nxt = fa.fa_page_trim(torch.tensor(count, **I32), cu, lens, table.cuda(), free, start, page)
    assert _errors() == ""
    # the same moves on the host, all rows read before one is written
    want = [t.clone() for t in before]
    a = 0
    place = lambda r, p: (int(table[r, p // page]), p % page)
    for r in range(N):
        for i in range(count[r]):
            (p0, i0), (p1, i1) = place(r, ctx[r] + path[a + i]), place(r, ctx[r] + i)
            for w, b in zip(want, before):
                if w.shape == (pages, page, H_kv, d):
                    w[p1, i1] = b[p0, i0]
                else:
                    w[p1, :, i1] = b[p0, :, i0]
        a += new[r]
    for got, w in zip(K + V + (Ke + Ve if q8 else []), want):
        assert torch.equal(raw(got), w)
    kept = [c + k for c, k in zip(ctx, count)]
    assert out.tolist() == kept
    back = [int(table[r, c]) for r in range(N) for c in range(-(-kept[r] // page), need[r])]
    assert nxt.tolist() == [at - len(back)]
    assert free[nxt.item():].tolist() == back + order[at:].tolist()
    assert free[:nxt.item()].tolist() == order[:nxt.item()].tolist()


def test_keep_head_major_and_wrong_paths():
    H_kv, d, page, pages, new, ctx = 2, 64, 8, 12, [6, 5, 4, 3], [10, 3, 20, 0]
    table = torch.arange(12, dtype=torch.int32).view(4, 3).cuda()
    base = [_rand(i, (pages, page, H_kv, d), torch.bfloat16) for i in range(2)]
    lens, cu = torch.tensor([a + b for a, b in zip(new, ctx)], **I32), _cu(new)
    good = [0, 3, 5, 0, 0, 0] + [1, 2, 4, 0, 0] + [0, 1, 2, 3] + [2, 0, 0]
    count = [3, 3, 4, 1]

    def keep(path, cnt, caches, t=table):
        caches = [c.clone(memory_format=torch.preserve_format) for c in caches]
        fa.fa_paged_keep(torch.tensor(path, **I32), torch.tensor(cnt, **I32), cu, lens, t, caches[:1], caches[1:])
        return caches

    want = keep(good, count, base)
    assert _errors() == ""
    hm = [c.transpose(1, 2).contiguous().transpose(1, 2) for c in base]
    got = keep(good, count, hm)
    assert got[0].stride() == hm[0].stride() and all(torch.equal(a, b) for a, b in zip(got, want))
    assert _errors() == ""
    # request 0 wrong in many ways: it is left alone, the others are moved
    for path0, c0 in (([0, 3, 3], 3), ([0, 5, 3], 3), ([0, 3, 6], 3), ([-1, 3, 5], 3), ([0, 3, 5], 7), ([0, 3, 5], -1)):
        got = keep(path0 + good[3:], [c0] + count[1:], base)
        assert "path" in _errors()
        for a, b, w in zip(got, base, want):
            assert torch.equal(a[:3], b[:3]) and torch.equal(a[3:], w[3:])
    # a page outside the cache: its rows stay, the others move
    t = table.clone()
    t[0, 1] = 99
    got = keep(good, count, base, t)
    assert "page" in _errors()
    assert all(torch.equal(a[3:], w[3:]) and torch.equal(a[:1], w[:1]) for a, w in zip(got, want))


def test_trim_refuses_what_does_not_fit():
    page, table = 4, torch.arange(6, dtype=torch.int32).view(2, 3).cuda()
    cu, lens = _cu([8, 3]), torch.tensor([10, 12], **I32)
    free = torch.arange(100, 110, **I32)
    for count in ([9, 0], [-1, 0], [0, 4]):
        f = free.clone()
        out, nxt = fa.fa_page_trim(torch.tensor(count, **I32), cu, lens, table, f, torch.tensor([6], **I32), page)
        assert "lengths" in _errors()
        assert out.tolist() == [10, 12] and nxt.tolist() == [6] and torch.equal(f, free)
    # more pages back than were taken
    f = free.clone()
    out, nxt = fa.fa_page_trim(torch.tensor([1, 0], **I32), cu, lens, table, f, torch.tensor([1], **I32), page)
    assert "free pages" in _errors()
    assert out.tolist() == [3, 9] and nxt.tolist() == [1] and torch.equal(f, free)
    # the list had run out: what comes back is all there is
    t = table.clone()
    t[0, 2] = -1
    out, nxt = fa.fa_page_trim(torch.tensor([1, 3], **I32), cu, lens, t, f, torch.tensor([13], **I32), page)
    assert _errors() == ""
    assert out.tolist() == [3, 12] and nxt.tolist() == [9] and f.tolist() == free.tolist()[:9] + [1]


class _Spec:
    """Requests answered with drafted tokens: every step a tree for each, of which a path is kept."""

    def __init__(self, quantised, dtype, rows, H, H_kv, d, page, pages, layers=2):
        self.H, self.H_kv, self.d, self.dt, self.layers = H, H_kv, d, DT[dtype], layers
        self.cache = fa.PagedKVCache(layers, pages, page, H_kv, d, rows, 40, dtype=self.dt, quantised=quantised)
        self.q8 = quantised
        self.kv = [[torch.zeros(layers, 0, H_kv, d, dtype=torch.float64) for _ in "KV"] for _ in range(rows)]
        self.gen = torch.Generator().manual_seed(11)

    def stored(self, x):
        if not self.q8:
            return x.double()
        code, exp = dr.quantise(x)
        return dr.numbers(code) * (2.0 ** (exp.double() - 127))[..., None]

    def step(self, new, parents=None, keep=None):
        T = sum(new)
        cu = _cu(new)
        ups = None if parents is None else torch.tensor(sum(parents, []), **I32)
        pos = self.cache.begin(cu, T, parents=ups)
        r = lambda h: torch.randn(self.layers, T, h, self.d, generator=self.gen).to(self.dt)
        Q, K, V = r(self.H), r(self.H_kv), r(self.H_kv)
        sK, sV = self.stored(K), self.stored(V)
        out = [self.cache.attend(l, Q[l].cuda(), K[l].cuda(), V[l].cuda()) for l in range(self.layers)]
        a = 0
        for i, n in enumerate(new):
            held = self.kv[i][0].shape[1]
            see, depth = dr.ancestors(parents[i] if parents else list(range(-1, n - 1)))
            assert pos[a:a + n].tolist() == [held + x for x in depth]
            vis = torch.cat([torch.ones(n, held, dtype=torch.bool), see], 1)
            for l in range(self.layers):
                k, v = (torch.cat([old[l], s[l, a:a + n]]) for old, s in zip(self.kv[i], (sK, sV)))
                o, lse, mag, e = dr.attend(Q[l, a:a + n].double(), k, v, vis, self.d ** -0.5)
                ref.check(f"layer {l} request {i}", out[l][0][a:a + n], o, mag, e, self.dt)
                ref.check_lse(out[l][1][:, a:a + n], lse, e)
            p = list(range(n)) if keep is None else keep[i]
            self.kv[i] = [torch.cat([old, s[:, [a + x for x in p]]], 1) for old, s in zip(self.kv[i], (sK, sV))]
            a += n
        if keep is not None:
            path = [x for p, n in zip(keep, new) for x in p + [0] * (n - len(p))]
            self.cache.accept(torch.tensor(path, **I32), torch.tensor([len(p) for p in keep], **I32))
        assert _errors() == ""
        lens = [x[0].shape[1] for x in self.kv]
        assert self.cache.lens.tolist() == lens
        page = self.cache.page_size
        used = [int(x) for row, n in zip(self.cache.block_table, lens) for x in row[: -(-n // page)]]
        assert sorted(used + self.cache.free_pages[self.cache.free_start.item():].tolist()) == list(range(self.cache.free_pages.numel()))


@pytest.mark.parametrize("quantised,dtype,H,H_kv,d,page", [
    (False, "bf16", 8, 2, 128, 16), (True, "bf16", 8, 2, 128, 16), (True, "f16", 4, 4, 64, 8), (False, "f32", 4, 2, 32, 5),
    (True, "f32", 4, 1, 64, 16), (True, "bf16", 4, 2, 256, 32),
])
def test_drafting_end_to_end(quantised, dtype, H, H_kv, d, page):
    run = _Spec(quantised, dtype, 3, H, H_kv, d, page, pages=90)
    run.step([30, 0, 7])
    run.step([12, 5, 12], [_parents(1, 12, "any"), _parents(2, 5, "chain"), _parents(3, 12, "roots")], [[0, 3], [0], []])
    run.step([12, 9, 1], [_parents(4, 12, "any"), _parents(5, 9, "star"), [-1]], [[0, 5, 9, 11], [0, 8], [0]])
    run.step([1, 1, 1])
    run.cache.release(1)
    run.kv[1] = [x[:, :0] for x in run.kv[1]]
    run.step([40, 40, 40], [_parents(i, 40, "any") for i in range(3)], [list(range(0, 40, 5)), [39], list(range(40))])
    run.step([2, 0, 3], keep=[[0], [], [0, 1]])


@pytest.mark.parametrize("quantised", [False, True])
def test_drafting_step_is_capturable(quantised):
    """begin, attend and accept captured once; every replay goes on from the last."""
    rows, H, H_kv, d, page, n = 3, 8, 2, 128, 16, 10
    caches = [fa.PagedKVCache(1, 60, page, H_kv, d, rows, 20, quantised=quantised) for _ in range(2)]
    gen = torch.Generator().manual_seed(1)
    r = lambda h: torch.randn(rows * n, h, d, generator=gen).bfloat16().cuda()
    cu = _cu([n] * rows)
    Q, K, V = r(H), r(H_kv), r(H_kv)
    parents = torch.tensor(sum((_parents(i, n, "any") for i in range(rows)), []), **I32)
    path, count = torch.zeros(rows * n, **I32), torch.zeros(rows, **I32)

    def step(c):
        pos = c.begin(cu, rows * n, parents=parents)
        out = c.attend(0, Q, K, V)
        c.accept(path, count)
        return (pos, *out)

    def fresh(seed):
        for t, h in ((Q, H), (K, H_kv), (V, H_kv)):
            t.copy_(r(h))
        parents.copy_(torch.tensor(sum((_parents(seed + i, n, "any") for i in range(rows)), []), **I32))
        p, c = [], []
        g = torch.Generator().manual_seed(seed)
        for _ in range(rows):
            k = int(torch.randint(0, 6, (1,), generator=g))
            p += sorted(torch.randperm(n, generator=g)[:k].tolist()) + [0] * (n - k)
            c.append(k)
        path.copy_(torch.tensor(p, **I32))
        count.copy_(torch.tensor(c, **I32))

    fresh(0)
    for c in caches:
        step(c)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(caches[0])
    for i in range(12):
        fresh(10 * i + 1)
        g.replay()
        want = step(caches[1])
        assert _errors() == ""
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        for name in ("lens", "free_start", "free_pages"):
            assert torch.equal(getattr(caches[0], name), getattr(caches[1], name)), name
