"""Exponents of an 8-bit cache, at every kernel that attends over one: tiles and pages of nothing but zeros, bytes
that nobody has written, rows whose sizes lie far apart, rows that fp16 cannot hold."""
import math

import pytest
import torch

import flashattention_backward_preprocess_gb300 as fa
from tests import draft_ref as dr
from tests import packed_ref as ref
from tests.test_draft_tree_gpu import I32, _check_tree, _parents
from tests.test_packed_gpu import DT, _cu
from tests.test_paged_q8_gpu import _check, _errors, _setup

pytestmark = pytest.mark.gpu

# dtype, H, H_kv, d, page_size, new tokens: few rows a request (many requests, few), 128-row tiles, a copy of the
# rows, CUDA cores
KERNELS = {
    "rows": ("bf16", 8, 2, 128, 16, [6] * 80), "rows_f16": ("f16", 4, 2, 64, 16, [12, 16]),
    "tiles": ("bf16", 8, 2, 128, 16, [40, 30]), "tiles_f16": ("f16", 4, 1, 128, 24, [35, 60]), "tiles_64": ("f16", 4, 2, 64, 16, [50, 40]),
    "tiles_256": ("bf16", 4, 2, 256, 16, [40, 3]), "tiles_f16_256": ("f16", 2, 1, 256, 8, [1, 70]),
    "copy": ("bf16", 8, 2, 128, 16, [300, 200]), "copy_f16": ("f16", 8, 2, 64, 32, [300, 220]), "simt": ("f32", 4, 2, 64, 16, [20, 30]),
}
# fp16's P where the rows are copied: packed_ref and test_paged_q8_kernels_gpu say why
P_STEP = {"copy_f16": 2.0 ** -25}


def _zero(caches, exps, page):
    for c, e in zip(caches, exps):
        c.view(torch.uint8)[page] = 0
        e[page] = 0


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("where", ["last", "first", "all", "cleared"])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 150), (False, 0)])
def test_tiles_of_zeros(kernel, where, causal, window):
    """Whole tiles of keys without a page, or of a cleared cache, some of whose columns the mask hides: keys of 0
    with values of 0."""
    dtype, H, H_kv, d, page, new = KERNELS[kernel]
    dt, ctx = DT[dtype], [(29 * i) % 70 + 128 for i in range(len(new))]
    Q, caches, exps, table, lens = _setup(9, new, ctx, H, H_kv, d, page, dt)
    cols = {"last": range(128 // page, table.shape[1]), "first": range(-(-128 // page))}.get(where, range(table.shape[1]))
    held = [min(-(-n // page), table.shape[1]) for n in lens.tolist()]
    asked = table.clone()
    for n in range(len(new)):
        for c in cols:
            if c < held[n]:
                _zero(caches, exps, int(table[n, c]))
                if where != "cleared":
                    asked[n, c] = -1
    O, LSE = fa.fa_paged_fwd(Q, *caches, asked, _cu(new), lens, causal=causal, window_size=window, K_exp=exps[0], V_exp=exps[1])
    assert ("page" in _errors()) == (where != "cleared")
    _check(O, LSE, Q, caches, exps, table, new, lens.tolist(), dt, causal, window, p_step=P_STEP.get(kernel, 0.0))


@pytest.mark.parametrize("kernel", KERNELS)
def test_tree_over_a_cleared_cache(kernel):
    dtype, H, H_kv, d, page, new = KERNELS[kernel]
    dt, ctx = DT[dtype], [(29 * i) % 7 for i in range(len(new))]
    Q, caches, exps, table, lens = _setup(9, new, ctx, H, H_kv, d, page, dt)
    _zero(caches, exps, slice(None))
    ups = [_parents(i, m, "any") for i, m in enumerate(new)]
    tree, _ = fa.fa_tree_mask(torch.tensor(sum(ups, []), **I32), _cu(new), torch.tensor(ctx, **I32), -(-max(new) // 64))
    O, LSE = fa.fa_paged_fwd(Q, *caches, table, _cu(new), lens, tree=tree, K_exp=exps[0], V_exp=exps[1])
    assert _errors() == ""
    assert (O == 0).all()
    _check_tree(O, LSE, Q, [dr.values(c, e) for c, e in zip(caches, exps)], table, new, lens.tolist(),
                [dr.ancestors(u)[0] for u in ups], dt)


@pytest.mark.parametrize("scale", [1e-38, 1e-30])
@pytest.mark.parametrize("kernel", ["tiles", "tiles_f16", "rows"])
def test_tiny_scale(kernel, scale):
    """A scale that leaves every score next to 0, masked columns among them."""
    dtype, H, H_kv, d, page, new = KERNELS[kernel]
    dt, ctx = DT[dtype], [(29 * i) % 70 for i in range(len(new))]
    Q, caches, exps, table, lens = _setup(9, new, ctx, H, H_kv, d, page, dt)
    for c, e in zip(caches, exps):
        e.copy_((e.int() - 20).clamp(min=97).to(torch.uint8))
    O, LSE = fa.fa_paged_fwd(Q, *caches, table, _cu(new), lens, scale=scale, K_exp=exps[0], V_exp=exps[1])
    assert _errors() == ""
    vals, a = [dr.values(c, e) for c, e in zip(caches, exps)], 0
    for i, (nq, nk) in enumerate(zip(new, lens.tolist())):
        k, v = (ref.gather_pages(x, table[i].cpu(), nk, page) for x in vals)
        o, lse, mag, e = ref.attend(Q[a:a + nq].double().cpu(), k, v, True, 0, scale)
        ref.check(f"O of request {i}", O[a:a + nq], o, mag, e, dt)
        ref.check_lse(LSE[:, a:a + nq], lse, e)
        a += nq


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 20), (False, 0)])
def test_bytes_that_nobody_has_written(kernel, causal, window):
    """Exponents of 255 and numbers of NaN in every slot that holds no key, those behind a last key among them."""
    dtype, H, H_kv, d, page, new = KERNELS[kernel]
    dt, ctx = DT[dtype], [(13 * i + 5) % 100 for i in range(len(new))]
    Q, caches, exps, table, lens = _setup(9, new, ctx, H, H_kv, d, page, dt)
    held = torch.zeros(exps[0].shape[0], page, dtype=torch.bool)
    for row, n in zip(table.cpu(), lens.tolist()):
        j = torch.arange(n)
        held[row.long()[j // page], j % page] = True
    for e in exps:
        e.masked_fill_(~held[:, None].cuda(), 255)
    O, LSE = fa.fa_paged_fwd(Q, *caches, table, _cu(new), lens, causal=causal, window_size=window, K_exp=exps[0], V_exp=exps[1])
    assert _errors() == ""
    _check(O, LSE, Q, caches, exps, table, new, lens.tolist(), dt, causal, window, p_step=P_STEP.get(kernel, 0.0))


@pytest.mark.parametrize("kernel", ["rows", "tiles", "tiles_256", "copy", "simt"])
@pytest.mark.parametrize("exponent", [97, 142, 157])
def test_zeros_beside_values_of_one_size(kernel, exponent):
    """Cleared pages and pages outside the cache beside values that are all small, or all large: the zeros do not
    cost the others' weights their bits."""
    dtype, H, H_kv, d, page, new = KERNELS[kernel]
    dt, ctx = DT[dtype], [(29 * i) % 70 + 300 for i in range(len(new))]
    Q, caches, exps, table, lens = _setup(9, new, ctx, H, H_kv, d, page, dt)
    exps[1].fill_(exponent)
    asked = table.clone()
    for n in range(len(new)):
        for col in [1, 3, *range(128 // page, 256 // page)]:  # two pages of a tile, and a whole one
            _zero(caches, exps, int(table[n, col]))
        asked[n, 3] = -1
    O, LSE = fa.fa_paged_fwd(Q, *caches, asked, _cu(new), lens, K_exp=exps[0], V_exp=exps[1])
    assert "page" in _errors()
    _check(O, LSE, Q, caches, exps, table, new, lens.tolist(), dt)


def _check_rows(O, LSE, q, k, v, vis, scale, dtype, lift=4):
    """packed_ref's bounds, of each row and head from the keys that it sees alone, and the fixed step of P.

    A score is off by d 2^-23 scale sum |q k|, its P by the factor exp of that, x_j.  P is an fp16 operand P 2^ev,
    ev the exponent of its key's V; the largest of them is 2^8 or more where numbers below 2^-14 are off by up to
    2^-25: O by 2^-33 max_j(P_j 2^ev_j) sum_j |V_jc| 2^-ev_j.  With top_j = max_c |V_jc|, 224 2^ev_j < top_j <=
    448 2^ev_j above the smallest exponent, so by 2^-32 max_j(P_j top_j) sum_j |V_jc| / top_j.  Where one factor
    serves a tile of keys, it is up to 2^lift times theirs."""
    nq, H, d = q.shape
    g = H // k.shape[1]
    for h in range(H):
        kh, vh = k[:, h // g], v[:, h // g]
        s = ((q[:, h] @ kh.T) * scale).masked_fill(~vis, -math.inf)
        lse = torch.logsumexp(s, 1)
        P = torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[:, None])
        x = torch.expm1((d * ref.STEP * scale * (q[:, h].abs() @ kh.abs().T)).clamp(max=80.0))
        e = len(kh) * ref.STEP + 2.0 ** -21
        want, A = P @ vh, P @ vh.abs()
        f32 = (P * x) @ vh.abs() + (P * x).sum(1, keepdim=True) * want.abs() + e * A
        top = vh.abs().amax(1).clamp(min=2.0 ** -40)
        f32 = f32 + 2.0 ** (lift - 32) * (P * top).amax(1, keepdim=True) * (vis.double() @ (vh.abs() / top[:, None]))
        tol = ref.U[dtype] * (want.abs() + A + f32) * 1.001 + f32 + (2.0 ** -24 if dtype == torch.float16 else 1e-30)
        worst = float(((O[:, h].double().cpu() - want).abs() / tol).max())
        assert worst <= 1.0, f"O of head {h}: {worst:.3g} times its bound"  # NaN fails too
        off = (LSE[h].double().cpu() - lse).abs() / ((P * x).sum(1) + e + 2.0 ** -22 * lse.abs())
        assert float(off.max()) <= 1.0, f"LSE of head {h}: {float(off.max()):.3g} times its bound"


def _check_requests(O, LSE, Q, caches, exps, table, lens, new, scale, dtype, sees=None, rows=lambda i: True, lift=4):
    """_check_rows of every request, of its new tokens numbered i with rows(i)."""
    vals, a = [dr.values(c, e) for c, e in zip(caches, exps)], 0
    for n, (nq, nk) in enumerate(zip(new, lens.tolist())):
        k, v = (ref.gather_pages(x, table[n].cpu(), nk, caches[0].shape[1]) for x in vals)
        vis = ref.visible(nq, nk, True, 0)
        if sees is not None:
            vis[:, nk - nq:] = sees[n]
        at = [i for i in range(nq) if rows(i)]
        _check_rows(O[a:a + nq][at], LSE[:, a:a + nq][:, at], Q[a:a + nq][at].double().cpu(), k, v, vis[at], scale, dtype, lift)
        a += nq


@pytest.mark.parametrize("new", [[1, 3], [40, 30], [300, 220]])
@pytest.mark.parametrize("d,page", [(128, 16), (64, 32), (256, 16)])
@pytest.mark.parametrize("which", ["large K", "small K", "large V"])
def test_fp16_queries_over_rows_of_a_wider_type(new, d, page, which):
    """A cache written from bf16 holds values above fp16's largest and below its smallest: fp16 queries see them
    as they are, whichever kernel the number of rows chooses."""
    H, H_kv, ctx = 8, 2, [(29 * i) % 70 + 100 for i in range(len(new))]
    Q, caches, exps, table, lens = _setup(9, new, ctx, H, H_kv, d, page, torch.bfloat16, spread=1)
    scale = d ** -0.5
    if which == "large V":  # on one row of every page, whose scores leave it no weight
        caches[0].view(torch.uint8)[:, 3] = 0x7e  # 448 in every column
        exps[0][:, :, 3] = 127
        exps[1][:, :, 3] = 139
        Q = -Q.abs()
    else:
        up, q_up = (20, -12) if which == "large K" else (-20, 12)
        exps[0].copy_((exps[0].int() + up).clamp(97, 157).to(torch.uint8))
        Q = Q.float() * 2.0 ** q_up
        scale *= 2.0 ** -(up + q_up)
    Q = Q.to(torch.float16)
    O, LSE = fa.fa_paged_fwd(Q, *caches, table, _cu(new), lens, K_exp=exps[0], V_exp=exps[1], scale=scale)
    assert _errors() == ""
    _check_requests(O, LSE, Q, caches, exps, table, lens, new, scale, torch.float16)


FAR = ["rows", "rows_f16", "tiles", "tiles_f16", "tiles_64", "tiles_256", "tiles_f16_256", "copy", "simt"]


@pytest.mark.parametrize("kernel", FAR)
@pytest.mark.parametrize("which", ["K", "V", "KV"])
@pytest.mark.parametrize("gap", [13, 16, 24, 34])
def test_rows_far_larger_than_the_others_that_nobody_sees(kernel, which, gap):
    """Drafted tokens whose K, V or both are 2^gap times everybody's and which none but themselves sees: the others'
    results are as exact as without them."""
    dtype, H, H_kv, d, page, new = KERNELS[kernel]
    dt, ctx = DT[dtype], [(29 * i) % 70 + 120 for i in range(len(new))]
    Q, caches, exps, table, lens = _setup(9, new, ctx, H, H_kv, d, page, dt, spread=1)
    ups, at = [], 0
    for n, m in enumerate(new):
        up, last = [], -1
        for i in range(m):
            up.append(last)
            if i % 7 != 2:
                last = i
                continue
            pg, row = int(table[n, (ctx[n] + i) // page]), (ctx[n] + i) % page
            for name, e in zip("KV", exps):
                if name in which:
                    e[pg, :, row] = (e[pg, :, row].int() + gap).clamp(max=157).to(torch.uint8)
            Q[at + i] = 0  # of what it sees itself every weight is alike
        ups.append(up)
        at += m
    tree, _ = fa.fa_tree_mask(torch.tensor(sum(ups, []), **I32), _cu(new), torch.tensor(ctx, **I32), -(-max(new) // 64))
    O, LSE = fa.fa_paged_fwd(Q, *caches, table, _cu(new), lens, tree=tree, K_exp=exps[0], V_exp=exps[1])
    assert _errors() == ""
    sees = [dr.ancestors(u)[0] for u in ups]
    lift = 14 if gap < 15 else 4
    for rows in (lambda i: i % 7 != 2, lambda i: i % 7 == 2):
        if dtype != "f16" or rows(0):  # fp16 has no room for the large rows' own O
            _check_requests(O, LSE, Q, caches, exps, table, lens, new, d ** -0.5, dt, sees, rows, lift)


@pytest.mark.parametrize("kernel", FAR)
@pytest.mark.parametrize("gap", [16, 30])
def test_rows_far_larger_than_the_others_without_weight(kernel, gap):
    """Cached rows of V 2^gap times the others', whose scores leave them no weight."""
    dtype, H, H_kv, d, page, new = KERNELS[kernel]
    dt, ctx = DT[dtype], [(29 * i) % 70 + 300 for i in range(len(new))]
    Q, caches, exps, table, lens = _setup(9, new, ctx, H, H_kv, d, page, dt, spread=1)
    Q = -Q.abs()
    for pg in table[:, [1, 9]].reshape(-1).tolist():
        caches[0].view(torch.uint8)[pg, 5] = 0x7e  # 448 in every column
        exps[0][pg, :, 5] = 123
        exps[1][pg, :, 5] = (exps[1][pg, :, 5].int() + gap).clamp(max=157).to(torch.uint8)
    O, LSE = fa.fa_paged_fwd(Q, *caches, table, _cu(new), lens, K_exp=exps[0], V_exp=exps[1])
    assert _errors() == ""
    _check_requests(O, LSE, Q, caches, exps, table, lens, new, d ** -0.5, dt)


@pytest.mark.parametrize("kernel", ["tiles", "tiles_64", "tiles_256", "copy", "simt", "rows"])
def test_every_exponent_that_is_written(kernel):
    """Exponents from end to end of what fa_paged_write_q8 writes, rows of zeros among them."""
    dtype, H, H_kv, d, page, new = KERNELS[kernel]
    dt, ctx = DT[dtype], [(29 * i) % 70 + 300 for i in range(len(new))]
    Q, caches, exps, table, lens = _setup(7, new, ctx, H, H_kv, d, page, dt, spread=0)
    g = torch.Generator().manual_seed(1)
    lo, hi = (112, 122) if dt == torch.float16 else (97, 157)
    exps[1].copy_(torch.randint(lo, hi + 1, exps[1].shape, generator=g).to(torch.uint8))
    exps[0].copy_(torch.randint(lo, 121, exps[0].shape, generator=g).to(torch.uint8))  # scores of moderate size
    for c in caches:
        c.view(torch.uint8)[c.view(torch.uint8) & 127 == 127] = 0
    _zero(caches, exps, int(table[0, 2]))
    Q = Q * 0.125
    O, LSE = fa.fa_paged_fwd(Q, *caches, table, _cu(new), lens, K_exp=exps[0], V_exp=exps[1])
    assert _errors() == ""
    _check_requests(O, LSE, Q, caches, exps, table, lens, new, d ** -0.5, dt, lift=14 if dt == torch.float16 else 4)


def test_fp16_queries_in_a_replayed_graph():
    """Each replay looks at the rows that the cache holds then: they fit fp16, do not, and do again."""
    dtype, H, H_kv, d, page, new = KERNELS["copy_f16"]
    Q, caches, exps, table, lens = _setup(9, new, [40, 100], H, H_kv, d, page, torch.bfloat16, spread=1)
    Q, args = Q.half(), (*caches, table, _cu(new), lens)
    fit = [e.clone() for e in exps]
    wide = [(fit[0].int() - 14).clamp(min=97).to(torch.uint8), fit[1]]
    want = []
    for values in (fit, wide):
        for e, x in zip(exps, values):
            e.copy_(x)
        want.append(fa.fa_paged_fwd(Q, *args, K_exp=exps[0], V_exp=exps[1]))
    assert not torch.equal(want[0][0], want[1][0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        O, LSE = fa.fa_paged_fwd(Q, *args, K_exp=exps[0], V_exp=exps[1])
    for i in (0, 1, 1, 0, 1, 0, 0):
        for e, x in zip(exps, (fit, wide)[i]):
            e.copy_(x)
        O.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(O, want[i][0]) and torch.equal(LSE, want[i][1])
    assert _errors() == ""
