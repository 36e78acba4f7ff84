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
