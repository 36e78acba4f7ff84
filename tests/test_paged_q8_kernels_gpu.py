"""The kernels that attention over an 8-bit cache chooses between, each at the sizes where it is taken: few
rows per request (one CTA per SM or several), 128-row tiles, a copy of the rows in the queries' type."""
import math

import pytest
import torch

import flashattention_backward_preprocess_gb300 as fa
from tests import draft_ref as dr
from tests.test_draft_tree_gpu import I32, _check_tree, _parents
from tests.test_packed_gpu import DT, _cu
from tests.test_paged_q8_gpu import _check, _errors, _setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,H,H_kv,d,page", [
    ("bf16", 8, 2, 128, 16), ("f16", 4, 1, 64, 32), ("bf16", 16, 1, 96, 48), ("f16", 3, 1, 32, 16), ("bf16", 4, 4, 128, 128),
    ("f16", 6, 2, 128, 80),
])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 30), (False, 0), (False, 25)])
def test_many_requests_of_few_rows(dtype, H, H_kv, d, page, causal, window):
    """More (request, head) pairs than half the SMs; several tokens, no tokens, no cached tokens among them."""
    dt, N = DT[dtype], 90
    new = [(1, 1, 2, 0, 1, 3)[i % 6] for i in range(N)]
    ctx = [(37 * i * i) % 400 if i % 7 else 0 for i in range(N)]
    Q, caches, exps, table, lens = _setup(1, new, ctx, H, H_kv, d, page, dt)
    args = (Q, *caches, table, _cu(new), lens)
    O, LSE = fa.fa_paged_fwd(*args, causal=causal, window_size=window, K_exp=exps[0], V_exp=exps[1])
    O2, LSE2 = fa.fa_paged_fwd(*args, causal=causal, window_size=window, K_exp=exps[0], V_exp=exps[1])
    assert _errors() == ""
    assert torch.equal(O, O2) and torch.equal(LSE, LSE2)
    _check(O, LSE, Q, caches, exps, table, new, lens.tolist(), dt, causal, window)


@pytest.mark.parametrize("dtype,H,H_kv,d,page,N,n", [
    ("bf16", 8, 2, 128, 16, 80, 6), ("f16", 4, 4, 64, 16, 3, 30), ("bf16", 2, 1, 128, 48, 2, 16), ("f16", 16, 1, 32, 32, 100, 2),
])
def test_trees_of_few_rows(dtype, H, H_kv, d, page, N, n):
    dt = DT[dtype]
    new = [n if i % 5 else n - 1 for i in range(N)]
    ctx = [(61 * i) % 300 if i % 4 else 0 for i in range(N)]
    Q, caches, exps, table, lens = _setup(5, new, ctx, H, H_kv, d, page, dt)
    ups = [_parents(i, m, "any") for i, m in enumerate(new)]
    tree, _ = fa.fa_tree_mask(torch.tensor(sum(ups, []), **I32), _cu(new), torch.tensor(ctx, **I32))
    O, LSE = fa.fa_paged_fwd(Q, *caches, table, _cu(new), lens, tree=tree, K_exp=exps[0], V_exp=exps[1])
    assert _errors() == ""
    _check_tree(O, LSE, Q, [dr.values(c, e) for c, e in zip(caches, exps)], table, new, lens.tolist(),
                [dr.ancestors(u)[0] for u in ups], dt)


SPREAD = [("bf16", 8, 2, 128, 16, [200, 140, 0, 150]), ("f16", 4, 1, 64, 8, [130, 400]), ("bf16", 8, 1, 256, 64, [90, 70]),
          ("f16", 16, 2, 96, 256, [64, 100]), ("bf16", 4, 1, 128, 128, [513, 1])]


@pytest.mark.parametrize("dtype,H,H_kv,d,page,new", SPREAD)
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 70), (False, 0), (False, 50)])
def test_many_rows(dtype, H, H_kv, d, page, new, causal, window):
    dt = DT[dtype]
    ctx = [77, 0, 9, 300][:len(new)]
    Q, caches, exps, table, lens = _setup(3, new, ctx, H, H_kv, d, page, dt)
    args = (Q, *caches, table, _cu(new), lens)
    O, LSE = fa.fa_paged_fwd(*args, causal=causal, window_size=window, K_exp=exps[0], V_exp=exps[1])
    assert _errors() == ""
    # These rows go through the kernel for caches of Q's type.  Its fp16 P is relative to the largest score of
    # the first tile in which the row sees a key, so that key's P is 1 and the row sum at least 1 (a higher
    # reference later on scales both alike); below 2^-14 fp16 has steps of 2^-24, half of which is 2^-25.
    # bf16 has P's relative precision down to 2^-126.
    _check(O, LSE, Q, caches, exps, table, new, lens.tolist(), dt, causal, window, p_step=2.0 ** -25 if dt == torch.float16 else 0.0)


def test_many_rows_tree_and_unset_workspace():
    """A tree of many rows; the copy's workspace holds NaN, of which nothing reaches the result."""
    dt, H, H_kv, d, page, new, ctx = torch.bfloat16, 8, 1, 128, 16, [100, 70], [33, 500]
    Q, caches, exps, table, lens = _setup(3, new, ctx, H, H_kv, d, page, dt)
    ups = [_parents(i, m, "any") for i, m in enumerate(new)]
    tree, _ = fa.fa_tree_mask(torch.tensor(sum(ups, []), **I32), _cu(new), torch.tensor(ctx, **I32), 2)
    junk = [torch.full((1 << 26,), math.nan, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    del junk
    O, LSE = fa.fa_paged_fwd(Q, *caches, table, _cu(new), lens, tree=tree, K_exp=exps[0], V_exp=exps[1])
    assert _errors() == ""
    _check_tree(O, LSE, Q, [dr.values(c, e) for c, e in zip(caches, exps)], table, new, lens.tolist(),
                [dr.ancestors(u)[0] for u in ups], dt)
    # with a window, rows before it are never looked at: their table entries may be anything
    table2 = table.clone()
    table2[1, :20] = -5
    O, LSE = fa.fa_paged_fwd(Q, *caches, table2, _cu(new), lens, window_size=100, K_exp=exps[0], V_exp=exps[1])
    assert _errors() == ""
    _check(O, LSE, Q, caches, exps, table, new, lens.tolist(), dt, True, 100)
    table2[0, 0] = 10 ** 6
    O, LSE = fa.fa_paged_fwd(Q, *caches, table2, _cu(new), lens, window_size=1000, K_exp=exps[0], V_exp=exps[1])
    assert "page" in _errors()


@pytest.mark.parametrize("new,window", [([1] * 90, 0), ([1, 2], 0), ([40, 40], 0), ([300, 300], 0), ([300, 300], 64)])
def test_a_cache_in_use_is_read_where_it_ends(new, window):
    """NaN numbers behind each request's last key, on its own last page, reach nobody."""
    dt, H, H_kv, d, page = torch.float16, 8, 2, 128, 16
    ctx = [(13 * i + 5) % 100 for i in range(len(new))]
    Q, caches, exps, table, lens = _setup(9, new, ctx, H, H_kv, d, page, dt)
    O, LSE = fa.fa_paged_fwd(Q, *caches, table, _cu(new), lens, window_size=window, K_exp=exps[0], V_exp=exps[1])
    assert _errors() == ""
    assert torch.isfinite(O).all() and torch.isfinite(LSE).all()
    # 2^-25: fp16's P in the kernel for caches of Q's type, as above
    _check(O, LSE, Q, caches, exps, table, new, lens.tolist(), dt, True, window, p_step=2.0 ** -25 if sum(new) >= 256 else 0.0)


def test_padded_batch_of_few_rows():
    """Rows of no request: set in new outputs, left as they were in given ones."""
    dt, H, H_kv, d, page, new = torch.bfloat16, 8, 2, 128, 16, [1] * 5
    Q, caches, exps, table, lens = _setup(9, new, [30, 0, 7, 100, 64], H, H_kv, d, page, dt)
    Q = torch.cat([Q[:1], Q, Q[:3]])
    cu = _cu([1] + new)[1:].contiguous()
    O, LSE = fa.fa_paged_fwd(Q, *caches, table, cu, lens, K_exp=exps[0], V_exp=exps[1])
    assert _errors() == ""
    for at in (slice(0, 1), slice(6, 9)):
        assert (O[at] == 0).all() and (LSE[:, at] == -math.inf).all()
    _check(O[1:6], LSE[:, 1:6], Q[1:6], caches, exps, table, new, lens.tolist(), dt)
    O2, LSE2 = torch.full_like(O, 3.0), torch.full_like(LSE, 4.0)
    fa.fa_paged_fwd(Q, *caches, table, cu, lens, O=O2, LSE=LSE2, K_exp=exps[0], V_exp=exps[1])
    assert (O2[[0, 6, 7, 8]] == 3).all() and (LSE2[:, [0, 6, 7, 8]] == 4).all() and torch.equal(O2[1:6], O[1:6])


def test_two_streams_at_once():
    """Two calls in flight on two streams do not share scratch."""
    dt, H, H_kv, d, page = torch.bfloat16, 8, 2, 128, 16
    jobs = []
    for seed, new, ctx in ((1, [1] * 60, [200] * 60), (2, [300, 200], [50, 900])):
        Q, caches, exps, table, lens = _setup(seed, new, ctx, H, H_kv, d, page, dt)
        jobs.append(((Q, *caches, table, _cu(new), lens), dict(K_exp=exps[0], V_exp=exps[1])))
    want = [fa.fa_paged_fwd(*a, **k) for a, k in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [[fa.fa_paged_fwd(*a, **k, stream=s) for _ in range(5)] for (a, k), s in zip(jobs, streams)]
    torch.cuda.synchronize()
    assert _errors() == ""
    for w, g in zip(want, got):
        for o, lse in g:
            assert torch.equal(o, w[0]) and torch.equal(lse, w[1])


@pytest.mark.parametrize("dtype,H,H_kv,d,page,new", [
    ("bf16", 8, 2, 128, 16, [1] * 60), ("f16", 4, 2, 64, 16, [1, 2]), ("bf16", 8, 2, 128, 16, [30, 20]), ("f16", 4, 1, 128, 24, [1, 1]),
    ("bf16", 8, 1, 128, 16, [100, 80]), ("f32", 4, 2, 64, 16, [1, 3]), ("bf16", 4, 2, 256, 64, [1, 2]),
])
def test_pages_outside_the_cache_read_as_zeros(dtype, H, H_kv, d, page, new):
    """Keys without a page keep their place in the softmax, as keys of 0 with values of 0; so do the rows of a
    cleared cache, whose exponents are 0."""
    dt, ctx = DT[dtype], [(29 * i) % 70 + 300 for i in range(len(new))]
    Q, caches, exps, table, lens = _setup(9, new, ctx, H, H_kv, d, page, dt)
    # request 0: a cleared page; request 1: pages outside the cache, one of them a whole tile of 128 keys long
    cleared = int(table[0, 1])
    for c, e in zip(caches, exps):
        c.view(torch.uint8)[cleared] = 0
        e[cleared] = 0
    gone = list(range(128 // page, 256 // page + 1))
    bad = table.clone()
    bad[1, gone] = torch.tensor([-1 if i % 2 else caches[0].shape[0] + i for i in gone], dtype=torch.int32).cuda()
    O, LSE = fa.fa_paged_fwd(Q, *caches, bad, _cu(new), lens, K_exp=exps[0], V_exp=exps[1])
    assert "page" in _errors()
    want = [c.clone() for c in caches]
    for c, e in zip(want, exps):
        c.view(torch.uint8)[table[1, gone].long()] = 0
    _check(O, LSE, Q, want, exps, table, new, lens.tolist(), dt)


@pytest.mark.parametrize("dtype,H,H_kv,d,page,N,n", [("bf16", 4, 1, 64, 16, 1000, 1), ("f16", 4, 2, 128, 32, 950, 2), ("bf16", 4, 1, 64, 16, 900, 9)])
def test_more_requests_than_a_cta_plans_for(dtype, H, H_kv, d, page, N, n):
    """Hundreds of requests: the plan is a kernel of its own."""
    dt = DT[dtype]
    new, ctx = [n if i % 9 else 0 for i in range(N)], [(7 * i) % 90 for i in range(N)]
    Q, caches, exps, table, lens = _setup(4, new, ctx, H, H_kv, d, page, dt)
    O, LSE = fa.fa_paged_fwd(Q, *caches, table, _cu(new), lens, K_exp=exps[0], V_exp=exps[1])
    assert _errors() == ""
    _check(O, LSE, Q, caches, exps, table, new, lens.tolist(), dt)
