"""NaN inside a sequence: rows that see one are NaN in O, LSE and the gradients, whether their item is
whole or cut into parts, and no other row is touched; a row without keys stays 0 and -inf whatever V
holds.  Rows that see no NaN are held to the bounds of tests/packed_ref.py on the clean data."""
import math

import pytest
import torch

import flashattention_backward_preprocess_gb300 as fa
from tests import packed_ref as ref
from tests.test_packed_gpu import DT, _cu, _packed, _paged, _rand

pytestmark = pytest.mark.gpu
PATHS = [("bf16", 4, 2, 64), ("bf16", 8, 2, 128), ("f16", 4, 2, 128), ("bf16", 4, 2, 256), ("f32", 4, 2, 64),
         ("bf16", 130, 1, 64)]
# (lengths, the sequence that holds the NaN): whole items; one row of keys long enough to be cut
WHOLE, CUT = ([70, 33, 150], [70, 33, 150], 2), ([2, 3, 1], [5, 4000, 1], 1)


def _check_rows(O, LSE, hit, clean, lq, lk, causal, dt):
    """`hit` [T_q, H]: the rows (per head) that must be NaN; the others against 64 bits of the clean data."""
    torch.cuda.synchronize()
    fa.fa_check_device()
    hit = hit.cpu()
    assert torch.isnan(O).all(2).cpu().equal(hit) and torch.isnan(O).any(2).cpu().equal(hit)
    assert torch.isnan(LSE).t().cpu().equal(hit)
    a = b = 0
    for nq, nk in zip(lq, lk):
        q, k, v = (x.double().cpu() for x in (clean[0][a:a + nq], clean[1][b:b + nk], clean[2][b:b + nk]))
        o, lse, mag, e = ref.attend(q, k, v, causal, 0, q.shape[2] ** -0.5)
        ok = ~hit[a:a + nq]
        ref.check(f"O of a sequence {nq}x{nk}", O[a:a + nq][ok.cuda()], o[ok], mag[ok], e, dt)
        ref.check_lse(LSE[:, a:a + nq].t()[ok.cuda()], lse.t()[ok], e)
        a, b = a + nq, b + nk


@pytest.mark.parametrize("dtype,H,H_kv,d", PATHS)
@pytest.mark.parametrize("lq,lk,n", [WHOLE, CUT], ids=["whole", "cut"])
@pytest.mark.parametrize("where", ["query", "key", "keys of a tile", "last key"])
@pytest.mark.parametrize("causal", [False, True])
def test_varlen_fwd_keeps_nan(dtype, H, H_kv, d, lq, lk, n, where, causal):
    dt, g = DT[dtype], H // H_kv
    clean = _packed(5, lq, lk, H, H_kv, d, dt)
    Q, K, V = (x.clone() for x in clean)
    q0, k0, nq, nk = sum(lq[:n]), sum(lk[:n]), lq[n], lk[n]
    hit = torch.zeros(sum(lq), H, dtype=torch.bool)
    if where == "query":
        Q[q0 + 1, H - 1, d // 2] = math.nan
        hit[q0 + 1, H - 1] = True
    else:
        keys = {"key": [nk // 2], "keys of a tile": list(range(min(128, nk))), "last key": [nk - 1]}[where]
        K[k0 + torch.tensor(keys), H_kv - 1, 0] = math.nan
        sees = ref.visible(nq, nk, causal, 0)[:, keys].any(1)
        hit[q0:q0 + nq, (H_kv - 1) * g:] = sees[:, None]
    O, LSE = fa.fa_varlen_fwd(Q, K, V, _cu(lq), _cu(lk), causal=causal)
    _check_rows(O, LSE, hit, clean, lq, lk, causal, dt)


@pytest.mark.parametrize("dtype,page", [("bf16", 16), ("bf16", 5), ("f32", 16)])
@pytest.mark.parametrize("where", ["query", "key"])
def test_paged_fwd_keeps_nan(dtype, page, where):
    """Single tokens: the request with the NaN is cut over the grid, the one beside it is not touched."""
    dt, new, total = DT[dtype], [1, 1], [3000, 40]
    H, H_kv, d = 8, 2, 64
    Q, K, V, table, lens = _paged(7, new, total, H, H_kv, d, page, dt)
    clean = Q.clone(), [(ref.gather_pages(x, table[n], total[n], page)) for n in range(2) for x in (K, V)]
    hit = torch.zeros(2, H, dtype=torch.bool)
    if where == "query":
        Q[0, 3, 1] = math.nan
        hit[0, 3] = True
    else:
        K[int(table[0, 1000 // page]), 1000 % page, 0, 5] = math.nan
        hit[0, :H // H_kv] = True
    O, LSE = fa.fa_paged_fwd(Q, K, V, table, _cu(new), lens)
    k, v = torch.cat([clean[1][0], clean[1][2]]), torch.cat([clean[1][1], clean[1][3]])
    _check_rows(O, LSE, hit, (clean[0], k, v), new, total, True, dt)


@pytest.mark.parametrize("dtype,H,H_kv,d", PATHS[:5])
@pytest.mark.parametrize("lq,lk", [([4, 9], [2, 9]), ([300], [200]), ([3], [1])])
def test_rows_without_keys_stay_zero(dtype, H, H_kv, d, lq, lk):
    """Causal, more queries than keys: the first rows see nothing, so no infinity of V reaches them."""
    dt = DT[dtype]
    Q, K, V = _packed(9, lq, lk, H, H_kv, d, dt)
    V[0] = math.inf
    O, LSE = fa.fa_varlen_fwd(Q, K, V, _cu(lq), _cu(lk), causal=True)
    torch.cuda.synchronize()
    fa.fa_check_device()
    none = lq[0] - lk[0]
    assert (O[:none] == 0).all() and (LSE[:, :none] == -math.inf).all()
    assert torch.isfinite(LSE[:, none:]).all()
    assert not torch.isfinite(O[none:lq[0]]).any()  # key 0 is seen by every row that sees one


@pytest.mark.parametrize("dtype,H,H_kv,d", PATHS[:5])
@pytest.mark.parametrize("deterministic", [False, True])
@pytest.mark.parametrize("where", ["query", "key"])
def test_varlen_bwd_keeps_nan(dtype, H, H_kv, d, deterministic, where):
    """Without a mask every pair of the sequence and head is seen: its gradients are NaN, others finite."""
    dt, lens, g = DT[dtype], [70, 33, 150], H // H_kv
    Q, K, V = _packed(5, lens, lens, H, H_kv, d, dt)
    dO = _rand(8, Q.shape, dt)
    rows, heads = slice(70, 103), slice((H_kv - 1) * g, H)
    want = [torch.zeros(x.shape[:2], dtype=torch.bool, device="cuda") for x in (Q, K, V)]
    want[1][rows, H_kv - 1] = want[2][rows, H_kv - 1] = True
    if where == "query":
        Q[75, H - 1, 3] = math.nan
        want[0][75, H - 1] = True
    else:
        K[80, H_kv - 1, 3] = math.nan
        want[0][rows, heads] = True
    O, LSE = fa.fa_varlen_fwd(Q, K, V, _cu(lens), _cu(lens))
    grads = fa.fa_varlen_bwd(dO, Q, K, V, O, LSE, _cu(lens), _cu(lens), deterministic=deterministic)
    torch.cuda.synchronize()
    fa.fa_check_device()
    for name, got, w in zip(("dQ", "dK", "dV"), grads, want):
        assert torch.isnan(got).any(2).equal(w) and torch.isnan(got).all(2).equal(w), name
