"""Plain 64-bit attention over packed sequences and paged caches, one sequence and head at a
time, with the elementwise error bounds its kernels are held to.

Bounds (u = eps / 2 of the tensors' type, the largest relative error of one rounding):
  * the kernels round P (and dS) to the tensors' type once before a product and the result
    once at the end, so with A_ic = sum_j P_ij |V_jc|
      |O - O64|   <= u (|O64| + A) + e A,
      |dV - dV64| <= u (|dV64| + sum_i P_ij |dO_ic|) + e (...)
      |dQ - dQ64| <= u (|dQ64| + scale sum_j |dS_ij| |K_jc|) + e (...), dK alike;
    fp32 tensors are not rounded in between: u = 2^-24;
  * e covers fp32 arithmetic: a product of n terms summed in fp32 is off by at most
    n 2^-23 sum |terms| (2^-23 per step: tensor cores may truncate), so a score is off by
    s_err = d 2^-23 scale sum |q k|, P by the factor exp(s_err) - 1, and a sum over the keys
    or rows of one tile list by n 2^-23; 2^-21 stands for exp2 and the division.
"""
import math

import torch

U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
STEP = 2.0 ** -23


def visible(nq, nk, causal, window):
    p = torch.arange(nq)[:, None] + (nk - nq)
    j = torch.arange(nk)[None, :]
    m = torch.ones(nq, nk, dtype=torch.bool)
    if causal:
        m &= j <= p
    if window > 0:
        m &= p - j < window
        if not causal:
            m &= j - p < window
    return m


def attend(q, k, v, causal, window, scale):
    """q [S_q, H, d], k, v [S_k, H_kv, d] in fp64 -> O, LSE [H, S_q], bound factors."""
    nq, H, d = q.shape
    nk, H_kv, _ = k.shape
    g = H // H_kv
    O = torch.zeros_like(q)
    LSE = torch.full((H, nq), -math.inf, dtype=torch.float64)
    A = torch.zeros_like(q)
    e = 0.0
    vis = visible(nq, nk, causal, window)
    for h in range(H):
        kh, vh = k[:, h // g], v[:, h // g]
        s = (q[:, h] @ kh.T) * scale
        s_err = d * STEP * scale * float((q[:, h].abs() @ kh.abs().T).max()) if nk and nq else 0.0
        s = s.masked_fill(~vis, -math.inf)
        lse = torch.logsumexp(s, 1) if nk else LSE[h]
        P = torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[:, None])
        O[:, h] = P @ vh.masked_fill(~vis.any(0)[:, None], 0.0)
        A[:, h] = P @ vh.abs().masked_fill(~vis.any(0)[:, None], 0.0)
        LSE[h] = lse
        e = max(e, 2 * math.expm1(s_err) + nk * STEP + 2.0 ** -21)
    return O, LSE, A, e


def grads(do, q, k, v, o, lse, causal, window, scale):
    """fp64 dQ, dK, dV of one sequence, the sums of absolute values, and e."""
    nq, H, d = q.shape
    nk, H_kv, _ = k.shape
    g = H // H_kv
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    aq, ak, av = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    vis = visible(nq, nk, causal, window)
    e = 0.0
    if nk and nq:
        for h in range(H):
            kh, vh = k[:, h // g], v[:, h // g]
            s = (q[:, h] @ kh.T) * scale
            s_err = d * STEP * scale * float((q[:, h].abs() @ kh.abs().T).max())
            L = torch.where(lse[h] == -math.inf, 0.0, lse[h])
            P = torch.exp((s - L[:, None]).masked_fill(~vis, -math.inf))
            D = (do[:, h] * o[:, h]).sum(1)
            dp = do[:, h] @ vh.T
            mag = do[:, h].abs() @ vh.abs().T + (do[:, h] * o[:, h]).abs().sum(1)[:, None]
            dS = P * (dp - D[:, None])
            dq[:, h] = scale * (dS @ kh)
            dk[:, h // g] += scale * (dS.T @ q[:, h])
            dv[:, h // g] += P.T @ do[:, h]
            # |dS| plus what fp32 may add to it, as sums of absolute terms
            rel = 2 * math.expm1(s_err) + (nq * g + nk) * STEP + 2.0 ** -21
            big = dS.abs() + P * mag  # one scale for the rounding of dS and for e
            aq[:, h] = scale * (dS.abs() @ kh.abs())
            ak[:, h // g] += scale * (dS.abs().T @ q[:, h].abs())
            av[:, h // g] += P.T @ do[:, h].abs()
            # fp32 part: kept apart in e through the ratio of the two sums
            r = float((big.sum() / dS.abs().sum().clamp(min=1e-30)))
            e = max(e, (rel + d * STEP) * max(1.0, min(r, 1e4)))
    return dq, dk, dv, aq, ak, av, e


def check(name, got, want, mag, e, dtype):
    """got within u (|want| + mag) + e mag of want, elementwise; infinities equal."""
    got, want, mag = got.double().cpu(), want.cpu(), mag.cpu()
    assert torch.isfinite(got).all(), f"{name}: not finite"
    tol = U[dtype] * (want.abs() + mag) * 1.001 + e * mag + 1e-30
    if dtype == torch.float16:
        tol = tol + 2.0 ** -24  # subnormal step
    worst = ((got - want).abs() / tol).max() if want.numel() else 0.0
    assert worst <= 1.0, f"{name}: {float(worst):.3g} times its bound"


def check_lse(got, want, e):
    got, want = got.double().cpu(), want.cpu()
    assert torch.equal(torch.isinf(got), torch.isinf(want)), "LSE: rows without keys differ"
    f = torch.isfinite(want)
    assert ((got - want)[f].abs() <= e + 2.0 ** -22 * want[f].abs()).all(), float((got - want)[f].abs().max())


def gather_pages(cache, table_row, n, page):
    """Rows of the first n keys of one request, [n, H_kv, d]."""
    held = table_row[: -(-n // page)].long()
    return cache[held].reshape(-1, *cache.shape[2:])[:n]
