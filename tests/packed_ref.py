"""Plain 64-bit attention over packed sequences and paged caches, one sequence and head at a
time, with the elementwise error bounds its kernels are held to.

Bounds (u = eps / 2 of the tensors' type, the largest relative error of one rounding):
  * the kernels round P (and dS) to the tensors' type once before a product and the result
    once at the end, so with A_ic = sum_j P_ij |V_jc|
      |O - O64|   <= u (|O64| + A) + e A,
      |dV - dV64| <= u (|dV64| + sum_i P_ij |dO_ic|) + e (...)
      |dQ - dQ64| <= u (|dQ64| + scale sum_j |dS_ij| |K_jc|) + e (...), dK alike (grads());
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
    """fp64 dQ, dK, dV of one sequence; for each the sum of magnitudes that a rounding of dS (P)
    scales with, and the one that fp32 arithmetic scales with; and e.

    dP and D are d-term fp32 sums and P carries the factor of its score's error, so
      |error of dS_ij| <= e P_ij (sum_c |dO_ic V_jc| + sum_c |dO_ic O_ic|) = e P_ij M_ij,
    which does not shrink with dS itself: where dP = D (a query with one key, for which O = V)
    dS is 0 and only that remains.  It reaches dQ as e scale sum_j P_ij M_ij |K_j|, dK alike.
    """
    nq, H, d = q.shape
    nk, H_kv, _ = k.shape
    g = H // H_kv
    out = [torch.zeros_like(x) for x in (q, k, v)]
    mag = [torch.zeros_like(x) for x in (q, k, v)]
    f32 = [torch.zeros_like(x) for x in (q, k, v)]
    vis = visible(nq, nk, causal, window)
    e = 0.0
    if nk and nq:
        for h in range(H):
            c = h // g
            kh, vh = k[:, c], v[:, c]
            s = (q[:, h] @ kh.T) * scale
            s_err = d * STEP * scale * float((q[:, h].abs() @ kh.abs().T).max())
            L = torch.where(lse[h] == -math.inf, 0.0, lse[h])
            P = torch.exp((s - L[:, None]).masked_fill(~vis, -math.inf))
            D = (do[:, h] * o[:, h]).sum(1)
            dS = P * (do[:, h] @ vh.T - D[:, None])
            M = P * (do[:, h].abs() @ vh.abs().T + (do[:, h] * o[:, h]).abs().sum(1)[:, None])
            out[0][:, h] = scale * (dS @ kh)
            out[1][:, c] += scale * (dS.T @ q[:, h])
            out[2][:, c] += P.T @ do[:, h]
            mag[0][:, h] = scale * (dS.abs() @ kh.abs())
            mag[1][:, c] += scale * (dS.abs().T @ q[:, h].abs())
            mag[2][:, c] += P.T @ do[:, h].abs()
            f32[0][:, h] = scale * (M @ kh.abs())
            f32[1][:, c] += scale * (M.T @ q[:, h].abs())
            f32[2][:, c] += P.T @ do[:, h].abs()
            # LSE is given in fp32 and scaled once more in fp32: 2^-22 |LSE| in the exponent
            l_err = 2.0 ** -22 * float(L.abs().max())
            e = max(e, 2 * math.expm1(s_err + l_err) + (d + nq * g + nk) * STEP + 2.0 ** -21)
    return out, mag, f32, e


def check(name, got, want, mag, e, dtype, f32=None):
    """got within u (|want| + mag + e f32) + e f32 of want, elementwise (f32: mag unless given)."""
    got, want, mag = got.double().cpu(), want.cpu(), mag.cpu()
    f32 = mag if f32 is None else f32.cpu()
    assert torch.isfinite(got).all(), f"{name}: not finite"
    tol = U[dtype] * (want.abs() + mag + e * f32) * 1.001 + e * f32 + 1e-30
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
