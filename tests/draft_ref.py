"""Plain 64-bit forms of the 8-bit cache and of trees of drafted tokens; the bounds are packed_ref's.

Attention over an 8-bit cache is compared with 64-bit attention over the values the cache stands for, which
every kernel reads without rounding, so the bounds of packed_ref hold unchanged: P is rounded to a 16-bit
type whose u is at most that of Q, O once to Q's type, and Q's row is scaled by a power of two.
"""
import math

import torch

from tests import packed_ref as ref

LIMITS = {torch.float32: (-30, 30, 448.0 * 2.0 ** 30), torch.bfloat16: (-30, 30, 448.0 * 2.0 ** 30),
          torch.float16: (-15, 8, 61440.0)}


def grid():
    """The finite e4m3 magnitudes, in the order of their codes 0..126."""
    out = []
    for code in range(127):
        e, m = code >> 3, code & 7
        out.append(math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10))
    return torch.tensor(out, dtype=torch.float64)


def quantise(x):
    """Codes (uint8) and exponent bytes of rows x [..., d], found by looking every element up among the
    e4m3 numbers."""
    lo, hi, most = LIMITS[x.dtype]
    x = x.double().cpu()
    finite = torch.isfinite(x)
    top = torch.where(finite, x.abs(), 0.0).amax(-1)
    e = torch.full(top.shape, hi, dtype=torch.int64)
    for c in range(hi, lo - 1, -1):
        e[top <= 448.0 * 2.0 ** c] = c
    y = torch.where(finite, x.clamp(-most, most), 0.0) * (2.0 ** -e.double())[..., None]
    g = grid()
    a = y.abs()
    up = torch.searchsorted(g, a.contiguous()).clamp(max=126)
    down = (up - 1).clamp(min=0)
    du, dd = g[up] - a, a - g[down]
    code = torch.where((dd < du) | ((dd == du) & (down % 2 == 0)), down, up)
    code = code | torch.where(torch.signbit(x), 128, 0)
    # 127 is NaN, whatever its sign
    return torch.where(finite, code, 127).to(torch.uint8), (e + 127).to(torch.uint8)


def numbers(codes):
    """fp64 numbers of e4m3 codes."""
    c = codes.long().cpu()
    mag = torch.cat([grid(), torch.tensor([math.nan], dtype=torch.float64)])[c & 127]
    return torch.where(c > 127, -mag, mag)


def values(cache, exp):
    """fp64 values [pages, page_size, H_kv, d] of an 8-bit cache."""
    return numbers(cache.view(torch.uint8)) * (2.0 ** (exp.double().cpu() - 127)).transpose(1, 2)[..., None]


def ancestors(parents):
    """[n, n] whether token i sees token k, and the number of ancestors of each, of one request."""
    n = len(parents)
    see = torch.eye(n, dtype=torch.bool)
    depth = [0] * n
    for i, p in enumerate(parents):
        if 0 <= p < i:
            see[i] |= see[p]
            depth[i] = depth[p] + 1
    return see, depth


def pack(see, words):
    """int64 masks [n, words] of see [n, n]."""
    out = torch.zeros(see.shape[0], words, dtype=torch.int64)
    for i, row in enumerate(see.tolist()):
        for k, s in enumerate(row):
            if s and k < 64 * words:
                out[i, k // 64] |= (1 << (k % 64)) - (1 << 64 if k % 64 == 63 else 0)
    return out


def attend(q, k, v, vis, scale):
    """q [S_q, H, d], k, v [S_k, H_kv, d] in fp64, vis [S_q, S_k] -> O, LSE, bound factors (packed_ref.attend)."""
    nq, H, d = q.shape
    nk, H_kv, _ = k.shape
    g = H // H_kv
    O, A = torch.zeros_like(q), torch.zeros_like(q)
    LSE = torch.full((H, nq), -math.inf, dtype=torch.float64)
    e = 0.0
    for h in range(H):
        kh, vh = k[:, h // g], v[:, h // g].masked_fill(~vis.any(0)[:, None], 0.0)
        s_err = d * ref.STEP * scale * float((q[:, h].abs() @ kh.abs().T).max()) if nk and nq else 0.0
        s = ((q[:, h] @ kh.T) * scale).masked_fill(~vis, -math.inf)
        lse = torch.logsumexp(s, 1) if nk else LSE[h]
        P = torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[:, None])
        O[:, h], A[:, h], LSE[h] = P @ vh, P @ vh.abs(), lse
        e = max(e, 2 * math.expm1(s_err) + nk * ref.STEP + 2.0 ** -21)
    return O, LSE, A, e
