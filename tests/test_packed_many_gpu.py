"""Packed calls over many sequences, at the plan's branches: more than 256 sequences or tiles (plan block
of 1024 threads), more than 1024 key tiles (bucket sort over several rounds), more than 2047 sequences in
a backward and 4096 in a forward (offsets in global memory), a long sequence among them whose tiles are
cut.  And the fp32 kernels at head dims 96 and 256.  Against 64 bits, bounds as in tests/packed_ref.py."""
import math

import pytest
import torch

import flashattention_backward_preprocess_gb300 as fa
from tests import packed_ref as ref
from tests.test_packed_bwd_gpu import _case, _check
from tests.test_packed_gpu import DT, SETS, _check_fwd, _cu, _packed

pytestmark = pytest.mark.gpu


def _short(N, seed=0):
    return [1 + (i * 31 + seed) % 20 for i in range(N)]


class _Padded:
    """The sequences of `lens` (starting at row `first`) as one padded batch in 64 bits, causal."""

    def __init__(self, lens, first, d):
        self.n, self.d = torch.tensor(lens), d
        m = max(lens)
        off = first + torch.tensor([0] + lens).cumsum(0)[:-1]
        self.at = off[:, None] + torch.arange(m)
        self.inside = torch.arange(m) < self.n[:, None]
        self.see = torch.ones(m, m).tril().bool() & self.inside[:, None, :, None] & self.inside[:, None, None, :]

    def take(self, x):  # [N, heads, m, d], zeros behind each sequence
        y = x.double().cpu()[self.at.clamp(max=x.shape[0] - 1)]
        return torch.where(self.inside[:, :, None, None], y, 0.0).transpose(1, 2)

    def rows(self, x):  # back to packed rows
        return x.transpose(1, 2)[self.inside]

    def forward(self, Q, K, V):
        q, k, v = (self.take(x) for x in (Q, K, V))
        g = q.shape[1] // k.shape[1]
        k, v = (x.repeat_interleave(g, 1) for x in (k, v))
        scale = self.d ** -0.5
        s = (q @ k.transpose(-1, -2)) * scale
        s_err = self.d * ref.STEP * scale * float((q.abs() @ k.abs().transpose(-1, -2)).max())
        s = s.masked_fill(~self.see, -math.inf)
        lse = torch.logsumexp(s, -1)
        P = torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[..., None])
        e = 2 * math.expm1(s_err) + q.shape[2] * ref.STEP + 2.0 ** -21
        return self.rows(P @ v), self.rows(P @ v.abs()), self.rows(lse[..., None])[..., 0].t(), e

    def check_grads(self, grads, dO, Q, K, V, O, LSE, dt):
        do, q, o = (self.take(x) for x in (dO, Q, O))
        k, v = (self.take(x) for x in (K, V))
        N, H, m, d = q.shape
        g, scale = H // k.shape[1], d ** -0.5
        kk, vv = (x.repeat_interleave(g, 1) for x in (k, v))
        t = lambda x: x.transpose(-1, -2)
        per_kv = lambda x: x.view(N, H // g, g, m, d).sum(2)
        L = torch.where(self.inside[:, None], LSE.double().cpu().t()[self.at.clamp(max=Q.shape[0] - 1)].transpose(1, 2), 0.0)
        s = (q @ t(kk)) * scale
        s_err = d * ref.STEP * scale * float((q.abs() @ t(kk).abs()).max())
        P = torch.exp((s - L[..., None]).masked_fill(~self.see, -math.inf))
        D = (do * o).sum(-1)[..., None]
        dS = P * (do @ t(vv) - D)
        M = P * (do.abs() @ t(vv).abs() + (do * o).abs().sum(-1)[..., None])
        e = 2 * math.expm1(s_err + 2.0 ** -22 * float(L.abs().max())) + (d + m * g + m) * ref.STEP + 2.0 ** -21
        first, last = int(self.at[0, 0]), int(self.at[0, 0] + self.n.sum())
        for name, got, want, mag, f32 in (
                ("dQ", grads[0], scale * dS @ kk, scale * dS.abs() @ kk.abs(), scale * M @ kk.abs()),
                ("dK", grads[1], per_kv(scale * t(dS) @ q), per_kv(scale * t(dS).abs() @ q.abs()), per_kv(scale * t(M) @ q.abs())),
                ("dV", grads[2], per_kv(t(P) @ do), per_kv(t(P) @ do.abs()), per_kv(t(P) @ do.abs()))):
            ref.check(f"{name} of {N} short sequences", got[first:last], *(self.rows(x) for x in (want, mag)), e, dt, self.rows(f32))


@pytest.mark.parametrize("dtype,H,H_kv,d", [("bf16", 2, 1, 64), ("f16", 2, 2, 128), ("bf16", 2, 1, 256), ("f32", 2, 1, 64)])
@pytest.mark.parametrize("N,long", [(300, 200), (900, 3500), (2500, 3500)])
@pytest.mark.parametrize("deterministic", [False, True])
def test_varlen_bwd_many_sequences(dtype, H, H_kv, d, N, long, deterministic):
    dt = DT[dtype]
    a, b = _short(N // 3), _short(N - N // 3, 7)
    lens = a + [long] + b
    args = _case(17, lens, lens, H, H_kv, d, dt, True, 0)
    cu = _cu(lens)
    torch.cuda.synchronize()
    grads = fa.fa_varlen_bwd(*args, cu, cu, causal=True, deterministic=deterministic)
    again = fa.fa_varlen_bwd(*args, cu, cu, causal=True, deterministic=deterministic)
    torch.cuda.synchronize()
    fa.fa_check_device()
    assert torch.equal(grads[1], again[1]) and torch.equal(grads[2], again[2])
    assert not deterministic or torch.equal(grads[0], again[0])
    _Padded(a, 0, d).check_grads(grads, *args, dt)
    _Padded(b, sum(a) + long, d).check_grads(grads, *args, dt)
    at = slice(sum(a), sum(a) + long)
    _check([x[at] for x in grads], *(x[at] for x in args[:5]), args[5][:, at], [long], [long], True, 0, dt)


@pytest.mark.parametrize("dtype,H,H_kv,d", [("bf16", 4, 2, 64), ("f32", 2, 1, 32)])
def test_varlen_fwd_many_sequences(dtype, H, H_kv, d):
    dt, long = DT[dtype], 2500
    a, b = _short(1500), _short(3500, 3)
    lens = a + [long] + b
    Q, K, V = _packed(19, lens, lens, H, H_kv, d, dt)
    O, LSE = fa.fa_varlen_fwd(Q, K, V, _cu(lens), _cu(lens), causal=True)
    torch.cuda.synchronize()
    fa.fa_check_device()
    for part, first in ((a, 0), (b, sum(a) + long)):
        o, mag, lse, e = _Padded(part, first, d).forward(Q, K, V)
        at = slice(first, first + sum(part))
        ref.check("O", O[at], o, mag, e, dt)
        ref.check_lse(LSE[:, at], lse, e)
    at = slice(sum(a), sum(a) + long)
    _check_fwd(O[at], LSE[:, at], Q[at], K[at], V[at], [long], [long], True, 0, dt)


@pytest.mark.parametrize("d", [96, 256])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 20)])
@pytest.mark.parametrize("deterministic", [False, True])
def test_fp32_other_head_dims(d, causal, window, deterministic):
    dt = torch.float32
    for n, (lq, lk) in enumerate(SETS + [([700], [900])]):
        args = _case(11 * n, lq, lk, 2, 1, d, dt, causal, window)
        dO, Q, K, V, O, LSE = args
        grads = fa.fa_varlen_bwd(*args, _cu(lq), _cu(lk), causal=causal, window_size=window, deterministic=deterministic)
        torch.cuda.synchronize()
        fa.fa_check_device()
        _check_fwd(O, LSE, Q, K, V, lq, lk, causal, window, dt)
        _check(grads, *args, lq, lk, causal, window, dt)


def test_scratch_of_many_short_sequences():
    """The backward of 4096 sequences takes little more than an fp32 accumulator of its rows."""
    N, H, H_kv, d = 4096, 8, 2, 64
    lens = [4 + i % 9 for i in range(N)]
    args = _case(23, lens, lens, H, H_kv, d, torch.bfloat16, True, 0)
    cu = _cu(lens)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    held = torch.cuda.memory_allocated()
    grads = fa.fa_varlen_bwd(*args, cu, cu, causal=True)
    torch.cuda.synchronize()
    fa.fa_check_device()
    T = sum(lens)
    outputs = sum(x.numel() * 2 for x in grads)
    padded = (T // 128 + N) * 128 * H * 8  # D and LSE
    assert torch.cuda.max_memory_allocated() - held <= outputs + T * H * d * 4 + padded + (96 << 20)
    _Padded(lens, 0, d).check_grads(grads, *args, torch.bfloat16)
