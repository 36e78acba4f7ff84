"""The packed backward on the GPU: against the 64-bit formula (tests/packed_ref.py), against
differences, through autograd, reproducible, captured into a graph, on another stream."""
import math

import pytest
import torch

import flashattention_backward_preprocess_gb300 as fa
from tests import packed_ref as ref
from tests.test_packed_gpu import DT, SETS, _cu, _packed, _rand

pytestmark = pytest.mark.gpu


def _case(seed, lq, lk, H, H_kv, d, dt, causal, window, extra_q=0, extra_k=0):
    Q, K, V = _packed(seed, lq, lk, H, H_kv, d, dt, extra_q, extra_k)
    dO = _rand(seed + 3, Q.shape, dt)
    dO[sum(lq):] = math.nan
    O, LSE = fa.fa_varlen_fwd(Q, K, V, _cu(lq), _cu(lk), causal=causal, window_size=window)
    return dO, Q, K, V, O, LSE


def _check(grads, dO, Q, K, V, O, LSE, lq, lk, causal, window, dt):
    a = b = 0
    d = Q.shape[2]
    for nq, nk in zip(lq, lk):
        do, q, o = (x[a:a + nq].double().cpu() for x in (dO, Q, O))
        k, v = (x[b:b + nk].double().cpu() for x in (K, V))
        lse = LSE[:, a:a + nq].double().cpu()
        want, mag, f32, e = ref.grads(do, q, k, v, o, lse, causal, window, 1 / math.sqrt(d))
        got = (grads[0][a:a + nq], grads[1][b:b + nk], grads[2][b:b + nk])
        for i, name in enumerate(("dQ", "dK", "dV")):
            ref.check(f"{name} of a sequence {nq}x{nk}", got[i], want[i], mag[i], e, dt, f32[i])
        a, b = a + nq, b + nk


@pytest.mark.parametrize("dtype,H,H_kv,d", [
    ("bf16", 4, 4, 64), ("bf16", 8, 2, 128), ("f16", 6, 2, 64), ("f16", 2, 2, 32), ("bf16", 7, 1, 96),
    ("bf16", 4, 2, 256), ("f32", 4, 2, 64), ("f32", 2, 1, 128),
])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 50), (False, 20)])
@pytest.mark.parametrize("deterministic", [False, True])
def test_varlen_bwd(dtype, H, H_kv, d, causal, window, deterministic):
    dt = DT[dtype]
    for n, (lq, lk) in enumerate(SETS):
        args = _case(11 * n, lq, lk, H, H_kv, d, dt, causal, window)
        grads = fa.fa_varlen_bwd(*args, _cu(lq), _cu(lk), causal=causal, window_size=window, deterministic=deterministic)
        torch.cuda.synchronize()
        fa.fa_check_device()
        _check(grads, *args, lq, lk, causal, window, dt)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 64), ("f32", 64)])
def test_varlen_bwd_deterministic_bits(dtype, d):
    dt = DT[dtype]
    lq = lk = [700, 3, 1300, 129]
    args = _case(2, lq, lk, 8, 2, d, dt, True, 0)
    one = fa.fa_varlen_bwd(*args, _cu(lq), _cu(lk), causal=True, deterministic=True)
    two = fa.fa_varlen_bwd(*args, _cu(lq), _cu(lk), causal=True, deterministic=True)
    plain = fa.fa_varlen_bwd(*args, _cu(lq), _cu(lk), causal=True)
    torch.cuda.synchronize()
    fa.fa_check_device()
    assert all(torch.equal(a, b) for a, b in zip(one, two))
    assert torch.equal(one[1], plain[1]) and torch.equal(one[2], plain[2])
    _check(one, *args, lq, lk, True, 0, dt)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 256), ("f32", 64)])
def test_varlen_bwd_other_sequences_do_not_leak(dtype, d):
    """NaN and infinities of a neighbour and behind the last sequence stay out of the gradients."""
    dt = DT[dtype]
    lens = [70, 30, 130]
    clean = _case(3, lens, lens, 4, 2, d, dt, False, 0)
    want = fa.fa_varlen_bwd(*clean, _cu(lens), _cu(lens), deterministic=True)
    dirty = [torch.cat([x, torch.full_like(x[:9], math.nan)]) for x in clean[:5]]
    LSE = torch.cat([clean[5], torch.full_like(clean[5][:, :9], math.nan)], 1)
    for x in dirty[:4]:
        x[70:100] = math.nan
    dirty[3][80] = math.inf
    got = fa.fa_varlen_bwd(*dirty, LSE, _cu(lens), _cu(lens), deterministic=True)
    torch.cuda.synchronize()
    fa.fa_check_device()
    for g, w in zip(got, want):
        assert torch.equal(g[:70], w[:70]) and torch.equal(g[100:230], w[100:230])
        assert (g[230:] == 0).all()  # rows of no sequence
    mine = [torch.full_like(x, 7) for x in got]
    fa.fa_varlen_bwd(*dirty, LSE, _cu(lens), _cu(lens), dQ=mine[0], dK=mine[1], dV=mine[2])
    assert all((x[230:] == 7).all() for x in mine)


def test_varlen_bwd_strided_views():
    """Gradients of a joint projection written into the slices of its gradient."""
    H, H_kv, d, lens = 8, 2, 64, [100, 1, 60]
    joint = _rand(1, (sum(lens), H + 2 * H_kv, d), torch.bfloat16)
    Q, K, V = joint[:, :H], joint[:, H:H + H_kv], joint[:, H + H_kv:]
    O, LSE = fa.fa_varlen_fwd(Q, K, V, _cu(lens), _cu(lens), causal=True)
    dO = _rand(2, O.shape, torch.bfloat16)
    want = fa.fa_varlen_bwd(dO, Q.contiguous(), K.contiguous(), V.contiguous(), O, LSE, _cu(lens), _cu(lens), causal=True,
                            deterministic=True)
    dj = torch.full_like(joint, 9)
    hm = dO.transpose(0, 1).contiguous().transpose(0, 1)
    fa.fa_varlen_bwd(hm, Q, K, V, O, LSE, _cu(lens), _cu(lens), causal=True, deterministic=True, dQ=dj[:, :H],
                     dK=dj[:, H:H + H_kv], dV=dj[:, H + H_kv:])
    assert torch.equal(dj, torch.cat(want, 1))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_varlen_bwd_empty_axes(dtype):
    """No query rows at all: dK = dV = 0.  No key rows at all: dQ = 0."""
    dt = DT[dtype]
    none, some = [0, 0], [5, 9]
    for lq, lk in ((none, some), (some, none)):
        args = _case(1, lq, lk, 4, 2, 64, dt, True, 0)
        grads = fa.fa_varlen_bwd(*args, _cu(lq), _cu(lk), causal=True)
        torch.cuda.synchronize()
        fa.fa_check_device()
        assert all((g == 0).all() for g in grads)
        if lk is none:
            assert (args[4] == 0).all() and (args[5] == -math.inf).all()


def test_varlen_matches_dense_backward():
    """Sequences of one length: the dense call on the same data."""
    N, S, H, H_kv, d = 3, 200, 4, 2, 64
    lens = [S] * N
    args = _case(4, lens, lens, H, H_kv, d, torch.float16, True, 0)
    got = fa.fa_varlen_bwd(*args, _cu(lens), _cu(lens), causal=True)
    dense = [x.view(N, S, -1, d).transpose(1, 2).contiguous() for x in args[:5]]
    lse = args[5].view(H, N, S).transpose(0, 1).contiguous()
    want = fa.fa_bwd(dense[0], dense[1], dense[2], dense[3], dense[4], lse, causal=True)
    for g, w in zip(got, want):
        w = w.transpose(1, 2).reshape(g.shape)
        assert (g - w).abs().max() <= 2 ** -8 * w.abs().max()


def test_varlen_bwd_against_differences():
    """fp32: the gradient of sum(O * dO) along random directions, by central differences in 64 bits."""
    lens = [37, 1, 70]
    dO, Q, K, V, O, LSE = _case(6, lens, lens, 2, 1, 32, torch.float32, True, 0)
    grads = fa.fa_varlen_bwd(dO, Q, K, V, O, LSE, _cu(lens), _cu(lens), causal=True)

    def f(q, k, v):
        s, a = 0.0, 0
        for n in lens:
            o = ref.attend(q[a:a + n], k[a:a + n], v[a:a + n], True, 0, 32 ** -0.5)[0]
            s += float((o * dO[a:a + n].double().cpu()).sum())
            a += n
        return s

    x = [t.double().cpu() for t in (Q, K, V)]
    for i in range(3):
        g = torch.Generator().manual_seed(i)
        dir = torch.randn(x[i].shape, generator=g, dtype=torch.float64)
        h = 1e-5
        up, down = ([t + s * h * dir if j == i else t for j, t in enumerate(x)] for s in (1, -1))
        want = (f(*up) - f(*down)) / (2 * h)
        got = float((grads[i].double().cpu() * dir).sum())
        # fp32 gradients: relative 1e-5 of the sum of magnitudes covers their rounding and h^2
        assert abs(got - want) <= 1e-5 * float((grads[i].double().cpu() * dir).abs().sum()), i


def test_flash_attention_varlen_autograd():
    """Values and gradients through autograd; expanded heads and unaligned views; padding rows."""
    lens, d = [33, 5, 80], 64
    T = sum(lens) + 4
    q = _rand(1, (T, 4, d), torch.bfloat16).requires_grad_()
    k1 = _rand(2, (T, 1, d), torch.bfloat16).requires_grad_()  # one head, expanded to two
    v = _rand(3, (T, 2, d + 1), torch.bfloat16).requires_grad_()
    cu = _cu(lens)
    out = fa.flash_attention_varlen(q, k1.expand(-1, 2, -1), v[..., 1:], cu, cu, causal=True)
    do = _rand(4, out.shape, torch.bfloat16)
    dq, dk1, dv = torch.autograd.grad(out, (q, k1, v), do)
    torch.cuda.synchronize()
    fa.fa_check_device()
    kk, vv = k1.detach().expand(-1, 2, -1).contiguous(), v.detach()[..., 1:].contiguous()
    O, LSE = fa.fa_varlen_fwd(q.detach(), kk, vv, cu, cu, causal=True)
    want = fa.fa_varlen_bwd(do, q.detach(), kk, vv, O, LSE, cu, cu, causal=True)
    n = sum(lens)
    assert torch.equal(out, O) and (out[n:] == 0).all() and (dq[n:] == 0).all() and (dv[n:] == 0).all()
    assert (dq - want[0]).abs().max() <= 2 ** -7 * want[0].abs().max()  # atomics: dQ alone may vary
    assert torch.equal(dv[..., 1:], want[2]) and (dv[..., 0] == 0).all()
    assert torch.equal(dk1, want[1].sum(1, keepdim=True)) or torch.allclose(
        dk1.float(), want[1].float().sum(1, keepdim=True), rtol=2 ** -7, atol=2 ** -7)


def test_captured_forward_and_backward_follow_the_lengths():
    """One graph, other lengths at every replay; two graphs of one stream replayed side by side."""
    T, H, d = 600, 4, 64
    Q, K, V, dO = (_rand(i, (T, H, d), torch.bfloat16) for i in range(4))
    cu = _cu([100, 400, 100])
    cap = torch.cuda.Stream()
    cap.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    with torch.cuda.stream(cap):
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=cap):
                O, LSE = fa.fa_varlen_fwd(Q, K, V, cu, cu, causal=True)
                outs.append((O, LSE, *fa.fa_varlen_bwd(dO, Q, K, V, O, LSE, cu, cu, causal=True, deterministic=True)))
            graphs.append(g)
    torch.cuda.current_stream().wait_stream(cap)
    for lens in ([100, 400, 100], [1, 598, 1], [300, 0, 250]):
        cu.copy_(_cu(lens))
        for x in outs[0] + outs[1]:
            x.zero_()
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for _ in range(5):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        fa.fa_check_device()
        O, LSE = fa.fa_varlen_fwd(Q, K, V, cu, cu, causal=True)
        want = (O, LSE, *fa.fa_varlen_bwd(dO, Q, K, V, O, LSE, cu, cu, causal=True, deterministic=True))
        n = sum(lens)
        for got in outs:
            assert torch.equal(got[1][:, :n], LSE[:, :n])
            assert all(torch.equal(got[i][:n], want[i][:n]) for i in (0, 2, 3, 4))


def test_calls_on_other_streams():
    """stream= as a torch stream and as a raw handle, two calls at once."""
    lens = [300, 20, 130]
    args = _case(8, lens, lens, 4, 2, 128, torch.bfloat16, True, 0)
    cu = _cu(lens)
    want = (fa.fa_varlen_fwd(*args[1:4], cu, cu, causal=True), fa.fa_varlen_bwd(*args, cu, cu, causal=True, deterministic=True))
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(4):
        for s in (s1, s2.cuda_stream):
            got.append((fa.fa_varlen_fwd(*args[1:4], cu, cu, causal=True, stream=s),
                        fa.fa_varlen_bwd(*args, cu, cu, causal=True, deterministic=True, stream=s)))
    torch.cuda.synchronize()
    fa.fa_check_device()
    for f, b in got:
        assert all(torch.equal(x, y) for x, y in zip(f + b, want[0] + want[1]))


def test_calls_from_new_threads():
    """A thread whose first CUDA work is the call itself."""
    import threading
    lens = [50, 20]
    args = _case(8, lens, lens, 2, 2, 64, torch.bfloat16, True, 0)
    cu = _cu(lens)
    calls = [lambda: fa.fa_varlen_fwd(*args[1:4], cu, cu, causal=True),
             lambda: fa.fa_varlen_bwd(*args, cu, cu, causal=True, deterministic=True)]
    torch.cuda.synchronize()
    for call in calls:
        want, got = call(), []
        t = threading.Thread(target=lambda: got.extend(call()))
        t.start()
        t.join()
        torch.cuda.synchronize()
        assert len(got) == len(want) and all(torch.equal(x, y) for x, y in zip(got, want))


def test_bad_lengths_leave_gradients_alone():
    args = _case(1, [10, 10], [10, 10], 2, 2, 64, torch.bfloat16, False, 0)
    good = _cu([10, 10])
    for dt in (torch.bfloat16, torch.float32):
        a = [x.to(dt) for x in args[:5]] + [args[5]]
        for cu in ([0, 15, 10], [-1, 5, 20], [0, 10, 21]):
            bad = torch.tensor(cu, dtype=torch.int32, device="cuda")
            for q, k in ((bad, good), (good, bad)):
                out = [torch.full_like(x, 4) for x in a[1:4]]
                fa.fa_varlen_bwd(*a, q, k, dQ=out[0], dK=out[1], dV=out[2])
                torch.cuda.synchronize()
                assert all((x == 4).all() for x in out)
                with pytest.raises(fa.FaError, match="sequence lengths"):
                    fa.fa_check_device()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 256), ("f32", 64)])
def test_offsets_past_32_bits(dtype, d):
    """Sequences behind element 2^31 of the packed tensors give the bits that they give alone."""
    H, lens, dt = 32, [130, 77], DT[dtype]
    n = sum(lens)
    T = (1 << 31) // (H * d) + 1000
    gen = torch.Generator().manual_seed(6)
    small = [torch.randn(n, H, d, generator=gen).to(dt).cuda() for _ in range(4)]
    cu = _cu(lens)
    out = []
    for first in (0, T - n):
        Q, K, V, dO = big = [torch.empty(first + n, H, d, dtype=dt, device="cuda") for _ in range(4)]
        for b, x in zip(big, small):
            b[first:] = x
        c = cu + first
        O, LSE = fa.fa_varlen_fwd(Q, K, V, c, c, causal=True)
        grads = fa.fa_varlen_bwd(dO, Q, K, V, O, LSE, c, c, causal=True, deterministic=True)
        assert first == 0 or not any(x[first - 1].any() or x[0].any() for x in (O, *grads))
        out.append([x[first:].clone() for x in (O, *grads)] + [LSE[:, first:].clone()])
        torch.cuda.synchronize()
        del Q, K, V, dO, big, b, O, LSE, grads
    fa.fa_check_device()
    torch.cuda.empty_cache()
    assert all(torch.equal(a, b) for a, b in zip(*out))
