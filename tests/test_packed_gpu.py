"""Packed and paged attention on the GPU against plain 64-bit attention (tests/packed_ref.py)."""
import math

import pytest
import torch

import flashattention_backward_preprocess_gb300 as fa
from tests import packed_ref as ref

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _cu(lens):
    return torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32).cuda()


def _rand(seed, shape, dtype, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).cuda()


def _packed(seed, lens_q, lens_k, H, H_kv, d, dtype, extra_q=0, extra_k=0):
    """Q, K, V with `extra` rows of NaN behind the last sequence."""
    Q = _rand(seed, (sum(lens_q) + extra_q, H, d), dtype)
    K = _rand(seed + 1, (sum(lens_k) + extra_k, H_kv, d), dtype)
    V = _rand(seed + 2, (sum(lens_k) + extra_k, H_kv, d), dtype)
    for x, n in ((Q, sum(lens_q)), (K, sum(lens_k)), (V, sum(lens_k))):
        x[n:] = math.nan
    return Q, K, V


def _check_fwd(O, LSE, Q, K, V, lens_q, lens_k, causal, window, dtype):
    a = b = 0
    d = Q.shape[2]
    for nq, nk in zip(lens_q, lens_k):
        q, k, v = (x.double().cpu() for x in (Q[a:a + nq], K[b:b + nk], V[b:b + nk]))
        o, lse, mag, e = ref.attend(q, k, v, causal, window, 1 / math.sqrt(d))
        ref.check(f"O of a sequence {nq}x{nk}", O[a:a + nq], o, mag, e, dtype)
        ref.check_lse(LSE[:, a:a + nq], lse, e)
        a, b = a + nq, b + nk


# lengths: one token, tile borders and one past them, empty sides, uneven sides
SETS = [
    ([1], [1]),
    ([1, 17, 64, 100, 33], [1, 17, 64, 100, 33]),
    ([128, 129, 127, 1, 300], [128, 129, 127, 1, 300]),
    ([5, 0, 200, 3, 0], [0, 7, 130, 260, 0]),
    ([40, 257], [333, 100]),
]


@pytest.mark.parametrize("dtype,H,H_kv,d", [
    ("bf16", 4, 4, 64), ("bf16", 8, 2, 128), ("f16", 6, 2, 64), ("f16", 2, 2, 32), ("bf16", 7, 1, 96),
    ("bf16", 4, 2, 256), ("f32", 4, 2, 64), ("f32", 2, 1, 128), ("bf16", 130, 1, 64),
])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 50), (False, 20)])
def test_varlen_fwd(dtype, H, H_kv, d, causal, window):
    dt = DT[dtype]
    for n, (lq, lk) in enumerate(SETS):
        if H > 100 and sum(lq) > 250:
            continue
        Q, K, V = _packed(11 * n, lq, lk, H, H_kv, d, dt)
        O, LSE = fa.fa_varlen_fwd(Q, K, V, _cu(lq), _cu(lk), causal=causal, window_size=window)
        torch.cuda.synchronize()
        fa.fa_check_device()
        _check_fwd(O, LSE, Q, K, V, lq, lk, causal, window, dt)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_varlen_fwd_long_and_split(dtype):
    """A long sequence beside short ones: items are cut by shares and joined; twice the same bits."""
    dt = DT[dtype]
    lq, lk = [3, 1, 2048 if dtype == "bf16" else 600, 9], [5000, 1, 2048 if dtype == "bf16" else 600, 77]
    Q, K, V = _packed(5, lq, lk, 8, 2, 128, dt)
    O, LSE = fa.fa_varlen_fwd(Q, K, V, _cu(lq), _cu(lk), causal=True)
    O2, LSE2 = fa.fa_varlen_fwd(Q, K, V, _cu(lq), _cu(lk), causal=True)
    torch.cuda.synchronize()
    fa.fa_check_device()
    assert torch.equal(O, O2) and torch.equal(LSE, LSE2)
    _check_fwd(O, LSE, Q, K, V, lq, lk, True, 0, dt)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_varlen_fwd_other_sequences_do_not_leak(dtype):
    """Infinities and NaN in a neighbour's rows and behind the last sequence stay there."""
    dt = DT[dtype]
    lens = [70, 30, 130]
    Q, K, V = _packed(3, lens, lens, 4, 2, 64, dt, extra_q=9, extra_k=9)
    bad = slice(70, 100)
    for x in (Q, K, V):
        x[bad] = math.nan
    V[75] = math.inf
    O, LSE = fa.fa_varlen_fwd(Q, K, V, _cu(lens), _cu(lens))
    torch.cuda.synchronize()
    for sl in (slice(0, 70), slice(100, 230)):
        q, k, v = (x[sl].double().cpu() for x in (Q, K, V))
        o, lse, mag, e = ref.attend(q, k, v, False, 0, 1 / 8)
        ref.check("O", O[sl], o, mag, e, dt)
        ref.check_lse(LSE[:, sl], lse, e)
    # rows of no sequence: set when the call allocates its outputs
    assert (O[230:] == 0).all() and (LSE[:, 230:] == -math.inf).all()
    # left as they were when the caller passes them
    O2, LSE2 = torch.full_like(O, 7), torch.full_like(LSE, 5)
    fa.fa_varlen_fwd(Q, K, V, _cu(lens), _cu(lens), O=O2, LSE=LSE2)
    assert (O2[230:] == 7).all() and (LSE2[:, 230:] == 5).all()
    assert torch.equal(O2[:70], O[:70])


def test_varlen_fwd_strided_views():
    """Q, K, V as slices of one projection, head-major memory, an output with padded rows."""
    H, H_kv, d, lens = 8, 2, 64, [100, 1, 60]
    T = sum(lens)
    joint = _rand(1, (T, H + 2 * H_kv, d), torch.bfloat16)
    Q, K, V = joint[:, :H], joint[:, H:H + H_kv], joint[:, H + H_kv:]
    O, LSE = fa.fa_varlen_fwd(Q.contiguous(), K.contiguous(), V.contiguous(), _cu(lens), _cu(lens), causal=True)
    O2, LSE2 = fa.fa_varlen_fwd(Q, K, V, _cu(lens), _cu(lens), causal=True)
    assert torch.equal(O, O2) and torch.equal(LSE, LSE2)
    hm = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (Q, K, V)]
    wide = torch.full((T, H + 1, d), 3.0, dtype=torch.bfloat16, device="cuda")
    O3, LSE3 = fa.fa_varlen_fwd(*hm, _cu(lens), _cu(lens), causal=True, O=wide[:, :H])
    assert torch.equal(O, O3) and torch.equal(LSE, LSE3) and (wide[:, H] == 3).all()
    Qf, Kf, Vf = (x.float() for x in (Q, K, V))
    assert torch.equal(fa.fa_varlen_fwd(Qf.contiguous(), Kf, Vf, _cu(lens), _cu(lens))[0],
                       fa.fa_varlen_fwd(Qf, Kf, Vf, _cu(lens), _cu(lens))[0])


def _paged(seed, new, total, H, H_kv, d, page, dtype, spare=2):
    need = [-(-t // page) for t in total]
    pages = sum(need) + spare
    g = torch.Generator().manual_seed(seed)
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(new), max(max(need), 1)), -1, dtype=torch.int32)
    at = 0
    K = _rand(seed + 1, (pages, page, H_kv, d), dtype)
    V = _rand(seed + 2, (pages, page, H_kv, d), dtype)
    for n, k in enumerate(need):
        table[n, :k] = order[at:at + k]
        at += k
        if total[n] % page:  # what stands behind a request's last key must not matter
            K[int(table[n, k - 1]), total[n] % page:] = math.nan
            V[int(table[n, k - 1]), total[n] % page:] = math.inf
    Q = _rand(seed + 3, (sum(new), H, d), dtype)
    return Q, K, V, table.cuda(), torch.tensor(total, dtype=torch.int32, device="cuda")


def _check_paged(O, LSE, Q, K, V, table, new, total, causal, window, dtype):
    a, d, page = 0, Q.shape[2], K.shape[1]
    for n, (nq, nk) in enumerate(zip(new, total)):
        k, v = (ref.gather_pages(x, table[n], nk, page).double().cpu() for x in (K, V))
        o, lse, mag, e = ref.attend(Q[a:a + nq].double().cpu(), k, v, causal, window, 1 / math.sqrt(d))
        ref.check(f"O of request {n}", O[a:a + nq], o, mag, e, dtype)
        ref.check_lse(LSE[:, a:a + nq], lse, e)
        a += nq


@pytest.mark.parametrize("dtype,H,H_kv,d,page", [
    ("bf16", 8, 2, 128, 16), ("bf16", 4, 4, 64, 8), ("f16", 8, 1, 64, 64), ("f16", 6, 2, 128, 128),
    ("bf16", 4, 2, 128, 256), ("bf16", 4, 1, 256, 32), ("f16", 2, 1, 256, 128), ("bf16", 4, 2, 32, 16),
    ("f32", 4, 2, 64, 16), ("bf16", 4, 2, 64, 3), ("f32", 2, 2, 128, 1),
])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 40), (False, 0)])
def test_paged_fwd(dtype, H, H_kv, d, page, causal, window):
    dt = DT[dtype]
    for new, total in (([1], [1]), ([1, 1, 1], [15, 16, 1000]), ([1, 40, 130, 0, 7], [300, 40, 257, 5, 129]),
                       ([3], [1])):
        Q, K, V, table, lens = _paged(21, new, total, H, H_kv, d, page, dt)
        O, LSE = fa.fa_paged_fwd(Q, K, V, table, _cu(new), lens, causal=causal, window_size=window)
        torch.cuda.synchronize()
        fa.fa_check_device()
        _check_paged(O, LSE, Q, K, V, table, new, total, causal, window, dt)


def test_paged_fwd_head_major_cache_and_freed_pages():
    """A [pages, H_kv, page, d] cache as a view; pages before the window need not exist."""
    new, total, page = [1, 20], [900, 700], 16
    Q, K, V, table, lens = _paged(4, new, total, 8, 2, 64, page, torch.bfloat16)
    O, LSE = fa.fa_paged_fwd(Q, K, V, table, _cu(new), lens, window_size=100)
    Kh, Vh = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (K, V))
    freed = table.clone()
    freed[0, : (900 - 100) // page] = -1
    freed[1, : (700 - 20 - 100) // page] = 10 ** 6
    O2, LSE2 = fa.fa_paged_fwd(Q, Kh, Vh, freed, _cu(new), lens, window_size=100)
    torch.cuda.synchronize()
    fa.fa_check_device()
    assert torch.equal(O, O2) and torch.equal(LSE, LSE2)
    O3, _ = fa.fa_paged_fwd(Q.float(), Kh.float(), Vh.float(), freed, _cu(new), lens, window_size=100)
    torch.cuda.synchronize()
    fa.fa_check_device()
    assert (O3 - O.float()).abs().max() < 0.05


def test_paged_fwd_many_requests_use_one_launch_shape():
    """More requests than CTAs, some without new tokens; split and whole items side by side."""
    new = [1 + (i % 3) for i in range(300)]
    new[7] = new[200] = 0
    total = [max(n, (i * 37) % 400) for i, n in enumerate(new)]
    total[100] = 6000
    Q, K, V, table, lens = _paged(9, new, total, 4, 1, 64, 32, torch.float16)
    O, LSE = fa.fa_paged_fwd(Q, K, V, table, _cu(new), lens)
    torch.cuda.synchronize()
    fa.fa_check_device()
    _check_paged(O, LSE, Q, K, V, table, new, total, True, 0, torch.float16)


def _slots_ref(ctx, new, table, free, start, page, T):
    table = [list(map(int, r)) for r in table]
    slots, pos, at, t = [-1] * T, [-1] * T, start, 0
    for n, (c, m) in enumerate(zip(ctx, new)):
        for col in range(-(-c // page), -(-(c + m) // page)):
            table[n][col] = int(free[at])
            at += 1
        for i in range(m):
            slots[t], pos[t] = table[n][(c + i) // page] * page + (c + i) % page, c + i
            t += 1
    return table, slots, pos, [c + m for c, m in zip(ctx, new)], at


@pytest.mark.parametrize("N,page,most_new,most_ctx", [(1, 16, 1, 0), (8, 16, 1, 100), (5, 1, 9, 7), (300, 8, 3, 60),
                                                      (700, 16, 40, 500), (2, 128, 3000, 1000), (1500, 16, 1, 64)])
def test_page_slots(N, page, most_new, most_ctx):
    g = torch.Generator().manual_seed(N)
    new = torch.randint(0, most_new + 1, (N,), generator=g).tolist()
    ctx = torch.randint(0, most_ctx + 1, (N,), generator=g).tolist()
    cols = -(-(most_ctx + most_new) // page) + 1
    free = torch.randperm(N * cols * 2, generator=g).to(torch.int32)
    table = torch.full((N, cols), -1, dtype=torch.int32)
    at = N * cols
    for n, c in enumerate(ctx):
        k = -(-c // page)
        table[n, :k] = free[at:at + k]
        at += k
    T = sum(new) + 5
    want = _slots_ref(ctx, new, table, free, 2, page, T)
    dev = table.cuda()
    cu = torch.tensor([0] + new).cumsum(0).to(torch.int32).cuda()
    args = (torch.tensor(ctx, dtype=torch.int32).cuda(), cu, dev, free.cuda(), torch.tensor([2], dtype=torch.int32).cuda(), page, T)
    for _ in range(2):  # the call changes nothing it reads
        slots, pos, lens, nxt = fa.fa_page_slots(*args)
        torch.cuda.synchronize()
        fa.fa_check_device()
        assert dev.tolist() == want[0] and slots.tolist() == want[1] and pos.tolist() == want[2]
        assert lens.tolist() == want[3] and nxt.tolist() == [want[4]]


def test_page_slots_runs_out():
    """Too few free pages or columns: -1 entries and slots, an error, nothing out of range."""
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.full((2, 4), -1, **i32)
    cu = torch.tensor([0, 40, 120], **i32)
    slots, _, lens, nxt = fa.fa_page_slots(torch.tensor([0, 0], **i32), cu, table, torch.tensor([5, 6, 9, 1], **i32),
                                           torch.tensor([0], **i32), 16, 120)
    torch.cuda.synchronize()
    with pytest.raises(fa.FaError, match="FA_ERR_INVALID_ARG"):
        fa.fa_check_device()
    fa.fa_check_device()  # cleared
    assert table.tolist() == [[5, 6, 9, -1], [1, -1, -1, -1]]
    assert slots[:40].tolist() == [p * 16 + i for p in (5, 6, 9) for i in range(16)][:40]
    assert slots[40:56].tolist() == [16 + i for i in range(16)] and (slots[56:] == -1).all()
    assert lens.tolist() == [40, 80] and nxt.tolist() == [8]


@pytest.mark.parametrize("dtype,d,page,H_kv", [("bf16", 128, 16, 8), ("f32", 32, 3, 2), ("f16", 96, 64, 1)])
def test_paged_write(dtype, d, page, H_kv):
    dt = DT[dtype]
    pages, T = 11, 77 if page > 4 else 20
    K, V = _rand(1, (T, H_kv, d), dt), _rand(2, (T, H_kv, d), dt)
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(3))[:T]
    slots[5], slots[9] = -1, -7
    Kc, Vc = _rand(4, (pages, page, H_kv, d), dt), _rand(5, (pages, page, H_kv, d), dt)
    want = []
    for new, c in ((K, Kc), (V, Vc)):
        w = c.cpu().clone().view(-1, H_kv, d)
        for t, s in enumerate(slots.tolist()):
            if s >= 0:
                w[s] = new[t].cpu()
        want.append(w.view(pages, page, H_kv, d))
    hm = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in (Kc, Vc)]
    fa.fa_paged_write(K, V, slots.cuda(), Kc, Vc)
    joint = torch.cat([K, V], 1)
    fa.fa_paged_write(joint[:, :H_kv], joint[:, H_kv:], slots.cuda(), *hm)
    torch.cuda.synchronize()
    fa.fa_check_device()
    for got, w in ((Kc, want[0]), (Vc, want[1]), (hm[0], want[0]), (hm[1], want[1])):
        assert torch.equal(got.cpu(), w)


def test_bad_lengths_and_pages_are_reported():
    """Device-side arguments that do not fit: nothing out of range is touched, the check names them."""
    Q, K, V = _packed(1, [10, 10], [10, 10], 2, 2, 64, torch.bfloat16)
    good = _cu([10, 10])
    for cu in ([0, 15, 10], [-1, 5, 20], [0, 10, 21], [0, 10, 2 ** 31 - 1]):
        bad = torch.tensor(cu, dtype=torch.int32, device="cuda")
        for q, k in ((bad, good), (good, bad)):
            O = torch.full_like(Q, 4)
            LSE = torch.full((2, 20), 4.0, device="cuda")
            fa.fa_varlen_fwd(Q, K, V, q, k, O=O, LSE=LSE)
            torch.cuda.synchronize()
            assert (O == 4).all() and (LSE == 4).all()
            with pytest.raises(fa.FaError, match="sequence lengths"):
                fa.fa_check_device()
    new, total = [1, 5], [40, 33]
    for dt in (torch.bfloat16, torch.float32):
        Q, K, V, table, lens = _paged(2, new, total, 2, 1, 64, 16, dt)
        whole, _ = fa.fa_paged_fwd(Q, K, V, table, _cu(new), lens)
        for id in (-1, K.shape[0], 2 ** 31 - 1, -2 ** 31):
            t = table.clone()
            t[0, 1] = id
            O, _ = fa.fa_paged_fwd(Q, K, V, t, _cu(new), lens)
            torch.cuda.synchronize()
            with pytest.raises(fa.FaError, match="page or slot"):
                fa.fa_check_device()
            assert torch.equal(O[1:], whole[1:])  # the other request
        too_long = torch.tensor([40, 16 * table.shape[1] + 1], dtype=torch.int32, device="cuda")
        fa.fa_paged_fwd(Q, K, V, table, _cu(new), too_long)
        torch.cuda.synchronize()
        with pytest.raises(fa.FaError, match="sequence lengths"):
            fa.fa_check_device()
    K, V = _rand(1, (3, 1, 64), torch.bfloat16), _rand(2, (3, 1, 64), torch.bfloat16)
    Kc = torch.zeros(2, 8, 1, 64, dtype=torch.bfloat16, device="cuda")
    Vc = torch.zeros_like(Kc)
    fa.fa_paged_write(K, V, torch.tensor([3, 16, 2 ** 62], device="cuda"), Kc, Vc)
    torch.cuda.synchronize()
    with pytest.raises(fa.FaError, match="page or slot"):
        fa.fa_check_device()
    assert torch.equal(Kc.view(16, 64)[3], K[0, 0]) and Kc.count_nonzero() == K[0].count_nonzero()


def test_strided_head_dimension_is_refused():
    Q, K, V = _packed(1, [8], [8], 2, 2, 128, torch.bfloat16)
    with pytest.raises(fa.FaError, match="Q: the head dimension must be contiguous"):
        fa.fa_varlen_fwd(Q[..., ::2], K[..., :64], V[..., :64], _cu([8]), _cu([8]))
    with pytest.raises(fa.FaError, match="strides: entry"):  # rows of 65 elements
        wide = torch.zeros(8, 2, 65, dtype=torch.bfloat16, device="cuda")
        fa.fa_varlen_fwd(wide[..., :64], K[..., :64], V[..., :64], _cu([8]), _cu([8]))
    with pytest.raises(fa.FaError, match="strides: entry"):  # broadcast heads
        fa.fa_varlen_fwd(Q, K[:, :1].expand(-1, 2, -1), V, _cu([8]), _cu([8]))


@pytest.mark.parametrize("N,H,H_kv,d", [(700, 8, 8, 64), (1500, 8, 2, 128), (600, 4, 4, 256)])
def test_varlen_fwd_many_short_sequences(N, H, H_kv, d):
    """Items of one key tile each, many per CTA, with the plan of one block and of every CTA."""
    lens = [1 + (i * 31) % 40 for i in range(N)]
    Q, K, V = _packed(13, lens, lens, H, H_kv, d, torch.bfloat16)
    cu = _cu(lens)
    O, LSE = fa.fa_varlen_fwd(Q, K, V, cu, cu, causal=True)
    for _ in range(5):
        O2, LSE2 = fa.fa_varlen_fwd(Q, K, V, cu, cu, causal=True)
        torch.cuda.synchronize()
        fa.fa_check_device()
        assert torch.equal(O, O2) and torch.equal(LSE, LSE2)
    # one padded batch in 64 bits
    m, off = max(lens), torch.tensor([0] + lens).cumsum(0)[:-1]
    at = (off[:, None] + torch.arange(m)).clamp(max=sum(lens) - 1)
    q, k, v = (x.double().cpu()[at].transpose(1, 2) for x in (Q, K, V))
    k, v = (x.repeat_interleave(H // H_kv, 1) for x in (k, v))
    s = (q @ k.transpose(-1, -2)) * d ** -0.5
    see = torch.ones(m, m).tril().bool()
    s = s.masked_fill(~see, -math.inf)
    lse = torch.logsumexp(s, -1)
    P = torch.exp(s - lse[..., None])
    s_err = d * ref.STEP * d ** -0.5 * float((q.abs() @ k.abs().transpose(-1, -2)).max())
    e = 2 * math.expm1(s_err) + m * ref.STEP + 2.0 ** -21
    inside = torch.arange(m) < torch.tensor(lens)[:, None]
    pick = lambda x: x.transpose(1, 2)[inside]
    ref.check("O", O, pick(P @ v), pick(P @ v.abs()), e, torch.bfloat16)
    ref.check_lse(LSE, lse.transpose(1, 2)[inside].t(), e)


def test_empty_head_dimension_is_refused():
    q = torch.zeros(4, 2, 0, dtype=torch.bfloat16, device="cuda")
    cu = _cu([4])
    cache = torch.zeros(2, 8, 2, 0, dtype=torch.bfloat16, device="cuda")
    table, lens = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.full((1,), 4, dtype=torch.int32, device="cuda")
    lse = torch.zeros(2, 4, device="cuda")
    for call in (lambda: fa.fa_varlen_fwd(q, q, q, cu, cu), lambda: fa.fa_varlen_bwd(q, q, q, q, q, lse, cu, cu),
                 lambda: fa.fa_paged_fwd(q, cache, cache, table, cu, lens)):
        with pytest.raises(fa.FaError, match=" d:"):
            call()


@pytest.mark.parametrize("dtype,page,H_kv,d", [("bf16", 16, 8, 128), ("bf16", 5, 8, 128), ("f16", 64, 4, 256)])
def test_paged_offsets_past_32_bits(dtype, page, H_kv, d):
    """Pages at the far end of a cache of more than 2^32 elements give what a small cache gives."""
    pages = (1 << 32) // (page * H_kv * d) + 20
    H, ctx, dt = 2 * H_kv, 3 * page + 2, DT[dtype]
    gen = torch.Generator().manual_seed(5)
    Q = torch.randn(1, H, d, generator=gen).to(dt).cuda()
    K, V = (torch.randn(ctx, H_kv, d, generator=gen).to(dt).cuda() for _ in range(2))
    lens, cu = torch.tensor([ctx], dtype=torch.int32, device="cuda"), _cu([1])
    out = []
    for n in (20, pages):
        caches = [torch.empty(n, page, H_kv, d, dtype=dt, device="cuda") for _ in range(2)]
        table = torch.tensor([[n - 1, n - 9, n - 2, n - 20]], dtype=torch.int32, device="cuda")
        at = torch.arange(ctx, device="cuda")
        slots = table[0, at // page].long() * page + at % page
        fa.fa_paged_write(K, V, slots, *caches)
        assert torch.equal(caches[0].view(-1, H_kv, d)[slots], K) and torch.equal(caches[1].view(-1, H_kv, d)[slots], V)
        out.append(fa.fa_paged_fwd(Q, *caches, table, cu, lens))
        torch.cuda.synchronize()
        del caches
    fa.fa_check_device()
    torch.cuda.empty_cache()
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
