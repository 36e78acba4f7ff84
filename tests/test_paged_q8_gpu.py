"""The 8-bit paged cache on the GPU: rows as written, read back, and attention over them."""
import math

import pytest
import torch

import flashattention_backward_preprocess_gb300 as fa
from tests import draft_ref as dr
from tests import packed_ref as ref
from tests.test_packed_gpu import DT, _cu, _rand

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


def _errors():
    torch.cuda.synchronize()
    try:
        fa.fa_check_device()
    except fa.FaError as e:
        assert e.status == 1
        return str(e)
    return ""


def _empty_cache(pages, page, H_kv, d, fill=0x31):
    c = [torch.full((pages, page, H_kv, d), fill, dtype=torch.uint8, device="cuda").view(F8) for _ in "KV"]
    e = [torch.full((pages, H_kv, page), 120, dtype=torch.uint8, device="cuda") for _ in "KV"]
    return c + e


def _rows(seed, T, H_kv, d, dtype):
    """Rows of all sizes: normal ones, zeros, the type's ends, halves between two e4m3 numbers."""
    x = _rand(seed, (T, H_kv, d), torch.float32)
    g = torch.Generator().manual_seed(seed + 1)
    x = x * torch.exp2(torch.randint(-24, 14, (T, H_kv, 1), generator=g).float()).cuda()
    flat = x.view(-1, d)
    n = flat.shape[0]
    flat[0] = 0.0
    flat[1 % n, 1:] = 0.0
    if n > 12:
        flat[2] *= 1e-30
        flat[3, 0], flat[3, 1] = 448.0, -449.0
        flat[4] = 0.0
        flat[4, :4] = torch.tensor([1.0625, -1.1875, 448.0, 2.0 ** -10])   # halves, and half of the smallest number
        flat[5, 3], flat[5, 4], flat[5, 5] = math.inf, -math.inf, math.nan
        flat[6] = math.nan
        flat[7] = math.inf
        flat[8, 0] = torch.finfo(dtype).max
        flat[9] = torch.finfo(dtype).max
        flat[10] = torch.finfo(dtype).tiny
        flat[11] = 65504.0
    return x.to(dtype)


@pytest.mark.parametrize("dtype,d,page,H_kv,T", [
    ("bf16", 128, 16, 8, 77), ("f16", 64, 32, 2, 50), ("f32", 32, 3, 2, 31), ("bf16", 96, 5, 1, 40), ("f16", 256, 64, 3, 70),
    ("f32", 256, 16, 1, 1), ("bf16", 32, 8, 4, 13), ("f32", 96, 7, 3, 20), ("bf16", 64, 128, 1, 300),
])
def test_write_and_read(dtype, d, page, H_kv, T):
    dt = DT[dtype]
    K, V = _rows(1, T, H_kv, d, dt), _rows(2, T, H_kv, d, dt)
    pages = -(-T // page) + 2
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(3))[:T]
    slots[T // 2] = -1
    Kc, Vc, Ke, Ve = _empty_cache(pages, page, H_kv, d)
    fa.fa_paged_write_q8(K, V, slots.cuda(), Kc, Vc, Ke, Ve)
    assert _errors() == ""
    live = [t for t in range(T) if t != T // 2]
    for x, c, e in ((K, Kc, Ke), (V, Vc, Ve)):
        code, exp = dr.quantise(x)
        want = torch.full((pages * page, H_kv, d), 0x31, dtype=torch.uint8)
        want_e = torch.full((pages * page, H_kv), 120, dtype=torch.uint8)
        want[slots[live]], want_e[slots[live]] = code[live], exp[live]
        got = c.view(torch.uint8).view(-1, H_kv, d).cpu()
        nan = (want & 127) == 127
        assert torch.equal((got & 127) == 127, nan)
        assert torch.equal(torch.where(nan, 0, got), torch.where(nan, 0, want))
        assert torch.equal(e.transpose(1, 2).reshape(-1, H_kv).cpu(), want_e)
    # back: exactly the values the numbers stand for; -1 and the same slot twice
    ask = torch.cat([slots, slots[:1], torch.tensor([-1])])
    k, v = fa.fa_paged_read_q8(Kc, Vc, Ke, Ve, ask.cuda(), dt)
    assert _errors() == ""
    for got, c, e in ((k, Kc, Ke), (v, Vc, Ve)):
        want = torch.where((ask >= 0)[:, None, None], dr.values(c, e).view(-1, H_kv, d)[ask.clamp(min=0)], 0.0)
        assert torch.equal(torch.nan_to_num(got.double().cpu(), nan=12345.0), torch.nan_to_num(want, nan=12345.0))


def test_write_error_bound():
    """Off by half a step of an e4m3 number at most, 2^-4 of the element or 2^-10 of the row's unit."""
    T, H_kv, d, page = 64, 4, 128, 16
    for dt in DT.values():
        K = _rand(5, (T, H_kv, d), dt)
        Kc, Vc, Ke, Ve = _empty_cache(T // page, page, H_kv, d)
        slots = torch.arange(T, device="cuda")
        fa.fa_paged_write_q8(K, K, slots, Kc, Vc, Ke, Ve)
        k, v = fa.fa_paged_read_q8(Kc, Vc, Ke, Ve, slots, dt)
        assert torch.equal(k, v)
        unit = K.double().abs().amax(-1, keepdim=True) / 224.0  # 2^e is less than that
        err = (k.double() - K.double()).abs()
        assert (err <= torch.maximum(K.double().abs() * 2.0 ** -4, unit * 2.0 ** -10)).all()


def test_write_and_read_strided():
    """Slices of a joint projection into head-major caches, and back into a strided output."""
    T, H_kv, d, page, pages = 45, 2, 64, 16, 5
    joint = _rand(1, (T, 3 * H_kv, d), torch.bfloat16)
    K, V = joint[:, :H_kv], joint[:, H_kv:2 * H_kv]
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(2))[:T].cuda()
    dense = _empty_cache(pages, page, H_kv, d)
    fa.fa_paged_write_q8(K.contiguous(), V.contiguous(), slots, *dense)
    byte = lambda t: t.view(torch.uint8)
    hm = [byte(c).transpose(1, 2).contiguous().transpose(1, 2).view(F8) for c in _empty_cache(pages, page, H_kv, d)[:2]]
    exps = _empty_cache(pages, page, H_kv, d)[2:]
    fa.fa_paged_write_q8(K, V, slots, *hm, *exps)
    for a, b in zip(dense, hm + exps):
        assert torch.equal(byte(a), byte(b)) if a.dtype == F8 else torch.equal(a, b)
    out = torch.zeros(T, 3 * H_kv, d, dtype=torch.bfloat16, device="cuda")
    fa.fa_paged_read_q8(*hm, *exps, slots, K=out[:, :H_kv], V=out[:, 2 * H_kv:])
    k, v = fa.fa_paged_read_q8(*dense, slots)
    assert torch.equal(out[:, :H_kv], k) and torch.equal(out[:, 2 * H_kv:], v) and (out[:, H_kv:2 * H_kv] == 0).all()
    assert _errors() == ""


def test_slots_outside_the_cache():
    T, H_kv, d, page, pages = 6, 2, 64, 4, 2
    K = _rand(1, (T, H_kv, d), torch.bfloat16)
    cache = _empty_cache(pages, page, H_kv, d)
    slots = torch.tensor([0, 8, 3, -5, 7, 2 ** 40], device="cuda")
    fa.fa_paged_write_q8(K, K, slots, *cache)
    assert "slot" in _errors()
    code, _ = dr.quantise(K)
    want = torch.full((8, H_kv, d), 0x31, dtype=torch.uint8)
    for t, s in ((0, 0), (2, 3), (4, 7)):
        want[s] = code[t]
    assert torch.equal(cache[0].view(torch.uint8).view(8, H_kv, d).cpu(), want)
    k, v = fa.fa_paged_read_q8(*cache, slots)
    assert "slot" in _errors()
    assert (k[[1, 3, 5]] == 0).all() and (v[[1, 3, 5]] == 0).all() and (k[0] != 0).any()
    for t in fa.fa_paged_read_q8(*cache, slots[:0]):
        assert t.shape == (0, H_kv, d)
    fa.fa_paged_write_q8(K[:0], K[:0], slots[:0], *cache)
    assert _errors() == ""


def _setup(seed, new, ctx, H, H_kv, d, page, dtype, spread=3):
    """An 8-bit cache of rows of many sizes, tables in any order, NaN numbers on pages of no request."""
    total = [a + b for a, b in zip(new, ctx)]
    need = [-(-t // page) for t in total]
    pages = sum(need) + 2
    Kc, Vc, Ke, Ve = _empty_cache(pages, page, H_kv, d, fill=0x7f)
    g = torch.Generator().manual_seed(seed)
    order = torch.randperm(pages, generator=g)
    table = torch.full((len(new), max(max(need), 1)), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n].int()
        at += n
    rows = [_rand(seed + 1 + i, (sum(total), H_kv, d), torch.float32) for i in range(2)]
    rows = [(x * torch.exp2(torch.randint(-spread, spread + 1, (sum(total), H_kv, 1), generator=g).float()).cuda() * 0.5).to(dtype)
            for x in rows]
    slots = torch.cat([table[i].long()[torch.arange(t) // page] * page + torch.arange(t) % page for i, t in enumerate(total)])
    fa.fa_paged_write_q8(*rows, slots.cuda(), Kc, Vc, Ke, Ve)
    Q = _rand(seed + 5, (sum(new), H, d), dtype)
    return Q, (Kc, Vc), (Ke, Ve), table.cuda(), torch.tensor(total, dtype=torch.int32).cuda()


def _check(O, LSE, Q, caches, exps, table, new, total, dtype, causal=True, window=0, p_step=0.0):
    """p_step: by how much a P is off at most where that is more than u P; with the row sum at least 1 it moves
    O by p_step times the sum of |V| over the keys that the row sees."""
    page, d = caches[0].shape[1], Q.shape[2]
    vals = [dr.values(c, e) for c, e in zip(caches, exps)]
    a = 0
    for i, (nq, nk) in enumerate(zip(new, total)):
        k, v = (ref.gather_pages(x, table[i].cpu(), nk, page) for x in vals)
        o, lse, mag, e = ref.attend(Q[a:a + nq].double().cpu(), k, v, causal, window, 1 / math.sqrt(d))
        size = torch.zeros_like(mag)
        if p_step:
            seen = torch.einsum("ij,jhc->ihc", ref.visible(nq, nk, causal, window).double(), v.abs())
            size = seen.repeat_interleave(Q.shape[1] // v.shape[1], 1) * p_step / e
        ref.check(f"O of request {i} ({nq} over {nk})", O[a:a + nq], o, mag, e, dtype, f32=mag + size)
        ref.check_lse(LSE[:, a:a + nq], lse, e)
        a += nq


ATTEND = [
    ("bf16", 8, 2, 128, 16), ("f16", 4, 4, 64, 32), ("bf16", 4, 1, 128, 128), ("f16", 16, 2, 128, 8), ("bf16", 6, 2, 256, 16),
    ("f16", 2, 2, 32, 16), ("bf16", 7, 1, 96, 64), ("f32", 4, 2, 64, 16), ("bf16", 4, 2, 128, 5), ("f32", 4, 1, 128, 3),
    ("bf16", 32, 1, 64, 16), ("f16", 130, 1, 64, 16), ("bf16", 5, 5, 128, 256), ("f16", 40, 2, 256, 64), ("bf16", 8, 1, 128, 24),
]
NEWS = [
    ([1], [0]), ([1, 1, 1, 1], [0, 15, 16, 500]), ([1, 0, 3, 1], [127, 40, 128, 255]), ([5, 1, 40, 0, 2], [0, 300, 77, 9, 129]),
    ([130, 1, 17], [3, 1000, 250]),
]


@pytest.mark.parametrize("dtype,H,H_kv,d,page", ATTEND)
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 40), (False, 0), (False, 30)])
def test_attend(dtype, H, H_kv, d, page, causal, window):
    dt = DT[dtype]
    for n, (new, ctx) in enumerate(NEWS):
        if H > 100 and sum(new) > 100:
            continue
        Q, caches, exps, table, lens = _setup(10 * n, new, ctx, H, H_kv, d, page, dt)
        O, LSE = fa.fa_paged_fwd(Q, *caches, table, _cu(new), lens, causal=causal, window_size=window, K_exp=exps[0], V_exp=exps[1])
        assert _errors() == ""
        _check(O, LSE, Q, caches, exps, table, new, lens.tolist(), dt, causal, window)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("new,ctx", [([1], [20000]), ([1] * 40, [37 * i % 900 for i in range(40)]), ([4, 1], [9000, 3]), ([300], [5000])])
def test_attend_split(dtype, new, ctx):
    """Long caches are cut over the CTAs and joined; twice the same bits; outputs passed in."""
    dt = DT[dtype]
    Q, caches, exps, table, lens = _setup(3, new, ctx, 8, 2, 128, 16, dt)
    args = (Q, *caches, table, _cu(new), lens)
    O, LSE = fa.fa_paged_fwd(*args, K_exp=exps[0], V_exp=exps[1])
    O2, LSE2 = torch.full_like(O, 3.0), torch.full_like(LSE, 4.0)
    fa.fa_paged_fwd(*args, O=O2, LSE=LSE2, K_exp=exps[0], V_exp=exps[1])
    assert _errors() == ""
    assert torch.equal(O, O2) and torch.equal(LSE, LSE2)
    _check(O, LSE, Q, caches, exps, table, new, lens.tolist(), dt)


def test_exponents_of_all_sizes():
    """Rows whose sizes differ by 2^20 and more, zero rows among them: each row counts with its own exponent."""
    new, ctx, H, H_kv, d, page = [1, 3], [700, 260], 8, 2, 128, 16
    for dt in (torch.bfloat16, torch.float16):
        Q, caches, exps, table, lens = _setup(7, new, ctx, H, H_kv, d, page, dt, spread=0)
        g = torch.Generator().manual_seed(1)
        lo, hi = (97, 157) if dt == torch.bfloat16 else (112, 122)
        for e, c in zip(exps, caches):
            e.copy_(torch.randint(lo, hi + 1, e.shape, generator=g).to(torch.uint8))
        # K of one size: scores of all sizes would leave one key each
        exps[0].fill_(120)
        caches[1].view(torch.uint8)[:, ::3] = 0
        Q, c = Q * 0.125, (caches[0], caches[1])
        c[0].view(torch.uint8).masked_fill_(c[0].view(torch.uint8) & 127 == 127, 0)
        c[1].view(torch.uint8).masked_fill_(c[1].view(torch.uint8) & 127 == 127, 0)
        O, LSE = fa.fa_paged_fwd(Q, *c, table, _cu(new), lens, K_exp=exps[0], V_exp=exps[1])
        assert _errors() == ""
        _check(O, LSE, Q, c, exps, table, new, lens.tolist(), dt)


def test_small_and_large_queries():
    """Rows of Q of any size in their type: the kernels' own scaling of them does not show."""
    new, ctx, H, H_kv, d, page = [2, 1], [50, 333], 4, 2, 128, 16
    for size in (1e-30, 1e-6, 1.0, 1e6, 1e30):
        dt = torch.bfloat16
        Q, caches, exps, table, lens = _setup(7, new, ctx, H, H_kv, d, page, dt, spread=1)
        Q = Q * size
        scale = min(d ** -0.5 / size, 3e38)
        O, LSE = fa.fa_paged_fwd(Q, *caches, table, _cu(new), lens, K_exp=exps[0], V_exp=exps[1], scale=scale)
        assert _errors() == ""
        a = 0
        vals = [dr.values(c, e) for c, e in zip(caches, exps)]
        for i, (nq, nk) in enumerate(zip(new, lens.tolist())):
            k, v = (ref.gather_pages(x, table[i].cpu(), nk, page) for x in vals)
            o, lse, mag, e = ref.attend(Q[a:a + nq].double().cpu(), k, v, True, 0, scale)
            ref.check("O", O[a:a + nq], o, mag, e, dt)
            ref.check_lse(LSE[:, a:a + nq], lse, e)
            a += nq


@pytest.mark.parametrize("dtype,H,page", [("bf16", 8, 16), ("f32", 8, 16), ("f16", 64, 16)])
def test_nan_reaches_the_rows_that_see_it(dtype, H, page):
    """A NaN number in K or V shows in the requests that see it and in no other."""
    dt, new, ctx, H_kv, d = DT[dtype], [1, 1, 2], [40, 300, 20], 2, 64
    for which in range(2):
        Q, caches, exps, table, lens = _setup(2, new, ctx, H, H_kv, d, page, dt)
        caches[which].view(torch.uint8)[int(table[1, 3]), 2, 1, 5] = 0x7f
        O, LSE = fa.fa_paged_fwd(Q, *caches, table, _cu(new), lens, K_exp=exps[0], V_exp=exps[1])
        assert _errors() == ""
        g = H // H_kv
        hit = O[1, g:]
        assert torch.isnan(hit).all() if which == 0 else torch.isnan(hit[:, 5]).all()
        assert torch.isnan(LSE[g:, 1]).all() == (which == 0)
        rest = torch.cat([O[:1], O[2:]])
        assert torch.isfinite(rest).all() and torch.isfinite(O[1, :g]).all()


def test_bad_pages_and_lengths_are_reported():
    new, ctx, H, H_kv, d, page = [1, 2], [100, 40], 4, 2, 64, 16
    for dt in (torch.bfloat16, torch.float32):
        Q, caches, exps, table, lens = _setup(2, new, ctx, H, H_kv, d, page, dt)
        good = fa.fa_paged_fwd(Q, *caches, table, _cu(new), lens, K_exp=exps[0], V_exp=exps[1])
        assert _errors() == ""
        for entry in (-1, caches[0].shape[0], 2 ** 31 - 1):
            t = table.clone()
            t[0, 2] = entry
            O, LSE = fa.fa_paged_fwd(Q, *caches, t, _cu(new), lens, K_exp=exps[0], V_exp=exps[1])
            assert "page" in _errors()
            assert torch.equal(O[1:], good[0][1:]) and torch.isfinite(O).all()
        # a window that leaves the page out does not look at it
        O, LSE = fa.fa_paged_fwd(Q, *caches, t, _cu(new), lens, window_size=20, K_exp=exps[0], V_exp=exps[1])
        assert _errors() == ""
        # longer than the table
        O, LSE = fa.fa_paged_fwd(Q, *caches, table[:, :3].contiguous(), _cu(new), lens, K_exp=exps[0], V_exp=exps[1])
        assert "lengths" in _errors()
        assert torch.equal(O[1:], good[0][1:])
        # lengths that do not fit: nothing is computed, new outputs are set
        O, LSE = fa.fa_paged_fwd(Q, *caches, table, torch.tensor([0, 3, 2], dtype=torch.int32, device="cuda"), lens,
                                 K_exp=exps[0], V_exp=exps[1])
        assert "lengths" in _errors()
        assert (O == 0).all() and (LSE == -math.inf).all()


def test_another_stream_and_captured():
    """On a stream of its own, and captured with lengths that change between replays."""
    new, H, H_kv, d, page, dt = [1, 1, 1], 8, 2, 128, 16, torch.bfloat16
    Q, caches, exps, table, lens = _setup(4, new, [300, 20, 150], H, H_kv, d, page, dt)
    cu = _cu(new)
    want = fa.fa_paged_fwd(Q, *caches, table, cu, lens, K_exp=exps[0], V_exp=exps[1])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = fa.fa_paged_fwd(Q, *caches, table, cu, lens, K_exp=exps[0], V_exp=exps[1], stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        O, LSE = fa.fa_paged_fwd(Q, *caches, table, cu, lens, K_exp=exps[0], V_exp=exps[1])
    for cut in ([0, 0, 0], [250, 3, 1], [299, 19, 149], [0, 20, 0]):
        short = lens - torch.tensor(cut, dtype=torch.int32, device="cuda")
        keep = lens.clone()
        want = fa.fa_paged_fwd(Q, *caches, table, cu, short, K_exp=exps[0], V_exp=exps[1])
        lens.copy_(short)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(O, want[0]) and torch.equal(LSE, want[1])
        lens.copy_(keep)
    assert _errors() == ""


def test_head_major_cache():
    new, ctx, H, H_kv, d, page, dt = [1, 7], [200, 90], 8, 2, 128, 16, torch.bfloat16
    Q, caches, exps, table, lens = _setup(6, new, ctx, H, H_kv, d, page, dt)
    hm = [c.view(torch.uint8).transpose(1, 2).contiguous().transpose(1, 2).view(F8) for c in caches]
    a = fa.fa_paged_fwd(Q, *caches, table, _cu(new), lens, K_exp=exps[0], V_exp=exps[1])
    b = fa.fa_paged_fwd(Q, *hm, table, _cu(new), lens, K_exp=exps[0], V_exp=exps[1])
    assert _errors() == ""
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype,page", [("bf16", 16), ("f32", 24)])
def test_offsets_past_32_bits(dtype, page):
    """Caches of more than 2^32 bytes each, a request on their last pages."""
    dt, H, H_kv, d = DT[dtype], 8, 8, 128
    pages = 2 ** 32 // (page * H_kv * d) + 40
    caches = [torch.zeros(pages, page, H_kv, d, dtype=torch.uint8, device="cuda").view(F8) for _ in "KV"]
    exps = [torch.zeros(pages, H_kv, page, dtype=torch.uint8, device="cuda") for _ in "KV"]
    nk = 15 * page + 3
    table = (pages - 1 - torch.arange(16)).to(torch.int32)[None].cuda()
    K, V = _rand(1, (nk, H_kv, d), dt), _rand(2, (nk, H_kv, d), dt)
    j = torch.arange(nk).cuda()
    slots = table[0].long()[j // page] * page + j % page
    fa.fa_paged_write_q8(K, V, slots, *caches, *exps)
    lens = torch.tensor([nk], dtype=torch.int32, device="cuda")
    for nq in (1, 70):
        Q = _rand(3, (nq, H, d), dt)
        O, LSE = fa.fa_paged_fwd(Q, *caches, table, _cu([nq]), lens, K_exp=exps[0], V_exp=exps[1])
        assert _errors() == ""
        small = [c[-16:].flip(0).contiguous() if c.dtype == torch.uint8 else c.view(torch.uint8)[-16:].flip(0).contiguous().view(F8)
                 for c in caches + exps]
        t = torch.arange(16, dtype=torch.int32, device="cuda")[None]
        want = fa.fa_paged_fwd(Q, small[0], small[1], t, _cu([nq]), lens, K_exp=small[2], V_exp=small[3])
        assert torch.equal(O, want[0]) and torch.equal(LSE, want[1])
    k, v = fa.fa_paged_read_q8(*caches, *exps, slots, dt)
    code, exp = dr.quantise(K)
    assert torch.equal(k.double().cpu(), dr.numbers(code) * (2.0 ** (exp.double() - 127))[..., None])
