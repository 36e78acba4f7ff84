"""Arguments that the calls around an 8-bit cache and trees of drafted tokens refuse (no GPU needed)."""
import ctypes

import pytest
import torch

import flashattention_backward_preprocess_gb300 as fa
from flashattention_backward_preprocess_gb300 import build, packed

P = [0x10000 * (i + 1) for i in range(16)]  # never dereferenced: checked before anything is launched


@pytest.fixture(scope="module")
def lib():
    build.build()
    return fa.load_library()


def _says(rc, arg, status=1):
    assert rc == status, rc
    assert fa.fa_last_error().startswith(arg + ":"), fa.fa_last_error()


def _fwd(lib, **kw):
    a = dict(Q=P[0], K=P[1], V=P[2], K_exp=P[3], V_exp=P[4], O=P[5], LSE=P[6], table=P[7], cu=P[8], lens=P[9], tree=P[10], words=1,
             N=2, T_q=8, pages=4, page=16, cols=2, H=8, H_kv=2, d=64, strides=None, scale=0.1, causal=1, window=0, fill=1,
             dtype=fa.FA_BF16, ws=P[11], ws_bytes=0, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.fa_paged_fwd_ex(*a.values())


@pytest.mark.parametrize("kw,arg", [
    (dict(K_exp=None), "K_exp"), (dict(V_exp=None), "V_exp"), (dict(K_exp=P[3] + 8), "K_exp"), (dict(V_exp=P[4] + 1), "V_exp"),
    (dict(causal=0), "causal"), (dict(window=5), "window_size"), (dict(window=-1), "window_size"), (dict(words=0), "tree_words"),
    (dict(words=1025), "tree_words"), (dict(tree=P[10] + 4), "tree"), (dict(Q=None), "Q"), (dict(K=P[1] + 8), "K_cache"),
    (dict(table=None), "block_table"), (dict(page=0), "page_size"), (dict(H=7), "H_kv"), (dict(T_q=-1), "T_q"),
    (dict(cols=0), "max_pages"), (dict(scale=0.0), "scale"), (dict(dtype=3), "dtype"),
])
def test_fwd_ex(lib, kw, arg):
    _says(_fwd(lib, **kw), arg)


def test_fwd_ex_strides_and_heads(lib):
    dense = [8 * 64, 64, 2 * 64 * 16, 128, 64, 2 * 64 * 16, 128, 64, 8 * 64, 64]
    # 8-bit entries count bytes: 8 elements are a whole piece of Q, half a piece of the cache
    for i, ok in ((1, True), (4, False), (7, False), (9, True)):
        s = list(dense)
        s[i] = 8
        rc = _fwd(lib, strides=(ctypes.c_longlong * 10)(*s), ws=None) if not ok else 0
        if not ok:
            _says(rc, "strides")
    _says(_fwd(lib, d=80), "d", 2)
    assert _fwd(lib, T_q=0) == 0
    need = lib.fa_paged_workspace_bytes_ex(2, 8, 8, 2, 64, 16, 2, fa.FA_BF16, 1)
    assert need > 0 and lib.fa_paged_workspace_bytes_ex(2, 8, 8, 3, 64, 16, 2, fa.FA_BF16, 1) == 0
    assert lib.fa_paged_workspace_bytes_ex(2, 8, 8, 2, 64, 16, 2, fa.FA_BF16, 0) == lib.fa_paged_workspace_bytes(2, 8, 8, 2, 64, 16, fa.FA_BF16)


def test_copy_of_the_rows_has_a_bound(lib):
    """Many rows per request: room for all that the tables name, up to 2 GB each of K and V."""
    at = lambda cols, T: lib.fa_paged_workspace_bytes_ex(4, T, 32, 8, 128, 16, cols, fa.FA_BF16, 1)
    few, many = at(512, 100), at(512, 4096)
    copy = 2 * 4 * 512 * 16 * 8 * 128 * 2
    assert few < 64 << 20 and copy < many < copy + (64 << 20)
    assert at(1 << 20, 4096) < 64 << 20


def test_write_and_read_q8(lib):
    w = lambda **kw: lib.fa_paged_write_q8(*{**dict(K=P[0], V=P[1], slots=P[2], Kc=P[3], Vc=P[4], Ke=P[5], Ve=P[6], T=3, pages=2, page=16,
                                                    H=2, d=64, st=None, dt=fa.FA_F16, s=None), **kw}.values())
    for kw, arg in ((dict(K=None), "K"), (dict(slots=P[2] + 4), "slots"), (dict(Kc=P[3] + 4), "K_cache"), (dict(Ke=None), "K_exp"),
                    (dict(Ve=P[6] + 2), "V_exp"), (dict(T=-1), "T"), (dict(pages=0), "num_pages"), (dict(page=0), "page_size"),
                    (dict(dt=9), "dtype"), (dict(H=0), "H")):
        _says(w(**kw), arg)
    _says(w(d=48), "d", 2)
    assert w(T=0) == 0
    _says(lib.fa_paged_read_q8(P[0], P[1], P[2], P[3], P[4], P[5], None, 3, 2, 16, 2, 64, None, fa.FA_F16, None), "V")


def test_tree_mask(lib):
    t = lambda **kw: lib.fa_tree_mask(*{**dict(up=P[0], cu=P[1], ctx=P[2], tree=P[3], pos=P[4], N=2, T=8, words=1, s=None), **kw}.values())
    for kw, arg in ((dict(up=None), "parents"), (dict(tree=P[3] + 4), "tree"), (dict(pos=None), "positions"), (dict(words=0), "words"),
                    (dict(words=2000), "words"), (dict(N=0), "N"), (dict(T=-2), "T"), (dict(tree=P[0]), "tree"), (dict(pos=P[0] + 28), "positions")):
        _says(t(**kw), arg)
    assert t(T=0) == 0


def test_keep_and_trim(lib):
    arr = lambda *p: (ctypes.c_void_p * len(p))(*p)
    k = lambda **kw: lib.fa_paged_keep(*{**dict(path=P[0], count=P[1], cu=P[2], lens=P[3], table=P[4], K=arr(P[5], P[6]), V=arr(P[7], P[8]),
                                                Ke=None, Ve=None, layers=2, N=2, T=8, pages=4, page=16, cols=2, H=2, d=64, st=None,
                                                dt=fa.FA_BF16, s=None), **kw}.values())
    for kw, arg in ((dict(path=None), "path"), (dict(K=None), "K_caches"), (dict(K=arr(P[5], None)), "K_caches"),
                    (dict(V=arr(P[7] + 8, P[8])), "V_caches"), (dict(Ke=arr(P[9], P[10])), "V_exps"), (dict(layers=0), "layers"),
                    (dict(Ke=arr(P[9], P[10]), Ve=arr(P[9], P[10] + 1)), "V_exps"), (dict(N=0), "N"), (dict(cols=0), "max_pages")):
        _says(k(**kw), arg)
    assert k(T=0) == 0
    t = lambda **kw: lib.fa_page_trim(*{**dict(count=P[0], cu=P[1], lens=P[2], table=P[3], free=P[4], start=P[5], out=P[6], next=P[7], N=2,
                                               n_free=10, page=16, cols=2, s=None), **kw}.values())
    for kw, arg in ((dict(count=None), "count"), (dict(free=None), "free_pages"), (dict(out=P[2]), "lens"), (dict(next=P[5]), "free_next"),
                    (dict(free=P[3] + 8), "free_pages"), (dict(N=0), "N"), (dict(page=0), "page_size"), (dict(n_free=-1), "num_free")):
        _says(t(**kw), arg)


# ---- the torch calls: shapes, types and devices
q = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
kv = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
i32 = lambda *v: torch.tensor(v, dtype=torch.int32)
cu, table, lens = i32(0, 5), torch.zeros(1, 2, dtype=torch.int32), i32(5)
cache = torch.zeros(3, 16, 2, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
exps = torch.zeros(3, 2, 16, dtype=torch.uint8)
slots = torch.arange(5)
plain = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)


@pytest.mark.parametrize("call,match", [
    (lambda: fa.fa_paged_fwd(q, cache, cache, table, cu, lens, K_exp=exps), "V_exp"),
    (lambda: fa.fa_paged_fwd(q, cache, cache, table, cu, lens), "K_cache"),
    (lambda: fa.fa_paged_fwd(q, plain, plain, table, cu, lens, K_exp=exps, V_exp=exps), "K_cache"),
    (lambda: fa.fa_paged_fwd(q, cache, cache, table, cu, lens, K_exp=exps, V_exp=exps.transpose(1, 2)), "V_exp"),
    (lambda: fa.fa_paged_fwd(q, cache, cache, table, cu, lens, K_exp=exps.int(), V_exp=exps), "K_exp"),
    (lambda: fa.fa_paged_fwd(q, plain, plain, table, cu, lens, tree=torch.zeros(4, 1, dtype=torch.int64)), "tree"),
    (lambda: fa.fa_paged_fwd(q, plain, plain, table, cu, lens, tree=torch.zeros(5, dtype=torch.int64)), "tree"),
    (lambda: fa.fa_paged_fwd(q, plain, plain, table, cu, lens, tree=torch.zeros(5, 1, dtype=torch.int32)), "tree"),
    (lambda: fa.fa_paged_write_q8(kv, kv, slots, plain, plain, exps, exps), "K_cache"),
    (lambda: fa.fa_paged_write_q8(kv, kv[:4], slots, cache, cache, exps, exps), "V"),
    (lambda: fa.fa_paged_write_q8(kv, kv, slots.int(), cache, cache, exps, exps), "slots"),
    (lambda: fa.fa_paged_write_q8(kv.double(), kv.double(), slots, cache, cache, exps, exps), "dtype"),
    (lambda: fa.fa_paged_read_q8(cache, cache, exps, exps, slots, torch.float64), "dtype"),
    (lambda: fa.fa_paged_read_q8(cache, cache, exps, exps, slots, torch.float32, K=kv), "K"),
    (lambda: fa.fa_paged_read_q8(cache, cache, exps, None, slots), "V_exp"),
    (lambda: fa.fa_tree_mask(i32(-1), cu, lens, 0), "words"),
    (lambda: fa.fa_tree_mask(i32(-1), cu, lens, 2 ** 32 + 1), "words"),
    (lambda: fa.fa_tree_mask(i32(-1).long(), cu, lens), "parents"),
    (lambda: fa.fa_tree_mask(i32(-1), cu, i32(1, 2)), "ctx_lens"),
    (lambda: fa.fa_tree_mask(i32(-1), cu, lens, 1, tree=torch.zeros(2, 1, dtype=torch.int64)), "tree"),
    (lambda: fa.fa_paged_keep(i32(0), i32(1), cu, lens, table, [], []), "V_caches"),
    (lambda: fa.fa_paged_keep(i32(0), i32(1), cu, lens, table, [plain], [plain, plain]), "V_caches"),
    (lambda: fa.fa_paged_keep(i32(0), i32(1), cu, lens, table, [plain, plain[:2]], [plain, plain]), "K_caches"),
    (lambda: fa.fa_paged_keep(i32(0), i32(1), cu, lens, table, [plain, plain.transpose(1, 2).contiguous().transpose(1, 2)],
                              [plain, plain]), "K_caches"),
    (lambda: fa.fa_paged_keep(i32(0), i32(1), cu, lens, table, [cache], [cache], [exps]), "K_exps"),
    (lambda: fa.fa_paged_keep(i32(0), i32(1, 2), cu, lens, table, [plain], [plain]), "count"),
    (lambda: fa.fa_page_trim(i32(1), cu, lens, table, i32(1, 2), i32(0), 2 ** 32), "page_size"),
    (lambda: fa.fa_page_trim(i32(1), cu, lens, table, i32(1, 2).long(), i32(0), 16), "free_pages"),
    # everything right but the device
    (lambda: fa.fa_paged_write_q8(kv, kv, slots, cache, cache, exps, exps), "device pointers"),
    (lambda: fa.fa_paged_read_q8(cache, cache, exps, exps, slots), "device pointers"),
    (lambda: fa.fa_tree_mask(i32(-1), cu, lens), "device pointers"),
    (lambda: fa.fa_paged_keep(i32(0), i32(1), cu, lens, table, [plain], [plain]), "device pointers"),
    (lambda: fa.fa_page_trim(i32(1), cu, lens, table, i32(1, 2), i32(0), 16), "device pointers"),
])
def test_torch_calls(call, match):
    with pytest.raises(fa.FaError, match=match):
        call()


def test_cache_out_of_order():
    c = fa.PagedKVCache(1, 4, 16, 2, 64, 1, 4, device="cpu", quantised=True)
    assert c.K[0].dtype == torch.float8_e4m3fn and c.K_exp[0].shape == (4, 2, 16)
    with pytest.raises(fa.FaError, match="begin"):
        c.attend(0, q, kv, kv)
    with pytest.raises(fa.FaError, match="begin"):
        c.accept(i32(0), i32(1))
