"""Refusals of the calls behind PagedKVCache.accept (no GPU needed)."""
import ctypes

import pytest
import torch

import flashattention_backward_preprocess_gb300 as fa
from flashattention_backward_preprocess_gb300 import build

P = [0x10000 * (i + 1) for i in range(9)]  # never dereferenced: checked before anything is launched
i32 = lambda *v: torch.tensor(v, dtype=torch.int32)


@pytest.mark.parametrize("kw,arg", [
    (dict(path=None), "path"), (dict(path=P[0] + 2), "path"), (dict(T=-1), "T"), (dict(count=None), "count"), (dict(free=None), "free_pages"),
    (dict(out=P[0] + 28), "lens"), (dict(next=P[0]), "free_next"), (dict(out=P[3]), "lens"), (dict(N=0), "N"), (dict(page=0), "page_size"),
    (dict(cols=0), "max_pages"), (dict(n_free=-1), "num_free"),
])
def test_library(kw, arg):
    build.build()
    a = dict(path=P[0], count=P[1], cu=P[2], lens=P[3], table=P[4], free=P[5], start=P[6], out=P[7], next=P[8], N=2, T=8, n_free=10,
             page=16, cols=2, stream=None)
    assert set(kw) <= set(a)
    assert fa.load_library().fa_page_trim_ex(*{**a, **kw}.values()) == 1
    assert fa.fa_last_error().startswith(arg + ":"), fa.fa_last_error()


@pytest.mark.parametrize("path,match", [(i32(0, 1).long(), "path"), (torch.zeros(2, 2, dtype=torch.int32)[:, 0], "path"), (i32(0), "device")])
def test_torch_call(path, match):
    with pytest.raises(fa.FaError, match=match):
        fa.fa_page_trim(i32(1), i32(0, 5), i32(5), torch.zeros(1, 2, dtype=torch.int32), i32(1, 2), i32(0), 16, path=path)


@pytest.mark.parametrize("K,V,Ke,Ve", [
    ((1, 2, 1), (3, 4, 5), None, None), ((1, 2, 3), (4, 2, 5), None, None), ((1, 2, 3), (4, 5, 6), (7, 8, 7), (9, 10, 11)),
    ((1, 2, 3), (4, 5, 6), (7, 8, 9), (10, 11, 8)), ((1, 2, 3), (4, 5, 6), (7, 8, 9), (10, 11, 1)),
])
def test_keep_refuses_a_tensor_given_twice(K, V, Ke, Ve):
    """Its rows would be moved by two blocks at once."""
    build.build()
    arr = lambda ps: None if ps is None else (ctypes.c_void_p * 3)(*(0x10000 * p for p in ps))
    rc = fa.load_library().fa_paged_keep(P[0], P[1], P[2], P[3], P[4], arr(K), arr(V), arr(Ke), arr(Ve), 3, 2, 8, 4, 16, 2, 2, 64, None,
                                         fa.FA_BF16, None)
    assert rc == 1
    assert fa.fa_last_error() == "K_caches: the same tensor is given twice"


@pytest.mark.parametrize("parents,words,match", [
    (i32(-1, 0, 1, 2), None, "parents"), (i32(-1, 0, 1, 2, 3, 4), None, "parents"), (i32(-1, 0, 1, 2, 3).long(), None, "parents"),
    (i32(-1, 0, 1, 2, 3), 0, "words"),
])
def test_begin_refuses_parents_before_anything_else(parents, words, match):
    cache = fa.PagedKVCache(1, 4, 16, 2, 64, 1, 4, device="cpu")
    with pytest.raises(fa.FaError, match=match):
        cache.begin(i32(0, 5), 5, parents=parents, words=words)
    assert cache.slots is None and cache.cu_q is None and cache.tree is None
