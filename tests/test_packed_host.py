"""Refusals of the packed and paged calls on the host (no GPU needed): nothing is enqueued, so
the pointers below are never dereferenced.  And the page look-up that every kernel goes through."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import flashattention_backward_preprocess_gb300 as fa
from flashattention_backward_preprocess_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = [0x10000 * (i + 1) for i in range(12)]


@pytest.fixture(scope="module")
def lib():
    build.build()
    return fa.load_library()


def _arr(x):
    return None if x is None else (ctypes.c_longlong * len(x))(*x)


def _varlen(lib, **kw):
    a = dict(Q=P[0], K=P[1], V=P[2], O=P[3], LSE=P[4], cu_q=P[5], cu_k=P[6], N=3, T_q=100, T_k=100, H=4, H_kv=2, d=64,
             strides=None, scale=0.125, causal=1, window=0, fill=0, dtype=fa.FA_BF16, ws=P[7], ws_bytes=0, stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    a["strides"] = _arr(a["strides"])
    return lib.fa_varlen_fwd(*a.values())


def _varlen_bwd(lib, **kw):
    a = dict(dO=P[0], Q=P[1], K=P[2], V=P[3], O=P[4], LSE=P[5], dQ=P[6], dK=P[7], dV=P[8], cu_q=P[9], cu_k=P[10], N=3, T_q=100,
             T_k=100, H=4, H_kv=2, d=64, strides=None, scale=0.125, causal=1, window=0, det=0, fill=0, dtype=fa.FA_BF16,
             ws=P[11], ws_bytes=0, stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    a["strides"] = _arr(a["strides"])
    return lib.fa_varlen_bwd(*a.values())


def _paged(lib, **kw):
    a = dict(Q=P[0], K=P[1], V=P[2], O=P[3], LSE=P[4], table=P[5], cu_q=P[6], seq_lens=P[7], N=3, T_q=10, num_pages=50,
             page_size=16, max_pages=8, H=4, H_kv=2, d=64, strides=None, scale=0.125, causal=1, window=0, fill=0,
             dtype=fa.FA_BF16, ws=P[8], ws_bytes=0, stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    a["strides"] = _arr(a["strides"])
    return lib.fa_paged_fwd(*a.values())


def _slots(lib, **kw):
    a = dict(ctx=P[0], cu_q=P[1], free=P[2], start=P[3], table=P[4], slots=P[5], pos=P[6], lens=P[7], nxt=P[8], N=3, T=10,
             num_free=50, page_size=16, max_pages=8, stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    return lib.fa_page_slots(*a.values())


def _write(lib, **kw):
    a = dict(K=P[0], V=P[1], slots=P[2], Kc=P[3], Vc=P[4], T=10, num_pages=50, page_size=16, H_kv=2, d=64, strides=None,
             dtype=fa.FA_BF16, stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    a["strides"] = _arr(a["strides"])
    return lib.fa_paged_write(*a.values())


COMMON = [(dict(H=0), "H"), (dict(H_kv=3), "H_kv"), (dict(d=0), "d"), (dict(dtype=9), "dtype"), (dict(scale=0.0), "scale"),
          (dict(scale=float("nan")), "scale"), (dict(causal=2), "causal"), (dict(window=-1), "window_size"),
          (dict(fill=2), "fill"), (dict(N=0), "N"), (dict(Q=None), "Q"), (dict(Q=P[0] + 8), "Q"), (dict(O=None), "O"),
          (dict(LSE=P[4] + 2), "LSE"), (dict(cu_q=None), "cu_q"), (dict(T_q=-1), "T_q")]


@pytest.mark.parametrize("kw,arg", COMMON + [
    (dict(K=None), "K"), (dict(V=P[2] + 4), "V"), (dict(cu_k=None), "cu_k"), (dict(T_k=2 ** 30), "T_k"),
    (dict(strides=[256, 64, 128, 64, 128, 64, 256, 0]), "strides"),
    (dict(strides=[256, 64, 128, 64, 128, 60, 256, 64]), "strides"),
    (dict(strides=[-256, 64, 128, 64, 128, 64, 256, 64]), "strides")])
def test_varlen_fwd_refuses(lib, kw, arg):
    assert _varlen(lib, **kw) == 1, kw
    assert fa.fa_last_error().startswith(arg + ":"), fa.fa_last_error()


@pytest.mark.parametrize("kw,arg", COMMON + [
    (dict(K=None), "K_cache"), (dict(V=P[2] + 4), "V_cache"), (dict(table=None), "block_table"),
    (dict(seq_lens=None), "seq_lens"), (dict(num_pages=0), "num_pages"), (dict(page_size=0), "page_size"),
    (dict(max_pages=0), "max_pages"), (dict(strides=[256, 64, 2048, 128, 64, 2048, 128, 64, 256, 4]), "strides")])
def test_paged_fwd_refuses(lib, kw, arg):
    assert _paged(lib, **kw) == 1, kw
    assert fa.fa_last_error().startswith(arg + ":"), fa.fa_last_error()


@pytest.mark.parametrize("kw,arg", [c for c in COMMON if "O" not in c[0] and "LSE" not in c[0]] + [
    (dict(dO=None), "dO"), (dict(O=P[4] + 8), "O"), (dict(LSE=None), "LSE"), (dict(K=None), "K"), (dict(V=P[3] + 4), "V"),
    (dict(dQ=None), "dQ"), (dict(dK=P[7] + 2), "dK"), (dict(dV=None), "dV"), (dict(cu_k=P[10] + 2), "cu_k"), (dict(det=2), "deterministic"),
    (dict(T_k=-5), "T_k"), (dict(strides=[256, 64, 256, 64, 128, 64, 128, 64, 256, 64, 256, 64, 128, 64, 128, 4]), "strides")])
def test_varlen_bwd_refuses(lib, kw, arg):
    assert _varlen_bwd(lib, **kw) == 1, kw
    assert fa.fa_last_error().startswith(arg + ":"), fa.fa_last_error()


def test_unsupported_head_dim(lib):
    assert _varlen_bwd(lib, d=80) == 2
    assert _varlen(lib, d=80) == 2 and _paged(lib, d=48) == 2 and _write(lib, d=80) == 2
    assert lib.fa_varlen_workspace_bytes(3, 100, 100, 4, 2, 80, fa.FA_BF16, 0) == 0
    assert lib.fa_varlen_workspace_bytes(0, 100, 100, 4, 2, 64, fa.FA_BF16, 0) == 0
    assert lib.fa_paged_workspace_bytes(3, 100, 4, 3, 64, 16, fa.FA_BF16) == 0


def test_no_rows_is_no_work(lib):
    """Empty packed axes are valid and need no tensors."""
    assert _varlen(lib, T_q=0, Q=None, O=None, LSE=None) == 0
    assert _paged(lib, T_q=0, Q=None, O=None, LSE=None) == 0
    assert _write(lib, T=0, K=None, V=None, slots=None) == 0
    assert _varlen_bwd(lib, T_q=0, T_k=0, dO=None, Q=None, K=None, V=None, O=None, LSE=None, dQ=None, dK=None, dV=None) == 0


@pytest.mark.parametrize("kw,arg", [
    (dict(ctx=None), "ctx_lens"), (dict(cu_q=P[1] + 1), "cu_q"), (dict(start=None), "free_start"), (dict(free=None), "free_pages"),
    (dict(table=None), "block_table"), (dict(slots=P[5] + 4), "slots"), (dict(pos=None), "positions"), (dict(lens=None), "seq_lens"),
    (dict(nxt=None), "free_next"), (dict(N=0), "N"), (dict(T=-1), "T"), (dict(page_size=0), "page_size"),
    (dict(max_pages=0), "max_pages"), (dict(num_free=-1), "num_free")])
def test_page_slots_refuses(lib, kw, arg):
    assert _slots(lib, **kw) == 1, kw
    assert fa.fa_last_error().startswith(arg + ":"), fa.fa_last_error()


@pytest.mark.parametrize("out,of", [
    ("lens", P[0]), ("nxt", P[3]), ("slots", P[1]), ("pos", P[2] + 64), ("lens", P[1] + 4), ("table", P[0] - 4)])
def test_page_slots_refuses_outputs_over_inputs(lib, out, of):
    assert _slots(lib, **{out: of}) == 1
    assert "must not overlap" in fa.fa_last_error()


@pytest.mark.parametrize("kw,arg", [
    (dict(K=None), "K"), (dict(V=P[1] + 2), "V"), (dict(slots=None), "slots"), (dict(Kc=None), "K_cache"), (dict(Vc=P[4] + 8), "V_cache"),
    (dict(T=-1), "T"), (dict(num_pages=0), "num_pages"), (dict(page_size=-1), "page_size"), (dict(H_kv=0), "H"), (dict(dtype=5), "dtype"),
    (dict(strides=[128, 64, 128, 64, 2048, 128, 64, 2048, 130, 64]), "strides")])
def test_paged_write_refuses(lib, kw, arg):
    assert _write(lib, **kw) == 1, kw
    assert fa.fa_last_error().startswith(arg + ":"), fa.fa_last_error()


def test_binding_refuses_before_the_library():
    """Shapes, types and devices that the torch calls check themselves."""
    q, k = torch.zeros(5, 4, 64, dtype=torch.bfloat16), torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 5], dtype=torch.int32)
    cache, table, lens = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 2, dtype=torch.int32), torch.tensor([5], dtype=torch.int32)
    cases = [
        (lambda: fa.fa_varlen_fwd(q, k, k, cu, cu), "tensors"),
        (lambda: fa.fa_varlen_fwd(q[0], k, k, cu, cu), "Q"),
        (lambda: fa.fa_varlen_fwd(q, k.float(), k, cu, cu), "K"),
        (lambda: fa.fa_varlen_fwd(q, k, k[:3], cu, cu), "V"),
        (lambda: fa.fa_varlen_fwd(q, k[..., :32], k, cu, cu), "K"),
        (lambda: fa.fa_varlen_fwd(q, k, k, cu.long(), cu), "cu_q"),
        (lambda: fa.fa_varlen_fwd(q, k, k, cu, cu[:1]), "cu_k"),
        (lambda: fa.fa_varlen_fwd(q.transpose(1, 2), k, k, cu, cu), "K"),
        (lambda: fa.fa_varlen_bwd(q, q, k, k, q, torch.zeros(4, 6), cu, cu), "LSE"),
        (lambda: fa.fa_varlen_bwd(q[:4], q, k, k, q, torch.zeros(4, 5), cu, cu), "dO"),
        (lambda: fa.fa_varlen_bwd(q, q, k, k, q, torch.zeros(4, 5), cu, cu, dV=q), "dV"),
        (lambda: fa.fa_varlen_bwd(q, q, k, k, q, torch.zeros(4, 5), cu, cu), "tensors"),
        (lambda: fa.fa_paged_fwd(q, cache[0], cache, table, cu, lens), "K_cache"),
        (lambda: fa.fa_paged_fwd(q, cache, cache, table[0], cu, lens), "block_table"),
        (lambda: fa.fa_paged_fwd(q, cache, cache, table, cu, lens.long()), "seq_lens"),
        (lambda: fa.fa_paged_fwd(q, cache, cache, table, cu, lens), "tensors"),
        (lambda: fa.fa_page_slots(lens.long(), cu, table, lens, lens, 16, 5), "ctx_lens"),
        (lambda: fa.fa_page_slots(lens, cu, table, lens, lens, 16, -5), "tokens"),
        (lambda: fa.fa_paged_write(k, k, lens, cache, cache), "slots"),
        (lambda: fa.fa_paged_write(k, k, torch.zeros(5, dtype=torch.int64), cache[..., :32], cache[..., :32]), "K_cache"),
    ]
    for call, arg in cases:
        with pytest.raises(fa.FaError) as e:
            call()
        assert e.value.status == 1 and f" {arg}:" in str(e.value), (arg, str(e.value))


PROGRAM = r"""
#include <cstdio>
#include <climits>
#include "packed.cuh"
using namespace fa;
int main() {
    const int row[4] = {3, -1, 7, 0};
    struct { int j, page, max_pages, pages, id; bool bad; } c[] = {
        {0, 16, 4, 8, 3, false}, {15, 16, 4, 8, 3, false}, {16, 16, 4, 8, 8, true}, {47, 16, 4, 8, 7, false},
        {32, 16, 4, 7, 7, true},            // one past the cache
        {63, 16, 4, 8, 0, false}, {64, 16, 4, 8, 8, true},   // behind the table
        {INT_MAX, 1, 4, 8, 8, true}, {2, 1, 4, 8, 7, false}, {0, 1, 4, INT_MAX, 3, false}};
    for (auto& x : c) {
        bool bad = false;
        const int id = page_of(row, x.j, x.page, x.max_pages, x.pages, &bad);
        if (id != x.id || bad != x.bad) { printf("key %d: page %d bad %d\n", x.j, id, (int)bad); return 1; }
    }
    const int wild[2] = {INT_MIN, INT_MAX};
    for (int e = 0; e < 2; ++e) {
        bool bad = false;
        if (page_of(wild, e, 1, 2, 100, &bad) != 100 || !bad) return 2;
    }
    return 0;
}
"""


def test_page_look_up(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    src = tmp_path / "pages.cu"
    src.write_text(PROGRAM)
    exe = tmp_path / "pages"
    csrc = os.path.join(ROOT, "flashattention_backward_preprocess_gb300", "csrc")
    r = subprocess.run([nvcc, "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a", "-I", csrc, "-I",
                        os.path.join(ROOT, "include"), str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
