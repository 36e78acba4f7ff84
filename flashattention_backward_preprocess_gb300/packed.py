"""Packed (variable-length) and paged attention: the entry points of include/fa.h that
take sequences of different lengths, as torch calls.

Tensors are token major: Q [T, H, d], K and V [T, H_kv, d], caches [pages, page_size, H_kv, d].
Any strides that are whole 16-byte pieces are taken as they are (slices of a joint QKV
projection, transposed caches); the head dimension is contiguous.  Lengths stay on the device:
no call here waits for the GPU.  Outputs that the caller does not pass are allocated, with the
rows of no sequence set to 0 (LSE: -inf); outputs passed in keep those rows as they were.
Scratch comes from PyTorch's allocator, one block per call, so calls on different streams and
captured graphs do not share it.

The calls are short beside their own checks when a step has few tokens, so the checks are
written for the common case (dense tensors, current device and stream) first.
"""
from __future__ import annotations

import ctypes
import functools
import math

import torch

from .binding import _DT, FaError, _check, load_library

_I32, _I64, _F32, _U8 = torch.int32, torch.int64, torch.float32, torch.uint8
_empty, _empty_like, _Tensor = torch.empty, torch.empty_like, torch.Tensor
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else (
    lambda i: torch.cuda.current_stream(i).cuda_stream)


def _scale(scale, d):
    if scale is None:
        return max(d, 1) ** -0.5  # the library refuses d = 0
    return float(scale)


def _refuse(name, reason):
    raise FaError(1, f"{name}: {reason}")


def _int32(name, v):
    """v as the C int it is passed as (ctypes would wrap it around)."""
    v = int(v)
    if not -2 ** 31 <= v < 2 ** 31:
        _refuse(name, f"must fit 32 bits, got {v}")
    return v


def _type(t):
    dt = _DT.get(t.dtype)
    if dt is None:
        _refuse("dtype", f"unsupported dtype {t.dtype}")
    return dt


def _same(name, t, shape, dtype):
    if t.shape != shape:
        _refuse(name, f"expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        _refuse(name, f"expected {dtype}, got {t.dtype}")


def _ints(name, t, shape, dtype=_I32):
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        _refuse(name, f"must be contiguous {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")


def _lse(t, shape):
    if t.shape != shape or t.dtype != _F32 or not t.is_contiguous():
        _refuse("LSE", f"must be contiguous float32 {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")


def _strides(*named):
    """Element strides of all but the last dimension of each (name, tensor)."""
    flat = []
    for name, t in named:
        if t.is_contiguous():
            size, dense = 1, []
            for n in reversed(t.shape[1:]):
                size *= n
                dense.append(max(size, 1))
            flat += reversed(dense)
            continue
        st = t.stride()
        if st[-1] != 1 and t.shape[-1] != 1:
            _refuse(name, "the head dimension must be contiguous")
        flat += [s if n > 1 else t.shape[-1] for s, n in zip(st[:-1], t.shape[:-1])]
    return (ctypes.c_longlong * len(flat))(*flat)


def _device(first, *rest):
    """The one CUDA device all given tensors are on."""
    dev = first.device
    i = first.get_device()
    for t in rest:
        if t is not None and t.get_device() != i:
            _refuse("tensors", f"expected one device, got {dev} and {t.device}")
    if not first.is_cuda:
        _refuse("tensors", f"device pointers required, got {dev}")
    return dev


def _call(dev, stream, body):
    """body(raw stream) with `dev` and `stream` as the current ones."""
    if stream is None:
        if dev.index == _current_device():
            return body(_raw_stream(dev.index))
        with torch.cuda.device(dev):
            return body(_raw_stream(dev.index))
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=dev)
    with torch.cuda.device(dev), torch.cuda.stream(stream):
        return body(stream.cuda_stream)


@functools.lru_cache(maxsize=4096)
def _varlen_ws(dev, *a):
    return max(int(load_library().fa_varlen_workspace_bytes(*a)), 1)


@functools.lru_cache(maxsize=4096)
def _paged_ws(dev, *a):
    return max(int(load_library().fa_paged_workspace_bytes(*a)), 1)


def _shape3(name, t):
    if t.dim() != 3:
        _refuse(name, f"must be 3-D [T, heads, d], got shape {tuple(t.shape)}")
    return t.shape


def _outputs(Q, T, H, O, LSE):
    """O, LSE and whether the call sets their rows of no sequence (it does when both are new)."""
    if O is None and LSE is None:
        o = _empty_like(Q) if Q.is_contiguous() else _empty(Q.shape, dtype=Q.dtype, device=Q.device)
        return o, _empty((H, T), dtype=_F32, device=Q.device), 1
    if LSE is None:
        LSE = torch.full((H, T), -math.inf, dtype=_F32, device=Q.device)
    else:
        _lse(LSE, (H, T))
    if O is None:
        O = torch.zeros(Q.shape, dtype=Q.dtype, device=Q.device)
    else:
        _same("O", O, Q.shape, Q.dtype)
    return O, LSE, 0


def fa_varlen_fwd(Q, K, V, cu_q, cu_k, scale: float | None = None, causal: bool = False, window_size: int = 0,
                  O=None, LSE=None, stream=None):
    """(O, LSE) of attention inside each packed sequence; see include/fa.h (fa_varlen_fwd)."""
    T_q, H, d = _shape3("Q", Q)
    T_k, H_kv, dk = _shape3("K", K)
    if dk != d or K.dtype != Q.dtype:
        _refuse("K", f"{K.dtype} {tuple(K.shape)} incompatible with Q {Q.dtype} {tuple(Q.shape)}")
    _same("V", V, K.shape, Q.dtype)
    N = cu_q.numel() - 1
    _ints("cu_q", cu_q, (N + 1,))
    _ints("cu_k", cu_k, (N + 1,))
    dt = _type(Q)
    dev = _device(Q, K, V, cu_q, cu_k, O, LSE)
    need = _varlen_ws(dev.index, N, T_q, T_k, H, H_kv, d, dt, 0)

    def body(st):
        o, lse, fill = _outputs(Q, T_q, H, O, LSE)
        ws = _empty(need, dtype=_U8, device=dev)
        _check(load_library().fa_varlen_fwd(
            Q.data_ptr(), K.data_ptr(), V.data_ptr(), o.data_ptr(), lse.data_ptr(), cu_q.data_ptr(), cu_k.data_ptr(),
            N, T_q, T_k, H, H_kv, d,
            None if Q.is_contiguous() and K.is_contiguous() and V.is_contiguous() and o.is_contiguous() else
            _strides(("Q", Q), ("K", K), ("V", V), ("O", o)),
            _scale(scale, d), int(bool(causal)), _int32("window_size", window_size), fill, dt, ws.data_ptr(),
            need, st))
        return o, lse

    return _call(dev, stream, body)


def fa_varlen_bwd(dO, Q, K, V, O, LSE, cu_q, cu_k, scale: float | None = None, causal: bool = False,
                  window_size: int = 0, deterministic: bool = False, dQ=None, dK=None, dV=None, stream=None):
    """(dQ, dK, dV) of attention inside each packed sequence; see include/fa.h (fa_varlen_bwd)."""
    T_q, H, d = _shape3("Q", Q)
    T_k, H_kv, dk = _shape3("K", K)
    if dk != d or K.dtype != Q.dtype:
        _refuse("K", f"{K.dtype} {tuple(K.shape)} incompatible with Q {Q.dtype} {tuple(Q.shape)}")
    _same("V", V, K.shape, Q.dtype)
    _same("dO", dO, Q.shape, Q.dtype)
    _same("O", O, Q.shape, Q.dtype)
    _lse(LSE, (H, T_q))
    N = cu_q.numel() - 1
    _ints("cu_q", cu_q, (N + 1,))
    _ints("cu_k", cu_k, (N + 1,))
    for name, t, like in (("dQ", dQ, Q), ("dK", dK, K), ("dV", dV, V)):
        if t is not None:
            _same(name, t, like.shape, Q.dtype)
    dt = _type(Q)
    dev = _device(Q, dO, K, V, O, LSE, cu_q, cu_k, dQ, dK, dV)
    need = _varlen_ws(dev.index, N, T_q, T_k, H, H_kv, d, dt, 1)

    def body(st):
        fill = int(dQ is None and dK is None and dV is None)
        new = torch.empty if fill else torch.zeros
        gq, gk, gv = (new(like.shape, dtype=like.dtype, device=dev) if t is None else t
                      for t, like in ((dQ, Q), (dK, K), (dV, V)))
        ws = _empty(need, dtype=_U8, device=dev)
        _check(load_library().fa_varlen_bwd(
            dO.data_ptr(), Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), LSE.data_ptr(), gq.data_ptr(),
            gk.data_ptr(), gv.data_ptr(), cu_q.data_ptr(), cu_k.data_ptr(), N, T_q, T_k, H, H_kv, d,
            None if all(map(_Tensor.is_contiguous, (dO, Q, K, V, O, gq, gk, gv))) else
            _strides(("dO", dO), ("Q", Q), ("K", K), ("V", V), ("O", O), ("dQ", gq), ("dK", gk), ("dV", gv)),
            _scale(scale, d), int(bool(causal)), _int32("window_size", window_size), int(bool(deterministic)),
            fill, dt, ws.data_ptr(), need, st))
        return gq, gk, gv

    return _call(dev, stream, body)


def _caches(K_cache, V_cache, dtype):
    if K_cache.dim() != 4 or K_cache.dtype != dtype:
        _refuse("K_cache", f"must be {dtype} [pages, page_size, H_kv, d], got {K_cache.dtype} {tuple(K_cache.shape)}")
    _same("V_cache", V_cache, K_cache.shape, dtype)
    return K_cache.shape


def _table(t, N):
    if t.dim() != 2:
        _refuse("block_table", f"must be 2-D [N, max_pages], got shape {tuple(t.shape)}")
    _ints("block_table", t, (N, t.shape[1]))
    return t.shape[1]


def fa_paged_fwd(Q, K_cache, V_cache, block_table, cu_q, seq_lens, scale: float | None = None, causal: bool = True,
                 window_size: int = 0, O=None, LSE=None, stream=None):
    """(O, LSE) of each request's newest tokens over its pages; see include/fa.h (fa_paged_fwd)."""
    T_q, H, d = _shape3("Q", Q)
    pages, page, H_kv, dk = _caches(K_cache, V_cache, Q.dtype)
    if dk != d:
        _refuse("K_cache", f"shape {tuple(K_cache.shape)} incompatible with Q {tuple(Q.shape)}")
    N = cu_q.numel() - 1
    _ints("cu_q", cu_q, (N + 1,))
    _ints("seq_lens", seq_lens, (N,))
    cols = _table(block_table, N)
    dt = _type(Q)
    dev = _device(Q, K_cache, V_cache, block_table, cu_q, seq_lens, O, LSE)
    need = _paged_ws(dev.index, N, T_q, H, H_kv, d, page, dt)

    def body(st):
        o, lse, fill = _outputs(Q, T_q, H, O, LSE)
        ws = _empty(need, dtype=_U8, device=dev)
        _check(load_library().fa_paged_fwd(
            Q.data_ptr(), K_cache.data_ptr(), V_cache.data_ptr(), o.data_ptr(), lse.data_ptr(), block_table.data_ptr(),
            cu_q.data_ptr(), seq_lens.data_ptr(), N, T_q, pages, page, cols, H, H_kv, d,
            None if Q.is_contiguous() and K_cache.is_contiguous() and V_cache.is_contiguous() and o.is_contiguous() else
            _strides(("Q", Q), ("K_cache", K_cache), ("V_cache", V_cache), ("O", o)),
            _scale(scale, d), int(bool(causal)), _int32("window_size", window_size), fill, dt, ws.data_ptr(),
            need, st))
        return o, lse

    return _call(dev, stream, body)


def fa_page_slots(ctx_lens, cu_q, block_table, free_pages, free_start, page_size: int, tokens: int, slots=None,
                  positions=None, seq_lens=None, free_next=None, stream=None):
    """(slots, positions, seq_lens, free_next) of a step's new tokens; new pages are entered into
    block_table in place; see include/fa.h (fa_page_slots)."""
    N = cu_q.numel() - 1
    _ints("cu_q", cu_q, (N + 1,))
    _ints("ctx_lens", ctx_lens, (N,))
    cols = _table(block_table, N)
    n_free = free_pages.numel()
    _ints("free_pages", free_pages, (n_free,))
    _ints("free_start", free_start, (1,))
    tokens, page_size = _int32("tokens", tokens), _int32("page_size", page_size)
    if tokens < 0:
        _refuse("tokens", f"must be >= 0, got {tokens}")
    dev = _device(ctx_lens, cu_q, block_table, free_pages, free_start, slots, positions, seq_lens, free_next)
    for name, t, shape, dtype in (("slots", slots, (tokens,), _I64), ("positions", positions, (tokens,), _I32),
                                  ("seq_lens", seq_lens, (N,), _I32), ("free_next", free_next, (1,), _I32)):
        if t is not None:
            _ints(name, t, shape, dtype)

    def body(st):
        out = (_empty(tokens, dtype=_I64, device=dev) if slots is None else slots,
               _empty(tokens, dtype=_I32, device=dev) if positions is None else positions,
               _empty_like(ctx_lens) if seq_lens is None else seq_lens,
               _empty_like(free_start) if free_next is None else free_next)
        _check(load_library().fa_page_slots(
            ctx_lens.data_ptr(), cu_q.data_ptr(), free_pages.data_ptr(), free_start.data_ptr(), block_table.data_ptr(),
            out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), out[3].data_ptr(), N, tokens, n_free,
            page_size, cols, st))
        return out

    return _call(dev, stream, body)


def fa_paged_write(K, V, slots, K_cache, V_cache, stream=None):
    """Writes K and V rows to their slots of the caches, in place; see include/fa.h (fa_paged_write)."""
    T, H_kv, d = _shape3("K", K)
    _same("V", V, K.shape, K.dtype)
    pages, page, hc, dc = _caches(K_cache, V_cache, K.dtype)
    if hc != H_kv or dc != d:
        _refuse("K_cache", f"shape {tuple(K_cache.shape)} incompatible with K {tuple(K.shape)}")
    _ints("slots", slots, (T,), _I64)
    dt = _type(K)
    dev = _device(K, V, slots, K_cache, V_cache)

    def body(st):
        _check(load_library().fa_paged_write(
            K.data_ptr(), V.data_ptr(), slots.data_ptr(), K_cache.data_ptr(), V_cache.data_ptr(), T, pages, page, H_kv, d,
            None if K.is_contiguous() and V.is_contiguous() and K_cache.is_contiguous() and V_cache.is_contiguous() else
            _strides(("K", K), ("V", V), ("K_cache", K_cache), ("V_cache", V_cache)), dt, st))
        return K_cache, V_cache

    return _call(dev, stream, body)
