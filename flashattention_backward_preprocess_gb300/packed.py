"""Packed (variable-length) and paged attention: the entry points of include/fa.h that
take sequences of different lengths, as torch calls.

Tensors are token major: Q [T, H, d], K and V [T, H_kv, d], caches [pages, page_size, H_kv, d].
Any strides that are whole 16-byte pieces are taken as they are (slices of a joint QKV
projection, transposed caches); the head dimension is contiguous.  Lengths stay on the device:
no call here waits for the GPU.  Outputs that the caller does not pass are allocated, with the
rows of no sequence set to 0 (LSE: -inf); outputs passed in keep those rows as they were.
Scratch comes from PyTorch's allocator, one block per call, so calls on different streams and
captured graphs do not share it.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math

import torch

from .binding import FaError, _check, _dtype, load_library

_NULL = contextlib.nullcontext()


def _refuse(name, reason):
    raise FaError(1, f"{name}: {reason}")


def _device_of(first, *rest):
    """The one CUDA device all given tensors are on."""
    dev = first.device
    for t in rest:
        if t is not None and t.device != dev:
            _refuse("tensors", f"expected one device, got {dev} and {t.device}")
    if dev.type != "cuda":
        _refuse("tensors", f"device pointers required, got {dev}")
    return dev


class _on:
    """The call's device and stream as the current ones; .handle is the stream's."""

    def __init__(self, dev, stream):
        self.dev = _NULL if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)
        if stream is None:
            self.stream, self.handle = _NULL, torch._C._cuda_getCurrentRawStream(dev.index)
        else:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(int(stream), device=dev)
            self.stream, self.handle = torch.cuda.stream(stream), stream.cuda_stream

    def __enter__(self):
        self.dev.__enter__()
        self.stream.__enter__()
        return self.handle

    def __exit__(self, *e):
        self.stream.__exit__(*e)
        self.dev.__exit__(*e)


def _rows(name, t, dims, shape=None, dtype=None):
    """Strides (elements) of all but the last dimension; a dimension of size one counts as dense."""
    if t.dim() != dims:
        _refuse(name, f"must be {dims}-D, got shape {tuple(t.shape)}")
    if shape is not None and t.shape != shape:
        _refuse(name, f"expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        _refuse(name, f"expected {dtype}, got {t.dtype}")
    if t.is_contiguous():
        size, out = 1, []
        for n in reversed(t.shape[1:]):
            size *= n
            out.append(max(size, 1))
        return out[::-1]
    st = t.stride()
    if st[-1] != 1 and t.shape[-1] != 1:
        _refuse(name, "the head dimension must be contiguous")
    return [s if n > 1 else t.shape[-1] for s, n in zip(st[:-1], t.shape[:-1])]


def _ints(name, t, shape, dtype=torch.int32):
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        _refuse(name, f"must be contiguous {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")


def _strides(*groups):
    flat = [s for g in groups for s in g]
    return (ctypes.c_longlong * len(flat))(*flat)


@functools.lru_cache(maxsize=4096)
def _varlen_ws(dev, *a):
    return int(load_library().fa_varlen_workspace_bytes(*a))


@functools.lru_cache(maxsize=4096)
def _paged_ws(dev, *a):
    return int(load_library().fa_paged_workspace_bytes(*a))


def _workspace(n, dev):
    return torch.empty(max(n, 1), dtype=torch.uint8, device=dev)


def _forward_outputs(Q, O, LSE):
    """O, LSE and whether the call sets their rows of no sequence (it does when both are new)."""
    T, H, _ = Q.shape
    if LSE is not None and (LSE.shape != (H, T) or LSE.dtype != torch.float32 or not LSE.is_contiguous()):
        _refuse("LSE", f"must be contiguous float32 {(H, T)}")
    if O is None and LSE is None:
        return Q.new_empty(Q.shape), torch.empty((H, T), dtype=torch.float32, device=Q.device), 1
    if O is None:
        O = Q.new_zeros(Q.shape)
    if LSE is None:
        LSE = torch.full((H, T), -math.inf, dtype=torch.float32, device=Q.device)
    return O, LSE, 0


def fa_varlen_fwd(Q, K, V, cu_q, cu_k, scale: float | None = None, causal: bool = False, window_size: int = 0,
                  O=None, LSE=None, stream=None):
    """(O, LSE) of attention inside each packed sequence; see include/fa.h (fa_varlen_fwd)."""
    qs = _rows("Q", Q, 3)
    T_q, H, d = Q.shape
    ks = _rows("K", K, 3, dtype=Q.dtype)
    T_k, H_kv, dk = K.shape
    if dk != d:
        _refuse("K", f"shape {tuple(K.shape)} incompatible with Q {tuple(Q.shape)}")
    vs = _rows("V", V, 3, K.shape, Q.dtype)
    N = cu_q.numel() - 1
    _ints("cu_q", cu_q, (N + 1,))
    _ints("cu_k", cu_k, (N + 1,))
    dt = _dtype(Q)
    dev = _device_of(Q, K, V, cu_q, cu_k, O, LSE)
    lib = load_library()
    with _on(dev, stream) as st:
        O, LSE, fill = _forward_outputs(Q, O, LSE)
        os_ = _rows("O", O, 3, Q.shape, Q.dtype)
        need = _varlen_ws(dev.index, N, T_q, T_k, H, H_kv, d, dt, 0)
        ws = _workspace(need, dev)
        _check(lib.fa_varlen_fwd(Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), LSE.data_ptr(),
                                 cu_q.data_ptr(), cu_k.data_ptr(), N, T_q, T_k, H, H_kv, d,
                                 _strides(qs, ks, vs, os_), 1.0 / math.sqrt(d) if scale is None else float(scale),
                                 int(bool(causal)), int(window_size), fill, dt, ws.data_ptr(), need, st))
    return O, LSE


def fa_varlen_bwd(dO, Q, K, V, O, LSE, cu_q, cu_k, scale: float | None = None, causal: bool = False,
                  window_size: int = 0, deterministic: bool = False, dQ=None, dK=None, dV=None, stream=None):
    """(dQ, dK, dV) of attention inside each packed sequence; see include/fa.h (fa_varlen_bwd)."""
    qs = _rows("Q", Q, 3)
    T_q, H, d = Q.shape
    ks = _rows("K", K, 3, dtype=Q.dtype)
    T_k, H_kv, dk = K.shape
    if dk != d:
        _refuse("K", f"shape {tuple(K.shape)} incompatible with Q {tuple(Q.shape)}")
    vs = _rows("V", V, 3, K.shape, Q.dtype)
    dos = _rows("dO", dO, 3, Q.shape, Q.dtype)
    os_ = _rows("O", O, 3, Q.shape, Q.dtype)
    if LSE.shape != (H, T_q) or LSE.dtype != torch.float32 or not LSE.is_contiguous():
        _refuse("LSE", f"must be contiguous float32 {(H, T_q)}, got {LSE.dtype} {tuple(LSE.shape)}")
    N = cu_q.numel() - 1
    _ints("cu_q", cu_q, (N + 1,))
    _ints("cu_k", cu_k, (N + 1,))
    dt = _dtype(Q)
    dev = _device_of(Q, dO, K, V, O, LSE, cu_q, cu_k, dQ, dK, dV)
    lib = load_library()
    with _on(dev, stream) as st:
        fill = int(dQ is None and dK is None and dV is None)
        new = torch.Tensor.new_empty if fill else torch.Tensor.new_zeros
        dQ = new(Q, Q.shape) if dQ is None else dQ
        dK = new(K, K.shape) if dK is None else dK
        dV = new(V, V.shape) if dV is None else dV
        dqs, dks, dvs = (_rows(n, t, 3, r.shape, Q.dtype) for n, t, r in (("dQ", dQ, Q), ("dK", dK, K), ("dV", dV, V)))
        need = _varlen_ws(dev.index, N, T_q, T_k, H, H_kv, d, dt, 1)
        ws = _workspace(need, dev)
        _check(lib.fa_varlen_bwd(dO.data_ptr(), Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), LSE.data_ptr(),
                                 dQ.data_ptr(), dK.data_ptr(), dV.data_ptr(), cu_q.data_ptr(), cu_k.data_ptr(), N, T_q,
                                 T_k, H, H_kv, d, _strides(dos, qs, ks, vs, os_, dqs, dks, dvs),
                                 1.0 / math.sqrt(d) if scale is None else float(scale), int(bool(causal)),
                                 int(window_size), int(bool(deterministic)), fill, dt, ws.data_ptr(), need, st))
    return dQ, dK, dV


def fa_paged_fwd(Q, K_cache, V_cache, block_table, cu_q, seq_lens, scale: float | None = None, causal: bool = True,
                 window_size: int = 0, O=None, LSE=None, stream=None):
    """(O, LSE) of each request's newest tokens over its pages; see include/fa.h (fa_paged_fwd)."""
    qs = _rows("Q", Q, 3)
    T_q, H, d = Q.shape
    ks = _rows("K_cache", K_cache, 4, dtype=Q.dtype)
    pages, page, H_kv, dk = K_cache.shape
    if dk != d:
        _refuse("K_cache", f"shape {tuple(K_cache.shape)} incompatible with Q {tuple(Q.shape)}")
    vs = _rows("V_cache", V_cache, 4, K_cache.shape, Q.dtype)
    N = cu_q.numel() - 1
    _ints("cu_q", cu_q, (N + 1,))
    _ints("seq_lens", seq_lens, (N,))
    if block_table.dim() != 2:
        _refuse("block_table", f"must be 2-D [N, max_pages], got shape {tuple(block_table.shape)}")
    _ints("block_table", block_table, (N, block_table.shape[1]))
    dt = _dtype(Q)
    dev = _device_of(Q, K_cache, V_cache, block_table, cu_q, seq_lens, O, LSE)
    lib = load_library()
    with _on(dev, stream) as st:
        O, LSE, fill = _forward_outputs(Q, O, LSE)
        os_ = _rows("O", O, 3, Q.shape, Q.dtype)
        need = _paged_ws(dev.index, N, T_q, H, H_kv, d, page, dt)
        ws = _workspace(need, dev)
        _check(lib.fa_paged_fwd(Q.data_ptr(), K_cache.data_ptr(), V_cache.data_ptr(), O.data_ptr(), LSE.data_ptr(),
                                block_table.data_ptr(), cu_q.data_ptr(), seq_lens.data_ptr(), N, T_q, pages, page,
                                block_table.shape[1], H, H_kv, d, _strides(qs, ks, vs, os_),
                                1.0 / math.sqrt(d) if scale is None else float(scale), int(bool(causal)),
                                int(window_size), fill, dt, ws.data_ptr(), need, st))
    return O, LSE


def fa_page_slots(ctx_lens, cu_q, block_table, free_pages, free_start, page_size: int, tokens: int, slots=None,
                  positions=None, seq_lens=None, free_next=None, stream=None):
    """(slots, positions, seq_lens, free_next) of a step's new tokens; new pages are entered into
    block_table in place; see include/fa.h (fa_page_slots)."""
    N = cu_q.numel() - 1
    _ints("cu_q", cu_q, (N + 1,))
    _ints("ctx_lens", ctx_lens, (N,))
    if block_table.dim() != 2:
        _refuse("block_table", f"must be 2-D [N, max_pages], got shape {tuple(block_table.shape)}")
    _ints("block_table", block_table, (N, block_table.shape[1]))
    _ints("free_pages", free_pages, (free_pages.numel(),))
    _ints("free_start", free_start, (1,))
    tokens = int(tokens)
    if tokens < 0:
        _refuse("tokens", f"must be >= 0, got {tokens}")
    dev = _device_of(ctx_lens, cu_q, block_table, free_pages, free_start, slots, positions, seq_lens, free_next)
    lib = load_library()
    with _on(dev, stream) as st:
        i32 = dict(dtype=torch.int32, device=dev)
        slots = torch.empty(tokens, dtype=torch.int64, device=dev) if slots is None else slots
        positions = torch.empty(tokens, **i32) if positions is None else positions
        seq_lens = torch.empty(N, **i32) if seq_lens is None else seq_lens
        free_next = torch.empty(1, **i32) if free_next is None else free_next
        _ints("slots", slots, (tokens,), torch.int64)
        _ints("positions", positions, (tokens,))
        _ints("seq_lens", seq_lens, (N,))
        _ints("free_next", free_next, (1,))
        _check(lib.fa_page_slots(ctx_lens.data_ptr(), cu_q.data_ptr(), free_pages.data_ptr(), free_start.data_ptr(),
                                 block_table.data_ptr(), slots.data_ptr(), positions.data_ptr(), seq_lens.data_ptr(),
                                 free_next.data_ptr(), N, tokens, free_pages.numel(), int(page_size),
                                 block_table.shape[1], st))
    return slots, positions, seq_lens, free_next


def fa_paged_write(K, V, slots, K_cache, V_cache, stream=None):
    """Writes K and V rows to their slots of the caches, in place; see include/fa.h (fa_paged_write)."""
    ks = _rows("K", K, 3)
    T, H_kv, d = K.shape
    vs = _rows("V", V, 3, K.shape, K.dtype)
    if K_cache.dim() != 4 or K_cache.shape[2:] != K.shape[1:]:
        _refuse("K_cache", f"shape {tuple(K_cache.shape)} incompatible with K {tuple(K.shape)}")
    kc = _rows("K_cache", K_cache, 4, dtype=K.dtype)
    vc = _rows("V_cache", V_cache, 4, K_cache.shape, K.dtype)
    _ints("slots", slots, (T,), torch.int64)
    dt = _dtype(K)
    dev = _device_of(K, V, slots, K_cache, V_cache)
    lib = load_library()
    with _on(dev, stream) as st:
        _check(lib.fa_paged_write(K.data_ptr(), V.data_ptr(), slots.data_ptr(), K_cache.data_ptr(), V_cache.data_ptr(),
                                  T, K_cache.shape[0], K_cache.shape[1], H_kv, d, _strides(ks, vs, kc, vc), dt, st))
    return K_cache, V_cache
