"""Attention with a sliding window and sinks, its gradients, and its cache of
constant size (the kda_window_* entry points of include/kda.h). Marshalling
only, in the manner of ``_linear``: q, k and v may be slices of a fused
projection, and every call takes ``stream``."""
from __future__ import annotations

import functools

import torch

from ._binding import _check, _dtype_code
from ._linear import _on_stream, _out, _packed, _plain, _ptr, _space, _stream, _view, load

_MOST = (1 << 31) - 1  # a longer window is as good as this one


def _counts(window: int, sinks: int) -> tuple:
    """The two as C ints, which would be given the low 32 bits of what they do not hold; the library refuses the rest."""
    if not -_MOST <= sinks <= _MOST:
        raise ValueError(f"sinks must be 0 to 128, got {sinks}")
    if window < -_MOST:
        raise ValueError(f"window must be 1 or more, got {window}")
    return min(window, _MOST), sinks


@functools.lru_cache(maxsize=256)
def _bytes(name: str, *sizes: int) -> int:
    if not all(-_MOST <= n <= _MOST for n in sizes):
        raise ValueError(f"the sizes must fit in 32 bits, got {sizes}")
    return int(getattr(load(), name + "_workspace_bytes")(*sizes))


def window_varlen_attention_workspace_bytes(N: int, T_total: int, H_q: int, H_k: int, d: int = 128) -> int:
    return _bytes("kda_window_varlen_attention", N, T_total, H_q, H_k, d)


def window_attention_backward_workspace_bytes(B: int, T: int, H_q: int, H_k: int, d: int = 128, sinks: int = 0,
                                              dtype=torch.bfloat16) -> int:
    return _bytes("kda_window_attention_backward", B, T, H_q, H_k, d, sinks, _dtype_code(torch.empty(0, dtype=dtype)))


def window_varlen_attention_backward_workspace_bytes(N: int, T_total: int, H_q: int, H_k: int, d: int = 128,
                                                     sinks: int = 0, dtype=torch.bfloat16) -> int:
    return _bytes("kda_window_varlen_attention_backward", N, T_total, H_q, H_k, d, sinks,
                  _dtype_code(torch.empty(0, dtype=dtype)))


def _inputs(q, k, v, lead: int, scale):
    """Checks q, k, v; returns (device index, lead shape, H_q, H_k, d, strides, scale)."""
    qs = _view(q, "q", lead)
    index, dtype, shape = q.get_device(), q.dtype, q.shape
    ks, vs = _view(k, "k", lead, dtype, index), _view(v, "v", lead, dtype, index)
    if k.shape != v.shape or k.shape[:-2] != shape[:-2] or k.shape[-1] != shape[-1]:
        raise ValueError("shape mismatch among q, k, v")
    d = shape[-1]
    return index, shape[:lead], shape[-2], k.shape[-2], d, (qs, ks, vs), d ** -0.5 if scale is None and d else scale or 0.0


def _attention(q, k, v, cu_seqlens, window, sinks, scale, out, lse, workspace, device_status):
    lib = load()
    window, sinks = _counts(window, sinks)
    packed = cu_seqlens is not None
    index, lead, hq, hk, d, strides, scale = _inputs(q, k, v, 1 if packed else 2, scale)
    out = _out(out, "out", q, q.shape, q.dtype, index)
    lse = _out(lse, "lse", q, q.shape[:-1], torch.float32, index)
    head = (q.data_ptr(), k.data_ptr(), v.data_ptr(), _dtype_code(q), *strides, scale, window, sinks,
            out.data_ptr(), lse.data_ptr())
    if packed:
        N, T = _packed(cu_seqlens, device_status, index), lead[0]
        ws, size = _space(workspace, _bytes("kda_window_varlen_attention", N, T, hq, hk, d), q)
        st = lib.kda_window_varlen_attention(*head, cu_seqlens.data_ptr(), N, T, hq, hk, d, ws.data_ptr(), size,
                                             _ptr(device_status), _stream(index))
    else:
        st = lib.kda_window_attention(*head, *lead, hq, hk, d, _stream(index))
    _check(lib, st)
    return out, lse


@_on_stream
def window_attention(q, k, v, *, window: int, sinks: int = 0, scale: float | None = None, out=None, lse=None):
    """Causal softmax attention over the last ``window`` tokens, the token's own
    included, and the first ``sinks`` (0 to 128): token i sees token j <= i where
    i - j < window or j < sinks.

    q: [B, T, H_q, d]; k, v: [B, T, H_k, d] (bf16 or fp32, the same type; d 64 or
    128); query head h reads key head h // (H_q // H_k). scale: positive,
    d ** -0.5 by default. Returns (o [B, T, H_q, d] in q's type, lse [B, T, H_q] fp32: the
    natural logarithm of the sum of e^score, which the gradients want)."""
    return _attention(q, k, v, None, window, sinks, scale, out, lse, None, None)


@_on_stream
def window_varlen_attention(q, k, v, cu_seqlens, *, window: int, sinks: int = 0, scale: float | None = None, out=None,
                            lse=None, workspace=None, device_status=None):
    """``window_attention`` over N sequences packed along the token axis: q
    [T_total, H_q, d]; k, v [T_total, H_k, d]; cu_seqlens: int32 [N + 1] on the
    device. ``device_status`` (int32 [1]) receives KDA_DEV_OK or
    KDA_DEV_BAD_CU_SEQLENS, in which case nothing else is written."""
    if cu_seqlens is None:
        raise ValueError("cu_seqlens is required")
    return _attention(q, k, v, cu_seqlens, window, sinks, scale, out, lse, workspace, device_status)


def _backward(q, k, v, out, lse, d_o, cu_seqlens, window, sinks, scale, workspace, device_status):
    lib = load()
    window, sinks = _counts(window, sinks)
    packed = cu_seqlens is not None
    index, lead, hq, hk, d, strides, scale = _inputs(q, k, v, 1 if packed else 2, scale)
    _plain(out, "out", q.dtype, index, q.shape)
    _plain(lse, "lse", torch.float32, index, q.shape[:-1])
    _plain(d_o, "d_o", q.dtype, index, q.shape)
    grads = {"dq": torch.empty_like(d_o),
             "dk": torch.empty(k.shape, dtype=q.dtype, device=q.device),
             "dv": torch.empty(v.shape, dtype=q.dtype, device=q.device)}
    head = (q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), d_o.data_ptr(), _dtype_code(q),
            *strides, scale, window, sinks, *(t.data_ptr() for t in grads.values()))
    if packed:
        N, T = _packed(cu_seqlens, device_status, index), lead[0]
        ws, size = _space(workspace, _bytes("kda_window_varlen_attention_backward", N, T, hq, hk, d, sinks, _dtype_code(q)), q)
        st = lib.kda_window_varlen_attention_backward(*head, cu_seqlens.data_ptr(), N, T, hq, hk, d, ws.data_ptr(), size,
                                                      _ptr(device_status), _stream(index))
    else:
        ws, size = _space(workspace, _bytes("kda_window_attention_backward", *lead, hq, hk, d, sinks, _dtype_code(q)), q)
        st = lib.kda_window_attention_backward(*head, *lead, hq, hk, d, ws.data_ptr(), size, _stream(index))
    _check(lib, st)
    return grads


@_on_stream
def window_attention_backward(q, k, v, out, lse, d_o, *, window: int, sinks: int = 0, scale: float | None = None,
                              workspace=None):
    """Gradients of ``window_attention`` for L = sum <d_o, o>; out and lse as it
    returned them, d_o in q's type, all three contiguous. Returns a dict: ``dq``,
    ``dk``, ``dv`` in q's type (dk and dv summed over the query heads of a key
    head)."""
    return _backward(q, k, v, out, lse, d_o, None, window, sinks, scale, workspace, None)


@_on_stream
def window_varlen_attention_backward(q, k, v, out, lse, d_o, cu_seqlens, *, window: int, sinks: int = 0,
                                     scale: float | None = None, workspace=None, device_status=None):
    """Gradients of ``window_varlen_attention`` (packed sequences): the dict of
    ``window_attention_backward``."""
    if cu_seqlens is None:
        raise ValueError("cu_seqlens is required")
    return _backward(q, k, v, out, lse, d_o, cu_seqlens, window, sinks, scale, workspace, device_status)


def _cache(k, k_cache, v_cache, slots, N: int, sinks: int, hk: int, d: int, device_status, index: int):
    """Checks a cache; returns (pool size, entries)."""
    _plain(k_cache, "k_cache", k.dtype, index)
    _plain(v_cache, "v_cache", k.dtype, index, k_cache.shape)
    if k_cache.dim() != 4 or k_cache.shape[2:] != (hk, d) or k_cache.shape[1] <= sinks:
        raise ValueError(f"k_cache and v_cache must be [P, sinks + window, {hk}, {d}] with a window of 1 or more, got "
                         f"{tuple(k_cache.shape)}")
    _plain(slots, "slots", torch.int32, index, (N,))
    if device_status is not None:
        _plain(device_status, "device_status", torch.int32, index)
    return k_cache.shape[:2]


@_on_stream
def window_cache_write(k, v, cu_seqlens, k_cache, v_cache, slots, *, sinks: int = 0, device_status=None):
    """Puts the keys and values of N packed prompts into their slots, for the
    decode steps behind them: of each its first ``sinks`` and its last ``window``
    tokens, where ``k_cache.shape[1]`` is sinks + window.

    k, v: [T_total, H_k, d]; cu_seqlens: int32 [N + 1]; k_cache, v_cache: [P,
    sinks + window, H_k, d] in k's type, updated in place; slots: int32 [N]
    (``-1 - s`` stands for slot s too, so the slots that start a state afresh
    serve here as they are). A slot outside [0, P) leaves its prompt out and sets
    KDA_DEV_BAD_SLOT in ``device_status``; after KDA_DEV_BAD_CU_SEQLENS nothing
    is written."""
    lib = load()
    _counts(1, sinks)
    ks = _view(k, "k", 1)
    index = k.get_device()
    vs = _view(v, "v", 1, k.dtype, index)
    if k.shape != v.shape:
        raise ValueError("shape mismatch between k and v")
    if cu_seqlens is None:
        raise ValueError("cu_seqlens is required")
    N, (T, hk, d) = _packed(cu_seqlens, device_status, index), k.shape
    pool, entries = _cache(k, k_cache, v_cache, slots, N, sinks, hk, d, device_status, index)
    _check(lib, lib.kda_window_cache_write(k.data_ptr(), v.data_ptr(), _dtype_code(k), ks, vs, cu_seqlens.data_ptr(),
                                           slots.data_ptr(), sinks, k_cache.data_ptr(), v_cache.data_ptr(), pool,
                                           entries, N, T, hk, d, _ptr(device_status), _stream(index)))


@_on_stream
def window_decode_step(q, k, v, k_cache, v_cache, slots, positions, *, sinks: int = 0, scale: float | None = None,
                       out=None, device_status=None):
    """One token per sequence: its key and value go into the slot's cache, its
    query attends over what the slot holds, itself included.

    q: [N, H_q, d]; k, v: [N, H_k, d]; k_cache, v_cache, slots, sinks: as for
    ``window_cache_write``; positions: int32 [N], the number of tokens that the
    sequence has before this one. Returns o [N, H_q, d]. A sequence with a slot
    outside [0, P) or a negative position is left out and sets KDA_DEV_BAD_SLOT
    or KDA_DEV_BAD_POSITION in ``device_status``."""
    lib = load()
    _counts(1, sinks)
    index, (N,), hq, hk, d, strides, scale = _inputs(q, k, v, 1, scale)
    pool, entries = _cache(k, k_cache, v_cache, slots, N, sinks, hk, d, device_status, index)
    _plain(positions, "positions", torch.int32, index, (N,))
    out = _out(out, "out", q, q.shape, q.dtype, index)
    _check(lib, lib.kda_window_decode_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), _dtype_code(q), *strides, scale,
                                           sinks, k_cache.data_ptr(), v_cache.data_ptr(), pool, entries,
                                           slots.data_ptr(), positions.data_ptr(), out.data_ptr(), N, hq, hk, d,
                                           _ptr(device_status), _stream(index)))
    return out
