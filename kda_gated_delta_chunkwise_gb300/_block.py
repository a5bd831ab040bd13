"""The norms around a block: of every head with a gate, and of the residual
stream (the kda_gated_norm* and kda_residual_norm* entry points of
include/kda.h). Marshalling only, in the manner of ``_linear``: slices of a
fused projection where the docstring says so, ``stream`` on every call."""
from __future__ import annotations

import functools
import math

import torch

from ._binding import _check, _dtype_code
from ._linear import NORMS, _kind, _on_stream, _out, _plain, _ptr, _space, _stream, _view, load

ACTIVATIONS = {"sigmoid": 0, "silu": 1}


def _gated_inputs(x, gate, weight, norm, activation):
    if x is None or x.dim() < 3:
        raise ValueError("x must be [.., H, d]")
    lead = x.dim() - 2
    xs = _view(x, "x", lead)
    index = x.get_device()
    gs = _view(gate, "gate", lead, x.dtype, index)
    if gate.shape != x.shape:
        raise ValueError("x and gate must have the same shape")
    d = x.shape[-1]
    if weight is not None:
        _plain(weight, "weight", torch.float32, index, (d,))
    return (index, math.prod(x.shape[:-2]), x.shape[-2], d, _dtype_code(x), xs, gs, _kind(NORMS, norm, "norm"),
            _kind(ACTIVATIONS, activation, "activation"))


@_on_stream
def gated_norm(x, gate, weight=None, *, norm: str = "rms", activation: str = "sigmoid", eps: float = 1e-6, out=None):
    """The norm of every head times a gate, behind a recurrence or an attention:
    weight * x / norm(x) * activation(gate).

    x, gate: [.., H, d], d 64 or 128 (bf16 or fp32, the same type; slices of a
    fused projection are taken as they are); weight: fp32 [d] or None; norm:
    "rms", "l2" or "none"; activation: "sigmoid" or "silu" (gate * sigmoid(gate)).
    Returns out, contiguous, in x's type; ``out`` may be x or gate itself."""
    lib = load()
    index, n, h, d, code, xs, gs, nk, act = _gated_inputs(x, gate, weight, norm, activation)
    out = _out(out, "out", x, x.shape, x.dtype, index)
    _check(lib, lib.kda_gated_norm(x.data_ptr(), gate.data_ptr(), code, xs, gs, _ptr(weight), nk, act, eps,
                                   out.data_ptr(), n, h, d, _stream(index)))
    return out


@functools.lru_cache(maxsize=None)
def _gated_bytes(d: int) -> int:
    return int(load().kda_gated_norm_backward_workspace_bytes(d))


@_on_stream
def gated_norm_backward(x, gate, d_out, weight=None, *, norm: str = "rms", activation: str = "sigmoid",
                        eps: float = 1e-6, workspace=None):
    """Gradients of ``gated_norm`` for L = sum <d_out, out> (d_out contiguous, in
    x's type). Returns a dict: ``dx``, ``dgate`` in x's type, ``dweight`` (fp32
    [d]; None without a weight)."""
    lib = load()
    index, n, h, d, code, xs, gs, nk, act = _gated_inputs(x, gate, weight, norm, activation)
    _plain(d_out, "d_out", x.dtype, index, x.shape)
    out = {"dx": torch.empty_like(d_out), "dgate": torch.empty_like(d_out),
           "dweight": None if weight is None else torch.empty_like(weight)}
    ws, size = (None, 0) if weight is None else _space(workspace, _gated_bytes(d), x)
    _check(lib, lib.kda_gated_norm_backward(x.data_ptr(), gate.data_ptr(), d_out.data_ptr(), code, xs, gs, _ptr(weight),
                                            nk, act, eps, *(_ptr(t) for t in out.values()), n, h, d, _ptr(ws), size,
                                            _stream(index)))
    return out


def _residual_inputs(stream, name, dtype, weight, branch_weight, channel_scale, branch_norm):
    if stream is None or stream.dim() < 1:
        raise ValueError(f"{name} must be [.., D]")
    index = stream.get_device()
    if index < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    _plain(stream, name, None, index)
    if stream.dtype != dtype and stream.dtype != torch.float32:
        raise TypeError(f"{name} must be {dtype} or torch.float32, got {stream.dtype}")
    D = stream.shape[-1]
    for t, n in ((weight, "weight"), (branch_weight, "branch_weight"), (channel_scale, "channel_scale")):
        if t is not None:
            _plain(t, n, torch.float32, index, (D,))
    return index, math.prod(stream.shape[:-1]), D, _dtype_code(stream), _kind(NORMS, branch_norm, "branch_norm")


@_on_stream
def residual_norm(residual, branch, weight=None, *, branch_norm: str = "none", branch_weight=None, channel_scale=None,
                  scale: float = 1.0, eps: float = 1e-6, hidden_out=None, out=None):
    """A block's branch added to the residual stream, and the norm that the next
    block reads: u = branch_weight * branch / norm(branch),
    hidden = residual + scale * channel_scale * u,
    out = weight * hidden / sqrt(mean hidden^2 + eps).

    residual: [.., D] contiguous, fp32 or branch's type; branch: [.., D] contiguous
    (bf16 or fp32), D a multiple of 8 up to 8192; weight, branch_weight,
    channel_scale: fp32 [D] or None (ones); branch_norm: "none" (no division),
    "rms" or "l2". Returns (hidden in residual's type, out in branch's);
    ``hidden_out`` may be residual itself, ``out`` branch."""
    lib = load()
    if branch is None:
        raise ValueError("branch is required")
    index, n, D, scode, bn = _residual_inputs(residual, "residual", branch.dtype, weight, branch_weight, channel_scale,
                                              branch_norm)
    _plain(branch, "branch", None, index, residual.shape)
    hidden_out = _out(hidden_out, "hidden_out", residual, residual.shape, residual.dtype, index)
    out = _out(out, "out", branch, branch.shape, branch.dtype, index)
    _check(lib, lib.kda_residual_norm(residual.data_ptr(), branch.data_ptr(), scode, _dtype_code(branch), _ptr(weight),
                                      bn, _ptr(branch_weight), _ptr(channel_scale), scale, eps, hidden_out.data_ptr(),
                                      out.data_ptr(), n, D, _stream(index)))
    return hidden_out, out


@functools.lru_cache(maxsize=None)
def _residual_bytes(D: int) -> int:
    return int(load().kda_residual_norm_backward_workspace_bytes(D))


@_on_stream
def residual_norm_backward(hidden, branch, d_out, d_hidden=None, weight=None, *, branch_norm: str = "none",
                           branch_weight=None, channel_scale=None, scale: float = 1.0, eps: float = 1e-6,
                           workspace=None):
    """Gradients of ``residual_norm`` for L = sum <d_out, out> + <d_hidden, hidden>,
    from the stored hidden (d_out in branch's type; d_hidden in hidden's, None:
    zero). Returns a dict: ``d_residual`` in hidden's type, ``d_branch`` in
    d_out's, ``dweight``, ``dbranch_weight``, ``dchannel_scale`` (fp32 [D]; None
    without that factor). ``branch`` may be None where branch_norm is "none" and
    neither branch_weight nor channel_scale is given."""
    lib = load()
    if d_out is None:
        raise ValueError("d_out is required")
    index, n, D, scode, bn = _residual_inputs(hidden, "hidden", d_out.dtype, weight, branch_weight, channel_scale,
                                              branch_norm)
    _plain(d_out, "d_out", None, index, hidden.shape)
    if branch is not None:
        _plain(branch, "branch", d_out.dtype, index, hidden.shape)
    if d_hidden is not None:
        _plain(d_hidden, "d_hidden", hidden.dtype, index, hidden.shape)
    out = {"d_residual": torch.empty_like(hidden),
           "d_branch": torch.empty_like(d_out),
           "dweight": None if weight is None else torch.empty_like(weight),
           "dbranch_weight": None if branch_weight is None else torch.empty_like(branch_weight),
           "dchannel_scale": None if channel_scale is None else torch.empty_like(channel_scale)}
    ws, size = None, 0
    if weight is not None or branch_weight is not None or channel_scale is not None:
        ws, size = _space(workspace, _residual_bytes(D), hidden)
    _check(lib, lib.kda_residual_norm_backward(hidden.data_ptr(), _ptr(branch), d_out.data_ptr(), _ptr(d_hidden), scode,
                                               _dtype_code(d_out), _ptr(weight), bn, _ptr(branch_weight),
                                               _ptr(channel_scale), scale, eps, *(_ptr(t) for t in out.values()), n, D,
                                               _ptr(ws), size, _stream(index)))
    return out
