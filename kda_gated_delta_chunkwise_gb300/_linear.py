"""Linear attention with a decay, and the norm and rotary positions in front
of it (the kda_linear_* and kda_qk_norm_rope* entry points of include/kda.h).

Marshalling only, like the rest of the binding: checks of shapes, types and
strides, outputs and workspaces through PyTorch, raw pointers and a CUDA
stream. There is no fallback.

q, k and v may be slices of a wider tensor (a fused projection): their last two
axes must be contiguous and their tokens evenly spaced. With ``stream`` the
outputs and the workspace are allocated for that stream; the inputs must be
ready on it.
"""
from __future__ import annotations

import contextlib
import functools
import math

import torch

from . import _binding
from ._binding import _check, _dtype_code, _need

# Host time counts for one token of one sequence: these stand for the
# binding's helpers of the same names without the objects they make per call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def load():
    return _binding._lib or _binding.load()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream

# decay kinds: one log decay per token and head, one per head, none
DECAYS = {"token": 0, "head": 1, "none": 2}
NORMS = {"none": 0, "l2": 1, "rms": 2}
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}


def _kind(kinds: dict, value: str, name: str) -> int:
    if value not in kinds:
        raise ValueError(f"{name} must be one of {sorted(kinds)}")
    return kinds[value]


_here = contextlib.nullcontext()


def _on(stream):
    return _here if stream is None else torch.cuda.stream(stream)


def _view(t, name: str, lead: int, dtype=None, device=None) -> int:
    """The token stride of ``t`` [*lead axes, H, d], whose heads are contiguous
    and whose tokens are evenly spaced over all lead axes."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dim() != lead + 2:
        raise ValueError(f"{name} must have {lead + 2} dimensions, got {t.dim()}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.is_contiguous() or t.numel() == 0:
        return 0
    H, d = t.shape[-2:]
    step, want, even = None, None, (t.stride(-1) == 1 or d == 1) and (H == 1 or t.stride(-2) == d)
    for a in range(lead - 1, -1, -1):  # from the innermost lead axis outwards
        if t.shape[a] == 1:
            continue
        if step is None:
            step = want = t.stride(a)
        even = even and step > 0 and t.stride(a) == want
        want *= t.shape[a]
    if not even:
        raise ValueError(f"{name} must be contiguous, or a slice whose heads are contiguous and whose tokens are "
                         "evenly spaced")
    return step or 0


def _check_decay(decay: str, log_decay, lead: tuple, H: int, dev):
    kind = _kind(DECAYS, decay, "decay")
    if decay == "none":
        return kind, None
    _need(log_decay, "log_decay", torch.float32, dev)
    want = tuple(lead) + (H,) if decay == "token" else (H,)
    if tuple(log_decay.shape) != want:
        raise ValueError(f"log_decay must be {want} for decay={decay!r}, got {tuple(log_decay.shape)}")
    return kind, log_decay


def _qkv(q, k, v, lead: int):
    """Checks q, k, v; returns (device, lead shape, H, d_k, d_v, the three token strides)."""
    qs = _view(q, "q", lead)
    dev = q.device
    ks, vs = _view(k, "k", lead, q.dtype, dev), _view(v, "v", lead, q.dtype, dev)
    H, dk = q.shape[-2:]
    dv = v.shape[-1]
    if k.shape != q.shape or v.shape[:-1] != q.shape[:-1]:
        raise ValueError("shape mismatch among q, k, v")
    return dev, tuple(q.shape[:lead]), H, dk, dv, (qs, ks, vs)


def _state(t, name: str, shape: tuple, dev):
    if t is not None:
        _need(t, name, torch.float32, dev)
        if tuple(t.shape) != shape:
            raise ValueError(f"{name} must be {shape}, got {tuple(t.shape)}")


def _out(t, name: str, shape: tuple, dtype, dev):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _need(t, name, dtype, dev)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _space(workspace, nbytes: int, dev):
    """The caller's workspace or a new one; (tensor, bytes)."""
    if workspace is None:
        return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev), nbytes
    _need(workspace, "workspace", None, dev)
    return workspace, workspace.numel() * workspace.element_size()


@functools.lru_cache(maxsize=256)
def _size(name: str, n: int, T: int, H: int, dk: int, dv: int, code: int) -> int:
    """Workspace bytes: a function of the sizes alone."""
    return int(getattr(load(), name + "_workspace_bytes")(n, T, H, dk, dv, code))


def _bytes(name: str, n: int, T: int, H: int, dk: int, dv: int, dtype) -> int:
    return _size(name, n, T, H, dk, dv, _dtype_code(torch.empty(0, dtype=dtype)))


def linear_prefill_workspace_bytes(B: int, T: int, H: int, dk: int = 128, dv: int = 128, dtype=torch.bfloat16) -> int:
    return _bytes("kda_linear_prefill", B, T, H, dk, dv, dtype)


def linear_varlen_prefill_workspace_bytes(N: int, T_total: int, H: int, dk: int = 128, dv: int = 128,
                                          dtype=torch.bfloat16) -> int:
    return _bytes("kda_linear_varlen_prefill", N, T_total, H, dk, dv, dtype)


def linear_prefill_backward_workspace_bytes(B: int, T: int, H: int, dk: int = 128, dv: int = 128,
                                            dtype=torch.bfloat16) -> int:
    return _bytes("kda_linear_prefill_backward", B, T, H, dk, dv, dtype)


def linear_varlen_prefill_backward_workspace_bytes(N: int, T_total: int, H: int, dk: int = 128, dv: int = 128,
                                                   dtype=torch.bfloat16) -> int:
    return _bytes("kda_linear_varlen_prefill_backward", N, T_total, H, dk, dv, dtype)


def _prefill(q, k, v, log_decay, cu_seqlens, initial_state, decay, scale, output_final_state, out, final_state,
             workspace, device_status, stream):
    lib = load()
    packed = cu_seqlens is not None
    dev, lead, H, dk, dv, strides = _qkv(q, k, v, 1 if packed else 2)
    code = _dtype_code(q)
    kind, g = _check_decay(decay, log_decay, lead, H, dev)
    if packed:
        _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
            raise ValueError("cu_seqlens must be one-dimensional with N + 1 entries")
        N, T = cu_seqlens.numel() - 1, lead[0]
        if device_status is not None:
            _need(device_status, "device_status", torch.int32, dev)
    else:
        N, T = lead
    _state(initial_state, "initial_state", (N, H, dk, dv), dev)
    name = "kda_linear_varlen_prefill" if packed else "kda_linear_prefill"
    with _on(stream):
        out = _out(out, "out", tuple(v.shape), v.dtype, dev)
        if final_state is not None or output_final_state:
            final_state = _out(final_state, "final_state", (N, H, dk, dv), torch.float32, dev)
        ws, size = _space(workspace, _size(name, N, T, H, dk, dv, code), dev)
    head = (_ptr(q), _ptr(k), _ptr(v), code, *strides, _ptr(g), kind, float(scale), _ptr(initial_state), _ptr(out),
            _ptr(final_state))
    if packed:
        st = lib.kda_linear_varlen_prefill(*head, _ptr(cu_seqlens), N, T, H, dk, dv, _ptr(ws), size,
                                           _ptr(device_status), _stream(stream))
    else:
        st = lib.kda_linear_prefill(*head, N, T, H, dk, dv, _ptr(ws), size, _stream(stream))
    _check(lib, st)
    return out, final_state


def linear_prefill(q, k, v, log_decay=None, initial_state=None, *, decay: str = "token", scale: float = 1.0,
                   output_final_state: bool = True, out=None, final_state=None, workspace=None, stream=None):
    """Linear attention with a decay over B equal-length sequences:
    S_t = e^{g_t} S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t.

    q, k: [B, T, H, d_k]; v: [B, T, H, d_v] (bf16 or fp32, the same type);
    log_decay: natural logarithms <= 0, fp32 [B, T, H] (decay="token"), [H]
    (decay="head") or None (decay="none"); -inf, or anything <= -128, resets
    the state; initial_state: [B, H, d_k, d_v] fp32 or None (zeros).
    Returns (o [B, T, H, d_v] in v's type, final_state fp32 or None).
    """
    return _prefill(q, k, v, log_decay, None, initial_state, decay, scale, output_final_state, out, final_state,
                    workspace, None, stream)


def linear_varlen_prefill(q, k, v, log_decay, cu_seqlens, initial_state=None, *, decay: str = "token",
                          scale: float = 1.0, output_final_state: bool = True, out=None, final_state=None,
                          workspace=None, device_status=None, stream=None):
    """``linear_prefill`` over N sequences packed along the token axis:
    q, k: [T_total, H, d_k]; v: [T_total, H, d_v]; log_decay [T_total, H]
    (decay="token"); cu_seqlens: int32 [N + 1] on the device; initial_state:
    [N, H, d_k, d_v]. ``device_status`` (int32 [1]) receives KDA_DEV_OK or
    KDA_DEV_BAD_CU_SEQLENS, in which case nothing else is written."""
    if cu_seqlens is None:
        raise ValueError("cu_seqlens is required")
    return _prefill(q, k, v, log_decay, cu_seqlens, initial_state, decay, scale, output_final_state, out, final_state,
                    workspace, device_status, stream)


def _backward(q, k, v, log_decay, d_o, cu_seqlens, initial_state, d_final_state, decay, scale, want_decay_grad,
              want_initial_state_grad, workspace, device_status, stream):
    lib = load()
    packed = cu_seqlens is not None
    dev, lead, H, dk, dv, strides = _qkv(q, k, v, 1 if packed else 2)
    code = _dtype_code(q)
    kind, g = _check_decay(decay, log_decay, lead, H, dev)
    _need(d_o, "d_o", q.dtype, dev)
    if d_o.shape != v.shape:
        raise ValueError(f"d_o must be {tuple(v.shape)}, got {tuple(d_o.shape)}")
    if packed:
        _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
            raise ValueError("cu_seqlens must be one-dimensional with N + 1 entries")
        N, T = cu_seqlens.numel() - 1, lead[0]
        if device_status is not None:
            _need(device_status, "device_status", torch.int32, dev)
    else:
        N, T = lead
    for t, n in ((initial_state, "initial_state"), (d_final_state, "d_final_state")):
        _state(t, n, (N, H, dk, dv), dev)
    name = "kda_linear_varlen_prefill_backward" if packed else "kda_linear_prefill_backward"
    with _on(stream):
        out = {"dq": torch.empty(q.shape, dtype=q.dtype, device=dev),
               "dk": torch.empty(k.shape, dtype=q.dtype, device=dev),
               "dv": torch.empty(v.shape, dtype=q.dtype, device=dev),
               "dlog_decay": torch.empty_like(g) if g is not None and want_decay_grad else None,
               "d_initial_state": torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev)
               if want_initial_state_grad else None}
        ws, size = _space(workspace, _size(name, N, T, H, dk, dv, code), dev)
    head = (_ptr(q), _ptr(k), _ptr(v), code, *strides, _ptr(g), kind, float(scale), _ptr(initial_state), _ptr(d_o),
            _ptr(d_final_state), _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dlog_decay"]),
            _ptr(out["d_initial_state"]))
    if packed:
        st = lib.kda_linear_varlen_prefill_backward(*head, _ptr(cu_seqlens), N, T, H, dk, dv, _ptr(ws), size,
                                                    _ptr(device_status), _stream(stream))
    else:
        st = lib.kda_linear_prefill_backward(*head, N, T, H, dk, dv, _ptr(ws), size, _stream(stream))
    _check(lib, st)
    return out


def linear_prefill_backward(q, k, v, log_decay, d_o, initial_state=None, d_final_state=None, *, decay: str = "token",
                            scale: float = 1.0, want_decay_grad: bool = True, want_initial_state_grad: bool = True,
                            workspace=None, stream=None):
    """Gradients of ``linear_prefill`` for L = sum <d_o, o> + <d_final_state, S_T>.

    d_o: o's shape and type; d_final_state: fp32 or None (zero). Returns a dict:
    ``dq``, ``dk``, ``dv`` in q's type, ``dlog_decay`` in log_decay's shape (fp32;
    None without a decay or when not wanted; with decay="head" the sum over
    every token) and ``d_initial_state`` (fp32; None when not wanted)."""
    return _backward(q, k, v, log_decay, d_o, None, initial_state, d_final_state, decay, scale, want_decay_grad,
                     want_initial_state_grad, workspace, None, stream)


def linear_varlen_prefill_backward(q, k, v, log_decay, d_o, cu_seqlens, initial_state=None, d_final_state=None, *,
                                   decay: str = "token", scale: float = 1.0, want_decay_grad: bool = True,
                                   want_initial_state_grad: bool = True, workspace=None, device_status=None,
                                   stream=None):
    """Gradients of ``linear_varlen_prefill`` (packed sequences): the dict of
    ``linear_prefill_backward``."""
    if cu_seqlens is None:
        raise ValueError("cu_seqlens is required")
    return _backward(q, k, v, log_decay, d_o, cu_seqlens, initial_state, d_final_state, decay, scale, want_decay_grad,
                     want_initial_state_grad, workspace, device_status, stream)


def linear_decode_step(q, k, v, log_decay, state, *, decay: str = "token", scale: float = 1.0, out=None, stream=None):
    """One token of ``linear_prefill`` per (sequence, head); ``state`` [N, H,
    d_k, d_v] fp32 is updated in place. q, k: [N, H, d_k]; v: [N, H, d_v];
    log_decay [N, H], [H] or None. Returns o [N, H, d_v]."""
    lib = load()
    dev, (N,), H, dk, dv, strides = _qkv(q, k, v, 1)
    code = _dtype_code(q)
    kind, g = _check_decay(decay, log_decay, (N,), H, dev)
    if state is None:
        raise ValueError("state is required")
    _state(state, "state", (N, H, dk, dv), dev)
    with _on(stream):
        out = _out(out, "out", tuple(v.shape), v.dtype, dev)
    _check(lib, lib.kda_linear_decode_step(_ptr(q), _ptr(k), _ptr(v), code, *strides, _ptr(g), kind, float(scale),
                                           _ptr(state), _ptr(out), N, H, dk, dv, _stream(stream)))
    return out


def linear_decode_step_slots(q, k, v, log_decay, state_pool, slots, *, decay: str = "token", scale: float = 1.0,
                             out=None, device_status=None, stream=None):
    """``linear_decode_step`` on ``state_pool[slots[n]]`` ([P, H, d_k, d_v] fp32,
    updated in place; slots int32 [N], ``-1 - s`` starts slot s from zeros). A
    slot outside [0, P) is skipped and sets KDA_DEV_BAD_SLOT in ``device_status``."""
    lib = load()
    dev, (N,), H, dk, dv, strides = _qkv(q, k, v, 1)
    code = _dtype_code(q)
    kind, g = _check_decay(decay, log_decay, (N,), H, dev)
    _need(slots, "slots", torch.int32, dev)
    _need(state_pool, "state_pool", torch.float32, dev)
    if slots.shape != (N,) or state_pool.dim() != 4 or tuple(state_pool.shape[1:]) != (H, dk, dv):
        raise ValueError("shape mismatch among q, k, v, slots, state_pool")
    if device_status is not None:
        _need(device_status, "device_status", torch.int32, dev)
    with _on(stream):
        out = _out(out, "out", tuple(v.shape), v.dtype, dev)
    _check(lib, lib.kda_linear_decode_step_slots(_ptr(q), _ptr(k), _ptr(v), code, *strides, _ptr(g), kind, float(scale),
                                                 _ptr(state_pool), _ptr(slots), state_pool.shape[0], _ptr(out), N, H,
                                                 dk, dv, _ptr(device_status), _stream(stream)))
    return out


# ---------------------------------------------------------------- norm and rotary positions
def rope_table(max_position: int, rotary: int, *, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
               original_max_position: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0, device=None):
    """Cosines and sines of position times frequency, [max_position, rotary]
    fp32 (rotary / 2 cosines, then rotary / 2 sines), computed in 64 bits.

    Channel pair i turns by base^(-2 i / rotary) per position. ``scaling``:
    "linear" divides every frequency by ``factor``; "ntk" scales the base so that
    the slowest pair is divided by ``factor`` and the fastest keeps its pace;
    "yarn" (Peng et al. 2023) divides the pairs that turn fewer than
    ``beta_slow`` times over ``original_max_position``, keeps those that turn
    more than ``beta_fast`` times, blends in between, and multiplies cosines and
    sines by 0.1 ln(factor) + 1."""
    if rotary <= 0 or rotary % 2 or max_position <= 0:
        raise ValueError("max_position must be positive and rotary a positive even number")
    if not factor >= 1.0:
        raise ValueError("factor must be at least 1")
    i = torch.arange(0, rotary, 2, dtype=torch.float64) / rotary
    gain = 1.0
    if scaling == "none":
        f = base ** -i
    elif scaling == "linear":
        f = base ** -i / factor
    elif scaling == "ntk":
        if rotary < 4:
            raise ValueError("scaling='ntk' needs at least two channel pairs")
        f = (base * factor ** (rotary / (rotary - 2))) ** -i
    elif scaling == "yarn":
        if original_max_position <= 0:
            raise ValueError("scaling='yarn' needs original_max_position")
        f = base ** -i
        turns = original_max_position * f / (2 * math.pi)
        keep = ((turns - beta_slow) / (beta_fast - beta_slow)).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
        gain = 0.1 * math.log(factor) + 1.0
    else:
        raise ValueError("scaling must be one of ['linear', 'none', 'ntk', 'yarn']")
    a = torch.arange(max_position, dtype=torch.float64)[:, None] * f
    table = (torch.cat([a.cos(), a.sin()], -1) * gain).float()
    if device is None:
        device = torch.device("cuda", torch.cuda.current_device())
    return table.to(device).contiguous()


@functools.lru_cache(maxsize=None)
def _weight_grad_bytes(d: int) -> int:
    return int(load().kda_qk_norm_rope_backward_workspace_bytes(d))


def _norm_rope_inputs(q, k, positions, table, q_weight, k_weight, norm, layout):
    if q is None or q.dim() < 3:
        raise ValueError("q must be [.., H_q, d]")
    lead = q.dim() - 2
    qs = _view(q, "q", lead)
    dev = q.device
    ks = _view(k, "k", lead, q.dtype, dev)
    if k.shape[:-2] != q.shape[:-2] or k.shape[-1] != q.shape[-1]:
        raise ValueError("q and k must have the same leading axes and head size")
    n, d = math.prod(q.shape[:-2]), q.shape[-1]
    rot, max_position = 0, 0
    if table is not None:
        _need(table, "rope_table", torch.float32, dev)
        _need(positions, "positions", torch.int32, dev)
        if table.dim() != 2 or positions.shape != q.shape[:-2]:
            raise ValueError("rope_table must be [max_position, rotary] and positions have q's leading axes")
        max_position, rot = table.shape
    elif positions is not None:
        raise ValueError("positions need a rope_table")
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None:
            _need(w, name, torch.float32, dev)
            if w.shape != (d,):
                raise ValueError(f"{name} must be {(d,)}, got {tuple(w.shape)}")
    return (dev, n, d, q.shape[-2], k.shape[-2], _dtype_code(q), qs, ks, max_position, rot,
            _kind(ROPE_LAYOUTS, layout, "layout"), _kind(NORMS, norm, "norm"))


def qk_norm_rope(q, k, positions=None, rope_table=None, q_weight=None, k_weight=None, *, norm: str = "rms",
                 eps: float = 1e-6, layout: str = "half", q_out=None, k_out=None, device_status=None, stream=None):
    """The norm of every query and key head and the rotary positions, in one
    pass: w * x / norm(x), then the first ``rope_table.shape[1]`` channels turned.

    q: [.., H_q, d], k: [.., H_k, d] (bf16 or fp32; slices of a fused projection
    are taken as they are); positions: int32 [..]; rope_table: see
    :func:`rope_table`, None for no rotation; q_weight, k_weight: fp32 [d] or
    None; norm: "l2" (x / sqrt(sum x^2 + eps)), "rms" (the mean instead of the
    sum) or "none"; layout: channel pairs (i, i + rotary / 2) ("half") or
    (2 i, 2 i + 1) ("interleaved"). q_out, k_out may be q, k themselves.
    Returns (q_out, k_out), contiguous, in q's type. A token whose position lies
    outside the table is left out and sets KDA_DEV_BAD_POSITION in
    ``device_status`` (int32 [1])."""
    lib = load()
    dev, n, d, hq, hk, code, qs, ks, P, rot, lay, nk = _norm_rope_inputs(q, k, positions, rope_table, q_weight,
                                                                         k_weight, norm, layout)
    if device_status is not None:
        _need(device_status, "device_status", torch.int32, dev)
    with _on(stream):
        q_out = _out(q_out, "q_out", tuple(q.shape), q.dtype, dev)
        k_out = _out(k_out, "k_out", tuple(k.shape), q.dtype, dev)
    _check(lib, lib.kda_qk_norm_rope(_ptr(q), _ptr(k), code, qs, ks, _ptr(positions), _ptr(rope_table), P, rot, lay,
                                     _ptr(q_weight), _ptr(k_weight), nk, float(eps), _ptr(q_out), _ptr(k_out), n, hq,
                                     hk, d, _ptr(device_status), _stream(stream)))
    return q_out, k_out


def qk_norm_rope_backward(q, k, dq_out, dk_out, positions=None, rope_table=None, q_weight=None, k_weight=None, *,
                          norm: str = "rms", eps: float = 1e-6, layout: str = "half", workspace=None,
                          device_status=None, stream=None):
    """Gradients of ``qk_norm_rope`` for L = sum <dq_out, q_out> + <dk_out, k_out>
    (dq_out, dk_out contiguous, in q's type). Returns a dict: ``dq``, ``dk`` in
    q's type, ``dq_weight``, ``dk_weight`` (fp32 [d]; None without that weight)."""
    lib = load()
    dev, n, d, hq, hk, code, qs, ks, P, rot, lay, nk = _norm_rope_inputs(q, k, positions, rope_table, q_weight,
                                                                         k_weight, norm, layout)
    for t, x, name in ((dq_out, q, "dq_out"), (dk_out, k, "dk_out")):
        _need(t, name, q.dtype, dev)
        if t.shape != x.shape:
            raise ValueError(f"{name} must be {tuple(x.shape)}, got {tuple(t.shape)}")
    if device_status is not None:
        _need(device_status, "device_status", torch.int32, dev)
    with _on(stream):
        out = {"dq": torch.empty(q.shape, dtype=q.dtype, device=dev),
               "dk": torch.empty(k.shape, dtype=q.dtype, device=dev),
               "dq_weight": None if q_weight is None else torch.empty(d, dtype=torch.float32, device=dev),
               "dk_weight": None if k_weight is None else torch.empty(d, dtype=torch.float32, device=dev)}
        ws, size = None, 0
        if q_weight is not None or k_weight is not None:
            ws, size = _space(workspace, _weight_grad_bytes(d), dev)
    _check(lib, lib.kda_qk_norm_rope_backward(_ptr(q), _ptr(k), _ptr(dq_out), _ptr(dk_out), code, qs, ks,
                                              _ptr(positions), _ptr(rope_table), P, rot, lay, _ptr(q_weight),
                                              _ptr(k_weight), nk, float(eps), _ptr(out["dq"]), _ptr(out["dk"]),
                                              _ptr(out["dq_weight"]), _ptr(out["dk_weight"]), n, hq, hk, d, _ptr(ws),
                                              size, _ptr(device_status), _stream(stream)))
    return out
