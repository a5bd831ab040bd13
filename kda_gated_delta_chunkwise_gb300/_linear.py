"""Linear attention with a decay, and the norm and rotary positions in front
of it (the kda_linear_* and kda_qk_norm_rope* entry points of include/kda.h).

Marshalling only, like the rest of the binding: checks of shapes, types and
strides, outputs and workspaces through PyTorch, raw pointers and a CUDA
stream. There is no fallback.

q, k and v may be slices of a wider tensor (a fused projection): their last two
axes must be contiguous and their tokens evenly spaced. A call runs on its
tensors' device, current or not. Every call also takes ``stream``, of that
device: it then runs there, its outputs and workspace are allocated for that
stream, and the inputs must be ready on it. They may be let go of after the call,
though they come from another stream.
"""
from __future__ import annotations

import functools
import math

import torch

from . import _binding
from ._binding import _check, _dtype_code

# Host time counts for one token of one sequence: these stand for the
# binding's helpers of the same names without the objects they make per call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def load():
    return _binding._lib or _binding.load()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(index: int):
    """The device's current stream."""
    return _raw_stream(index) if _raw_stream is not None else torch.cuda.current_stream(index).cuda_stream


# decay kinds: one log decay per token and head, one per head, none
DECAYS = {"token": 0, "head": 1, "none": 2}
NORMS = {"none": 0, "l2": 1, "rms": 2}
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}


def _kind(kinds: dict, value: str, name: str) -> int:
    if value not in kinds:
        raise ValueError(f"{name} must be one of {sorted(kinds)}")
    return kinds[value]


def _plain(t, name: str, dtype, index: int, shape=None):
    """Checks a contiguous tensor on CUDA device ``index``."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")


def _view(t, name: str, lead: int, dtype=None, index: int = -1) -> int:
    """The token stride of ``t`` [*lead axes, H, d] (0: contiguous), whose heads
    are contiguous and whose tokens are evenly spaced over all lead axes."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dim() != lead + 2:
        raise ValueError(f"{name} must have {lead + 2} dimensions, got {t.dim()}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if index >= 0 and t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
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


def _check_decay(decay: str, log_decay, lead: tuple, H: int, index: int):
    if decay == "none":
        return 2, None
    kind = _kind(DECAYS, decay, "decay")
    _plain(log_decay, "log_decay", torch.float32, index)
    want = (*lead, H) if kind == 0 else (H,)
    if log_decay.shape != want:
        raise ValueError(f"log_decay must be {tuple(want)} for decay={decay!r}, got {tuple(log_decay.shape)}")
    return kind, log_decay


def _qkv(q, k, v, lead: int):
    """Checks q, k, v; returns (device index, lead shape, H, d_k, d_v, the three token strides)."""
    qs = _view(q, "q", lead)
    index, dtype, shape = q.get_device(), q.dtype, q.shape
    ks, vs = _view(k, "k", lead, dtype, index), _view(v, "v", lead, dtype, index)
    if k.shape != shape or v.shape[:-1] != shape[:-1]:
        raise ValueError("shape mismatch among q, k, v")
    return index, shape[:lead], shape[-2], shape[-1], v.shape[-1], (qs, ks, vs)


def _state(t, name: str, shape: tuple, index: int):
    if t is not None:
        _plain(t, name, torch.float32, index, shape)


def _out(t, name: str, like, shape, dtype, index: int):
    if t is None:
        if like.shape == shape and like.dtype == dtype and like.is_contiguous():
            return torch.empty_like(like)  # the same tensor, half a microsecond sooner
        return torch.empty(shape, dtype=dtype, device=like.device)
    _plain(t, name, dtype, index, torch.Size(shape))
    return t


def _space(workspace, nbytes: int, like):
    """The caller's workspace or a new one; (tensor, bytes)."""
    if workspace is None:
        return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=like.device), nbytes
    _plain(workspace, "workspace", None, like.get_device())
    return workspace, workspace.numel() * workspace.element_size()


@functools.lru_cache(maxsize=256)
def _size(name: str, n: int, T: int, H: int, dk: int, dv: int, code: int) -> int:
    """Workspace bytes: a function of the sizes alone."""
    return int(getattr(load(), name + "_workspace_bytes")(n, T, H, dk, dv, code))


def _bytes(name: str, n: int, T: int, H: int, dk: int, dv: int, dtype) -> int:
    return _size(name, n, T, H, dk, dv, _dtype_code(torch.empty(0, dtype=dtype)))


def _on_stream(f):
    """Runs ``f`` on q's device, with its ``stream`` current where one is given, so that what it allocates belongs to
    that stream. A launch goes to the current device, whatever the pointers and the stream's handle belong to."""
    @functools.wraps(f)
    def g(*args, stream=None, **kw):
        q = args[0] if args else kw.get("q")
        index = q.get_device() if isinstance(q, torch.Tensor) else -1  # -1: not a CUDA tensor, refused by f
        if stream is not None:
            if index >= 0 and stream.device.index != index:
                raise ValueError(f"stream is on {stream.device}, q on cuda:{index}")
            with torch.cuda.stream(stream):
                out = f(*args, **kw)
            for t in (*args, *kw.values()):  # the allocator keeps their memory until the stream is past the call
                if isinstance(t, torch.Tensor):
                    t.record_stream(stream)
            return out
        if index >= 0 and index != torch.cuda.current_device():
            with torch.cuda.device(index):
                return f(*args, **kw)
        return f(*args, **kw)
    return g


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
             workspace, device_status):
    lib = load()
    packed = cu_seqlens is not None
    index, lead, H, dk, dv, strides = _qkv(q, k, v, 1 if packed else 2)
    code = _dtype_code(q)
    kind, g = _check_decay(decay, log_decay, lead, H, index)
    if packed:
        N, T = _packed(cu_seqlens, device_status, index), lead[0]
    else:
        N, T = lead
    _state(initial_state, "initial_state", (N, H, dk, dv), index)
    name = "kda_linear_varlen_prefill" if packed else "kda_linear_prefill"
    out = _out(out, "out", v, v.shape, v.dtype, index)
    if final_state is not None or output_final_state:
        final_state = _out(final_state, "final_state", v if initial_state is None else initial_state, (N, H, dk, dv),
                           torch.float32, index)
    ws, size = _space(workspace, _size(name, N, T, H, dk, dv, code), v)
    head = (q.data_ptr(), k.data_ptr(), v.data_ptr(), code, *strides, _ptr(g), kind, scale, _ptr(initial_state),
            out.data_ptr(), _ptr(final_state))
    if packed:
        st = lib.kda_linear_varlen_prefill(*head, cu_seqlens.data_ptr(), N, T, H, dk, dv, ws.data_ptr(), size,
                                           _ptr(device_status), _stream(index))
    else:
        st = lib.kda_linear_prefill(*head, N, T, H, dk, dv, ws.data_ptr(), size, _stream(index))
    _check(lib, st)
    return out, final_state


def _packed(cu_seqlens, device_status, index: int) -> int:
    """Checks the arguments of a packed batch; returns the number of sequences."""
    _plain(cu_seqlens, "cu_seqlens", torch.int32, index)
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be one-dimensional with N + 1 entries")
    if device_status is not None:
        _plain(device_status, "device_status", torch.int32, index)
    return cu_seqlens.numel() - 1


@_on_stream
def linear_prefill(q, k, v, log_decay=None, initial_state=None, *, decay: str = "token", scale: float = 1.0,
                   output_final_state: bool = True, out=None, final_state=None, workspace=None):
    """Linear attention with a decay over B equal-length sequences:
    S_t = e^{g_t} S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t.

    q, k: [B, T, H, d_k]; v: [B, T, H, d_v] (bf16 or fp32, the same type);
    log_decay: natural logarithms <= 0, fp32 [B, T, H] (decay="token"), [H]
    (decay="head") or None (decay="none"); -inf, or anything <= -128, resets
    the state, a NaN makes it NaN up to the next reset; initial_state: [B, H, d_k, d_v] fp32 or None (zeros).
    Returns (o [B, T, H, d_v] in v's type, final_state fp32 or None).
    """
    return _prefill(q, k, v, log_decay, None, initial_state, decay, scale, output_final_state, out, final_state,
                    workspace, None)


@_on_stream
def linear_varlen_prefill(q, k, v, log_decay, cu_seqlens, initial_state=None, *, decay: str = "token",
                          scale: float = 1.0, output_final_state: bool = True, out=None, final_state=None,
                          workspace=None, device_status=None):
    """``linear_prefill`` over N sequences packed along the token axis:
    q, k: [T_total, H, d_k]; v: [T_total, H, d_v]; log_decay [T_total, H]
    (decay="token"); cu_seqlens: int32 [N + 1] on the device; initial_state:
    [N, H, d_k, d_v]. ``device_status`` (int32 [1]) receives KDA_DEV_OK or
    KDA_DEV_BAD_CU_SEQLENS, in which case nothing else is written."""
    if cu_seqlens is None:
        raise ValueError("cu_seqlens is required")
    return _prefill(q, k, v, log_decay, cu_seqlens, initial_state, decay, scale, output_final_state, out, final_state,
                    workspace, device_status)


def _backward(q, k, v, log_decay, d_o, cu_seqlens, initial_state, d_final_state, decay, scale, want_decay_grad,
              want_initial_state_grad, workspace, device_status):
    lib = load()
    packed = cu_seqlens is not None
    index, lead, H, dk, dv, strides = _qkv(q, k, v, 1 if packed else 2)
    code = _dtype_code(q)
    kind, g = _check_decay(decay, log_decay, lead, H, index)
    _plain(d_o, "d_o", q.dtype, index, v.shape)
    if packed:
        N, T = _packed(cu_seqlens, device_status, index), lead[0]
    else:
        N, T = lead
    for t, n in ((initial_state, "initial_state"), (d_final_state, "d_final_state")):
        _state(t, n, (N, H, dk, dv), index)
    name = "kda_linear_varlen_prefill_backward" if packed else "kda_linear_prefill_backward"
    out = {"dq": torch.empty(q.shape, dtype=q.dtype, device=q.device),
           "dk": torch.empty(k.shape, dtype=q.dtype, device=q.device),
           "dv": torch.empty(v.shape, dtype=q.dtype, device=q.device),
           "dlog_decay": torch.empty_like(g) if g is not None and want_decay_grad else None,
           "d_initial_state": torch.empty((N, H, dk, dv), dtype=torch.float32, device=q.device)
           if want_initial_state_grad else None}
    ws, size = _space(workspace, _size(name, N, T, H, dk, dv, code), q)
    head = (q.data_ptr(), k.data_ptr(), v.data_ptr(), code, *strides, _ptr(g), kind, scale, _ptr(initial_state),
            d_o.data_ptr(), _ptr(d_final_state), *(_ptr(t) for t in out.values()))
    if packed:
        st = lib.kda_linear_varlen_prefill_backward(*head, cu_seqlens.data_ptr(), N, T, H, dk, dv, ws.data_ptr(), size,
                                                    _ptr(device_status), _stream(index))
    else:
        st = lib.kda_linear_prefill_backward(*head, N, T, H, dk, dv, ws.data_ptr(), size, _stream(index))
    _check(lib, st)
    return out


@_on_stream
def linear_prefill_backward(q, k, v, log_decay, d_o, initial_state=None, d_final_state=None, *, decay: str = "token",
                            scale: float = 1.0, want_decay_grad: bool = True, want_initial_state_grad: bool = True,
                            workspace=None):
    """Gradients of ``linear_prefill`` for L = sum <d_o, o> + <d_final_state, S_T>.

    d_o: o's shape and type; d_final_state: fp32 or None (zero). Returns a dict:
    ``dq``, ``dk``, ``dv`` in q's type, ``dlog_decay`` in log_decay's shape (fp32;
    None without a decay or when not wanted; with decay="head" the sum over
    every token) and ``d_initial_state`` (fp32; None when not wanted)."""
    return _backward(q, k, v, log_decay, d_o, None, initial_state, d_final_state, decay, scale, want_decay_grad,
                     want_initial_state_grad, workspace, None)


@_on_stream
def linear_varlen_prefill_backward(q, k, v, log_decay, d_o, cu_seqlens, initial_state=None, d_final_state=None, *,
                                   decay: str = "token", scale: float = 1.0, want_decay_grad: bool = True,
                                   want_initial_state_grad: bool = True, workspace=None, device_status=None):
    """Gradients of ``linear_varlen_prefill`` (packed sequences): the dict of
    ``linear_prefill_backward``."""
    if cu_seqlens is None:
        raise ValueError("cu_seqlens is required")
    return _backward(q, k, v, log_decay, d_o, cu_seqlens, initial_state, d_final_state, decay, scale, want_decay_grad,
                     want_initial_state_grad, workspace, device_status)


@_on_stream
def linear_decode_step(q, k, v, log_decay, state, *, decay: str = "token", scale: float = 1.0, out=None):
    """One token of ``linear_prefill`` per (sequence, head); ``state`` [N, H,
    d_k, d_v] fp32 is updated in place. q, k: [N, H, d_k]; v: [N, H, d_v];
    log_decay [N, H], [H] or None. Returns o [N, H, d_v]."""
    lib = load()
    index, (N,), H, dk, dv, strides = _qkv(q, k, v, 1)
    kind, g = _check_decay(decay, log_decay, (N,), H, index)
    _plain(state, "state", torch.float32, index, (N, H, dk, dv))
    out = _out(out, "out", v, v.shape, v.dtype, index)
    _check(lib, lib.kda_linear_decode_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), _dtype_code(q), *strides, _ptr(g),
                                           kind, scale, state.data_ptr(), out.data_ptr(), N, H, dk, dv,
                                           _stream(index)))
    return out


@_on_stream
def linear_decode_step_slots(q, k, v, log_decay, state_pool, slots, *, decay: str = "token", scale: float = 1.0,
                             out=None, device_status=None):
    """``linear_decode_step`` on ``state_pool[slots[n]]`` ([P, H, d_k, d_v] fp32,
    updated in place; slots int32 [N], ``-1 - s`` starts slot s from zeros). A
    slot outside [0, P) is skipped and sets KDA_DEV_BAD_SLOT in ``device_status``."""
    lib = load()
    index, (N,), H, dk, dv, strides = _qkv(q, k, v, 1)
    kind, g = _check_decay(decay, log_decay, (N,), H, index)
    _plain(slots, "slots", torch.int32, index, (N,))
    _plain(state_pool, "state_pool", torch.float32, index)
    pool = state_pool.shape
    if len(pool) != 4 or pool[1:] != (H, dk, dv):
        raise ValueError(f"state_pool must be [P, {H}, {dk}, {dv}], got {tuple(pool)}")
    if device_status is not None:
        _plain(device_status, "device_status", torch.int32, index)
    out = _out(out, "out", v, v.shape, v.dtype, index)
    _check(lib, lib.kda_linear_decode_step_slots(q.data_ptr(), k.data_ptr(), v.data_ptr(), _dtype_code(q), *strides,
                                                 _ptr(g), kind, scale, state_pool.data_ptr(), slots.data_ptr(),
                                                 pool[0], out.data_ptr(), N, H, dk, dv, _ptr(device_status),
                                                 _stream(index)))
    return out


# ---------------------------------------------------------------- norm and rotary positions
def rope_table(max_position: int, rotary: int, *, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
               original_max_position: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0, device=None):
    """Cosines and sines of position times frequency, [max_position, rotary]
    fp32 (rotary / 2 cosines, then rotary / 2 sines), computed in 64 bits.

    Channel pair i turns by base^(-2 i / rotary) per position. ``scaling``:
    "linear" divides every frequency by ``factor``; "ntk" scales the base so that
    the slowest pair is divided by ``factor`` and the fastest keeps its pace;
    "yarn" (Peng et al. 2023) divides by ``factor`` the frequencies of the pairs
    that turn fewer than ``beta_slow`` times over ``original_max_position``, keeps
    those of the pairs that turn more than ``beta_fast`` times, blends in between
    in proportion to the number of turns, as the paper's formula does, and
    multiplies cosines and sines by 0.1 ln(factor) + 1. (A model that was trained
    with the blend in proportion to the pair's index i needs a table made by that
    rule: the two agree outside the blend alone.)"""
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
        if not 0.0 <= beta_slow < beta_fast < math.inf:
            raise ValueError("scaling='yarn' needs 0 <= beta_slow < beta_fast")
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


def _norm_rope_inputs(q, k, positions, table, q_weight, k_weight, norm, layout, device_status):
    if q is None or q.dim() < 3:
        raise ValueError("q must be [.., H_q, d]")
    lead = q.dim() - 2
    qs = _view(q, "q", lead)
    index, shape = q.get_device(), q.shape
    ks = _view(k, "k", lead, q.dtype, index)
    if k.shape[:-2] != shape[:-2] or k.shape[-1] != shape[-1]:
        raise ValueError("q and k must have the same leading axes and head size")
    n, d = (shape[0] if lead == 1 else math.prod(shape[:-2])), shape[-1]
    rot, max_position = 0, 0
    if table is not None:
        _plain(table, "rope_table", torch.float32, index)
        _plain(positions, "positions", torch.int32, index)
        if table.dim() != 2 or positions.shape != shape[:-2]:
            raise ValueError("rope_table must be [max_position, rotary] and positions have q's leading axes")
        max_position, rot = table.shape
    elif positions is not None:
        raise ValueError("positions need a rope_table")
    if q_weight is not None:
        _plain(q_weight, "q_weight", torch.float32, index, (d,))
    if k_weight is not None:
        _plain(k_weight, "k_weight", torch.float32, index, (d,))
    if device_status is not None:
        _plain(device_status, "device_status", torch.int32, index)
    return (index, n, d, shape[-2], k.shape[-2], _dtype_code(q), qs, ks, max_position, rot,
            _kind(ROPE_LAYOUTS, layout, "layout"), _kind(NORMS, norm, "norm"))


@_on_stream
def qk_norm_rope(q, k, positions=None, rope_table=None, q_weight=None, k_weight=None, *, norm: str = "rms",
                 eps: float = 1e-6, layout: str = "half", q_out=None, k_out=None, device_status=None):
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
    index, n, d, hq, hk, code, qs, ks, P, rot, lay, nk = _norm_rope_inputs(q, k, positions, rope_table, q_weight,
                                                                           k_weight, norm, layout, device_status)
    q_out = _out(q_out, "q_out", q, q.shape, q.dtype, index)
    k_out = _out(k_out, "k_out", k, k.shape, q.dtype, index)
    _check(lib, lib.kda_qk_norm_rope(q.data_ptr(), k.data_ptr(), code, qs, ks, _ptr(positions), _ptr(rope_table), P, rot,
                                     lay, _ptr(q_weight), _ptr(k_weight), nk, eps, q_out.data_ptr(), k_out.data_ptr(),
                                     n, hq, hk, d, _ptr(device_status), _stream(index)))
    return q_out, k_out


@_on_stream
def qk_norm_rope_backward(q, k, dq_out, dk_out, positions=None, rope_table=None, q_weight=None, k_weight=None, *,
                          norm: str = "rms", eps: float = 1e-6, layout: str = "half", workspace=None,
                          device_status=None):
    """Gradients of ``qk_norm_rope`` for L = sum <dq_out, q_out> + <dk_out, k_out>
    (dq_out, dk_out contiguous, in q's type). Returns a dict: ``dq``, ``dk`` in
    q's type, ``dq_weight``, ``dk_weight`` (fp32 [d]; None without that weight)."""
    lib = load()
    index, n, d, hq, hk, code, qs, ks, P, rot, lay, nk = _norm_rope_inputs(q, k, positions, rope_table, q_weight,
                                                                           k_weight, norm, layout, device_status)
    _plain(dq_out, "dq_out", q.dtype, index, q.shape)
    _plain(dk_out, "dk_out", q.dtype, index, k.shape)
    out = {"dq": torch.empty(q.shape, dtype=q.dtype, device=q.device),
           "dk": torch.empty(k.shape, dtype=q.dtype, device=q.device),
           "dq_weight": None if q_weight is None else torch.empty_like(q_weight),
           "dk_weight": None if k_weight is None else torch.empty_like(k_weight)}
    ws, size = None, 0
    if q_weight is not None or k_weight is not None:
        ws, size = _space(workspace, _weight_grad_bytes(d), q)
    _check(lib, lib.kda_qk_norm_rope_backward(q.data_ptr(), k.data_ptr(), dq_out.data_ptr(), dk_out.data_ptr(), code, qs,
                                              ks, _ptr(positions), _ptr(rope_table), P, rot, lay, _ptr(q_weight),
                                              _ptr(k_weight), nk, eps, *(_ptr(t) for t in out.values()), n, hq, hk, d,
                                              _ptr(ws), size, _ptr(device_status), _stream(index)))
    return out
