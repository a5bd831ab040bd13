"""What the linear-attention and query/key norm entry points refuse, before
anything is launched, and the host-made rotary table. No GPU."""
import ctypes
import math

import pytest
import torch

import kda_gated_delta_chunkwise_gb300 as kda
from kda_gated_delta_chunkwise_gb300 import build

P = ctypes.c_void_p(0x1000)
OK, INVALID, UNSUPPORTED, CUDA, WORKSPACE = 0, 1, 2, 3, 5
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    build.build()
    return kda.load()


def _prefill(lib, q=P, dtype=1, qs=0, ks=0, vs=0, g=P, decay=0, scale=1.0, o=P, B=1, T=4, H=2, dk=128, dv=128, ws=P,
             size=BIG, s0=None):
    return lib.kda_linear_prefill(q, P, P, dtype, qs, ks, vs, g, decay, scale, s0, o, None, B, T, H, dk, dv, ws, size,
                                  None)


def _backward(lib, d_o=P, dq=P, dg=P, decay=0, ws=P, size=BIG, **kw):
    a = dict(dtype=1, B=1, T=4, H=2, dk=128, dv=128)
    a.update(kw)
    return lib.kda_linear_prefill_backward(P, P, P, a["dtype"], 0, 0, 0, P, decay, 1.0, None, d_o, None, dq, P, P, dg,
                                           None, a["B"], a["T"], a["H"], a["dk"], a["dv"], ws, size, None)


def test_prefill_refusals(lib):
    assert _prefill(lib, dtype=7) == INVALID
    assert _prefill(lib, decay=3) == INVALID
    assert _prefill(lib, H=0) == INVALID
    assert _prefill(lib, B=-1) == INVALID and _prefill(lib, T=-1) == INVALID
    assert _prefill(lib, dk=96) == UNSUPPORTED and b"64 or 128" in lib.kda_last_error()
    assert _prefill(lib, dv=0) == INVALID
    assert _prefill(lib, scale=math.nan) == INVALID and _prefill(lib, scale=math.inf) == INVALID
    assert _prefill(lib, q=None) == INVALID and b"q must not be NULL" in lib.kda_last_error()
    assert _prefill(lib, q=ctypes.c_void_p(0x1008)) == INVALID and b"16-byte" in lib.kda_last_error()
    assert _prefill(lib, o=None) == INVALID
    assert _prefill(lib, g=None) == INVALID and _prefill(lib, g=ctypes.c_void_p(0x1002)) == INVALID
    assert _prefill(lib, s0=ctypes.c_void_p(0x1004)) == INVALID
    assert _prefill(lib, qs=255) == INVALID and _prefill(lib, qs=260) == INVALID  # below H * d; off 16 bytes
    assert _prefill(lib, ks=-256) == INVALID and _prefill(lib, vs=8) == INVALID
    assert _prefill(lib, B=1 << 16, T=1 << 16) == UNSUPPORTED
    assert _prefill(lib, B=1, T=1 << 30, H=1 << 12) == UNSUPPORTED
    assert _prefill(lib, ws=None) == WORKSPACE and _prefill(lib, size=16) == WORKSPACE
    assert _prefill(lib, ws=ctypes.c_void_p(0x1010)) == WORKSPACE
    assert _prefill(lib, B=0) == OK


def test_varlen_refusals(lib):
    def call(cu=P, N=2, T=10, status=None, size=BIG):
        return lib.kda_linear_varlen_prefill(P, P, P, 1, 0, 0, 0, P, 0, 1.0, None, P, None, cu, N, T, 2, 128, 128, P,
                                             size, status, None)
    assert call(cu=None) == INVALID and call(cu=ctypes.c_void_p(0x1002)) == INVALID
    assert call(status=ctypes.c_void_p(0x1002)) == INVALID
    assert call(N=-1) == INVALID and call(T=-1) == INVALID
    assert call(size=0) == WORKSPACE
    assert call(N=0) == OK


def test_backward_refusals(lib):
    assert _backward(lib, d_o=None) == INVALID and _backward(lib, dq=None) == INVALID
    assert _backward(lib, dg=ctypes.c_void_p(0x1002)) == INVALID
    assert _backward(lib, decay=9) == INVALID
    assert _backward(lib, dk=32) == UNSUPPORTED
    assert _backward(lib, ws=None) == WORKSPACE and _backward(lib, size=256) == WORKSPACE
    assert _backward(lib, B=0) == OK


def test_decode_refusals(lib):
    def call(q=P, decay=0, g=P, state=P, slots=P, pool=4, N=1, H=2, dk=128, status=None, qs=0):
        return lib.kda_linear_decode_step_slots(q, P, P, 1, qs, 0, 0, g, decay, 1.0, state, slots, pool, P, N, H, dk,
                                                128, status, None)
    assert call(slots=None) == INVALID and call(pool=0) == INVALID
    assert call(state=None) == INVALID and call(q=None) == INVALID and call(g=None) == INVALID
    assert call(status=ctypes.c_void_p(0x1001)) == INVALID
    assert call(pool=1 << 30, H=8) == UNSUPPORTED
    assert call(dk=16) == UNSUPPORTED and call(N=-2) == INVALID and call(qs=4) == INVALID
    assert lib.kda_linear_decode_step(P, P, P, 1, 0, 0, 0, P, 0, 1.0, None, P, 1, 2, 128, 128, None) == INVALID
    assert lib.kda_linear_decode_step(P, P, P, 1, 0, 0, 0, P, 0, 1.0, P, P, 0, 2, 128, 128, None) == OK


def test_norm_rope_refusals(lib):
    def call(dtype=1, qs=0, pos=P, table=P, maxp=10, rot=64, layout=0, wq=None, norm=2, eps=1e-6, qo=P, n=3, hq=2, hk=2,
             d=128, status=None, q=P):
        return lib.kda_qk_norm_rope(q, P, dtype, qs, 0, pos, table, maxp, rot, layout, wq, None, norm, eps, qo, P, n,
                                    hq, hk, d, status, None)
    assert call(dtype=5) == INVALID and call(norm=3) == INVALID and call(layout=2) == INVALID
    assert call(d=96) == UNSUPPORTED and call(d=0) == INVALID
    assert call(rot=24) == UNSUPPORTED and call(rot=256) == INVALID and call(rot=-16) == INVALID
    assert call(maxp=0) == INVALID and call(pos=None) == INVALID and call(table=None) == INVALID
    assert call(eps=0.0) == INVALID and call(eps=math.nan) == INVALID
    assert call(qs=100) == INVALID and call(q=None) == INVALID and call(qo=None) == INVALID
    assert call(n=-1) == INVALID and call(hq=-1) == INVALID
    assert call(wq=ctypes.c_void_p(0x1002)) == INVALID and call(status=ctypes.c_void_p(0x1002)) == INVALID
    assert call(n=0) == OK

    def back(dw=P, ws=P, size=BIG, dy=P):
        return lib.kda_qk_norm_rope_backward(P, P, dy, P, 1, 0, 0, P, P, 10, 64, 0, P, P, 2, 1e-6, P, P, dw, dw, 3, 2,
                                             2, 128, ws, size, None, None)
    assert back(dy=None) == INVALID and back(ws=None) == WORKSPACE and back(size=8) == WORKSPACE


def test_workspace_sizes(lib):
    f = kda.linear_prefill_workspace_bytes
    assert 0 < f(1, 64, 2) < f(1, 4096, 2) and f(-1, 64, 2) == 0 and f(1, 64, 0) == 0
    assert kda.linear_prefill_backward_workspace_bytes(1, 4096, 2) > f(1, 4096, 2)
    assert kda.linear_varlen_prefill_workspace_bytes(3, 0, 2) > 0


def test_python_refusals():
    x = torch.zeros(1, 4, 2, 128)
    with pytest.raises(ValueError, match="CUDA"):
        kda.linear_prefill(x, x, x, torch.zeros(1, 4, 2))
    with pytest.raises(ValueError, match="CUDA"):
        kda.qk_norm_rope(x, x)
    with pytest.raises(ValueError):
        kda.linear_prefill(None, x, x)
    with pytest.raises(ValueError, match="dimensions"):
        kda.linear_varlen_prefill(x, x, x, None, torch.zeros(2))


def test_rope_table():
    t = kda.rope_table(50, 8, base=100.0, device="cpu")
    assert t.shape == (50, 8) and t.dtype == torch.float32
    for pos, i in ((0, 0), (7, 1), (49, 3)):
        a = pos * 100.0 ** (-2 * i / 8)
        assert abs(t[pos, i].item() - math.cos(a)) < 1e-6 and abs(t[pos, 4 + i].item() - math.sin(a)) < 1e-6
    lin = kda.rope_table(50, 8, base=100.0, scaling="linear", factor=2.0, device="cpu")
    assert torch.allclose(lin[::2], t[:25], atol=1e-6)
    ntk = kda.rope_table(50, 8, base=100.0, scaling="ntk", factor=4.0, device="cpu")
    assert torch.allclose(ntk[:, 0], t[:, 0]) and torch.allclose(ntk[::4, 3], t[:13, 3], atol=1e-6)
    yarn = kda.rope_table(512, 16, scaling="yarn", factor=8.0, original_max_position=64, device="cpu")
    gain = 0.1 * math.log(8.0) + 1
    slow = kda.rope_table(512, 16, scaling="linear", factor=8.0, device="cpu")
    assert torch.allclose(yarn[:, 7], gain * slow[:, 7], atol=1e-6)
    for bad in (dict(scaling="other"), dict(factor=0.5), dict(scaling="yarn"), dict(scaling="ntk", rotary=2)):
        with pytest.raises(ValueError):
            kda.rope_table(**{**dict(max_position=10, rotary=16, device="cpu"), **bad})
    with pytest.raises(ValueError):
        kda.rope_table(10, 7, device="cpu")
