"""What window attention, its cache, the norms around a block and the rotary
positions of several axes refuse, before anything is launched. No GPU."""
import ctypes
import math

import pytest
import torch

import kda_gated_delta_chunkwise_gb300 as kda
from kda_gated_delta_chunkwise_gb300 import build

P = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1002)
OK, INVALID, UNSUPPORTED, CUDA, WORKSPACE = 0, 1, 2, 3, 5
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    build.build()
    return kda.load()


def _forward(lib, q=P, dtype=1, qs=0, ks=0, vs=0, scale=1.0, window=8, sinks=2, o=P, lse=P, B=1, T=4, hq=4, hk=2, d=128):
    return lib.kda_window_attention(q, P, P, dtype, qs, ks, vs, scale, window, sinks, o, lse, B, T, hq, hk, d, None)


def test_forward_refusals(lib):
    assert _forward(lib, dtype=7) == INVALID
    assert _forward(lib, hq=0) == INVALID and _forward(lib, hk=0) == INVALID and _forward(lib, hq=3) == INVALID
    assert b"multiple of H_k" in lib.kda_last_error()
    assert _forward(lib, hq=-4, hk=-2) == INVALID
    assert _forward(lib, d=96) == UNSUPPORTED and _forward(lib, d=0) == INVALID
    assert _forward(lib, B=-1) == INVALID and _forward(lib, T=-1) == INVALID
    assert _forward(lib, window=0) == INVALID and _forward(lib, window=-5) == INVALID
    assert _forward(lib, sinks=-1) == INVALID and _forward(lib, sinks=129) == UNSUPPORTED
    assert _forward(lib, scale=0.0) == INVALID and _forward(lib, scale=-1.0) == INVALID
    assert _forward(lib, scale=math.nan) == INVALID and _forward(lib, scale=math.inf) == INVALID
    assert _forward(lib, q=None) == INVALID and _forward(lib, q=ctypes.c_void_p(0x1008)) == INVALID
    assert _forward(lib, o=None) == INVALID and _forward(lib, lse=ODD) == INVALID
    assert _forward(lib, qs=511) == INVALID and _forward(lib, qs=516) == INVALID and _forward(lib, ks=128) == INVALID
    assert _forward(lib, vs=-256) == INVALID
    assert _forward(lib, B=1 << 16, T=1 << 16) == UNSUPPORTED
    assert _forward(lib, B=1, T=1 << 30, hq=1 << 12) == UNSUPPORTED
    assert _forward(lib, B=1, T=(1 << 30) + 1, hq=1, hk=1) == UNSUPPORTED
    assert _forward(lib, B=0) == OK and _forward(lib, T=0) == OK


def test_varlen_refusals(lib):
    def call(cu=P, N=2, T=10, status=None, ws=P, size=BIG):
        return lib.kda_window_varlen_attention(P, P, P, 1, 0, 0, 0, 1.0, 8, 2, P, P, cu, N, T, 4, 2, 128, ws, size, status,
                                               None)
    assert call(cu=None) == INVALID and call(cu=ODD) == INVALID and call(status=ODD) == INVALID
    assert call(N=-1) == INVALID and call(T=-1) == INVALID
    assert call(ws=None) == WORKSPACE and call(size=16) == WORKSPACE and call(ws=ctypes.c_void_p(0x1010)) == WORKSPACE
    assert call(N=0) == OK and call(N=0, T=0) == OK


def test_backward_refusals(lib):
    def call(out=P, lse=P, d_o=P, dq=P, dk=P, window=8, ws=P, size=BIG, d=128, T=300):
        return lib.kda_window_attention_backward(P, P, P, out, lse, d_o, 1, 0, 0, 0, 1.0, window, 2, dq, dk, P, 1, T, 4, 2,
                                                 d, ws, size, None)
    for name in ("out", "lse", "d_o", "dq", "dk"):
        assert call(**{name: None}) == INVALID and call(**{name: ODD}) == INVALID
    assert call(window=0) == INVALID and call(d=32) == UNSUPPORTED
    assert call(ws=None) == WORKSPACE and call(size=256) == WORKSPACE
    assert call(T=0) == OK


def test_cache_refusals(lib):
    def write(k=P, cu=P, slots=P, sinks=2, kc=P, pool=4, entries=10, N=2, T=5, hk=2, d=128, ks=0, status=None):
        return lib.kda_window_cache_write(k, P, 1, ks, 0, cu, slots, sinks, kc, P, pool, entries, N, T, hk, d, status, None)
    assert write(k=None) == INVALID and write(cu=None) == INVALID and write(slots=ODD) == INVALID and write(kc=None) == INVALID
    assert write(entries=2) == INVALID and write(entries=-1) == INVALID and write(pool=0) == INVALID
    assert write(sinks=129, entries=200) == UNSUPPORTED and write(sinks=-1) == INVALID and write(d=16) == UNSUPPORTED
    assert write(ks=64) == INVALID and write(status=ODD) == INVALID and write(N=-1) == INVALID
    assert write(N=70000) == UNSUPPORTED and write(N=0) == OK

    def step(q=P, slots=P, positions=P, entries=10, N=2, hq=4, hk=2, scale=1.0, o=P, vc=P, qs=0):
        return lib.kda_window_decode_step(q, P, P, 1, qs, 0, 0, scale, 2, P, vc, 4, entries, slots, positions, o, N, hq, hk,
                                          128, None, None)
    assert step(q=None) == INVALID and step(slots=None) == INVALID and step(positions=ODD) == INVALID
    assert step(entries=2) == INVALID and step(hq=5) == INVALID and step(scale=math.inf) == INVALID
    assert step(o=None) == INVALID and step(vc=None) == INVALID and step(qs=8) == INVALID
    assert step(N=1 << 30) == UNSUPPORTED and step(N=0) == OK


def test_gated_refusals(lib):
    def call(x=P, gate=P, dtype=1, xs=0, gs=0, w=P, norm=2, act=0, eps=1e-6, out=P, n=3, h=2, d=128):
        return lib.kda_gated_norm(x, gate, dtype, xs, gs, w, norm, act, eps, out, n, h, d, None)
    assert call(dtype=5) == INVALID and call(norm=3) == INVALID and call(act=2) == INVALID
    assert call(d=96) == UNSUPPORTED and call(d=0) == INVALID and call(n=-1) == INVALID and call(h=-1) == INVALID
    assert call(eps=0.0) == INVALID and call(eps=math.nan) == INVALID
    assert call(x=None) == INVALID and call(gate=ODD) == INVALID and call(w=ODD) == INVALID and call(out=None) == INVALID
    assert call(xs=100) == INVALID and call(gs=260) == INVALID
    assert call(n=1 << 31, h=1) == UNSUPPORTED and call(n=1 << 40, h=1 << 30) == UNSUPPORTED
    assert call(n=0) == OK and call(h=0) == OK

    def back(dy=P, dx=P, dw=P, ws=P, size=BIG):
        return lib.kda_gated_norm_backward(P, P, dy, 1, 0, 0, P, 2, 0, 1e-6, dx, P, dw, 3, 2, 128, ws, size, None)
    assert back(dy=None) == INVALID and back(dx=ODD) == INVALID and back(dw=ODD) == INVALID
    assert back(ws=None) == WORKSPACE and back(size=8) == WORKSPACE


def test_residual_refusals(lib):
    def call(x=P, b=P, st=1, dt=1, w=P, bn=0, wb=None, c=None, scale=1.0, eps=1e-6, h=P, y=P, n=3, D=256):
        return lib.kda_residual_norm(x, b, st, dt, w, bn, wb, c, scale, eps, h, y, n, D, None)
    assert call(st=3) == INVALID and call(dt=-1) == INVALID and call(st=1, dt=0) == UNSUPPORTED
    assert call(bn=4) == INVALID and call(eps=0.0) == INVALID and call(scale=math.nan) == INVALID
    assert call(n=-1) == INVALID and call(n=1 << 31) == UNSUPPORTED
    assert call(D=0) == INVALID and call(D=100) == UNSUPPORTED and call(D=8200) == UNSUPPORTED
    assert call(x=None) == INVALID and call(b=ODD) == INVALID and call(h=None) == INVALID and call(y=ODD) == INVALID
    assert call(w=ODD) == INVALID and call(wb=ODD) == INVALID and call(c=ODD) == INVALID
    assert call(n=0) == OK

    def back(h=P, b=P, dy=P, dh=None, bn=0, wb=None, dx=P, db=P, dw=P, dwb=None, ws=P, size=BIG):
        return lib.kda_residual_norm_backward(h, b, dy, dh, 1, 1, P, bn, wb, None, 1.0, 1e-6, dx, db, dw, dwb, None, 3, 256,
                                              ws, size, None)
    assert back(h=None) == INVALID and back(dy=None) == INVALID and back(dh=ODD) == INVALID
    assert back(dx=None) == INVALID and back(db=ODD) == INVALID and back(dw=ODD) == INVALID
    assert back(b=None, bn=2) == INVALID and back(b=None, wb=P) == INVALID and back(b=None, dwb=P) == INVALID
    assert back(ws=None) == WORKSPACE and back(size=64) == WORKSPACE


def test_axes_refusals(lib):
    def call(axes=2, pairs=bytes(32), rot=64, pos=P, table=P, d=128, n=3):
        return lib.kda_qk_norm_rope_axes(P, P, 1, 0, 0, pos, axes, pairs, table, 10, rot, 0, None, None, 2, 1e-6, P, P, n, 2, 2,
                                         d, None, None)
    assert call(axes=0) == INVALID and call(axes=5) == UNSUPPORTED
    assert call(pairs=None) == INVALID and call(pairs=bytes([0] * 31 + [2])) == INVALID
    assert b"pair_axis[31] is 2" in lib.kda_last_error()
    assert call(rot=0) == INVALID and call(rot=24) == UNSUPPORTED and call(rot=1 << 20) == INVALID
    assert call(pos=None) == INVALID and call(table=None) == INVALID
    assert call(n=0) == OK


def test_python_refusals():
    x = torch.zeros(1, 4, 2, 128)
    for call in (lambda: kda.window_attention(x, x, x, window=4), lambda: kda.gated_norm(x, x),
                 lambda: kda.residual_norm(x, x), lambda: kda.window_cache_write(x[0], x[0], None, x, x, None),
                 lambda: kda.qk_norm_rope_axes(x, x, torch.zeros(2, 1, 4).int(), torch.zeros(9, 64), [0, 1] * 16)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="entries"):
        kda.qk_norm_rope_axes(x, x, torch.zeros(2, 1, 4).int(), torch.zeros(9, 64), [0] * 31)
    with pytest.raises(ValueError, match="pair_axis"):
        kda.qk_norm_rope_axes(x, x, torch.zeros(2, 1, 4).int(), torch.zeros(9, 64), [-1] * 32)
    with pytest.raises(ValueError, match="required"):
        kda.qk_norm_rope_axes(x, x, None, torch.zeros(9, 64), [0] * 32)
    with pytest.raises(ValueError, match="required"):
        kda.window_varlen_attention(x[0], x[0], x[0], None, window=3)
    with pytest.raises(ValueError, match="branch"):
        kda.residual_norm(x, None)


def test_workspace_sizes(lib):
    assert kda.window_varlen_attention_workspace_bytes(3, 0, 4, 2) > 0
    assert kda.window_varlen_attention_workspace_bytes(-1, 10, 4, 2) == 0
    f = kda.window_attention_backward_workspace_bytes
    assert 0 < f(1, 64, 4, 2) < f(1, 4096, 4, 2) < f(1, 4096, 4, 2, 128, 64)
    assert f(1, 64, 4, 3) == 0 and f(1, 64, 4, 2, 128, 129) == 0 and f(1, 4096, 4, 2, 128, 64, torch.float32) > f(1, 4096, 4, 2, 128, 64)
