"""Gates far below zero, where the sigmoid runs to nothing: gated_norm and its
gradients against 64 bits, element by element, relative to each value.

Tolerances. fp32: e^g from the accurate exponential is within 2 ulp, the norm's
reciprocal root within 2 ulp, and seven products or quotients of half an ulp each
round what they make: below 8 ulp of 2^-23, 1e-6. bf16: the result's rounding is
2^-8 at most; the approximate exponential's argument, up to 125, is rounded at
2^-24 of itself twice, 1.5e-5 of the value, and fp32's other roundings are below
that: 2^-8 + 2^-14. Where the true value lies below fp32's normal numbers (2^-126)
it may be anything up to that."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
TOL = {F32: 1e-6, BF: 2.0 ** -8 + 2.0 ** -14}
GATES = [-20.0, -60.0, -75.0, -79.5, -80.5, -82.0, -86.0, -95.0, -1e4, -1e20, -1e30, -1e36]


def check(name, x, ref, tol):
    x = x.double().cpu()
    assert torch.isfinite(x).all(), name
    off = (x - ref).abs() - tol * ref.abs()
    assert (off <= 2.0 ** -126).all(), (name, float(off.max()))


def make(dtype, gates, d):
    gen = torch.Generator().manual_seed(d)
    n = len(gates)
    x, dy = ((0.5 + torch.rand(n, 2, d, generator=gen)).to(dtype) for _ in range(2))  # nothing cancels but in dx
    g = torch.tensor(gates).to(dtype).view(n, 1, 1).expand(n, 2, d).contiguous()
    return x, g, dy, 0.5 + torch.rand(d, generator=gen)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("act", ["sigmoid", "silu"])
def test_values_and_slopes(kda, dtype, d, act):
    x, g, dy, w = make(dtype, GATES + [torch.finfo(dtype).min], d)
    kw = dict(norm="none", activation=act)
    y = kda.gated_norm(x.cuda(), g.cuda(), w.cuda(), **kw)
    got = kda.gated_norm_backward(x.cuda(), g.cuda(), dy.cuda(), w.cuda(), **kw)
    x, g, dy, w = (t.double() for t in (x, g, dy, w))
    s = torch.exp(g) / (1 + torch.exp(g))
    a, da = (g * s, s * (1 + g * (1 - s))) if act == "silu" else (s, s * (1 - s))
    check("out", y, x * w * a, TOL[dtype])
    check("dx", got["dx"], w * a * dy, TOL[dtype])
    check("dgate", got["dgate"], x * w * da * dy, TOL[dtype])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("norm", ["rms", "l2", "none"])
@pytest.mark.parametrize("low", ["min", "-inf"])
def test_a_closed_gate_lets_nothing_through(kda, dtype, act, norm, low):
    low = -math.inf if low == "-inf" else torch.finfo(dtype).min
    x, g, dy, w = (t.cuda() for t in make(dtype, [1.0, low, -1.0, low], 128))
    g[0, 0, ::3] = low
    y = kda.gated_norm(x, g, w, norm=norm, activation=act)
    got = kda.gated_norm_backward(x, g, dy, w, norm=norm, activation=act)
    shut = g == low
    assert torch.isfinite(y).all() and all(torch.isfinite(t).all() for t in got.values())
    assert not y[shut].any() and not got["dgate"][shut].any()
    assert not got["dx"][1].any() and not got["dx"][3].any()
    open_ = kda.gated_norm_backward(x[::2].contiguous(), g[::2].contiguous(), dy[::2].contiguous(), w, norm=norm,
                                    activation=act)  # rows behind a closed gate add nothing to the weight's gradient
    assert torch.equal(got["dx"][::2], open_["dx"])
    assert (got["dweight"] - open_["dweight"]).abs().max() <= 1e-6 * open_["dweight"].abs().max()
