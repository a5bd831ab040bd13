"""Gradients of window attention where one token holds most of a row's weight: a
sink, as in trained models, or a token near by. There ds = p (dp - D) is far smaller
than dp, so that D must be exact to the digits that cancel.

Tolerances (relative 2-norm). bf16: the results are rounded, 1.66e-3 in the root mean
square, and so are the weights and ds as operands, ds of the heavy token at most as
large as all others together: below sqrt(1 + 1 + 1) 1.66e-3 = 2.9e-3, bound 5e-3, as
without a peak. fp32: a score is off by 2^-22 |q| |k| scale at most, 6e-6 here, a
weight by as much relative to itself; dp and D by 2^-22 each, of which 1 / (1 - p)
remains in their difference: 6e-6 + 2^-21 / (1 - p)."""
import pytest
import torch

import _window_ref as W

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def peaked(T, Hq, Hk, d, dtype, level, where, seed):
    """q, k, v, d_o whose heavy score is `level`; the others' are below 3 for the most part."""
    gen = torch.Generator().manual_seed(seed)
    q, d_o = torch.randn(T, Hq, d, generator=gen), torch.randn(T, Hq, d, generator=gen)
    k, v = torch.randn(T, Hk, d, generator=gen), torch.randn(T, Hk, d, generator=gen)
    if where == "sink":
        u = torch.ones(d) / d ** 0.5
        q = q + 8 * u
        k[0] = level * d ** 0.5 / 8 * u
    else:  # the token `where` behind
        to = k.roll(where, 0).repeat_interleave(Hq // Hk, 1)
        q = q + level * d ** 0.5 * to / to.pow(2).sum(-1, keepdim=True)
    return [x.to(dtype).cuda() for x in (q, k, v, d_o)]


def close(name, x, ref, tol):
    x, ref = x.double(), ref.double()
    assert torch.isfinite(x).all(), name
    err, size = float((x - ref).norm()), float(ref.norm())
    assert err <= tol * size, (name, err / size)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("level", [0.0, 5.0, 7.0, 8.5, 9.5])
@pytest.mark.parametrize("T,window,sinks,where", [(600, 256, 4, "sink"), (1300, 300, 1, "sink"), (700, 500, 128, "sink"),
                                                  (600, 256, 4, 3), (600, 600, 0, 70), (400, 100, 0, 0)])
def test_gradients(kda, dtype, d, level, T, window, sinks, where):
    q, k, v, d_o = peaked(T, 4, 2, d, dtype, level, where, T)
    o, lse = kda.window_attention(q[None], k[None], v[None], window=window, sinks=sinks)
    g = kda.window_attention_backward(q[None], k[None], v[None], o, lse, d_o[None], window=window, sinks=sinks)
    ref = W.gradients(q, k, v, d_o, window, sinks, d ** -0.5)
    s = torch.einsum("ihd,jhd->hij", q.double(), k.double().repeat_interleave(2, 1)) * d ** -0.5
    top = s.masked_fill(~W.visible(T, window, sinks, "cuda"), -torch.inf).softmax(-1).amax(-1)[:, T // 2:].mean()
    tol = 5e-3 if dtype == BF else 6e-6 + 2.0 ** -21 / (1 - float(top))
    for n in g:
        close(f"{n} at a weight of {float(top):.2f}", g[n][0], ref[n], tol)


@pytest.mark.parametrize("d", [64, 128])
def test_packed(kda, d):
    lens = [130, 0, 700, 1, 401]
    parts = [peaked(m, 4, 2, d, BF, 8.0, "sink", m) for m in lens if m]
    q, k, v, d_o = (torch.cat(x) for x in zip(*parts))
    cu = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    o, lse = kda.window_varlen_attention(q, k, v, cu, window=120, sinks=4)
    g = kda.window_varlen_attention_backward(q, k, v, o, lse, d_o, cu, window=120, sinks=4)
    ref = [W.gradients(*x, 120, 4, d ** -0.5) for x in parts]
    for n in g:
        close(n, g[n], torch.cat([r[n] for r in ref]), 5e-3)


def test_a_weight_next_to_one(kda):
    """999 parts in 1000 at the sink: what is left of ds is still right."""
    q, k, v, d_o = peaked(900, 2, 1, 128, BF, 13.0, "sink", 5)
    o, lse = kda.window_attention(q[None], k[None], v[None], window=256, sinks=4)
    g = kda.window_attention_backward(q[None], k[None], v[None], o, lse, d_o[None], window=256, sinks=4)
    ref = W.gradients(q, k, v, d_o, 256, 4, 128 ** -0.5)
    for n in g:
        close(n, g[n][0], ref[n], 5e-3)
