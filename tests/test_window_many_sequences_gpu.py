"""Window attention over thousands of short sequences with many sinks, long ones among
them, whose far queries' parts lie all over the batch. Tolerances as in
test_window_gpu.py: fp32 1e-5, bf16 3.2e-3 for o and 5e-3 for the gradients."""
import pytest
import torch

import _window_ref as W

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
TOL = {F32: (1e-5, 1e-5), BF: (3.2e-3, 5e-3)}


def reference(lens, q, k, v, d_o, window, sinks, scale):
    """Sequences of one length at a time, in 64 bits."""
    at = torch.tensor([0, *lens]).cumsum(0)[:-1].tolist()
    out = {n: torch.zeros(x.shape, dtype=torch.float64, device="cuda") for n, x in (("o", q), ("dq", q), ("dk", k), ("dv", v))}
    group = q.shape[1] // k.shape[1]
    for m in sorted(set(lens) - {0}):
        pick = torch.stack([torch.arange(a, a + m) for a, x in zip(at, lens) if x == m]).cuda()
        a, b, c = (x[pick].double().requires_grad_() for x in (q, k, v))
        s = torch.einsum("nihd,njhd->nhij", a, b.repeat_interleave(group, 2)) * scale
        s = s.masked_fill(~W.visible(m, window, sinks, "cuda"), -torch.inf)
        o = torch.einsum("nhij,njhd->nihd", s.softmax(-1), c.repeat_interleave(group, 2))
        o.backward(d_o[pick].double())
        for n, x in (("o", o.detach()), ("dq", a.grad), ("dk", b.grad), ("dv", c.grad)):
            out[n][pick] = x
    return out


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("lens,window,sinks", [
    ([0, 3, 17, 1, 24, 9] * 700, 5, 128), ([40, 2, 8] * 1200, 1, 128), ([16] * 500 + [2500] + [16, 0] * 300 + [1300, 5, 3100], 7, 128),
    ([300, 20] * 40 + [1100], 1023, 100), ([16] * 4096, 16, 128)],
    ids=["ragged", "window 1", "long ones among them", "one behind its window", "none behind its window"])
def test_gradients(kda, dtype, lens, window, sinks):
    Hq, Hk, d = 4, 2, 64
    q, k, v, d_o = W.inputs(lens, Hq, Hk, d, dtype)
    cu = torch.tensor([0, *lens], dtype=torch.int64).cumsum(0).int().cuda()
    kw = dict(window=window, sinks=sinks)
    o, lse = kda.window_varlen_attention(q, k, v, cu, **kw)
    g = kda.window_varlen_attention_backward(q, k, v, o, lse, d_o, cu, **kw)
    ref = reference(lens, q, k, v, d_o, window, sinks, d ** -0.5)
    for n, x in (("o", o), *g.items()):
        err, size = float((x.double() - ref[n]).norm()), float(ref[n].norm())
        assert torch.isfinite(x).all() and err <= TOL[dtype][n != "o"] * size, (n, err / size)
    # equal lengths need no table, and give the same bits
    if len(set(lens)) == 1:
        cut = [x.unflatten(0, (len(lens), lens[0])) for x in (q, k, v, o, lse, d_o)]
        e = kda.window_attention_backward(*cut, **kw)
        assert all(torch.equal(e[n].flatten(0, 1), g[n]) for n in g)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_the_same_bits_as_equal_lengths(kda, dtype):
    B, T, window, sinks = 200, 70, 20, 128
    q, k, v, d_o = W.inputs([T] * B, 4, 2, 128, dtype)
    kw = dict(window=window, sinks=sinks)
    cut = [x.unflatten(0, (B, T)) for x in (q, k, v, d_o)]
    o, lse = kda.window_attention(*cut[:3], **kw)
    a = kda.window_attention_backward(*cut[:3], o, lse, cut[3], **kw)
    cu = torch.arange(0, B * T + 1, T, dtype=torch.int32, device="cuda")
    b = kda.window_varlen_attention_backward(q, k, v, o.flatten(0, 1), lse.flatten(0, 1), d_o, cu, **kw)
    assert all(torch.equal(a[n].flatten(0, 1), b[n]) for n in a)
