"""Window attention with sinks in 64 bits, from its definition: every score, the
mask, softmax, gradients by reverse mode."""
import math

import torch


def visible(T, window, sinks, device="cpu"):
    i, j = torch.arange(T, device=device)[:, None], torch.arange(T, device=device)[None]
    return (j <= i) & ((i - j < window) | (j < sinks))


def attention(q, k, v, window, sinks, scale):
    """q [T, Hq, d], k, v [T, Hk, d] float64 -> o [T, Hq, d], lse [T, Hq]."""
    T, Hq, _ = q.shape
    if T == 0:
        return q.clone(), q[..., 0].clone()
    group = Hq // k.shape[1]
    k, v = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
    s = torch.einsum("ihd,jhd->hij", q, k) * scale
    s = s.masked_fill(~visible(T, window, sinks, q.device), -math.inf)
    return torch.einsum("hij,jhd->ihd", torch.softmax(s, -1), v), torch.logsumexp(s, -1).t()


def gradients(q, k, v, d_o, window, sinks, scale):
    q, k, v = (x.double().detach().requires_grad_() for x in (q, k, v))
    o, _ = attention(q, k, v, window, sinks, scale)
    o.backward(d_o.double())
    return {"dq": q.grad, "dk": k.grad, "dv": v.grad}


def entry(p, window, sinks):
    return p if p < sinks else sinks + (p - sinks) % window


def inputs(lens, Hq, Hk, d, dtype, seed=0, fused=False, sharp=1.5):
    """q, k, v, d_o of packed sequences, on the GPU; fused: slices of one tensor."""
    gen = torch.Generator().manual_seed(seed)
    T = sum(lens)
    if fused:
        p = torch.randn(T, Hq + 2 * Hk, d, generator=gen).to(dtype).cuda()
        q, k, v = p[:, :Hq], p[:, Hq:Hq + Hk], p[:, Hq + Hk:]
    else:
        q = (sharp * torch.randn(T, Hq, d, generator=gen)).to(dtype).cuda()
        k, v = (torch.randn(T, Hk, d, generator=gen).to(dtype).cuda() for _ in range(2))
    return q, k, v, torch.randn(T, Hq, d, generator=gen).to(dtype).cuda()
