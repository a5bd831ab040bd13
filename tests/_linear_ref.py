"""Linear attention with a decay, and the head norm with rotary positions, in
64 bits from their definitions, for the tests: token by token, gradients by
torch's reverse mode. Shares nothing with the package's kernels.

Tolerances (relative L2 over a tensor), from the arithmetic the entry points
document:
  * fp32 results: operands split so that a product is off by at most 2^-22,
    sums of n <= 512 products in fp32 (sqrt(n) 2^-24 = 1.3e-6), a decay factor
    off by 2^-22, two or three such steps in a row: below 5e-6, bound 1e-5;
  * the log decay's gradient: a running sum of up to 512 row dots, each off by
    about 5e-7 of itself, errors adding as sqrt(512): 1.2e-5, bound 2e-5;
  * bf16 results: the rounding of the result, of the scores and of the state
    (each 2^-8 at most, 1.66e-3 in the root mean square): 2.9e-3, bound 5e-3.
"""
import torch

TOL = {torch.float32: 1e-5, torch.bfloat16: 5e-3}
TOL_DECAY = 2e-5


def recurrence(q, k, v, g, s0, scale):
    """One sequence: q, k [T, H, dk], v [T, H, dv], g [T, H] or None, s0 [H, dk, dv] or None, all 64-bit."""
    T, H, dk = q.shape
    S = torch.zeros(H, dk, v.shape[-1], dtype=torch.float64) if s0 is None else s0
    out = []
    for t in range(T):
        if g is not None:
            a = g[t].exp()[:, None, None]
            S = torch.where(a == 0, torch.zeros_like(S), a * S)
        S = S + k[t][:, :, None] * v[t][:, None, :]
        out.append(scale * torch.einsum("hkv,hk->hv", S, q[t]))
    return (torch.stack(out) if out else v.new_zeros(0, H, v.shape[-1])), S


def forward(q, k, v, g, s0, scale, lens=None):
    """Batched [B, T, H, d], or packed [T_total, H, d] with the sequence lengths; any dtype in, 64-bit out."""
    q, k, v = (x.detach().cpu().double() for x in (q, k, v))
    s0 = None if s0 is None else s0.detach().cpu().double()
    g = None if g is None else g.detach().cpu().double()
    return run64(q, k, v, g, s0, scale, lens)


def run64(q, k, v, g, s0, scale, lens=None):
    if lens is None:
        parts = [(q[b], k[b], v[b], None if g is None else g if g.dim() == 1 else g[b]) for b in range(q.shape[0])]
    else:
        parts, at = [], 0
        for n in lens:
            parts.append((q[at:at + n], k[at:at + n], v[at:at + n],
                          None if g is None else g if g.dim() == 1 else g[at:at + n]))
            at += n
    os, ss = [], []
    for i, (a, b, c, d) in enumerate(parts):
        if d is not None and d.dim() == 1:
            d = d.expand(a.shape[0], -1)
        o, s = recurrence(a, b, c, d, None if s0 is None else s0[i], scale)
        os.append(o)
        ss.append(s)
    return (torch.stack(os) if lens is None else torch.cat(os)), torch.stack(ss)


def gradients(q, k, v, g, s0, scale, d_o, dsT, lens=None):
    """The gradients of sum <d_o, o> + <dsT, S_T>, 64-bit, by reverse mode."""
    ins = {}
    for n, x in (("dq", q), ("dk", k), ("dv", v), ("dlog_decay", g), ("d_initial_state", s0)):
        if x is not None:
            ins[n] = x.detach().cpu().double().requires_grad_()
    o, S = run64(ins["dq"], ins["dk"], ins["dv"], ins.get("dlog_decay"), ins.get("d_initial_state"), scale, lens)
    L = (o * d_o.detach().cpu().double()).sum()
    if dsT is not None:
        L = L + (S * dsT.detach().cpu().double()).sum()
    names = list(ins)
    got = torch.autograd.grad(L, [ins[n] for n in names], allow_unused=True)
    return {n: torch.zeros_like(ins[n]) if x is None else x for n, x in zip(names, got)}


def rel(x, ref):
    x, ref = x.detach().cpu().double(), ref.detach().cpu().double()
    assert x.shape == ref.shape, (x.shape, ref.shape)
    assert bool(torch.isfinite(x).all())
    d = float((x - ref).norm())
    n = float(ref.norm())
    return d / n if n else d


def close(name, x, ref, tol):
    r = rel(x, ref)
    assert r <= tol, f"{name}: relative L2 {r:.2e} > {tol:.1e}"


def norm_rope(x, w, pos, table, norm, eps, layout):
    """64-bit norm and rotation of [n, H, d]."""
    y = x
    if norm != "none":
        ss = (x * x).sum(-1, keepdim=True)
        y = x / ((ss / x.shape[-1] if norm == "rms" else ss) + eps).sqrt()
    if w is not None:
        y = y * w
    if table is None:
        return y
    rot = table.shape[1]
    h = rot // 2
    row = table[pos.long()]
    c, s = row[:, None, :h], row[:, None, h:]
    a, rest = y[..., :rot], y[..., rot:]
    if layout == "half":
        u, z = a[..., :h], a[..., h:]
        a = torch.cat([u * c - z * s, z * c + u * s], -1)
    else:
        u, z = a[..., 0::2], a[..., 1::2]
        a = torch.stack([u * c - z * s, z * c + u * s], -1).flatten(-2)
    return torch.cat([a, rest], -1)
