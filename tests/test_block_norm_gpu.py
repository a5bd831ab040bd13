"""The norms around a block, forward and backward, against 64 bits.

Tolerances (relative 2-norm): fp32, sums of up to 8192 squares in trees and a
handful of products (below 1e-6; the accurate exponential of the gate 2^-22),
bound 3e-6; sums over the rows for the weights' gradients, up to 3,000 terms,
1e-5. bf16, one rounding of the result: 2^-9 at most per element, 1.66e-3 in the
root mean square, bound 2.5e-3."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
TOL = {F32: 3e-6, BF: 2.5e-3}
EPS = 1e-5


def close(name, x, ref, tol):
    x, ref = x.double().cpu(), ref.double()
    assert x.shape == ref.shape, name
    assert torch.isfinite(x).all(), name
    err, size = float((x - ref).norm()), float(ref.norm())
    assert err <= tol * size + 1e-30, (name, err / max(size, 1e-30))


def normed(x, norm, eps):
    if norm == "none":
        return x
    ss = x.pow(2).sum(-1, keepdim=True)
    return x / ((ss / x.shape[-1] if norm == "rms" else ss) + eps).sqrt()


def leaf(x):
    return None if x is None else x.double().requires_grad_()


def gated_ref(x, g, w, norm, act, eps):
    y = normed(x, norm, eps) * (torch.sigmoid(g) if act == "sigmoid" else g * torch.sigmoid(g))
    return y if w is None else y * w


def check_gated(kda, lead, h, d, dtype, norm, act, weight=True, fused=False, seed=0, eps=EPS, size=1.0, gate_size=3.0):
    gen = torch.Generator().manual_seed(seed)
    x = (size * torch.randn(*lead, h, d, generator=gen)).to(dtype)
    g, dy = (gate_size * torch.randn(*lead, h, d, generator=gen)).to(dtype), torch.randn(*lead, h, d, generator=gen).to(dtype)
    w = 1 + 0.3 * torch.randn(d, generator=gen) if weight else None
    xc, gc, wc = x.cuda(), g.cuda(), None if w is None else w.cuda()
    if fused:
        p = torch.cat([torch.zeros_like(xc), xc, gc], -2)
        xc, gc = p[..., h:2 * h, :], p[..., 2 * h:, :]
    kw = dict(norm=norm, activation=act, eps=eps)
    y = kda.gated_norm(xc, gc, wc, **kw)
    got = kda.gated_norm_backward(xc, gc, dy.cuda(), wc, **kw)
    x64, g64, w64 = leaf(x), leaf(g), leaf(w)
    ref = gated_ref(x64, g64, w64, norm, act, eps)
    assert y.dtype == dtype and y.is_contiguous()
    close("out", y, ref.detach(), TOL[dtype])
    ref.backward(dy.double())
    close("dx", got["dx"], x64.grad, TOL[dtype])
    close("dgate", got["dgate"], g64.grad, TOL[dtype])
    if weight:
        close("dweight", got["dweight"], w64.grad, 1e-5)
    else:
        assert got["dweight"] is None


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("norm", ["none", "l2", "rms"])
@pytest.mark.parametrize("act", ["sigmoid", "silu"])
def test_gated_kinds(kda, dtype, d, norm, act):
    check_gated(kda, (37,), 5, d, dtype, norm, act)
    check_gated(kda, (2, 9), 3, d, dtype, norm, act, weight=False, fused=True)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n,h", [(1, 1), (1, 32), (3, 7), (130, 1), (257, 16), (1000, 3)])
def test_gated_shapes(kda, dtype, n, h):
    check_gated(kda, (n,), h, 128, dtype, "rms", "sigmoid", seed=n)
    check_gated(kda, (n,), h, 64, dtype, "rms", "silu", fused=True, seed=n)


def test_gated_range(kda):
    for size in (1e-15, 1e-4, 1e12):
        check_gated(kda, (20,), 2, 128, F32, "rms", "sigmoid", size=size, eps=1e-30)
    # gates far out: the sigmoid runs to 0 and 1, its slope to nothing
    check_gated(kda, (20,), 2, 128, F32, "rms", "silu", gate_size=30.0)
    x, w = torch.randn(4, 1, 64, device="cuda"), torch.ones(64, device="cuda")
    g = torch.tensor([-1e4, -100.0, 100.0, 1e4], device="cuda").view(4, 1, 1).expand(4, 1, 64).contiguous()
    for act in ("sigmoid", "silu"):
        y = kda.gated_norm(x, g, w, activation=act)
        d = kda.gated_norm_backward(x, g, x, w, activation=act)
        assert torch.isfinite(y).all() and all(torch.isfinite(t).all() for t in d.values())
        assert y[:2].abs().max() < 1e-30 and d["dx"][:2].abs().max() < 1e-30
    zero = kda.gated_norm(torch.zeros_like(x), g, w)
    assert not zero.any()


def test_gated_in_place_and_the_same_bits(kda):
    x, g = (torch.randn(500, 8, 128, device="cuda").to(BF) for _ in range(2))
    w = torch.rand(128, device="cuda")
    y = kda.gated_norm(x, g, w)
    a, b = kda.gated_norm_backward(x, g, y, w), kda.gated_norm_backward(x, g, y, w)
    assert all(torch.equal(a[n], b[n]) for n in a)
    x2, g2 = x.clone(), g.clone()
    assert torch.equal(kda.gated_norm(x2, g, w, out=x2), y) and torch.equal(kda.gated_norm(x, g2, w, out=g2), y)


def residual_ref(x, b, w, wb, c, scale, branch_norm, eps):
    u = normed(b, branch_norm, eps)
    u = u if wb is None else u * wb
    h = x + scale * (u if c is None else u * c)
    y = normed(h, "rms", eps)
    return h, y if w is None else y * w


def check_residual(kda, lead, D, dtype, stream, branch_norm="none", weight=True, bweight=False, channel=False, scale=0.7,
                   dh=True, seed=0, eps=EPS):
    gen = torch.Generator().manual_seed(seed)

    def rand(*s, size=1.0):
        return size * torch.randn(*s, generator=gen)
    x, b = rand(*lead, D, size=2.0).to(stream), rand(*lead, D).to(dtype)
    w = 1 + 0.3 * rand(D) if weight else None
    wb = 1 + 0.3 * rand(D) if bweight else None
    c = 0.5 + 0.1 * rand(D) if channel else None
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    kw = dict(branch_norm=branch_norm, branch_weight=cu(wb), channel_scale=cu(c), scale=scale, eps=eps)
    h, y = kda.residual_norm(x.cuda(), b.cuda(), cu(w), **kw)
    x64, b64, w64, wb64, c64 = map(leaf, (x, b, w, wb, c))
    rh, ry = residual_ref(x64, b64, w64, wb64, c64, scale, branch_norm, eps)
    assert h.dtype == stream and y.dtype == dtype
    close("hidden", h, rh.detach(), TOL[stream])
    close("out", y, ry.detach(), TOL[dtype])
    # the gradients are those at the stored sum
    dy, dhid = rand(*lead, D).to(dtype), rand(*lead, D).to(stream) if dh else None
    reads = branch_norm != "none" or bweight or channel
    got = kda.residual_norm_backward(h, b.cuda() if reads else None, dy.cuda(), cu(dhid), cu(w), **kw)
    h64 = h.cpu().double().requires_grad_()
    out = normed(h64, "rms", eps)
    (out if w is None else out * w64).backward(dy.double())
    g = h64.grad if dhid is None else h64.grad + dhid.double()
    u = normed(b64, branch_norm, eps)
    u = u if wb is None else u * wb64
    (scale * (u if c is None else u * c64)).backward(g)
    close("d_residual", got["d_residual"], g, TOL[stream])
    close("d_branch", got["d_branch"], b64.grad, TOL[dtype])
    for n, t in (("dweight", w64), ("dbranch_weight", wb64), ("dchannel_scale", c64)):
        if t is None:
            assert got[n] is None
        else:
            close(n, got[n], t.grad, 1e-5)


TYPES = [(F32, F32), (BF, BF), (BF, F32)]


@pytest.mark.parametrize("dtype,stream", TYPES)
@pytest.mark.parametrize("branch_norm", ["none", "rms", "l2"])
@pytest.mark.parametrize("bweight", [False, True])
@pytest.mark.parametrize("channel", [False, True])
def test_residual_kinds(kda, dtype, stream, branch_norm, bweight, channel):
    check_residual(kda, (33,), 640, dtype, stream, branch_norm, True, bweight, channel)
    check_residual(kda, (2, 3), 256, dtype, stream, branch_norm, False, bweight, channel, dh=False)


@pytest.mark.parametrize("dtype,stream", TYPES)
@pytest.mark.parametrize("D", [8, 16, 64, 248, 256, 264, 512, 520, 1000, 1024, 2048, 2056, 4096, 4104, 8184, 8192])
@pytest.mark.parametrize("n", [1, 5, 700])
def test_residual_shapes(kda, dtype, stream, D, n):
    check_residual(kda, (n,), D, dtype, stream, "rms", True, True, True, seed=D + n)


def test_residual_in_place_and_the_same_bits(kda):
    x, b = (torch.randn(300, 2048, device="cuda").to(BF) for _ in range(2))
    w = torch.rand(2048, device="cuda")
    h, y = kda.residual_norm(x, b, w)
    x2, b2 = x.clone(), b.clone()
    h2, y2 = kda.residual_norm(x2, b2, w, hidden_out=x2, out=b2)
    assert h2 is x2 and y2 is b2 and torch.equal(h, h2) and torch.equal(y, y2)
    kw = dict(branch_norm="rms", branch_weight=w, channel_scale=w)
    a, c = (kda.residual_norm_backward(h, b, y, h, w, **kw) for _ in range(2))
    assert all(torch.equal(a[n], c[n]) for n in a)


def test_no_tokens(kda):
    e, w = torch.zeros(0, 4, 128, device="cuda"), torch.ones(128, device="cuda")
    assert kda.gated_norm(e, e, w).shape == e.shape
    assert not kda.gated_norm_backward(e, e, e, w)["dweight"].any()
    z, w = torch.zeros(0, 64, device="cuda"), torch.ones(64, device="cuda")
    assert kda.residual_norm(z, z, w)[0].shape == z.shape
    d = kda.residual_norm_backward(z, z, z, None, w, branch_weight=w, channel_scale=w)
    assert not d["dweight"].any() and not d["dbranch_weight"].any() and not d["dchannel_scale"].any()


def test_gradients_against_differences(kda):
    gen = torch.Generator().manual_seed(4)
    x, g, dy = (torch.randn(6, 2, 64, generator=gen) for _ in range(3))
    w = 1 + 0.2 * torch.randn(64, generator=gen)
    got = kda.gated_norm_backward(x.cuda(), g.cuda(), dy.cuda(), w.cuda(), activation="silu", eps=EPS)
    args = [t.double() for t in (x, g, w)]
    for at, name in enumerate(("dx", "dgate", "dweight")):
        u = torch.randn(args[at].shape, generator=gen, dtype=torch.float64)

        def loss(h):
            a = list(args)
            a[at] = a[at] + h * u
            return float((gated_ref(*a, "rms", "silu", EPS) * dy).sum())
        diff = (loss(1e-5) - loss(-1e-5)) / 2e-5
        mine = float((got[name].cpu().double() * u).sum())
        size = float(got[name].cpu().double().norm() * u.norm()) / math.sqrt(u.numel())
        assert abs(mine - diff) <= 1e-4 * size, (name, mine, diff)
    h, b, dy, dh = (torch.randn(5, 96, generator=gen) for _ in range(4))
    w, wb, c = (1 + 0.2 * torch.randn(96, generator=gen) for _ in range(3))
    got = kda.residual_norm_backward(h.cuda(), b.cuda(), dy.cuda(), dh.cuda(), w.cuda(), branch_norm="rms",
                                     branch_weight=wb.cuda(), channel_scale=c.cuda(), scale=0.3, eps=EPS)
    # x is what makes the sum h
    x = h.double() - residual_ref(torch.zeros(5, 96).double(), b.double(), None, wb.double(), c.double(), 0.3, "rms", EPS)[0]
    args = [t.double() for t in (x, b, w, wb, c)]
    for at, name in enumerate(("d_residual", "d_branch", "dweight", "dbranch_weight", "dchannel_scale")):
        u = torch.randn(args[at].shape, generator=gen, dtype=torch.float64)

        def loss(s):
            a = list(args)
            a[at] = a[at] + s * u
            hid, out = residual_ref(*a, 0.3, "rms", EPS)
            return float((out * dy).sum() + (hid * dh).sum())
        diff = (loss(1e-5) - loss(-1e-5)) / 2e-5
        mine = float((got[name].cpu().double() * u).sum())
        size = float(got[name].cpu().double().norm() * u.norm()) / math.sqrt(u.numel())
        assert abs(mine - diff) <= 1e-4 * size, (name, mine, diff)


def test_captured_and_on_a_given_stream(kda):
    x, g = (torch.randn(300, 4, 128, device="cuda").to(BF) for _ in range(2))
    w, wd = torch.rand(128, device="cuda"), torch.rand(512, device="cuda")

    def all_of_it(**kw):
        y = kda.gated_norm(x, g, w, **kw)
        d = kda.gated_norm_backward(x, g, y, w, **kw)
        h, out = kda.residual_norm(x.flatten(1), y.flatten(1), wd, branch_norm="rms", **kw)
        r = kda.residual_norm_backward(h, y.flatten(1), out, None, wd, branch_norm="rms", **kw)
        return [y, *d.values(), h, out, *(t for t in r.values() if t is not None)]
    first = [t.clone() for t in all_of_it()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    on_s = all_of_it(stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, on_s))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = all_of_it()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(first, out))
