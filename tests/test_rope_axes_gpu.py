"""The head norm with rotary positions of several axes against 64 bits, and bit
for bit against the one-axis call where the axes agree. Tolerances as in
test_qk_norm_rope_gpu.py: fp32 2e-6, weight gradients 5e-6, bf16 2.5e-3."""
import pytest
import torch

import _linear_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
TOL = {F32: 2e-6, BF: 2.5e-3}


def rotated(x, pos, table, pair_axis, layout):
    """x [n, H, d] float64, pos [axes, n]: every pair of channels turned by its axis' angle."""
    pairs = len(pair_axis)
    c, s = (torch.stack([table[pos[a].long(), i + at] for i, a in enumerate(pair_axis)], -1)[:, None] for at in (0, pairs))
    a, rest = x[..., :2 * pairs], x[..., 2 * pairs:]
    if layout == "half":
        u, w = a[..., :pairs], a[..., pairs:]
        return torch.cat([u * c - w * s, w * c + u * s, rest], -1)
    u, w = a[..., 0::2], a[..., 1::2]
    return torch.cat([torch.stack([u * c - w * s, w * c + u * s], -1).flatten(-2), rest], -1)


def check(kda, n, hq, hk, d, dtype, pair_axis, axes, norm="rms", layout="half", weight=True, fused=False, seed=0, P=50):
    gen = torch.Generator().manual_seed(seed)
    q, k = torch.randn(n, hq, d, generator=gen).to(dtype), torch.randn(n, hk, d, generator=gen).to(dtype)
    dq, dk = torch.randn(n, hq, d, generator=gen).to(dtype), torch.randn(n, hk, d, generator=gen).to(dtype)
    wq, wk = (1 + 0.3 * torch.randn(d, generator=gen) for _ in range(2)) if weight else (None, None)
    pos = torch.randint(0, P, (axes, n), generator=gen).int()
    table = kda.rope_table(P, 2 * len(pair_axis), device="cpu")
    cu = lambda x: None if x is None else x.cuda()  # noqa: E731
    qc, kc = q.cuda(), k.cuda()
    if fused:
        p = torch.cat([qc, kc, kc], 1)
        qc, kc = p[:, :hq], p[:, hq:hq + hk]
    kw = dict(norm=norm, layout=layout)
    yq, yk = kda.qk_norm_rope_axes(qc, kc, pos.cuda(), table.cuda(), pair_axis, cu(wq), cu(wk), **kw)
    got = kda.qk_norm_rope_axes_backward(qc, kc, dq.cuda(), dk.cuda(), pos.cuda(), table.cuda(), pair_axis, cu(wq), cu(wk), **kw)
    for x, w, y, dy, nm in ((q, wq, yq, dq, "q"), (k, wk, yk, dk, "k")):
        x64, w64 = x.double().requires_grad_(), None if w is None else w.double().requires_grad_()
        ref = rotated(R.norm_rope(x64, w64, None, None, norm, 1e-6, layout), pos, table.double(), pair_axis, layout)
        R.close(nm, y, ref.detach(), TOL[dtype])
        ref.backward(dy.double())
        R.close("d" + nm, got["d" + nm], x64.grad, TOL[dtype])
        if w is not None:
            R.close("d" + nm + "_weight", got["d" + nm + "_weight"], w64.grad, 5e-6)


def sections(*n):
    return [a for a, m in enumerate(n) for _ in range(m)]


AXES = [("blocks of four", 128, sections(16, 24, 24), 3), ("blocks", 128, sections(17, 23, 24), 3),
        ("in turn", 128, [i % 3 for i in range(64)], 3), ("two", 64, [0, 1] * 8, 2), ("four", 64, sections(4, 12, 8, 8), 4),
        ("part of the head", 128, sections(3, 5), 2), ("one", 64, [0] * 32, 1), ("an axis unused", 64, [2] * 8 + [0] * 8, 3)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("name,d,pair_axis,axes", AXES, ids=[a[0] for a in AXES])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_axes(kda, dtype, name, d, pair_axis, axes, layout):
    check(kda, 37, 5, 2, d, dtype, pair_axis, axes, layout=layout)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n,hq,hk", [(1, 1, 1), (1, 32, 8), (130, 1, 9), (257, 16, 16)])
def test_shapes(kda, dtype, n, hq, hk):
    check(kda, n, hq, hk, 128, dtype, sections(16, 24, 24), 3, seed=n, fused=True)
    check(kda, n, hq, hk, 64, dtype, [i % 3 for i in range(16)], 3, "l2", "interleaved", weight=False, seed=n)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("pair_axis", [sections(32, 32), [i % 2 for i in range(64)]])
def test_equal_positions_are_one_axis(kda, dtype, pair_axis):
    q, k = (torch.randn(300, 4, 128, device="cuda").to(dtype) for _ in range(2))
    w = torch.rand(128, device="cuda")
    pos = torch.randint(0, 90, (300,), device="cuda").int()
    table = kda.rope_table(90, 128)
    two = torch.stack([pos, pos])
    a, b = kda.qk_norm_rope(q, k, pos, table, w, w), kda.qk_norm_rope_axes(q, k, two, table, pair_axis, w, w)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    a, b = (kda.qk_norm_rope_backward(q, k, k, q, pos, table, w, w),
            kda.qk_norm_rope_axes_backward(q, k, k, q, two, table, pair_axis, w, w))
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_bad_positions_are_left_out(kda):
    q, k = (torch.randn(50, 4, 128, device="cuda").to(BF) for _ in range(2))
    pos = torch.randint(0, 30, (3, 50), device="cuda").int()
    bad = pos.clone()
    bad[0, 3], bad[2, 17], bad[1, 40] = -1, 30, 1 << 30
    table, pa = kda.rope_table(30, 128), sections(16, 24, 24)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    good = kda.qk_norm_rope_axes(q, k, pos, table, pa, device_status=st)
    assert st.item() == kda.KDA_DEV_OK
    out = [torch.full_like(x, 5.0) for x in (q, k)]
    kda.qk_norm_rope_axes(q, k, bad, table, pa, q_out=out[0], k_out=out[1], device_status=st)
    assert st.item() == kda.KDA_DEV_BAD_POSITION
    keep = [i for i in range(50) if i not in (3, 17, 40)]
    for a, b in zip(good, out):
        assert torch.equal(a[keep], b[keep]) and (b[[3, 17, 40]] == 5).all()
    w = torch.ones(128, device="cuda")
    g = kda.qk_norm_rope_axes_backward(q, k, q, k, bad, table, pa, w, w, device_status=st)
    assert st.item() == kda.KDA_DEV_BAD_POSITION
    h = kda.qk_norm_rope_axes_backward(q[keep], k[keep], q[keep], k[keep], pos[:, keep].contiguous(), table, pa, w, w)
    assert torch.allclose(g["dq_weight"], h["dq_weight"], rtol=1e-5, atol=1e-5)


def test_batched_and_no_tokens(kda):
    q, k = (torch.randn(2, 9, 3, 128, device="cuda") for _ in range(2))
    pos = torch.randint(0, 30, (3, 2, 9), device="cuda").int()
    table, pa = kda.rope_table(30, 128), sections(16, 24, 24)
    a = kda.qk_norm_rope_axes(q, k, pos, table, pa)
    b = kda.qk_norm_rope_axes(q.flatten(0, 1), k.flatten(0, 1), pos.flatten(1), table, pa)
    assert all(torch.equal(x.flatten(0, 1), y) for x, y in zip(a, b))
    e = torch.zeros(0, 3, 128, device="cuda")
    assert kda.qk_norm_rope_axes(e, e, torch.zeros(3, 0, dtype=torch.int32, device="cuda"), table, pa)[0].shape == e.shape
