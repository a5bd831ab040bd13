"""The head norm with rotary positions, forward and backward, against 64 bits.

Tolerances (relative L2): fp32, a sum of 128 squares and a handful of products
in fp32 (below 5e-7), bound 2e-6; weight gradients, sums of up to 4,000 terms in
a tree (below 1e-6), bound 5e-6; bf16, the one rounding of the result, 2^-8 at
most per element (1.66e-3 in the root mean square), bound 2.5e-3."""
import math

import pytest
import torch

import _linear_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
TOL = {F32: 2e-6, BF: 2.5e-3}


def _inputs(n, hq, hk, d, dtype, weight=True, P=100, rot=None, seed=0):
    gen = torch.Generator().manual_seed(seed)
    q, k = torch.randn(n, hq, d, generator=gen).to(dtype), torch.randn(n, hk, d, generator=gen).to(dtype)
    wq, wk = (1 + 0.3 * torch.randn(d, generator=gen) for _ in range(2)) if weight else (None, None)
    pos = torch.randint(0, P, (n,), generator=gen).int()
    table = None
    if rot is None or rot > 0:
        import kda_gated_delta_chunkwise_gb300 as kda
        table = kda.rope_table(P, rot or d, device="cpu")
    return q, k, pos if table is not None else None, table, wq, wk


def _cu(x):
    return None if x is None else x.cuda()


def _check(kda, q, k, pos, table, wq, wk, norm, layout, eps=1e-6):
    yq, yk = kda.qk_norm_rope(*map(_cu, (q, k, pos, table, wq, wk)), norm=norm, layout=layout, eps=eps)
    gen = torch.Generator().manual_seed(9)
    dq, dk = (torch.randn(x.shape, generator=gen).to(x.dtype) for x in (q, k))
    got = kda.qk_norm_rope_backward(*map(_cu, (q, k, dq, dk, pos, table, wq, wk)), norm=norm, layout=layout, eps=eps)
    for x, w, y, dy, n in ((q, wq, yq, dq, "q"), (k, wk, yk, dk, "k")):
        x64 = x.double().requires_grad_()
        w64 = None if w is None else w.double().requires_grad_()
        ref = R.norm_rope(x64, w64, pos, None if table is None else table.double(), norm, eps, layout)
        assert y.dtype == x.dtype and y.is_contiguous()
        R.close(n, y, ref, TOL[x.dtype])
        ref.backward(dy.double())
        R.close("d" + n, got["d" + n], x64.grad, TOL[x.dtype])
        if w is not None:
            R.close("d" + n + "_weight", got["d" + n + "_weight"], w64.grad, 5e-6)
        else:
            assert got["d" + n + "_weight"] is None


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("norm", ["none", "l2", "rms"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_kinds(kda, dtype, d, norm, layout):
    for rot in (16, 48, 64, d):
        _check(kda, *_inputs(37, 5, 2, d, dtype, rot=rot, seed=rot), norm, layout)


@pytest.mark.parametrize("n,hq,hk", [(1, 1, 1), (1, 32, 32), (3, 7, 1), (130, 1, 9), (257, 16, 16), (2, 33, 17)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_shapes(kda, n, hq, hk, dtype):
    _check(kda, *_inputs(n, hq, hk, 128, dtype, seed=n), "rms", "half")
    _check(kda, *_inputs(n, hq, hk, 64, dtype, weight=False, rot=32, seed=n), "l2", "interleaved")


def test_no_rotation_and_zero_rows(kda):
    q, k, pos, table, wq, wk = _inputs(20, 4, 2, 128, F32, rot=0)
    q[3] = 0
    k[:] = 0
    _check(kda, q, k, None, None, wq, wk, "rms", "half")
    yq, yk = kda.qk_norm_rope(q.cuda(), k.cuda(), norm="l2")
    assert not yq[3].any() and not yk.any()


def test_infinity_outside_the_rotated_part_stays_there(kda):
    q, k, pos, table, _, _ = _inputs(4, 2, 2, 128, F32, weight=False, rot=64)
    q[0, 0, 100] = math.inf
    for layout in ("half", "interleaved"):
        yq, _ = kda.qk_norm_rope(*map(_cu, (q, k, pos, table)), norm="none", layout=layout)
        assert yq[0, 0, 100] == math.inf
        assert torch.isfinite(torch.cat([yq[0, 0, :100], yq[0, 0, 101:]])).all()


def test_slices_in_place_batched_and_the_same_bits(kda):
    gen = torch.Generator().manual_seed(3)
    p = torch.randn(2, 9, 10, 128, generator=gen).to(BF).cuda()
    q, k = p[:, :, :4], p[:, :, 4:7]
    pos = torch.arange(18).view(2, 9).int().cuda()
    table = kda.rope_table(18, 128)
    a = kda.qk_norm_rope(q, k, pos, table, norm="l2")
    qc, kc = q.contiguous(), k.contiguous()
    b = kda.qk_norm_rope(qc, kc, pos, table, norm="l2", q_out=qc, k_out=kc)
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and b[0] is qc
    w = torch.rand(128, device="cuda")
    q2, k2 = (torch.randn(3000, 16, 128, device="cuda").to(BF) for _ in range(2))
    pos2 = torch.randint(0, 18, (3000,), device="cuda").int()
    x = kda.qk_norm_rope_backward(q2, k2, k2, q2, pos2, table, w, w)
    y = kda.qk_norm_rope_backward(q2, k2, k2, q2, pos2, table, w, w)
    assert all(torch.equal(x[n], y[n]) for n in x)


def test_bad_positions_are_left_out(kda):
    q, k, pos, table, wq, wk = _inputs(50, 4, 2, 128, BF, P=30)
    good = pos.clone()
    pos[[3, 17]] = torch.tensor([-1, 30]).int()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    qo, ko = (torch.full(x.shape, 5.0, dtype=BF, device="cuda") for x in (q, k))
    kda.qk_norm_rope(*map(_cu, (q, k, pos, table, wq, wk)), q_out=qo, k_out=ko, device_status=st)
    ok = kda.qk_norm_rope(*map(_cu, (q, k, good, table, wq, wk)), device_status=st)
    assert st.item() == kda.KDA_DEV_OK
    kda.qk_norm_rope(*map(_cu, (q, k, pos, table, wq, wk)), device_status=st)
    assert st.item() == kda.KDA_DEV_BAD_POSITION
    keep = [i for i in range(50) if i not in (3, 17)]
    assert (qo[[3, 17]] == 5).all() and (ko[[3, 17]] == 5).all()
    assert torch.equal(qo[keep], ok[0][keep]) and torch.equal(ko[keep], ok[1][keep])
    kda.qk_norm_rope_backward(*map(_cu, (q, k, q, k, pos, table, wq, wk)), device_status=st)
    assert st.item() == kda.KDA_DEV_BAD_POSITION


def test_no_tokens(kda):
    q, k = torch.zeros(0, 4, 128, device="cuda"), torch.zeros(0, 2, 128, device="cuda")
    w = torch.ones(128, device="cuda")
    yq, yk = kda.qk_norm_rope(q, k, None, None, w, w)
    assert yq.shape == q.shape and yk.shape == k.shape
    d = kda.qk_norm_rope_backward(q, k, q, k, None, None, w, w)
    assert not d["dq_weight"].any() and not d["dk_weight"].any()


def test_gradients_against_differences(kda):
    q, k, pos, table, wq, wk = _inputs(6, 3, 2, 64, F32, rot=32)
    gen = torch.Generator().manual_seed(2)
    dq, dk = (torch.randn(x.shape, generator=gen) for x in (q, k))
    got = kda.qk_norm_rope_backward(*map(_cu, (q, k, dq, dk, pos, table, wq, wk)), norm="l2")
    for x, w, dy, n in ((q, wq, dq, "q"), (k, wk, dk, "k")):
        def loss(a, b):
            return float((R.norm_rope(a, b, pos, table.double(), "l2", 1e-6, "half") * dy).sum())
        for name, at in (("d" + n, 0), ("d" + n + "_weight", 1)):
            args = [x.double(), w.double()]
            u = torch.randn(args[at].shape, generator=gen, dtype=torch.float64)
            h = 1e-5
            hi, lo = list(args), list(args)
            hi[at], lo[at] = args[at] + h * u, args[at] - h * u
            diff = (loss(*hi) - loss(*lo)) / (2 * h)
            mine = float((got[name].cpu().double() * u).sum())
            size = float(got[name].cpu().double().norm() * u.norm()) / math.sqrt(u.numel())
            assert abs(mine - diff) <= 1e-4 * size, (name, mine, diff)
