"""Rows of every size under an eps of every size, each row by itself against 64
bits; tolerances as in test_qk_norm_rope_gpu (rows are scaled by powers of ten,
which changes no relative error)."""
import pytest
import torch

import _linear_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
TOL = {F32: 2e-6, BF: 2.5e-3}
SIZES = [0.0, 1e-18, 1e-9, 1.0, 1e9, 1e13, 1e17]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("norm", ["l2", "rms"])
@pytest.mark.parametrize("eps", [1e-6, 1e-30])
@pytest.mark.parametrize("weight", [True, False])
def test_rows_of_every_size(kda, dtype, d, norm, eps, weight):
    gen = torch.Generator().manual_seed(6)
    n = len(SIZES)
    x = (torch.randn(n, 1, d, generator=gen) * torch.tensor(SIZES)[:, None, None]).to(dtype)
    dy = torch.randn(n, 1, d, generator=gen).to(dtype)
    w = 1 + 0.3 * torch.randn(d, generator=gen) if weight else None
    pos, table = torch.arange(n, dtype=torch.int32), kda.rope_table(n, d, device="cpu")
    kw = dict(norm=norm, eps=eps)
    wc = None if w is None else w.cuda()
    y, _ = kda.qk_norm_rope(x.cuda(), x.cuda(), pos.cuda(), table.cuda(), wc, wc, **kw)
    got = kda.qk_norm_rope_backward(x.cuda(), x.cuda(), dy.cuda(), dy.cuda(), pos.cuda(), table.cuda(), wc, wc, **kw)
    x64 = x.double().requires_grad_()
    ref = R.norm_rope(x64, None if w is None else w.double(), pos, table.double(), norm, eps, "half")
    ref.backward(dy.double())
    for i, size in enumerate(SIZES):
        R.close(f"y at {size}", y[i], ref[i], TOL[dtype])
        R.close(f"dx at {size}", got["dq"][i], x64.grad[i], TOL[dtype])
