"""Large inputs under decays of every strength between none and one that forgets
a chunk: scores and outputs far from 1, results still numbers, with the
tolerances of the reference file (everything here is a product and a sum, so
they hold at any scale)."""
import pytest
import torch

import _linear_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("size", [1e-6, 1e3, 1e5, 1e7])
@pytest.mark.parametrize("rate", [0.1, 0.2, 0.3, 0.42, 0.5])
def test_large_inputs(kda, size, rate):
    gen = torch.Generator().manual_seed(4)
    q, k, v, d_o = ((torch.randn(1, 300, 2, 128, generator=gen) * size).to(BF) for _ in range(4))
    g = -rate * (0.9 + 0.2 * torch.rand(1, 300, 2, generator=gen))
    o, S = kda.linear_prefill(*(x.cuda() for x in (q, k, v, g)), scale=0.3)
    ro, rS = R.forward(q, k, v, g, None, 0.3)
    R.close("o", o, ro, R.TOL[BF])
    R.close("S", S, rS, R.TOL[F32])
    got = kda.linear_prefill_backward(*(x.cuda() for x in (q, k, v, g, d_o)), scale=0.3, want_decay_grad=False)
    ref = R.gradients(q, k, v, g, None, 0.3, d_o, None)
    for n in ("dq", "dk", "dv"):
        R.close(n, got[n], ref[n], R.TOL[BF])
