"""Slow decays over long sequences: what the first tokens and the initial state
leave after 131,072 tokens, where an error that comes out the same for every
token or block adds up.

Tolerances (relative L2). The initial state is rounded once for every block: 2048
blocks of 64 tokens, 2^-24 at most each and 0.3 of it in the root mean square,
adding as a random walk: 0.8e-6; its decay is off by 2^-40 octaves a token
(0.8e-7 in all) and the blocks' factors by 2^-24 of what they take off: 1e-6 in
all, bound 3e-6. What the first token wrote also passes the factors that join a
segment's parts, 16 of them, off by 2^-22 each: 4e-6 more, bound 1e-5.
"""
import pytest
import torch

import _linear_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
T = 131072


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 128), (F32, 64), (BF, 64)])
@pytest.mark.parametrize("rate", [1e-5, 3e-6, 1e-6, 3e-8])
def test_the_initial_state_after_a_long_sequence(kda, dtype, d, rate):
    gen = torch.Generator("cuda").manual_seed(2)
    x = torch.zeros(1, T, 2, d, dtype=dtype, device="cuda")
    s0 = torch.randn(1, 2, d, d, generator=gen, device="cuda")
    g = torch.tensor([-rate, -0.7 * rate], device="cuda")
    ref = s0.double() * (g.double() * T).exp()[None, :, None, None]
    _, S = kda.linear_prefill(x, x, x, g, s0, decay="head")
    R.close("S", S, ref, 3e-6)
    for want in (True, False):
        r = kda.linear_prefill_backward(x, x, x, g, x, None, s0, decay="head", want_decay_grad=want)
        R.close("d_initial_state", r["d_initial_state"], ref, 3e-6)
    _, S = kda.linear_prefill(x, x, x, g.expand(1, T, 2).contiguous(), s0)
    R.close("S", S, ref, 3e-6)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_the_first_token_after_a_long_sequence(kda, dtype, d):
    gen = torch.Generator("cuda").manual_seed(3)
    k, v = (torch.zeros(1, T, 2, d, dtype=dtype, device="cuda") for _ in range(2))
    for x in (k, v):
        x[:, 0] = torch.randn(1, 2, d, generator=gen, device="cuda").to(dtype)
    g = torch.tensor([-1e-5, -3e-6], device="cuda")
    _, S = kda.linear_prefill(k, k, v, g, decay="head")
    first = k[0, 0].double()[:, :, None] * v[0, 0].double()[:, None, :]
    R.close("S", S[0], first * (g.double() * (T - 1)).exp()[:, None, None], R.TOL[F32])
