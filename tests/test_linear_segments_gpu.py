"""Sequences long enough to be cut into segments of every length, in one packed
batch that works on its longest segments first: the same bits as each sequence's
own call, and the results of the fp32 kernels, which cut them otherwise.

Tolerances: those of the reference file, 5e-3 for bf16 results (the fp32 call's
own error is far below it); for states, where both sides have an error of up to
1e-5, twice that.
"""
import pytest
import torch

import _linear_ref as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,lens", [(16, [1, 16385, 513, 2049, 0, 5000, 512]), (2, [4097, 1025, 130])])
@pytest.mark.parametrize("kind", ["token", "none"])
def test_packed_segments(kda, H, lens, kind):
    n, total = len(lens), sum(lens)
    gen = torch.Generator("cuda").manual_seed(11)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")
    q, v, d_o = (normal(total, H, 128).bfloat16() for _ in range(3))
    k = (normal(total, H, 128) * 128 ** -0.5).bfloat16()
    g = -torch.rand(total, H, generator=gen, device="cuda") * 0.1 if kind == "token" else None
    if g is None:
        q = q * 0.1  # without a decay the state grows with the square root of the length
    s0 = normal(n, H, 128, 128) * 0.1
    at = [0] + torch.tensor(lens).cumsum(0).tolist()
    cu = torch.tensor(at, dtype=torch.int32, device="cuda")
    o, S = kda.linear_varlen_prefill(q, k, v, g, cu, s0, decay=kind)
    d = kda.linear_varlen_prefill_backward(q, k, v, g, d_o, cu, s0, decay=kind, want_decay_grad=False)
    for i, (a, b) in enumerate(zip(at, at[1:])):
        if a == b:
            assert torch.equal(S[i], s0[i]) and not d["d_initial_state"][i].any()
            continue
        one = [None if x is None else x[None, a:b] for x in (q, k, v, g)]
        o1, S1 = kda.linear_prefill(*one, s0[i:i + 1], decay=kind)
        assert torch.equal(o[a:b], o1[0]) and torch.equal(S[i], S1[0])
        d1 = kda.linear_prefill_backward(*one, d_o[None, a:b], s0[i:i + 1], decay=kind, want_decay_grad=False)
        assert all(torch.equal(d[x][a:b], d1[x][0]) for x in ("dq", "dk", "dv"))
        assert torch.equal(d["d_initial_state"][i], d1["d_initial_state"][0])
    o32, S32 = kda.linear_varlen_prefill(q.float(), k.float(), v.float(), g, cu, s0, decay=kind)
    R.close("o", o, o32.double().cpu(), R.TOL[torch.bfloat16])
    R.close("S", S, S32.double().cpu(), 2 * R.TOL[torch.float32])
