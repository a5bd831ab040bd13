"""Many short segments behind longer ones on every CTA, where the roles of the
state pass run furthest apart: the same bits as each sequence's own call, in
which no CTA has more than one of its segments of a kind.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _inputs(total, H, n, seed):
    gen = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")
    q, v, d_o = (normal(total, H, 128).bfloat16() for _ in range(3))
    k = (normal(total, H, 128) * 128 ** -0.5).bfloat16()
    # decays that differ by token and head, so that another part's factor shows
    g = -torch.rand(total, H, generator=gen, device="cuda") * torch.linspace(1e-3, 0.05, H, device="cuda")
    return q, k, v, g, d_o, normal(n, H, 128, 128) * 0.1


def test_prompts_packed_with_short_sequences(kda):
    gen = torch.Generator().manual_seed(3)
    lens = torch.cat([torch.randint(260, 321, (20,), generator=gen), torch.randint(1, 65, (500,), generator=gen)])
    lens = lens[torch.randperm(520, generator=gen)].tolist()
    at = [0] + torch.tensor(lens).cumsum(0).tolist()
    q, k, v, g, d_o, s0 = _inputs(at[-1], 32, 520, 4)
    cu = torch.tensor(at, dtype=torch.int32, device="cuda")
    for _ in range(3):
        o, S = kda.linear_varlen_prefill(q, k, v, g, cu, s0, scale=0.3)
        d = kda.linear_varlen_prefill_backward(q, k, v, g, d_o, cu, s0, s0, scale=0.3, want_decay_grad=False)
        for i, (a, b) in enumerate(zip(at, at[1:])):
            one = [x[None, a:b] for x in (q, k, v, g)]
            o1, S1 = kda.linear_prefill(*one, s0[i:i + 1], scale=0.3)
            assert torch.equal(o[a:b], o1[0]) and torch.equal(S[i], S1[0]), (i, b - a)
            d1 = kda.linear_prefill_backward(*one, d_o[None, a:b], s0[i:i + 1], s0[i:i + 1], scale=0.3,
                                             want_decay_grad=False)
            assert all(torch.equal(d[n][a:b], d1[n][0]) for n in ("dq", "dk", "dv")), (i, b - a)
            assert torch.equal(d["d_initial_state"][i], d1["d_initial_state"][0]), (i, b - a)


def test_equal_lengths_with_a_short_second_segment(kda):
    B, T, H = 48, 576, 16
    q, k, v, g, d_o, s0 = _inputs(B * T, H, B, 5)
    q, k, v, d_o = (x.view(B, T, H, 128) for x in (q, k, v, d_o))
    g = g.view(B, T, H)
    for _ in range(3):
        o, S = kda.linear_prefill(q, k, v, g, s0, scale=0.3)
        d = kda.linear_prefill_backward(q, k, v, g, d_o, s0, s0, scale=0.3, want_decay_grad=False)
        for i in range(B):
            one = slice(i, i + 1)
            o1, S1 = kda.linear_prefill(q[one], k[one], v[one], g[one], s0[one], scale=0.3)
            assert torch.equal(o[one], o1) and torch.equal(S[one], S1), i
            d1 = kda.linear_prefill_backward(q[one], k[one], v[one], g[one], d_o[one], s0[one], s0[one], scale=0.3,
                                             want_decay_grad=False)
            assert all(torch.equal(d[n][one], d1[n]) for n in ("dq", "dk", "dv", "d_initial_state")), i
