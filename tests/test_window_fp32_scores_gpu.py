"""fp32 window attention at scores from ones to thousands, against 64 bits. The
tolerance is that of a score, by the size of q and k (_split_model.bound): relative
2-norm for o, absolute for lse, which is rounded besides (2^-24 of itself); for dv,
whose weights are made from a score and lse, one of each and D apart, three times o's and
2^-23 |lse|."""
import pytest
import torch

import _split_model as M
import _window_ref as W

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sharp,d,scale", M.CASES)
def test_scores_of_all_sizes(kda, sharp, d, scale):
    q, k, v, d_o = W.inputs([300], 2, 1, d, torch.float32, 3, sharp=sharp)
    s = scale or d ** -0.5
    tol = M.bound(q, k, s)
    kw = dict(window=100, sinks=4, scale=scale)
    o, lse = kda.window_attention(q[None], k[None], v[None], **kw)
    ro, rl = W.attention(q.double(), k.double(), v.double(), 100, 4, s)
    err = float((o[0].double() - ro).norm() / ro.norm())
    assert err <= tol, (err, tol)
    assert ((lse[0].double() - rl).abs() <= tol + 2.0 ** -24 * rl.abs()).all()
    g = kda.window_attention_backward(q[None], k[None], v[None], o, lse, d_o[None], **kw)
    ref = W.gradients(q, k, v, d_o, 100, 4, s)["dv"]
    err = float((g["dv"][0].double() - ref).norm() / ref.norm())
    assert err <= 3 * tol + 2.0 ** -23 * float(rl.abs().max()), (err, tol)


@pytest.mark.parametrize("group", [2, 8, 16])
@pytest.mark.parametrize("sharp,d,scale", M.CASES)
def test_decode(kda, sharp, d, scale, group):
    """Up to eight query heads to a key head by fp32 products, above by split ones; scores in powers of two, rounded
    twice on the way there, 2^-23 of themselves."""
    gen = torch.Generator().manual_seed(group)
    q = (sharp * torch.randn(3, group, d, generator=gen)).cuda()
    k, v = (torch.randn(3, 1, d, generator=gen).cuda() for _ in range(2))
    kc, vc = (torch.randn(3, 300, 1, d, generator=gen).cuda() for _ in range(2))
    slots, pos = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([2, 0, 1], [5, 299, 7000]))
    s = scale or d ** -0.5
    o = kda.window_decode_step(q, k, v, kc, vc, slots, pos, sinks=4, scale=scale)
    for n, (slot, count) in enumerate(((2, 6), (0, 300), (1, 300))):
        x = torch.einsum("hd,jd->hj", q[n].double(), kc[slot, :count, 0].double()) * s
        ref = x.softmax(-1) @ vc[slot, :count, 0].double()
        err = float((o[n].double() - ref).norm() / ref.norm())
        assert err <= M.bound(q, kc, s) + 2.0 ** -23 * float(x.abs().max()), err
