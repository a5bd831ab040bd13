"""The tolerance of test_window_fp32_scores_gpu.py: a model of the kernels' split
products stays within it, and one that has lost a product does not."""
import pytest
import torch

import _split_model as M
import _window_ref as W


@pytest.mark.parametrize("sharp,d,scale", M.CASES)
def test_a_lost_product_is_seen(sharp, d, scale):
    scale = scale or d ** -0.5
    gen = torch.Generator().manual_seed(3)
    q = sharp * torch.randn(300, 2, d, generator=gen)
    k, v = (torch.randn(300, 1, d, generator=gen) for _ in range(2))
    see = W.visible(300, 100, 4)

    def attend(s):
        s = (s * scale).masked_fill(~see, -torch.inf)
        return torch.einsum("hij,jd->hid", s.softmax(-1), v[:, 0].double()), s
    exact, s0 = attend(torch.einsum("ihd,jhd->hij", q.double(), k.double().repeat_interleave(2, 1)))

    def off(lost):
        o, s = attend(M.scores(q, k, lost))
        return float((o - exact).norm() / exact.norm()), float((s - s0)[:, see].abs().max())
    tol = M.bound(q, k, scale)
    assert max(off(None)) <= 0.5 * tol  # half of it left for the sums
    for lost in ("lo hi", "hi lo"):
        assert off(lost)[0] > 2 * tol
