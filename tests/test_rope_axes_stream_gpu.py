"""Axes given as a tensor, on a given stream: only what lies on the device is kept for it."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("axes", [lambda a: a, bytes, torch.tensor, lambda a: torch.tensor(a).cuda(), lambda a: torch.tensor(a).numpy()],
                         ids=["list", "bytes", "tensor", "device tensor", "array"])
def test_axes_of_any_kind(kda, axes):
    q, k = (torch.randn(7, h, 64, device="cuda") for h in (4, 2))
    table, pos = kda.rope_table(30, 64), torch.randint(0, 30, (3, 7), dtype=torch.int32, device="cuda")
    pairs = [i % 3 for i in range(32)]
    want = kda.qk_norm_rope_axes(q, k, pos, table, pairs)
    back = kda.qk_norm_rope_axes_backward(q, k, *want, pos, table, pairs)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = kda.qk_norm_rope_axes(q, k, pos, table, axes(pairs), stream=s)
    grads = kda.qk_norm_rope_axes_backward(q, k, *got, pos, table, axes(pairs), stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert all(torch.equal(back[n], grads[n]) for n in ("dq", "dk"))
