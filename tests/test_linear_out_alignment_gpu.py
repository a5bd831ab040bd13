"""Outputs that are aligned to 16 bytes alone, as the interface asks: the
tensor-core kernels store 32 bytes at a time where they may."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_linear_prefill_into_an_output_at_16_bytes(kda):
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(1, 300, 2, 128, generator=gen, device="cuda").bfloat16() for _ in range(3))
    g = -torch.rand(1, 300, 2, generator=gen, device="cuda") * 0.1
    room = torch.zeros(q.numel() + 8, dtype=torch.bfloat16, device="cuda")
    out = room[8:].view_as(q)
    assert out.data_ptr() % 32 == 16
    o, _ = kda.linear_prefill(q, k, v, g)
    kda.linear_prefill(q, k, v, g, out=out)
    assert torch.equal(o, out)
