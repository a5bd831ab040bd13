"""Inputs from one stream, the call on another, the inputs let go of at once:
their memory is not handed out again before the call has read it."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_inputs_let_go_of_after_a_call_on_a_side_stream(kda):
    gen = torch.Generator("cuda").manual_seed(1)

    def make():
        return [torch.randn(2, 2048, 8, 128, generator=gen, device="cuda").bfloat16() for _ in range(3)]
    inputs = make()
    want, _ = kda.linear_prefill(*inputs, decay="none", scale=0.01)
    side, ahead = torch.cuda.Stream(), torch.randn(8192, 8192, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(20):  # work in front of the call
            ahead @ ahead
    got, _ = kda.linear_prefill(*inputs, decay="none", scale=0.01, stream=side)
    shape = inputs[0].shape
    del inputs
    others = [torch.full(shape, 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    assert len(others) == 8 and torch.equal(got, want)
