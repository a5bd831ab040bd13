"""Calls on no sequences: the status and the per-head gradient are written all the same."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _status():
    return torch.full((1,), 9, dtype=torch.int32, device="cuda")


def _used(n):
    """Leaves memory that is not zero where the next tensor of n floats is likely to come from."""
    torch.full((n,), 7.0, device="cuda")


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_head_gradient_of_no_sequences_is_zero(kda, dtype, d):
    H = 300
    g = torch.zeros(H, device="cuda")
    x = torch.zeros(0, 5, H, d, dtype=dtype, device="cuda")
    _used(H)
    r = kda.linear_prefill_backward(x, x, x, g, x, decay="head")
    assert not r["dlog_decay"].any() and r["dq"].shape == x.shape and r["d_initial_state"].shape == (0, H, d, d)
    p, cu, st = x.reshape(0, H, d), torch.zeros(1, dtype=torch.int32, device="cuda"), _status()
    _used(H)
    r = kda.linear_varlen_prefill_backward(p, p, p, g, p, cu, decay="head", device_status=st)
    assert not r["dlog_decay"].any() and st.item() == kda.KDA_DEV_OK


def test_status_of_no_sequences(kda):
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    for tokens, want in ((0, kda.KDA_DEV_OK), (5, kda.KDA_DEV_BAD_CU_SEQLENS)):
        x, g = torch.zeros(tokens, 2, 128, dtype=BF, device="cuda"), torch.zeros(tokens, 2, device="cuda")
        out = torch.full_like(x, 5.0)
        st = _status()
        kda.linear_varlen_prefill(x, x, x, g, cu, out=out, device_status=st)
        assert st.item() == want and (out == 5).all()
        st = _status()
        kda.linear_varlen_prefill_backward(x, x, x, g, x, cu, device_status=st)
        assert st.item() == want
    x, g = torch.zeros(0, 2, 128, dtype=BF, device="cuda"), torch.zeros(0, 2, device="cuda")
    pool, slots, st = torch.zeros(3, 2, 128, 128, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda"), _status()
    kda.linear_decode_step_slots(x, x, x, g, pool, slots, device_status=st)
    assert st.item() == kda.KDA_DEV_OK and not pool.any()
