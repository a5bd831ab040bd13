"""The groups and batches of test_window_wide_gpu.py within the bounds that
test_window_gpu.py derives for the same kernels: bf16 3.2e-3 for o, 5e-3 for the
gradients (there 4e-3 and 6e-3)."""
import pytest
import torch

import test_window_wide_gpu as wide
from test_window_gpu import TOL_G, TOL_O
from test_window_wide_gpu import test_decode_of_a_wide_group_at_the_last_position, test_groups_and_batches  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _tight(monkeypatch):
    for dtype in (torch.bfloat16, torch.float32):
        monkeypatch.setitem(wide.TOL, dtype, (TOL_O[dtype], TOL_G[dtype]))
