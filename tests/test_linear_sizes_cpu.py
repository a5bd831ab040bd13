"""Sizes whose products pass 64 bits are refused like all others that are too
large, by the workspace functions and by the calls, before any launch. No GPU."""
import ctypes

import pytest

import kda_gated_delta_chunkwise_gb300 as kda
from kda_gated_delta_chunkwise_gb300 import build

P = ctypes.c_void_p(0x1000)
UNSUPPORTED = 2
M = 2 ** 31 - 1
SIZES = [(M, 1, M), (1 << 30, 1, 1 << 30), (1 << 30, 0, 1 << 30), (M, 1, 1 << 28), (M, M, M)]


@pytest.fixture(scope="module")
def lib():
    build.build()
    return kda.load()


@pytest.mark.parametrize("n,tokens,heads", SIZES)
def test_prefill_sizes_beyond_64_bits(lib, n, tokens, heads):
    for name in ("prefill", "varlen_prefill", "prefill_backward", "varlen_prefill_backward"):
        assert getattr(lib, f"kda_linear_{name}_workspace_bytes")(n, tokens, heads, 128, 128, 1) == 0, name
    big = (1 << 63) - 1
    assert lib.kda_linear_prefill(P, P, P, 1, 0, 0, 0, P, 0, 1.0, None, P, None, n, tokens, heads, 128, 128, None, big,
                                  None) == UNSUPPORTED
    assert lib.kda_linear_varlen_prefill(P, P, P, 1, 0, 0, 0, P, 0, 1.0, None, P, None, P, n, tokens, heads, 128, 128,
                                         None, big, None, None) == UNSUPPORTED


def test_sizes_that_still_fit(lib):
    assert lib.kda_linear_varlen_prefill_workspace_bytes(1 << 10, 0, 1 << 6, 128, 128, 1) > 0
    assert lib.kda_linear_prefill_workspace_bytes(1, 64, 1 << 20, 64, 64, 0) > 0


def test_decode_sizes_beyond_64_bits(lib):
    assert lib.kda_linear_decode_step(P, P, P, 1, 0, 0, 0, P, 0, 1.0, P, P, M, M, 128, 128, None) == UNSUPPORTED
    assert lib.kda_linear_decode_step(P, P, P, 1, 0, 0, 0, P, 0, 1.0, P, P, M, 1, 128, 128, None) == UNSUPPORTED
