"""The sizes beyond which window attention and its cache refuse: those whose index
arithmetic would leave the kernels' types. No GPU."""
import ctypes

import pytest

import kda_gated_delta_chunkwise_gb300 as kda
from kda_gated_delta_chunkwise_gb300 import build

P = ctypes.c_void_p(0x1000)
OK, UNSUPPORTED = 0, 2


@pytest.fixture(scope="module")
def lib():
    build.build()
    return kda.load()


@pytest.mark.parametrize("heads", [1025, 1 << 20, 1 << 27, (1 << 31) - 1])
def test_heads_of_a_cache(lib, heads):
    assert lib.kda_window_cache_write(P, P, 1, 0, 0, P, P, 0, P, P, 4, 8, 1, 4, heads, 128, None, None) == UNSUPPORTED
    assert b"heads" in lib.kda_last_error()
    assert lib.kda_window_decode_step(P, P, P, 1, 0, 0, 0, 1.0, 0, P, P, 4, 8, P, P, P, 1, heads, heads, 128, None,
                                      None) == UNSUPPORTED
    assert lib.kda_window_decode_step(P, P, P, 1, 0, 0, 0, 1.0, 0, P, P, 4, 8, P, P, P, 1, heads, 1, 128, None,
                                      None) == UNSUPPORTED


def test_prompts_of_a_cache_write(lib):
    assert lib.kda_window_cache_write(P, P, 1, 0, 0, P, P, 0, P, P, 4, 8, 65536, 4, 2, 128, None, None) == UNSUPPORTED


def test_heads_of_attention(lib):
    def call(hq, hk, B=1, T=4):
        return lib.kda_window_attention(P, P, P, 1, 0, 0, 0, 1.0, 8, 0, P, P, B, T, hq, hk, 128, None)
    assert call(1025, 1025) == UNSUPPORTED and call(1 << 20, 1) == UNSUPPORTED
    assert call(1024, 1024, T=1 << 30) == UNSUPPORTED  # tiles times heads
    assert call(1024, 1024, B=0) == OK
    assert lib.kda_window_attention_backward_workspace_bytes(1, 4, 1025, 1025, 128, 4, 1) == 0
    assert lib.kda_window_attention_backward_workspace_bytes(1, 1 << 30, 1024, 1024, 128, 4, 1) == 0
