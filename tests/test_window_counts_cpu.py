"""Counts that a C int does not hold are refused, not cut to their low 32 bits. No GPU."""
import pytest
import torch

import kda_gated_delta_chunkwise_gb300 as kda

X = torch.zeros(1, 4, 2, 128)
ROW, CACHE, INTS = X[0], torch.zeros(2, 9, 2, 128), torch.zeros(4, dtype=torch.int32)
CALLS = {
    "window_attention": lambda **kw: kda.window_attention(X, X, X, **{"window": 4, **kw}),
    "window_varlen_attention": lambda **kw: kda.window_varlen_attention(ROW, ROW, ROW, INTS, **{"window": 4, **kw}),
    "window_attention_backward": lambda **kw: kda.window_attention_backward(X, X, X, X, X[..., 0], X, **{"window": 4, **kw}),
    "window_varlen_attention_backward": lambda **kw: kda.window_varlen_attention_backward(
        ROW, ROW, ROW, ROW, ROW[..., 0], ROW, INTS, **{"window": 4, **kw}),
    "window_cache_write": lambda **kw: kda.window_cache_write(ROW, ROW, INTS, CACHE, CACHE, INTS, **kw),
    "window_decode_step": lambda **kw: kda.window_decode_step(ROW, ROW, ROW, CACHE, CACHE, INTS, INTS, **kw),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("sinks", [1 << 32, (1 << 32) + 4, -(1 << 32), 1 << 31, 1 << 70])
def test_sinks(name, sinks):
    with pytest.raises(ValueError, match="sinks"):
        CALLS[name](sinks=sinks)


@pytest.mark.parametrize("name", [n for n in CALLS if "attention" in n])
def test_windows(name):
    for window in (-(1 << 32) + 5, -(1 << 40), -(1 << 31) - 1):
        with pytest.raises(ValueError, match="window"):
            CALLS[name](window=window)
    with pytest.raises(ValueError, match="CUDA"):  # a long one is as good as any other
        CALLS[name](window=1 << 40)


@pytest.mark.parametrize("sizes", [(1 << 32, 64, 4, 2), (1, (1 << 32) + 64, 4, 2), (1, 64, (1 << 32) + 4, 2), (1, 64, 4, 2, 128, 1 << 32)])
def test_workspace_sizes(sizes):
    for f in (kda.window_attention_backward_workspace_bytes, kda.window_varlen_attention_backward_workspace_bytes):
        with pytest.raises(ValueError, match="32 bits"):
            f(*sizes)
    if len(sizes) == 4:
        with pytest.raises(ValueError, match="32 bits"):
            kda.window_varlen_attention_workspace_bytes(*sizes)
