"""The rows that the gradients of sinks are gathered in (win_near_row, win_far_row):
no two sums share one, all lie in the workspace, and that grows with the tokens,
whatever the number of sequences and sinks. No GPU."""
import random

import pytest
import torch

import kda_gated_delta_chunkwise_gb300 as kda
from kda_gated_delta_chunkwise_gb300 import build


def _rows(lens, window, sinks, queries):
    """As the kernels place them: (rows of the near sums, rows of the parts)."""
    tokens, rows = sum(lens), min(len(lens) * sinks, sum(lens))
    near, part, row, start = [], [], 0, 0
    for m in lens:
        each = min(sinks, m) if m > window else 0
        near += range(row, row + each)
        for first in range(0, m, queries):
            if m > window and min(first + queries, m) > window:  # some query of the part is behind the window
                at = row if first // queries == window // queries else rows + ((start + first) // queries - 1) * sinks
                part += range(at, at + each)
        row, start = row + each, start + m
    return near, part, rows, rows + tokens // queries * sinks


@pytest.mark.parametrize("queries", [256, 1024])
def test_no_two_sums_share_a_row(queries):
    rng = random.Random(queries)
    for _ in range(400):
        longest = rng.choice([3, 40, 300, 2000, 6000])
        lens = [int(longest ** rng.random()) - rng.randrange(2) for _ in range(rng.choice([1, 2, 7, 60]))]
        lens = [max(0, m) for m in lens]
        if not sum(lens):
            continue
        near, part, near_rows, part_rows = _rows(lens, rng.choice([1, 2, 7, 100, 255, 256, 1023, 1500]), rng.choice([1, 4, 100, 128]), queries)
        for rows, most in ((near, near_rows), (part, part_rows)):
            assert len(set(rows)) == len(rows)
            assert not rows or (min(rows) >= 0 and max(rows) < most)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,T", [(4096, 65536), (65536, 65536), (1, 65536), (60000, 1000), (4096, 4096)])
def test_the_workspace_grows_with_the_tokens(dtype, N, T):
    build.build()
    hq = hk = 16
    d, sinks = 128, 128
    both = 2 * T * hk * d * 4  # dk and dv of every token in fp32
    size = kda.window_varlen_attention_backward_workspace_bytes(N, T, hq, hk, d, sinks, dtype)
    small = 2 * 4 * T * hq + 16 * (T // 256 + N) + 8 * (N + 1) + 4096  # lse and D, the tables
    assert 0 < size <= 2.5 * both + small
    equal = kda.window_attention_backward_workspace_bytes(N, 16, hq, hk, d, sinks, dtype)
    assert 0 < equal <= 2.5 * (2 * N * 16 * hk * d * 4) + 8 * N * 16 * hq + 4096
    # few sinks of few sequences need few rows
    assert kda.window_varlen_attention_backward_workspace_bytes(2, 1 << 20, hq, hk, d, 4, dtype) <= 8 * (1 << 20) * hq + (1 << 29)
