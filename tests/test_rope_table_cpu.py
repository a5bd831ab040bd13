"""The "yarn" table: the blend by the number of turns, and the bounds it takes. No GPU."""
import math

import pytest

import kda_gated_delta_chunkwise_gb300 as kda


def test_yarn_blends_in_proportion_to_the_turns():
    n, rot, base, factor, fast, slow = 4096, 64, 10000.0, 4.0, 32.0, 1.0
    t = kda.rope_table(3, rot, base=base, scaling="yarn", factor=factor, original_max_position=n, beta_fast=fast,
                       beta_slow=slow, device="cpu")
    gain, blended = 0.1 * math.log(factor) + 1.0, 0
    for i in range(rot // 2):
        f = base ** (-2 * i / rot)
        keep = min(1.0, max(0.0, (n * f / (2 * math.pi) - slow) / (fast - slow)))
        blended += 0.0 < keep < 1.0
        f = f * keep + f / factor * (1.0 - keep)
        assert abs(t[2, i].item() - gain * math.cos(2 * f)) < 1e-6
        assert abs(t[2, rot // 2 + i].item() - gain * math.sin(2 * f)) < 1e-6
    assert blended >= 8


@pytest.mark.parametrize("fast,slow", [(1.0, 1.0), (1.0, 32.0), (32.0, -1.0), (math.nan, 1.0), (32.0, math.nan),
                                       (math.inf, 1.0)])
def test_yarn_refuses_bounds_without_a_blend_between_them(fast, slow):
    with pytest.raises(ValueError, match="beta_slow < beta_fast"):
        kda.rope_table(8, 64, scaling="yarn", factor=4.0, original_max_position=64, beta_fast=fast, beta_slow=slow,
                       device="cpu")
