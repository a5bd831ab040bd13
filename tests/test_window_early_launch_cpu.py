"""The kernels of window attention's gradients start while the one before them still
runs, so what that one writes is not read-only for them: no loads through the
read-only path, and no wait left out but where the kernel in front has waited."""
import os
import re

import pytest

import kda_gated_delta_chunkwise_gb300 as package

CSRC = os.path.join(os.path.dirname(package.__file__), "csrc")


def _kernels(name):
    """The bodies of a file's kernels, without comments."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    parts = re.split(r"__global__ void[^\n]*\n?\s*", text)[1:]
    return {re.match(r"(?:__launch_bounds__\([^)]*\)\s*)?(\w+)", p).group(1): p.split("\n}\n", 1)[0] for p in parts}


@pytest.mark.parametrize("name", ["kda_window.cu", "kda_window_tc.cu"])
def test_nothing_through_the_read_only_path(name):
    kernels = _kernels(name)
    assert len(kernels) >= 4
    for kernel, body in kernels.items():
        assert not re.search(r"__ldg|ld\.global\.nc|__ldcs|__restrict__", body), kernel


@pytest.mark.parametrize("name,front,behind", [("kda_window.cu", "win_dkv_kernel", "win_dq_kernel"),
                                               ("kda_window_tc.cu", "win_dkv_tc_kernel", "win_dq_tc_kernel")])
def test_who_reads_without_a_wait(name, front, behind):
    """dq reads lse and D without a wait: dk and dv's kernel waits for them before it lets dq start, and reads them behind
    that; dq waits before it ends, since whoever comes next waits for it alone."""
    kernels = _kernels(name)
    first = kernels[front]
    assert first.index("await_previous();") < first.index("let_next_start();")
    assert first.index("await_previous();") < min(m.start() for m in re.finditer(r"p\.(delta|lse2|lse_h)\b", first))
    assert "await_previous();" in kernels[behind][kernels[behind].rindex("store_rows" if "tc" in name else "p.dq"):]
