"""The roles of lin_state_tc_kernel (loads, weights, conversion in two groups,
MMA, accumulators out) and their barriers as a model, on the CPU.

The factor that joins two parts of a block goes from the warp of the weights to
the accumulator warps through a ring that has no barrier of its own: the others
have to keep its writer from coming round to an entry before its reader. Every
role's own steps have a fixed order and a wait can only be opened by others, so
the reader's worst case is the schedule in which it moves only when nobody else
can: whatever may be written before a read has then been written.
"""
import os
import re

import pytest

import kda_gated_delta_chunkwise_gb300 as package

SOURCE = os.path.join(os.path.dirname(package.__file__), "csrc", "kda_linear_tc.cu")


def _constant(text, name):
    return int(re.search(rf"constexpr int {name} = (\d+);", text).group(1))


def _from_source():
    with open(SOURCE) as f:
        text = f.read()
    ring = re.search(r"__shared__ float join\[(\w+)\]", text).group(1)
    return (int(ring) if ring.isdigit() else _constant(text, ring)), _constant(text, "ST_STAGES")


TOKENS, PART = 64, 256  # of a tile and of a part


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.done = count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.done = self.count, self.done + 1

    def passes(self, parity):  # as mbarrier.try_wait.parity
        return (self.done & 1) != parity


def _parts(items):
    """(first part of its block, tiles) of every part in turn."""
    return [(p0 == 0, -(-(min(n, p0 + PART) - p0) // TOKENS)) for n in items for p0 in range(0, n, PART)]


def _run(items, ring, stages):
    """Runs the roles; yields (part, what its reader found, whether the value counts)."""
    parts = _parts(items)
    full, conv, empty = ([Barrier(1) for _ in range(n)] for n in (6, stages, stages))
    acc_full, acc_empty, w_full = ([Barrier(1) for _ in range(2)] for _ in range(3))
    w_empty = [Barrier(2) for _ in range(2)]
    join, found = [None] * ring, []

    def loads():
        n = 0
        for _, tiles in parts:
            for _ in range(tiles):
                yield empty[n % stages], ((n // stages) & 1) ^ 1
                full[n % 6].arrive()
                n += 1

    def weights():
        for q in range(len(parts)):
            yield w_empty[q & 1], ((q >> 1) & 1) ^ 1
            join[q % ring] = q
            w_full[q & 1].arrive()

    def convert(group):
        n = 0
        for q, (_, tiles) in enumerate(parts):
            yield w_full[q & 1], (q >> 1) & 1
            for _ in range(tiles):
                if n & 1 == group:
                    yield full[n % 6], (n // 6) & 1
                    conv[n % stages].arrive()
                n += 1
            w_empty[q & 1].arrive()

    def mma():
        n = 0
        for q, (_, tiles) in enumerate(parts):
            yield acc_empty[q & 1], ((q >> 1) & 1) ^ 1
            for _ in range(tiles):
                yield conv[n % stages], (n // stages) & 1
                empty[n % stages].arrive()
                n += 1
            acc_full[q & 1].arrive()

    def out():
        for q, (first, _) in enumerate(parts):
            yield acc_full[q & 1], (q >> 1) & 1
            found.append((q, join[q % ring], not first))
            acc_empty[q & 1].arrive()

    roles = [loads(), weights(), convert(0), convert(1), mma(), out()]  # the reader last
    waits = [next(r, None) for r in roles]
    while any(w is not None for w in waits):
        for i, w in enumerate(waits):
            if w is not None and w[0].passes(w[1]):
                waits[i] = next(roles[i], None)
                break
        else:
            pytest.fail("the roles wait for one another")
    assert len(found) == len(parts)
    return found


@pytest.mark.parametrize("items", [
    [260] * 4 + [1] * 40, [512] + [1] * 12, [300] * 20, [512, 64] * 10, [320, 1, 1, 1, 1, 257, 1, 1, 1, 1],
    [512] * 6, [2048, 5, 513, 5, 5, 5, 5], [1] * 30, [4096, 1, 4095, 1],
])
def test_every_part_is_joined_with_its_own_factor(items):
    ring, stages = _from_source()
    wrong = [(q, x) for q, x, counts in _run(items, ring, stages) if counts and x != q]
    assert not wrong, f"part, the part whose factor it was joined with: {wrong}"


def test_the_model_finds_a_ring_that_is_too_short():
    assert any(counts and x != q for q, x, counts in _run([512] + [1] * 12, 4, 3))
    assert all(x == q for q, x, _ in _run([512] + [1] * 12, 7, 3))
