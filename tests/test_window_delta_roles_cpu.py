"""The roles of the kernel that makes D of the window attention's gradients
(win_delta_tc_kernel) and their barriers as a model, on the CPU, in random orders:
the way of test_window_roles_cpu.py."""
import re

import pytest

from test_window_roles_cpu import Item, Model, SOURCE, _always

STAGES = re.search(r"struct Bd \{.*?STAGES = D == 128 \? (\d+) : (\d+);", open(SOURCE).read(), re.S).groups()


def _delta(items, seed, stages, waits_for_rows=True):
    m = Model(seed)
    QF, OF, QE = m.barrier(), m.barrier(), m.barrier(2)
    PF, L = m.ring(2), m.ring(2, 4)
    KF, KE = m.ring(stages), m.ring(stages, 2)
    ring, at, made = [None] * stages, {"Q": None, "dO": None}, [[None, None], [None, None]]  # S, dP of each context

    def uses(item, w, j):
        far, begin, mine = item.halves[w]
        return mine > 0 and (bool(far) if j < item.far else begin <= j <= begin + mine - far - 1)

    def loads():
        slot, phase = 0, 1
        for k, item in enumerate(items):
            yield QE.wait(k + 1)
            at["Q"] = at["dO"] = k
            QF.arrive()
            for j in range(2 * item.tiles):
                yield KE[slot].wait(phase)
                ring[slot] = (k, j)
                KF[slot].arrive()
                if j == 0:
                    OF.arrive()
                slot += 1
                if slot == stages:
                    slot, phase = 0, phase ^ 1

    def products(w):
        slot, phase, n = 0, 0, 0

        def step():
            nonlocal slot, phase
            slot += 1
            if slot == stages:
                slot, phase = 0, phase ^ 1

        for k, item in enumerate(items):
            yield QF.wait(k)
            yield OF.wait(k)
            for j in range(item.tiles):
                pair = []
                for _ in range(2):  # K and V
                    yield KF[slot].wait(phase)
                    if uses(item, w, j):
                        pair.append(slot)
                    else:
                        m.issue(_always, KE[slot])
                    step()
                if not pair:
                    continue
                n += 1
                if waits_for_rows:
                    yield L[w].wait(n)
                for values in (0, 1):
                    def go(k=k, j=j, values=values, where=pair[values]):
                        assert ring[where] == (k, 2 * j + values) and at["dO" if values else "Q"] == k
                        made[w][values] = (k, j)
                    m.issue(go, *([PF[w]] if values else []), KE[pair[values]])
            m.issue(_always, QE)

    def rows(w):
        n = 0
        for k, item in enumerate(items):
            for j in range(item.tiles):
                if not uses(item, w, j):
                    continue
                yield PF[w].wait(n)
                n += 1
                for _ in range(2 if j >= item.far or item.kw > 64 else 1):
                    assert made[w] == [(k, j), (k, j)]
                    yield _always
                    assert made[w] == [(k, j), (k, j)]
                L[w].arrive()
                yield _always

    m.roles = {"loads": loads(), "products 0": products(0), "products 1": products(1),
               **{f"rows {w} {i}": rows(w) for w in (0, 1) for i in range(4)}}
    return m.run()


@pytest.mark.parametrize("stages", STAGES)
@pytest.mark.parametrize("T,window,sinks", [
    (600, 65, 128), (600, 1, 0), (1, 5, 2), (129, 7, 100), (700, 100, 3), (600, 128, 4), (2000, 300, 128), (600, 599, 4),
    (257, 1000, 0), (2500, 1024, 4), (513, 64, 128), (1500, 200, 128), (900, 899, 128), (300, 1, 128)])
def test_delta(T, window, sinks, stages):
    items = [Item(f, T, window, sinks) for f in range(0, T, 256)] * 3
    for seed in range(8):
        assert _delta(items, seed, int(stages)) is None, seed


def _fails(*args, **kw):
    try:
        return _delta(*args, **kw) is not None
    except AssertionError:
        return True


def test_the_model_finds_a_missing_wait():
    items = [Item(f, 900, 300, 4) for f in range(0, 900, 256)]
    assert any(_fails(items, seed, 3, waits_for_rows=False) for seed in range(20))

