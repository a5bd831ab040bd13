"""The roles of the tensor-core kernels of window attention and their barriers as
models, on the CPU: loads, products, softmax and epilogue, run in random orders in
which one role may lag behind all others. A barrier tells its waiters only the
parity of its phase, so one that comes two phases ahead of a waiter, or takes an
arrival that belongs to the next phase, would stop the kernel or let a product read
what is not there yet. Products are executed in the order of their issue, at any
time after it, and their commits with them.
"""
import os
import random
import re
from collections import deque

import pytest

import kda_gated_delta_chunkwise_gb300 as package

SOURCE = os.path.join(os.path.dirname(package.__file__), "csrc", "kda_window_tc.cu")


def _numbers(struct, *names):
    """The stages that the source gives its rings."""
    with open(SOURCE) as f:
        text = f.read().split(f"struct {struct} {{", 1)[1].split("\n};", 1)[0]
    return [int(re.search(rf"\b{n} = (\d+)", text).group(1)) for n in names]


class Barrier:
    def __init__(self, count=1):
        self.count, self.left, self.done = count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.done = self.count, self.done + 1

    def wait(self, phase):  # as mbarrier.try_wait.parity
        return lambda: (self.done & 1) != (phase & 1)


class Model:
    def __init__(self, seed):
        self.random, self.pipe, self.roles, self.barriers = random.Random(seed), deque(), {}, []

    def barrier(self, count=1):
        self.barriers.append(Barrier(count))
        return self.barriers[-1]

    def ring(self, n, count=1):
        return [self.barrier(count) for _ in range(n)]

    def run(self):
        """Until every role is through; None, or those that wait for one another."""
        waits = {}
        for name, role in self.roles.items():
            wait = next(role, None)
            if wait:
                waits[name] = wait
        slow = self.random.choice([None, "pipe", *self.roles])
        while waits or self.pipe:
            ready = [n for n, w in waits.items() if w()] + ["pipe"] * bool(self.pipe)
            if not ready:
                return sorted(waits)
            fast = [n for n in ready if n != slow]
            name = self.random.choice(fast if fast and self.random.random() < .97 else ready)
            if name == "pipe":
                self.pipe.popleft()()
                continue
            wait = next(self.roles[name], None)
            if wait:
                waits[name] = wait
            else:
                del waits[name]
        assert all(b.left == b.count for b in self.barriers), "a barrier ends within a phase"
        return None

    def issue(self, check, *commits):
        def execute():
            check()
            for b in commits:
                b.arrive()
        self.pipe.append(execute)


def _always():
    return True


# ------------------------------------------------------------------- gradients: dk, dv
def _dkv(items, seed, q_stages, o_stages):
    """``items``: the steps of every tile of keys."""
    m = Model(seed)
    KF, KE, SF, PE, DF, XF = (m.barrier(c) for c in (1, 2, 1, 1, 1, 1))
    SL, PR, DR, AE, XE = (m.barrier(8) for _ in range(5))
    AF = m.barrier(2)
    QF, QE, OF, OE = m.ring(q_stages), m.ring(q_stages), m.ring(o_stages), m.ring(o_stages, 2)
    LF, LE = m.ring(2), m.ring(2, 8)
    at = {"S": None, "dP": None, "D": None, "P": [None] * 8, "dS": [None] * 8, "lse": [None] * 2,
          "Q": [None] * q_stages, "dO": [None] * o_stages}

    def loads():
        n = 0
        for k, steps in enumerate(items):
            yield KE.wait(k + 1)
            KF.arrive()
            for _ in range(steps):
                yield QE[n % q_stages].wait(n // q_stages + 1)
                at["Q"][n % q_stages] = n
                QF[n % q_stages].arrive()
                yield OE[n % o_stages].wait(n // o_stages + 1)
                at["dO"][n % o_stages] = n
                OF[n % o_stages].arrive()
                n += 1

    def vectors():
        for n in range(sum(items)):
            yield LE[n & 1].wait((n >> 1) + 1)
            at["lse"][n & 1] = n
            LF[n & 1].arrive()
            yield XE.wait(n + 1)
            at["D"] = n
            XF.arrive()

    def holds(**want):
        def check():
            for name, (where, n) in want.items():
                got = at[name] if where is None else at[name][where] if where >= 0 else set(at[name])
                assert got == (n if where is None or where >= 0 else {n}), (name, got, n)
        return check

    def set_to(name, n, check):
        def go():
            check()
            at[name] = n
        return go

    def products(second):
        n = 0

        def ahead(j):
            if not second:
                yield QF[j % q_stages].wait(j // q_stages)
                yield LF[j & 1].wait(j >> 1)
                m.issue(set_to("S", j, holds(Q=(j % q_stages, j))), SF)
            else:
                yield OF[j % o_stages].wait(j // o_stages)
                yield XF.wait(j)
                m.issue(set_to("dP", j, holds(dO=(j % o_stages, j), D=(None, j))), DF, OE[j % o_stages])

        for k, steps in enumerate(items):
            yield KF.wait(k)
            yield from ahead(n)
            if steps == 1:
                m.issue(_always, KE)
            for j in range(steps):
                more = j + 1 < steps
                if not second:
                    if more:
                        yield SL.wait(n)
                        yield from ahead(n + 1)
                        if j + 2 == steps:
                            m.issue(_always, KE)
                    yield OF[n % o_stages].wait(n // o_stages)
                    yield PR.wait(n)
                else:
                    yield QF[n % q_stages].wait(n // q_stages)
                    yield DR.wait(n)
                if j == 0:
                    yield AE.wait(k + 1)
                if not second:
                    m.issue(holds(dO=(n % o_stages, n), P=(-1, n)), PE, OE[n % o_stages])
                else:
                    m.issue(holds(Q=(n % q_stages, n), dS=(-1, n)), QE[n % q_stages])
                    if more:
                        yield from ahead(n + 1)
                        if j + 2 == steps:
                            m.issue(_always, KE)
                if not more:
                    m.issue(_always, AF)
                n += 1

    def weights(i):
        n = 0
        for k, steps in enumerate(items):
            for _ in range(steps):
                yield SF.wait(n)
                holds(S=(None, n), lse=(n & 1, n))()
                yield _always
                holds(S=(None, n))()
                SL.arrive()
                yield _always
                holds(lse=(n & 1, n))()
                yield PE.wait(n + 1)
                at["P"][i] = n
                LE[n & 1].arrive()
                yield _always
                PR.arrive()
                yield DF.wait(n)
                holds(dP=(None, n), D=(None, n))()
                yield _always
                holds(dP=(None, n), D=(None, n))()
                at["dS"][i] = n
                XE.arrive()
                yield _always
                DR.arrive()
                n += 1
            yield AF.wait(k)
            AE.arrive()

    m.roles = {"loads": loads(), "vectors": vectors(), "S, dV": products(False), "dP, dK": products(True),
               **{f"weights {i}": weights(i) for i in range(8)}}
    return m.run()


# ------------------------------------------------------------------- gradients: dq
def _dq(items, seed, k_stages, v_stages, made_barriers=2):
    m = Model(seed)
    QF, DF, AF = (m.barrier() for _ in range(3))
    QE, DL, AE = m.barrier(2), m.barrier(8), m.barrier(8)
    SF, DR = m.ring(2), m.ring(made_barriers, 8)
    KF, KE, VF, VE = m.ring(k_stages), m.ring(k_stages), m.ring(v_stages), m.ring(v_stages)
    at = {"Q": None, "K": [None] * k_stages, "V": [None] * v_stages, "S": [None] * 2, "dP": None,
          "dS": [[None] * 8, [None] * 8], "dQ": None}

    def loads():
        n = 0
        for k, steps in enumerate(items):
            yield QE.wait(k + 1)
            at["Q"] = k
            QF.arrive()
            for _ in range(steps):
                yield KE[n % k_stages].wait(n // k_stages + 1)
                at["K"][n % k_stages] = n
                KF[n % k_stages].arrive()
                yield VE[n % v_stages].wait(n // v_stages + 1)
                at["V"][n % v_stages] = n
                VF[n % v_stages].arrive()
                n += 1

    def made(n):
        return DR[n % made_barriers], n // made_barriers

    def scores_and_dq():
        n = 0
        for k, steps in enumerate(items):
            yield QF.wait(k)

            def scores(i, k=k):
                yield KF[i % k_stages].wait(i // k_stages)

                def go():
                    assert at["Q"] == k and at["K"][i % k_stages] == i
                    at["S"][i & 1] = i
                m.issue(go, SF[i & 1])
            yield from scores(n)
            if steps == 1:
                m.issue(_always, QE)
            for j in range(steps):
                if j + 1 < steps:
                    yield from scores(n + 1)
                    if j + 2 == steps:
                        m.issue(_always, QE)
                barrier, phase = made(n)
                yield barrier.wait(phase)
                if j == 0:
                    yield AE.wait(k + 1)

                def dq(n=n, k=k):
                    assert at["K"][n % k_stages] == n and at["dS"][n & 1] == [n] * 8
                    at["dQ"] = k
                m.issue(dq, KE[n % k_stages])
                if j + 1 == steps:
                    m.issue(_always, AF)
                n += 1

    def dp():
        n = 0
        for k, steps in enumerate(items):
            yield QF.wait(k)
            for j in range(steps):
                yield VF[n % v_stages].wait(n // v_stages)
                if n > 0:
                    yield DL.wait(n - 1)

                def go(n=n, k=k):
                    assert at["Q"] == k and at["V"][n % v_stages] == n
                    at["dP"] = n
                m.issue(go, DF, VE[n % v_stages])
                if j + 1 == steps:
                    m.issue(_always, QE)
                n += 1

    def weights(i):
        n = 0
        for k, steps in enumerate(items):
            for _ in range(steps):
                yield SF[n & 1].wait(n >> 1)
                yield DF.wait(n)
                assert at["S"][n & 1] == n and at["dP"] == n
                yield _always
                assert at["S"][n & 1] == n and at["dP"] == n
                DL.arrive()
                yield _always
                at["dS"][n & 1][i] = n
                yield _always
                made(n)[0].arrive()
                n += 1
            yield AF.wait(k)
            assert at["dQ"] == k
            yield _always
            assert at["dQ"] == k
            AE.arrive()

    m.roles = {"loads": loads(), "S, dQ": scores_and_dq(), "dP": dp(), **{f"weights {i}": weights(i) for i in range(8)}}
    return m.run()


STEPS = [[1], [1] * 5, [3, 1, 2, 5, 1, 1, 4], [9] * 4, [2] * 4]


@pytest.mark.parametrize("items", STEPS, ids=str)
def test_gradients_of_keys_and_values(items):
    stages = _numbers("Bw", "QS", "OS")
    for seed in range(150):
        assert _dkv(items, seed, *stages) is None, seed


@pytest.mark.parametrize("items", STEPS, ids=str)
def test_gradients_of_queries(items):
    stages = _numbers("Bq", "KS", "VS")
    for seed in range(150):
        assert _dq(items, seed, *stages) is None, seed


def test_the_model_finds_one_barrier_of_ds_too_few():
    def fails(seed):
        try:
            return _dq([9] * 4, seed, 3, 2, made_barriers=1) is not None
        except AssertionError:
            return True
    assert any(fails(seed) for seed in range(400))


# ------------------------------------------------------------------- forward
class Item:
    """256 queries from ``first`` on: the key tiles that either half of them wants."""

    def __init__(self, first, T, window, sinks):
        rows = min(256, T - first)
        last = first + rows - 1
        self.far = int(sinks > 0 and last >= window)
        self.kw = (min(sinks, last - window + 1) + 15) & ~15 if self.far else 0
        near0 = max(0, first - window + 1) >> 7
        self.tiles = self.far + (first >> 7) - near0 + 1 + (rows > 128)
        self.halves = []
        for w in (0, 1):
            i0 = first + 128 * w
            far = int(self.far and min(i0 + 127, T - 1) >= window)
            begin = self.far + (max(0, i0 - window + 1) >> 7) - near0
            end = self.far + (i0 >> 7) - near0
            self.halves.append((far, begin, far + end - begin + 1 if rows > 128 * w else 0))


def _forward(T, window, sinks, seed, stages, copies=3):
    items = [Item(f, T, window, sinks) for f in range(0, T, 256)] * copies
    m = Model(seed)
    QF, QE = m.barrier(), m.barrier(2)
    SF, PF, PV, OF, OE = m.ring(4), m.ring(4, 4), m.ring(2), m.ring(2), m.ring(2, 4)
    KF, KE = m.ring(stages), m.ring(stages, 2)
    ring, queries = [None] * stages, [None]
    S, P, O = [None] * 4, [[None] * 4 for _ in range(4)], [None] * 2

    def loads():
        slot, phase = 0, 1
        for k, item in enumerate(items):
            yield QE.wait(k + 1)
            queries[0] = k
            QF.arrive()
            for j in range(2 * item.tiles):  # K and V in turn
                yield KE[slot].wait(phase)
                ring[slot] = (k, j >> 1, j & 1)
                KF[slot].arrive()
                slot += 1
                if slot == stages:
                    slot, phase = 0, phase ^ 1

    def products(w):
        cur = [0, 0]  # the ring's slot and its phase
        after, epilogues = [0, 0], 0

        def step():
            cur[0] += 1
            if cur[0] == stages:
                cur[0], cur[1] = 0, cur[1] ^ 1

        def skip(tiles):  # those of the other half
            for _ in range(2 * tiles):
                yield KF[cur[0]].wait(cur[1])
                KE[cur[0]].arrive()
                step()

        for k, item in enumerate(items):
            far, begin, mine = item.halves[w]
            others, lead = item.far - far, begin - item.far
            keys = [min(item.kw, 64), item.kw - 64] if far else [64, 64]

            def tile(n, far=far, begin=begin):
                return (0 if n == 0 else begin + n - 1) if far else begin + n

            def expect(slot, what, k=k):
                def check():
                    assert ring[slot] == (k, *what) and queries[0] == k
                return check

            def scores(n, u, slot):
                def go(check=expect(slot, (tile(n), 0)), k=k):
                    check()
                    S[2 * w + u] = (k, n)
                m.issue(go, SF[2 * w + u])
            yield QF.wait(k)
            if mine == 0:
                m.issue(_always, QE)
                yield from skip(item.tiles)
                continue
            yield from skip(others + (0 if far else lead))
            yield KF[cur[0]].wait(cur[1])
            scores(0, 0, cur[0])
            if keys[1] > 0:
                scores(0, 1, cur[0])
            m.issue(_always, KE[cur[0]])
            step()
            if mine == 1:
                m.issue(_always, QE)
            for n in range(mine):
                few, more, values = far and n == 0, n + 1 < mine, cur[0]
                yield KF[values].wait(cur[1])
                step()
                for u in (0, 1):
                    if not few or keys[u] > 0:
                        yield PF[2 * w + u].wait(after[u])
                        after[u] += 1
                        if n == 0 and u == 0:
                            epilogues += 1
                            yield OE[w].wait(epilogues)

                        def weigh(n=n, u=u, k=k, there=(values, (k, tile(n), 1))):
                            assert ring[there[0]] == there[1] and P[2 * w + u] == [(k, n)] * 4
                            O[w] = k
                        m.issue(weigh, PV[w])
                    if u == 1:
                        m.issue(_always, KE[values])
                        if not more:
                            m.issue(_always, OF[w])
                    if more:
                        if u == 0:
                            if few:
                                yield from skip(lead)
                            yield KF[cur[0]].wait(cur[1])
                        scores(n + 1, u, cur[0])
                if more:
                    m.issue(_always, KE[cur[0]])
                    step()
                    if n + 2 == mine:
                        m.issue(_always, QE)
            yield from skip(item.tiles - others - lead - mine)

    def softmax(w, i):
        seen, epilogues = [0, 0], 0
        for k, item in enumerate(items):
            far, _, mine = item.halves[w]
            if mine == 0:
                continue
            for h in range(2 * mine):
                u, n = h & 1, h >> 1
                if far and n == 0 and 64 * u >= item.kw:
                    continue
                yield SF[2 * w + u].wait(seen[u])
                assert S[2 * w + u] == (k, n)
                seen[u] += 1
                yield _always
                if h > 0 and m.random.random() < .3:  # the maximum grew: the sums so far are scaled
                    yield PV[w].wait(sum(seen))
                assert S[2 * w + u] == (k, n)
                P[2 * w + u][i] = (k, n)
                PF[2 * w + u].arrive()
            yield OF[w].wait(epilogues)
            assert O[w] == k
            epilogues += 1
            yield _always
            assert O[w] == k
            OE[w].arrive()

    m.roles = {"loads": loads(), "products 0": products(0), "products 1": products(1),
               **{f"softmax {w} {i}": softmax(w, i) for w in (0, 1) for i in range(4)}}
    return m.run()


@pytest.mark.parametrize("stages", re.findall(r"STAGES = D == 128 \? (\d+) : (\d+);", open(SOURCE).read())[0])
@pytest.mark.parametrize("T,window,sinks", [
    (600, 65, 128), (600, 1, 0), (1, 5, 2), (129, 7, 100), (700, 100, 3), (600, 128, 4), (2000, 300, 128), (600, 599, 4),
    (257, 1000, 0), (3000, 1024, 4), (513, 64, 128), (1500, 200, 128), (900, 899, 128), (300, 1, 128)])
def test_forward(T, window, sinks, stages):
    for seed in range(8):
        assert _forward(T, window, sinks, seed, int(stages)) is None, seed
