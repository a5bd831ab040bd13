"""window_cache_write of thousands of prompts: what lands where, and that its work
grows with the tokens, not with prompts times prompts."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def reference(k, v, lens, slots, kc, vc, sinks):
    entries = kc.shape[1]
    window = entries - sinks
    src, slot, at = [], [], []
    start = 0
    for m, s in zip(lens, slots):
        s = s if s >= 0 else -1 - s
        if s < kc.shape[0]:
            for p in [*range(min(sinks, m)), *range(max(min(sinks, m), m - window), m)]:
                src.append(start + p), slot.append(s), at.append(p if p < sinks else sinks + (p - sinks) % window)
        start += m
    src, slot, at = (torch.tensor(x, dtype=torch.long, device="cuda") for x in (src, slot, at))
    kc[slot, at], vc[slot, at] = k[src], v[src]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N,longest,entries,sinks", [(1, 5000, 64, 4), (3, 3, 2052, 4), (255, 60, 20, 3), (256, 60, 20, 0), (257, 60, 20, 3),
                                                     (5000, 30, 12, 5), (65535, 2, 2, 1), (4000, 700, 40, 39)])
def test_many_prompts(kda, dtype, N, longest, entries, sinks):
    gen = torch.Generator().manual_seed(N)
    lens = (torch.rand(N, generator=gen) ** 3 * (longest + 1)).long().tolist()
    lens[N // 2] = longest
    T = sum(lens)
    k, v = (torch.randn(T, 1, 64, generator=gen).to(dtype).cuda() for _ in range(2))
    kc, vc = (torch.full((N + 2, entries, 1, 64), x, dtype=dtype, device="cuda") for x in (3.0, 4.0))
    slots = torch.randperm(N + 2, generator=gen)[:N]
    slots[::3] = -1 - slots[::3]
    cu = torch.tensor([0, *lens]).cumsum(0).int().cuda()
    rk, rv = kc.clone(), vc.clone()
    st = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    kda.window_cache_write(k, v, cu, kc, vc, slots.int().cuda(), sinks=sinks, device_status=st)
    reference(k, v, lens, slots.tolist(), rk, rv, sinks)
    assert st.item() == kda.KDA_DEV_OK
    assert torch.equal(kc, rk) and torch.equal(vc, rv)


def test_bad_slots_and_offsets_among_many(kda):
    N, entries = 3000, 10
    lens = [(i * 7) % 13 for i in range(N)]
    T = sum(lens)
    k, v = (torch.randn(T, 2, 64, device="cuda") for _ in range(2))
    slots = list(range(N))
    empty = lens.index(0, 1000)
    slots[17], slots[1500], slots[empty] = N, -1 - N, 1 << 30
    kc, vc = (torch.zeros(N, entries, 2, 64, device="cuda") for _ in range(2))
    rk, rv = kc.clone(), vc.clone()
    cu = torch.tensor([0, *lens]).cumsum(0).int().cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kda.window_cache_write(k, v, cu, kc, vc, torch.tensor(slots, dtype=torch.int32, device="cuda"), sinks=2, device_status=st)
    reference(k, v, lens, slots, rk, rv, 2)
    assert st.item() == kda.KDA_DEV_BAD_SLOT and torch.equal(kc, rk) and torch.equal(vc, rv)
    # a bad slot of a prompt without tokens alone is told too
    slots = list(range(N))
    slots[empty] = N
    kda.window_cache_write(k, v, cu, kc, vc, torch.tensor(slots, dtype=torch.int32, device="cuda"), sinks=2, device_status=st)
    assert st.item() == kda.KDA_DEV_BAD_SLOT
    kc.zero_(), vc.zero_()
    good = torch.arange(N, dtype=torch.int32, device="cuda")
    for i, x in ((0, 1), (N, T - 1), (1234, -5), (2000, 1 << 30), (2999, -(1 << 31))):
        bad = cu.clone()
        bad[i] = x
        kda.window_cache_write(k, v, bad, kc, vc, good, sinks=2, device_status=st)
        assert st.item() == kda.KDA_DEV_BAD_CU_SEQLENS and not kc.any() and not vc.any(), i


def test_time_grows_with_the_tokens(kda):
    """4096 prompts of 16 tokens: as many bytes as 32 prompts of 2048, whose time they may take ten times of."""
    entries, sinks = 2052, 4

    def time(N, m):
        k, v = (torch.randn(N * m, 1, 128, device="cuda").to(BF) for _ in range(2))
        kc, vc = (torch.zeros(N, entries, 1, 128, device="cuda", dtype=BF) for _ in range(2))
        cu = torch.arange(0, N * m + 1, m, dtype=torch.int32, device="cuda")
        slots = torch.arange(N, dtype=torch.int32, device="cuda")
        best = float("inf")
        for _ in range(5):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(4):
                kda.window_cache_write(k, v, cu, kc, vc, slots, sinks=sinks)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b) / 4)
        return best
    few, many = time(32, 2048), time(4096, 16)
    assert many <= 10 * max(few, 0.02), (few, many)
