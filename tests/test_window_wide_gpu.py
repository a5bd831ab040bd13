"""Window attention at the edges of its sizes: unusual groups of heads, many empty
sequences, positions up to the last, offsets past 2^31 elements. Tolerances as in
test_window_gpu.py: fp32 1e-5; bf16 4e-3 for o (p and the result rounded, 2^-9 of each element at
most, 1.7e-3 in the root mean square, together 2.4e-3), 6e-3 for the gradients (two such factors more)."""
import pytest
import torch

import _window_ref as W

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
TOL = {F32: (1e-5, 1e-5), BF: (4e-3, 6e-3)}


def close(name, x, ref, tol):
    x, ref = x.double(), ref.double()
    assert x.shape == ref.shape and torch.isfinite(x).all(), name
    err, size = float((x - ref).norm()), float(ref.norm())
    assert err <= tol * size + 1e-30, (name, err / max(size, 1e-30))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("Hq,Hk,d,lens,window,sinks", [
    (1024, 1, 64, [70], 20, 3), (600, 200, 128, [40], 20, 128), (7, 1, 128, [600], 100, 17), (20, 2, 64, [600], 255, 1),
    (12, 2, 128, [400], 33, 0), (4, 2, 128, [1500], 1, 128),
    (6, 2, 128, [0] * 50 + [1] * 40 + [3, 0, 300, 0, 0, 129] + [0] * 3000 + [64, 65], 50, 5),
], ids=["1024 over 1", "600 over 200", "7 over 1", "20 over 2", "12 over 2", "far only", "empty ones"])
def test_groups_and_batches(kda, dtype, Hq, Hk, d, lens, window, sinks):
    q, k, v, d_o = W.inputs(lens, Hq, Hk, d, dtype)
    cu = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    o, lse = kda.window_varlen_attention(q, k, v, cu, window=window, sinks=sinks)
    g = kda.window_varlen_attention_backward(q, k, v, o, lse, d_o, cu, window=window, sinks=sinks)
    ref, grads = [], {"dq": [], "dk": [], "dv": []}
    for a, b, c, e in zip(*(x.split(lens) for x in (q, k, v, d_o))):
        if len(a):
            ref.append(W.attention(a.double(), b.double(), c.double(), window, sinks, d ** -0.5)[0])
            for n, x in W.gradients(a, b, c, e, window, sinks, d ** -0.5).items():
                grads[n].append(x)
    close("o", o, torch.cat(ref), TOL[dtype][0])
    for n in grads:
        close(n, g[n], torch.cat(grads[n]), TOL[dtype][1])


@pytest.mark.parametrize("dtype", [F32, BF])
def test_decode_of_a_wide_group_at_the_last_position(kda, dtype):
    N, Hq, d, entries = 3, 1024, 128, 70
    gen = torch.Generator().manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=gen).to(dtype).cuda()  # noqa: E731
    kc, vc, q, k, v = rand(N, entries, 1, d), rand(N, entries, 1, d), rand(N, Hq, d), rand(N, 1, d), rand(N, 1, d)
    slots = torch.arange(N, dtype=torch.int32, device="cuda")
    pos = torch.tensor([2 ** 31 - 1, 0, 69], dtype=torch.int32, device="cuda")
    o = kda.window_decode_step(q, k, v, kc, vc, slots, pos, sinks=4)
    at = W.entry(2 ** 31 - 1, entries - 4, 4)
    assert torch.equal(kc[0, at], k[0]) and torch.equal(kc[1, 0], k[1]) and torch.equal(kc[2, 69], k[2])
    for n, count in enumerate((entries, 1, 70)):
        p = torch.softmax(torch.einsum("hd,jd->hj", q[n].double(), kc[n, :count, 0].double()) * d ** -0.5, -1)
        close("o", o[n], p @ vc[n, :count, 0].double(), TOL[dtype][0])


def test_offsets_past_two_to_the_31(kda):
    """The end of 66,000 tokens of 256 heads, against its last tokens alone: rows a window behind the cut's
    start see the same keys, keys a window in front of its end the same queries."""
    T, Hq, Hk, d, window, cut = 66000, 256, 2, 128, 64, 400
    gen = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda H: torch.randn(1, T, H, d, generator=gen, device="cuda", dtype=BF)  # noqa: E731
    q, d_o, k, v = rand(Hq), rand(Hq), rand(Hk), rand(Hk)
    o, lse = kda.window_attention(q, k, v, window=window)
    g = kda.window_attention_backward(q, k, v, o, lse, d_o, window=window)
    tail = [x[0, -cut:] for x in (q, k, v, d_o)]
    heads = slice(Hq - 2, Hq)
    ref, _ = W.attention(tail[0][:, heads].double(), *(x[:, -1:].double() for x in tail[1:3]), window, 0, d ** -0.5)
    close("o", o[0, -cut + window:, heads], ref[window:], TOL[BF][0])
    grads = W.gradients(*tail, window, 0, d ** -0.5)
    close("dq", g["dq"][0, -cut + window:], grads["dq"][window:], TOL[BF][1])
    for n in ("dk", "dv"):
        close(n, g[n][0, -cut + window:], grads[n][window:], TOL[BF][1])


def test_a_pool_past_two_to_the_31(kda):
    """The last slot of a pool of 2.2e9 elements: the bits that a pool of one slot gives."""
    pool, entries, Hk, d = 2100, 2052, 4, 128
    q, k, v, _ = W.inputs([300], 8, Hk, d, BF)
    cu, pos = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 299], [299]))
    outs = []
    for slots in (pool, 1):
        kc, vc = (torch.zeros(slots, entries, Hk, d, dtype=BF, device="cuda") for _ in range(2))
        at = torch.tensor([slots - 1], dtype=torch.int32, device="cuda")
        kda.window_cache_write(k[:299], v[:299], cu, kc, vc, at, sinks=4)
        o = kda.window_decode_step(q[299:], k[299:], v[299:], kc, vc, at, pos, sinks=4)
        assert slots == 1 or not kc[:-1].any()
        outs.append((o, kc[-1].clone(), vc[-1].clone()))
    assert torch.equal(outs[0][1][:300], k)
    assert all(torch.equal(a, b) for a, b in zip(*outs))
