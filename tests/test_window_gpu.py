"""Window attention with sinks, its gradients and its cache against 64 bits.

Tolerances (relative 2-norm unless said otherwise).
fp32: an operand in two tf32 parts keeps 22 bits, so a score is off by about
2^-22 |q| |k| scale sqrt(1 / d) ... 1e-6 at the sizes here, a weight by as much
relative to itself, sums of them in fp32 by 2^-24 a step: bound 1e-5; lse, whose
error is the scores', 1e-5 absolute.
bf16: roundings to 8 bits are off by 2^-9 at most and 1.66e-3 in the root mean
square. o: the result's and the weights' as operands, independent: 2.35e-3 in
all, bound 3.2e-3. Gradients: the result's, the weights', and the stored o's,
which enters ds = p (dp - D) through D, where dp and D are each larger than
their difference: three of them and a factor of 1.7, bound 5e-3."""
import math

import pytest
import torch

import _window_ref as W

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
TOL_O = {F32: 1e-5, BF: 3.2e-3}
TOL_G = {F32: 1e-5, BF: 5e-3}


def close(name, x, ref, tol):
    x, ref = x.double(), ref.double()
    assert x.shape == ref.shape, name
    assert torch.isfinite(x).all(), name
    err, size = float((x - ref).norm()), float(ref.norm())
    assert err <= tol * size, (name, err / max(size, 1e-30))


def check(kda, lens, Hq, Hk, d, dtype, window, sinks, seed=0, fused=False, packed=None, grads=True, scale=None):
    q, k, v, d_o = W.inputs(lens, Hq, Hk, d, dtype, seed, fused)
    kw = dict(window=window, sinks=sinks, scale=scale)
    packed = len(set(lens)) > 1 if packed is None else packed
    cu = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32, device="cuda")

    def cut(x):
        return x.unflatten(0, (len(lens), lens[0]))
    if packed:
        o, lse = kda.window_varlen_attention(q, k, v, cu, **kw)
        g = kda.window_varlen_attention_backward(q, k, v, o, lse, d_o, cu, **kw) if grads else {}
    else:
        o, lse = kda.window_attention(cut(q), cut(k), cut(v), **kw)
        g = kda.window_attention_backward(cut(q), cut(k), cut(v), o, lse, cut(d_o), **kw) if grads else {}
        o, lse, g = o.flatten(0, 1), lse.flatten(0, 1), {n: x.flatten(0, 1) for n, x in g.items()}
    assert o.dtype == dtype and o.is_contiguous() and lse.dtype == F32
    ref = {n: [] for n in ("o", "lse", "dq", "dk", "dv")}
    at = 0
    for m in (m for m in lens if m):
        a = [x[at:at + m] for x in (q, k, v, d_o)]
        ro, rl = W.attention(*(x.double() for x in a[:3]), window, sinks, scale or d ** -0.5)
        ref["o"].append(ro), ref["lse"].append(rl)
        if grads:
            for n, x in W.gradients(*a, window, sinks, scale or d ** -0.5).items():
                ref[n].append(x)
        at += m
    ref = {n: torch.cat(x) for n, x in ref.items() if x}
    close("o", o, ref["o"], TOL_O[dtype])
    assert (lse.double() - ref["lse"]).abs().max() <= 1e-5 * (1 + ref["lse"].abs().max())
    for n, x in g.items():
        assert x.dtype == dtype and x.is_contiguous()
        if ref[n].norm() < 1e-12:  # every token sees itself alone
            assert not x.any(), n
        else:
            close(n, x, ref[n], TOL_G[dtype])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [1, 2, 31, 64, 65, 127, 128, 129, 255, 256, 257, 300, 513, 700])
def test_lengths(kda, dtype, d, T):
    check(kda, [T], 2, 1, d, dtype, window=100, sinks=3, seed=T)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 5), (2, 0), (16, 1), (63, 0), (64, 4), (65, 128), (127, 17), (128, 0),
                                          (128, 4), (129, 100), (256, 128), (257, 33), (599, 4), (600, 0), (601, 4),
                                          (1 << 40, 4), (300, 128)])
def test_windows_and_sinks(kda, dtype, window, sinks):
    check(kda, [600], 2, 2, 128 if window % 2 else 64, dtype, window, sinks, seed=sinks)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (3, 3), (4, 1), (5, 1), (6, 2), (16, 2), (15, 3)])
@pytest.mark.parametrize("d", [64, 128])
def test_heads(kda, dtype, Hq, Hk, d):
    check(kda, [200, 200], Hq, Hk, d, dtype, window=70, sinks=4, seed=Hq)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[5], [1, 1, 1], [0, 300, 0, 1, 129, 0], [256, 512], [257, 3, 640, 64, 0], [40] * 30])
def test_packed(kda, dtype, d, lens):
    check(kda, lens, 4, 2, d, dtype, window=90, sinks=5, seed=len(lens), packed=True)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_slices_of_a_projection(kda, dtype):
    check(kda, [150, 150], 4, 2, 128, dtype, 60, 4, fused=True)
    check(kda, [70, 230, 1], 4, 2, 64, dtype, 60, 4, fused=True)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_scales_and_large_scores(kda, dtype):
    check(kda, [300], 2, 1, 128, dtype, 100, 4, scale=0.01)
    check(kda, [300], 2, 1, 64, dtype, 100, 4, scale=0.5)
    # scores of hundreds: one key takes all, the weights of the others underflow
    q, k, v, _ = W.inputs([300], 2, 1, 128, dtype, 3, sharp=40.0)
    o, lse = kda.window_attention(q[None], k[None], v[None], window=100, sinks=4, scale=1.0)
    ro, rl = W.attention(q.double(), k.double(), v.double(), 100, 4, 1.0)
    # a score of 4000 in fp32 is off by 2^-22 |q| |k| = 1e-3, and its weight by as much relative to itself
    close("o", o[0], ro, 5e-3)
    assert (lse[0].double() - rl).abs().max() <= 2e-6 * rl.abs().max()


def test_rising_scores(kda):
    """Keys whose scores rise with their position, so that every tile brings a new maximum, and falling ones."""
    T, d = 700, 128
    for dtype in (F32, BF):
        for sign in (1, -1):
            k = torch.zeros(T, 1, d, device="cuda")
            k[:, 0, 0] = sign * torch.arange(T, device="cuda") * 0.25
            q = torch.zeros(T, 1, d, device="cuda")
            q[:, 0, 0] = 1.0
            v = torch.randn(T, 1, d, device="cuda")
            q, k, v = (x.to(dtype) for x in (q, k, v))
            o, lse = kda.window_attention(q[None], k[None], v[None], window=300, sinks=2, scale=1.0)
            ro, rl = W.attention(q.double(), k.double(), v.double(), 300, 2, 1.0)
            close("o", o[0], ro, TOL_O[dtype])
            assert (lse[0].double() - rl).abs().max() <= 2e-5 * (1 + rl.abs().max())


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [64, 128])
def test_the_same_bits_alone_and_packed_and_again(kda, dtype, d):
    lens = [130, 0, 513, 64, 300]
    q, k, v, d_o = W.inputs(lens, 4, 2, d, dtype)
    cu = torch.tensor([0, 130, 130, 643, 707, 1007], dtype=torch.int32, device="cuda")
    kw = dict(window=100, sinks=4)
    o, lse = kda.window_varlen_attention(q, k, v, cu, **kw)
    g = kda.window_varlen_attention_backward(q, k, v, o, lse, d_o, cu, **kw)
    o2, lse2 = kda.window_varlen_attention(q, k, v, cu, **kw)
    g2 = kda.window_varlen_attention_backward(q, k, v, o, lse, d_o, cu, **kw)
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and all(torch.equal(g[n], g2[n]) for n in g)
    at = 0
    for m in lens:
        a = [x[None, at:at + m].contiguous() for x in (q, k, v)]
        oa, la = kda.window_attention(*a, **kw)
        assert torch.equal(oa[0], o[at:at + m]) and torch.equal(la[0], lse[at:at + m])
        ga = kda.window_attention_backward(*a, oa, la, d_o[None, at:at + m].contiguous(), **kw)
        assert all(torch.equal(ga[n][0], g[n][at:at + m]) for n in g)
        at += m


@pytest.mark.parametrize("dtype", [F32, BF])
def test_another_sequences_nan_stays_there(kda, dtype):
    lens = [70, 100, 45]
    q, k, v, d_o = W.inputs(lens, 2, 2, 128, dtype)
    cu = torch.tensor([0, 70, 170, 215], dtype=torch.int32, device="cuda")
    kw = dict(window=50, sinks=4)
    o, lse = kda.window_varlen_attention(q, k, v, cu, **kw)
    g = kda.window_varlen_attention_backward(q, k, v, o, lse, d_o, cu, **kw)
    for t in (q, k, v, d_o):
        t[70:170] = math.nan
    o2, lse2 = kda.window_varlen_attention(q, k, v, cu, **kw)
    keep = torch.tensor([*range(70), *range(170, 215)], device="cuda")
    assert torch.equal(o[keep], o2[keep]) and torch.equal(lse[keep], lse2[keep])
    g2 = kda.window_varlen_attention_backward(q, k, v, o2, lse2, d_o, cu, **kw)
    assert all(torch.equal(g[n][keep], g2[n][keep]) for n in g)
    # nor does one key head's reach another's
    q, k, v, d_o = W.inputs([200], 4, 2, 128, dtype)
    a = kda.window_attention(q[None], k[None], v[None], **kw)
    v[:, 1] = math.inf
    b = kda.window_attention(q[None], k[None], v[None], **kw)
    assert torch.equal(a[0][:, :, :2], b[0][:, :, :2])


@pytest.mark.parametrize("dtype", [F32, BF])
def test_bad_offsets_write_nothing(kda, dtype):
    q, k, v, d_o = W.inputs([300], 2, 1, 128, dtype)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for bad in ([0, 200, 100, 300], [0, 100, 200, 299], [1, 100, 200, 300], [0, 400, 200, 300]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        out, lse = torch.full_like(q, 7.0), torch.full((300, 2), 7.0, device="cuda")
        kda.window_varlen_attention(q, k, v, cu, window=50, sinks=2, out=out, lse=lse, device_status=st)
        assert st.item() == kda.KDA_DEV_BAD_CU_SEQLENS and (out == 7).all() and (lse == 7).all()
        st.zero_()
        kda.window_varlen_attention_backward(q, k, v, out, lse, d_o, cu, window=50, sinks=2, device_status=st)
        assert st.item() == kda.KDA_DEV_BAD_CU_SEQLENS
    cu = torch.tensor([0, 100, 100, 300], dtype=torch.int32, device="cuda")
    kda.window_varlen_attention(q, k, v, cu, window=50, sinks=2, device_status=st)
    assert st.item() == kda.KDA_DEV_OK


def test_no_tokens(kda):
    z = torch.zeros(2, 0, 4, 128, device="cuda", dtype=BF)
    o, lse = kda.window_attention(z, z, z, window=5)
    assert o.shape == z.shape and lse.shape == (2, 0, 4)
    g = kda.window_attention_backward(z, z, z, o, lse, z, window=5, sinks=2)
    assert g["dq"].shape == z.shape
    e = torch.zeros(0, 4, 128, device="cuda", dtype=BF)
    st = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    for cu in ([0], [0, 0, 0]):
        kda.window_varlen_attention(e, e, e, torch.tensor(cu, dtype=torch.int32, device="cuda"), window=5, device_status=st)
        assert st.item() == kda.KDA_DEV_OK
    x = torch.zeros(3, 4, 128, device="cuda", dtype=BF)
    kda.window_varlen_attention(x, x, x, torch.tensor([0], dtype=torch.int32, device="cuda"), window=5, device_status=st)
    assert st.item() == kda.KDA_DEV_BAD_CU_SEQLENS


def test_gradients_against_differences(kda):
    q, k, v, d_o = W.inputs([90], 2, 1, 64, F32)
    o, lse = kda.window_attention(q[None], k[None], v[None], window=40, sinks=3)
    g = kda.window_attention_backward(q[None], k[None], v[None], o, lse, d_o[None], window=40, sinks=3)
    gen = torch.Generator().manual_seed(1)
    args = [x.double() for x in (q, k, v)]
    for n, name in enumerate(("dq", "dk", "dv")):
        u = torch.randn(args[n].shape, generator=gen, dtype=torch.float64).cuda()

        def loss(h):
            a = list(args)
            a[n] = a[n] + h * u
            return float((W.attention(*a, 40, 3, 64 ** -0.5)[0] * d_o.double()).sum())
        diff = (loss(1e-5) - loss(-1e-5)) / 2e-5
        mine = float((g[name][0].double() * u).sum())
        size = float(g[name].double().norm() * u.norm()) / math.sqrt(u.numel())
        assert abs(mine - diff) <= 1e-4 * size, (name, mine, diff)


# ---------------------------------------------------------------- the cache
def ref_write(kc, vc, k, v, lens, slots, window, sinks):
    at = 0
    for n, m in enumerate(lens):
        s = slots[n] if slots[n] >= 0 else -1 - slots[n]
        for p in range(m):
            if p < sinks or p >= m - window:
                e = W.entry(p, window, sinks)
                kc[s, e], vc[s, e] = k[at + p], v[at + p]
        at += m


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d,Hk", [(64, 1), (128, 3)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (7, 0), (8, 3), (64, 4), (100, 128)])
def test_cache_write(kda, dtype, d, Hk, window, sinks):
    lens = [0, 1, 3, 5, 8, 9, 20, 64, 200, 333]
    _, k, v, _ = W.inputs(lens, Hk, Hk, d, dtype, fused=True)
    cu = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    slots = [11, 0, -3, 5, -8, 9, 1, 3, 4, 10]
    kc, vc = (torch.full((12, window + sinks, Hk, d), x, dtype=dtype, device="cuda") for x in (3.0, 4.0))
    rk, rv = kc.clone(), vc.clone()
    st = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    kda.window_cache_write(k, v, cu, kc, vc, torch.tensor(slots, dtype=torch.int32, device="cuda"), sinks=sinks,
                           device_status=st)
    ref_write(rk, rv, k, v, lens, slots, window, sinks)
    assert st.item() == kda.KDA_DEV_OK
    assert torch.equal(kc, rk) and torch.equal(vc, rv)


def test_cache_write_bad_slots_and_offsets(kda):
    lens = [4, 6, 5]
    _, k, v, _ = W.inputs(lens, 1, 1, 64, F32)
    kc, vc = (torch.zeros(3, 9, 1, 64, device="cuda") for _ in range(2))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 4, 10, 15], dtype=torch.int32, device="cuda")
    slots = torch.tensor([2, 3, -5], dtype=torch.int32, device="cuda")
    kda.window_cache_write(k, v, cu, kc, vc, slots, sinks=1, device_status=st)
    assert st.item() == kda.KDA_DEV_BAD_SLOT and kc[2].any() and not kc[:2].any()
    kc.zero_()
    slots = torch.tensor([2, 1, 0], dtype=torch.int32, device="cuda")
    for bad in ([0, 4, 3, 15], [0, 4, 10, 14], [2, 4, 10, 15], [0, 99, 10, 15]):
        kda.window_cache_write(k, v, torch.tensor(bad, dtype=torch.int32, device="cuda"), kc, vc, slots, device_status=st)
        assert st.item() == kda.KDA_DEV_BAD_CU_SEQLENS and not kc.any()


def decode_ref(q, k, v, kc, vc, slots, positions, sinks, scale):
    window = kc.shape[1] - sinks
    o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    G = q.shape[1] // k.shape[1]
    for n, (s, p) in enumerate(zip(slots, positions)):
        s = s if s >= 0 else -1 - s
        e = W.entry(p, window, sinks)
        kc[s, e], vc[s, e] = k[n], v[n]
        m = min(p + 1, window + sinks)
        kk, vv = (x[s, :m].double().repeat_interleave(G, 1) for x in (kc, vc))
        a = torch.softmax(torch.einsum("hd,jhd->hj", q[n].double(), kk) * scale, -1)
        o[n] = torch.einsum("hj,jhd->hd", a, vv)
    return o


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d,Hq,Hk", [(128, 1, 1), (128, 8, 2), (64, 6, 2), (64, 5, 1), (128, 16, 1), (64, 17, 1), (128, 40, 1),
                                     (128, 24, 8)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 2), (16, 0), (100, 4), (700, 128)])
def test_decode(kda, dtype, d, Hq, Hk, window, sinks):
    gen = torch.Generator().manual_seed(window)
    positions = [0, 1, 2, 6, 7, 15, 16, 17, 99, 103, 104, 105, 500, 1000, 123456789, (1 << 31) - 1]
    N = len(positions)
    p = torch.randn(N, Hq + 2 * Hk, d, generator=gen).to(dtype).cuda()
    q, k, v = p[:, :Hq], p[:, Hq:Hq + Hk], p[:, Hq + Hk:]
    kc, vc = (torch.randn(N + 2, window + sinks, Hk, d, generator=gen).to(dtype).cuda() for _ in range(2))
    slots = torch.randperm(N + 2, generator=gen)[:N].tolist()
    slots[3] = -1 - slots[3]
    for n, pos in enumerate(positions):  # what holds no token is not read
        s = slots[n] if slots[n] >= 0 else -1 - slots[n]
        kc[s, pos:], vc[s, pos:] = math.nan, math.nan
    rk, rv = kc.clone(), vc.clone()
    ref = decode_ref(q, k, v, rk, rv, slots, positions, sinks, d ** -0.5)
    st = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    o = kda.window_decode_step(q, k, v, kc, vc, torch.tensor(slots, dtype=torch.int32, device="cuda"),
                               torch.tensor(positions, dtype=torch.int32, device="cuda"), sinks=sinks, device_status=st)
    assert st.item() == kda.KDA_DEV_OK
    close("o", o, ref, TOL_O[dtype])
    assert torch.equal(kc.nan_to_num(9.0), rk.nan_to_num(9.0)) and torch.equal(vc.nan_to_num(9.0), rv.nan_to_num(9.0))


@pytest.mark.parametrize("N", [1, 3, 40, 200])
def test_decode_batches(kda, N):
    """Few sequences go to clusters of CTAs, many to one each."""
    gen = torch.Generator().manual_seed(N)
    q, k, v = (torch.randn(N, h, 128, generator=gen).to(BF).cuda() for h in (8, 2, 2))
    kc, vc = (torch.randn(N, 604, 2, 128, generator=gen).to(BF).cuda() for _ in range(2))
    slots, positions = list(range(N)), [(n * 37) % 900 for n in range(N)]
    ref = decode_ref(q, k, v, kc.clone(), vc.clone(), slots, positions, 4, 128 ** -0.5)
    at = dict(slots=torch.arange(N, dtype=torch.int32, device="cuda"),
              positions=torch.tensor(positions, dtype=torch.int32, device="cuda"))
    o = kda.window_decode_step(q, k, v, kc, vc, **at, sinks=4)
    close("o", o, ref, TOL_O[BF])
    assert torch.equal(o, kda.window_decode_step(q, k, v, kc, vc, **at, sinks=4))


def test_decode_leaves_out_bad_sequences(kda):
    q, k, v = (torch.randn(4, 2, 64, device="cuda") for _ in range(3))
    kc, vc = (torch.zeros(3, 8, 2, 64, device="cuda") for _ in range(2))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((4, 2, 64), 5.0, device="cuda")
    slots = torch.tensor([0, 3, 1, 2], dtype=torch.int32, device="cuda")
    pos = torch.tensor([0, 0, -1, 0], dtype=torch.int32, device="cuda")
    kda.window_decode_step(q, k, v, kc, vc, slots, pos, sinks=2, out=out, device_status=st)
    assert st.item() == kda.KDA_DEV_BAD_SLOT | kda.KDA_DEV_BAD_POSITION
    assert (out[1:3] == 5).all() and not kc[1].any() and torch.allclose(out[[0, 3]], v[[0, 3]])


@pytest.mark.parametrize("dtype", [F32, BF])
def test_prompt_then_tokens(kda, dtype):
    """A prompt prefilled, its keys and values put into the cache, then token by token: what one prefill of all of it gives."""
    lens, more, window, sinks, Hq, Hk, d = [3, 50, 130], 40, 32, 4, 4, 2, 128
    full = [m + more for m in lens]
    q, k, v, _ = W.inputs(full, Hq, Hk, d, dtype)
    at = [0, *torch.tensor(full).cumsum(0).tolist()]
    pick = torch.cat([torch.arange(a, a + m) for a, m in zip(at, lens)]).cuda()
    cu = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    cu_full = torch.tensor(at, dtype=torch.int32, device="cuda")
    whole, _ = kda.window_varlen_attention(q, k, v, cu_full, window=window, sinks=sinks)
    part, _ = kda.window_varlen_attention(q[pick], k[pick], v[pick], cu, window=window, sinks=sinks)
    close("prompt", part, whole[pick], TOL_O[dtype])
    kc, vc = (torch.zeros(3, window + sinks, Hk, d, dtype=dtype, device="cuda") for _ in range(2))
    slots = torch.tensor([1, 2, 0], dtype=torch.int32, device="cuda")
    kda.window_cache_write(k[pick], v[pick], cu, kc, vc, slots, sinks=sinks)
    pos = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for i in range(more):
        now = torch.tensor([a + m + i for a, m in zip(at, lens)], device="cuda")
        o = kda.window_decode_step(q[now], k[now], v[now], kc, vc, slots, pos + i, sinks=sinks)
        close("token", o, whole[now], 2 * TOL_O[dtype])


@pytest.mark.parametrize("dtype", [F32, BF])
def test_captured_and_replayed(kda, dtype):
    lens = [100, 300]
    q, k, v, d_o = W.inputs(lens, 4, 2, 128, dtype)
    cu = torch.tensor([0, 100, 400], dtype=torch.int32, device="cuda")
    kc, vc = (torch.zeros(2, 68, 2, 128, dtype=dtype, device="cuda") for _ in range(2))
    slots = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    pos = torch.tensor([100, 300], dtype=torch.int32, device="cuda")

    def all_of_it():
        o, lse = kda.window_varlen_attention(q, k, v, cu, window=64, sinks=4)
        g = kda.window_varlen_attention_backward(q, k, v, o, lse, d_o, cu, window=64, sinks=4)
        kda.window_cache_write(k, v, cu, kc, vc, slots, sinks=4)
        return [o, lse, *g.values(), kda.window_decode_step(q[:2], k[:2], v[:2], kc, vc, slots, pos, sinks=4)]
    first = [x.clone() for x in all_of_it()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        all_of_it()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = all_of_it()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(first, out))
    q.mul_(0.5)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip([x.clone() for x in out], all_of_it()))


def test_on_a_given_stream(kda):
    q, k, v, d_o = W.inputs([200], 4, 2, 128, BF)
    a = kda.window_attention(q[None], k[None], v[None], window=64, sinks=4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = kda.window_attention(q[None], k[None], v[None], window=64, sinks=4, stream=s)
    g = kda.window_attention_backward(q[None], k[None], v[None], *b, d_o[None], window=64, sinks=4, stream=s)
    s.synchronize()
    h = kda.window_attention_backward(q[None], k[None], v[None], *a, d_o[None], window=64, sinks=4)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and all(torch.equal(g[n], h[n]) for n in g)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_into_an_output_at_16_bytes(kda, dtype):
    q, k, v, _ = W.inputs([300], 2, 1, 128, dtype)
    a = kda.window_attention(q[None], k[None], v[None], window=100, sinks=3)
    pad = 16 // q.element_size()
    out = torch.zeros(q.numel() + pad, dtype=dtype, device="cuda")[pad:].view(1, *q.shape)
    lse = torch.zeros(601, device="cuda")[1:].view(1, 300, 2)
    assert out.data_ptr() % 32 == 16
    kda.window_attention(q[None], k[None], v[None], window=100, sinks=3, out=out, lse=lse)
    assert torch.equal(a[0], out) and torch.equal(a[1], lse)
