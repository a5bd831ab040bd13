"""Linear attention with a decay against the 64-bit recurrence, at the sizes,
decays and layouts where it can go wrong."""
import math

import pytest
import torch

import _linear_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _decay(kind, lead, H, gen, strength=0.1):
    if kind == "none":
        return None
    if kind == "head":
        return -torch.rand(H, generator=gen) * strength
    return -torch.nn.functional.softplus(torch.randn(*lead, H, generator=gen)) * strength


def _inputs(lead, H, dk, dv, dtype, kind="token", n_states=None, seed=0, strength=0.1):
    gen = torch.Generator().manual_seed(seed)
    q = torch.randn(*lead, H, dk, generator=gen).to(dtype)
    k = torch.nn.functional.normalize(torch.randn(*lead, H, dk, generator=gen), dim=-1).to(dtype)
    v = torch.randn(*lead, H, dv, generator=gen).to(dtype)
    g = _decay(kind, lead, H, gen, strength)
    n = lead[0] if n_states is None else n_states
    s0 = torch.randn(n, H, dk, dv, generator=gen) * 0.1
    return q, k, v, g, s0


def _cu(x):
    return None if x is None else x.cuda()


def _check_forward(kda, q, k, v, g, s0, kind, scale=0.3):
    o, S = kda.linear_prefill(*map(_cu, (q, k, v, g, s0)), decay=kind, scale=scale)
    ro, rS = R.forward(q, k, v, g, s0, scale)
    assert o.dtype == v.dtype and S.dtype == F32
    R.close("o", o, ro, R.TOL[v.dtype])
    R.close("S", S, rS, R.TOL[F32])


@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 512, 513, 700])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_lengths(kda, T, dtype):
    _check_forward(kda, *_inputs((2, T), 3, 128, 128, dtype, seed=T), "token")


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", ["token", "head", "none"])
def test_sizes_types_and_decays(kda, dk, dv, dtype, kind):
    q, k, v, g, s0 = _inputs((1, 333), 2, dk, dv, dtype, kind, seed=1)
    _check_forward(kda, q, k, v, g, s0, kind)
    _check_forward(kda, q, k, v, g, None, kind)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strong_decays_and_resets(kda, dtype):
    """-inf and strong log decays in the middle, at a block's ends and in a row, next to tokens that keep everything."""
    q, k, v, g, s0 = _inputs((1, 600), 2, 128, 128, dtype, seed=2, strength=0.02)
    for t in (0, 63, 64, 200, 201, 255, 256, 511, 512, 513):
        g[0, t] = -math.inf
    g[0, 300:310] = -60.0
    g[0, 400:420, 0] = 0.0
    g[0, 430, 1] = -1e30
    _check_forward(kda, q, k, v, g, s0, "token")


def test_a_reset_at_the_first_token_drops_even_a_nan_state(kda):
    q, k, v, g, _ = _inputs((1, 70), 2, 128, 128, BF, seed=3)
    g[:, 0] = -math.inf
    s0 = torch.full((1, 2, 128, 128), math.nan)
    o, S = kda.linear_prefill(*map(_cu, (q, k, v, g, s0)))
    ro, rS = R.forward(q, k, v, g, None, 1.0)
    R.close("o", o, ro, R.TOL[BF])
    R.close("S", S, rS, R.TOL[F32])


def test_decay_that_forgets_everything_and_nothing(kda):
    for strength in (0.0, 30.0):
        _check_forward(kda, *_inputs((1, 300), 2, 128, 128, BF, seed=4, strength=strength), "token")


def test_no_tokens_copies_the_state(kda):
    q, k, v, g, s0 = _inputs((2, 0), 2, 128, 128, BF, n_states=2)
    o, S = kda.linear_prefill(*map(_cu, (q, k, v, g, s0)))
    assert o.shape == (2, 0, 2, 128) and torch.equal(S.cpu(), s0)
    _, S = kda.linear_prefill(*map(_cu, (q, k, v, g)))
    assert not S.any()
    o, S = kda.linear_prefill(*(x[:0].cuda() for x in (q, k, v, g)), s0[:0].cuda())
    assert S.shape == (0, 2, 128, 128)


@pytest.mark.parametrize("dtype,dk,dv", [(BF, 128, 128), (F32, 64, 128), (BF, 64, 64)])
def test_packed(kda, dtype, dk, dv):
    """Ragged lengths with empty sequences, one-token ones and block edges; every sequence equals its own call, and what
    its neighbours hold (NaN here) does not reach it."""
    lens = [1, 0, 64, 129, 300, 0, 63, 513, 2, 257, 0]
    N, Tt = len(lens), sum(lens)
    q, k, v, g, s0 = _inputs((Tt,), 2, dk, dv, dtype, n_states=N, seed=5)
    cu = torch.tensor([0] + lens).cumsum(0).int().cuda()
    st = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    o, S = kda.linear_varlen_prefill(*map(_cu, (q, k, v, g)), cu, s0.cuda(), scale=0.3, device_status=st)
    ro, rS = R.forward(q, k, v, g, s0, 0.3, lens)
    assert st.item() == kda.KDA_DEV_OK
    R.close("o", o, ro, R.TOL[dtype])
    R.close("S", S, rS, R.TOL[F32])
    at = [0] + torch.tensor(lens).cumsum(0).tolist()
    for n in (0, 3, 4, 7, 9):
        a, b = at[n], at[n + 1]
        o1, S1 = kda.linear_prefill(*(x[None, a:b].cuda() for x in (q, k, v, g)), s0[n:n + 1].cuda(), scale=0.3)
        assert torch.equal(o[a:b], o1[0]) and torch.equal(S[n], S1[0])
    a, b = at[4], at[5]
    bad = [x.clone() for x in (q, k, v, g)]
    for x in bad:
        x[:a] = math.nan
        x[b:] = math.nan
    o2, S2 = kda.linear_varlen_prefill(*map(_cu, bad), cu, s0.cuda(), scale=0.3)
    assert torch.equal(o2[a:b], o[a:b]) and torch.equal(S2[4], S[4])


def test_packed_bad_offsets_write_nothing(kda):
    q, k, v, g, s0 = _inputs((100,), 2, 128, 128, BF, n_states=2, seed=6)
    for cu in ([0, 60, 99], [0, 101, 100], [1, 50, 100], [0, -4, 100]):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full((100, 2, 128), 5.0, dtype=BF, device="cuda")
        fin = torch.full((2, 2, 128, 128), 5.0, device="cuda")
        kda.linear_varlen_prefill(*map(_cu, (q, k, v, g)), torch.tensor(cu).int().cuda(), s0.cuda(), out=out,
                                  final_state=fin, device_status=st)
        assert st.item() == kda.KDA_DEV_BAD_CU_SEQLENS
        assert (out == 5).all() and (fin == 5).all()
        d = kda.linear_varlen_prefill_backward(*map(_cu, (q, k, v, g)), v.cuda(), torch.tensor(cu).int().cuda(),
                                               s0.cuda(), device_status=st)
        assert st.item() == kda.KDA_DEV_BAD_CU_SEQLENS and set(d) >= {"dq", "dk", "dv"}


@pytest.mark.parametrize("dtype", [BF, F32])
def test_slices_of_a_fused_projection(kda, dtype):
    H, d, B, T = 3, 128, 2, 150
    gen = torch.Generator().manual_seed(8)
    p = torch.randn(B, T, 3 * H, d, generator=gen).to(dtype).cuda()
    q, k, v = p[:, :, :H], p[:, :, H:2 * H], p[:, :, 2 * H:]
    g = _decay("token", (B, T), H, gen).cuda()
    a = kda.linear_prefill(q, k, v, g, scale=0.1)
    b = kda.linear_prefill(q.contiguous(), k.contiguous(), v.contiguous(), g, scale=0.1)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    do = torch.randn(B, T, H, d, generator=gen).to(dtype).cuda()
    x = kda.linear_prefill_backward(q, k, v, g, do, scale=0.1)
    y = kda.linear_prefill_backward(q.contiguous(), k.contiguous(), v.contiguous(), g, do, scale=0.1)
    assert all(torch.equal(x[n], y[n]) for n in x)
    q1, k1, v1 = (t[:, 7] for t in (q, k, v))
    s1, s2 = a[1].clone(), a[1].clone()
    o1 = kda.linear_decode_step(q1, k1, v1, g[:, 7].contiguous(), s1)
    o2 = kda.linear_decode_step(q1.contiguous(), k1.contiguous(), v1.contiguous(), g[:, 7].contiguous(), s2)
    assert torch.equal(o1, o2) and torch.equal(s1, s2)


@pytest.mark.parametrize("dtype,dk,dv,T", [(BF, 128, 128, 4096), (F32, 64, 64, 1000)])
def test_same_bits_twice_in_place_and_on_a_side_stream(kda, dtype, dk, dv, T):
    q, k, v, g, s0 = map(_cu, _inputs((2, T), 4, dk, dv, dtype, seed=9))
    o, S = kda.linear_prefill(q, k, v, g, s0)
    s = s0.clone()
    o2, S2 = kda.linear_prefill(q, k, v, g, s, final_state=s)
    assert torch.equal(o, o2) and torch.equal(S, S2) and S2 is s
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o3, S3 = kda.linear_prefill(q, k, v, g, s0, stream=side)
    do = torch.randn(v.shape, device="cuda").to(dtype)
    side.wait_stream(torch.cuda.current_stream())
    a = kda.linear_prefill_backward(q, k, v, g, do, s0, s0, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    b = kda.linear_prefill_backward(q, k, v, g, do, s0, s0)
    assert torch.equal(o, o3) and torch.equal(S, S3)
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_graph_capture(kda):
    q, k, v, g, s0 = map(_cu, _inputs((1, 500), 4, 128, 128, BF, seed=10))
    o, S = kda.linear_prefill(q, k, v, g, s0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o2, S2 = kda.linear_prefill(q, k, v, g, s0)
    o2.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(S, S2)


def test_offsets_past_32_bits(kda):
    """More than 2^31 elements in q: the last tokens, whose decay forgets all but the last few before them."""
    T, H, d = 540_000, 32, 128
    torch.manual_seed(0)
    q, k, v = (torch.randn(1, T, H, d, dtype=BF, device="cuda") for _ in range(3))
    assert q.numel() > 2 ** 31
    g = torch.full((H,), -2.0, device="cuda")
    o, S = kda.linear_prefill(q, k, v, g, decay="head", scale=0.1)
    n = 80
    ro, rS = R.forward(*(x[:, -n:] for x in (q, k, v)), g, None, 0.1)
    R.close("o", o[:, -40:], ro[:, -40:], R.TOL[BF])
    R.close("S", S, rS, R.TOL[F32])


@pytest.mark.parametrize("heads", [(1, 3), (300, 4)])  # the sliced and the whole-row kernel
@pytest.mark.parametrize("dtype,dk,dv", [(BF, 128, 128), (F32, 64, 64), (BF, 128, 64), (F32, 64, 128)])
@pytest.mark.parametrize("kind", ["token", "head", "none"])
def test_decode(kda, heads, dtype, dk, dv, kind):
    N, H = heads
    q, k, v, g, s0 = _inputs((N,), H, dk, dv, dtype, kind, seed=11)
    if kind == "token":
        g[0, 0] = -math.inf
        s0[0, 0] = math.nan  # gone with the reset
    ref = s0.clone()
    if kind == "token":
        ref[0, 0] = 0
    st = s0.cuda()
    o = kda.linear_decode_step(q.cuda(), k.cuda(), v.cuda(), _cu(g), st, decay=kind, scale=0.2)
    g1 = g if g is None or g.dim() == 1 else g[:, None]
    ro, rS = R.forward(q[:, None], k[:, None], v[:, None], g1, ref, 0.2)
    R.close("o", o, ro[:, 0], R.TOL[dtype])
    R.close("S", st, rS, 1e-6)  # one multiply and one add per element


def test_decode_slots(kda):
    N, H, P = 5, 2, 9
    q, k, v, g, pool = _inputs((N,), H, 128, 128, BF, n_states=P, seed=12)
    slots = torch.tensor([3, -1 - 8, 0, 9, -1 - 400])  # a fresh one, two bad ones
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    p = pool.cuda()
    out = torch.full((N, H, 128), 5.0, dtype=BF, device="cuda")
    o = kda.linear_decode_step_slots(*map(_cu, (q, k, v, g)), p, slots.int().cuda(), out=out, device_status=st)
    assert st.item() == kda.KDA_DEV_BAD_SLOT
    s0 = torch.stack([pool[3], torch.zeros_like(pool[8]), pool[0]])
    ro, rS = R.forward(q[:3, None], k[:3, None], v[:3, None], g[:3, None], s0, 1.0)
    R.close("o", o[:3], ro[:, 0], R.TOL[BF])
    R.close("S", p[[3, 8, 0]], rS, 1e-6)
    assert (o[3:] == 5).all()
    rest = [i for i in range(P) if i not in (3, 8, 0)]
    assert torch.equal(p[rest].cpu(), pool[rest])


def test_decode_goes_on_from_prefill(kda):
    """A prompt, then tokens one by one, as one call over all of them."""
    q, k, v, g, _ = map(_cu, _inputs((2, 130), 3, 128, 128, BF, seed=13))
    o, S = kda.linear_prefill(q, k, v, g)
    o1, s = kda.linear_prefill(*(x[:, :120].contiguous() for x in (q, k, v, g)))
    for t in range(120, 130):
        ot = kda.linear_decode_step(q[:, t], k[:, t], v[:, t], g[:, t].contiguous(), s)
        R.close("o", ot, o[:, t], 2 * R.TOL[BF])
    R.close("S", s, S, 2 * R.TOL[F32])


# ---------------------------------------------------------------- gradients
def _check_backward(kda, q, k, v, g, s0, dsT, kind, lens=None, scale=0.3, seed=0):
    d_o = torch.randn(v.shape, generator=torch.Generator().manual_seed(seed)).to(v.dtype)
    kw = dict(decay=kind, scale=scale)
    if lens is None:
        got = kda.linear_prefill_backward(*map(_cu, (q, k, v, g, d_o, s0, dsT)), **kw)
    else:
        cu = torch.tensor([0] + lens).cumsum(0).int().cuda()
        got = kda.linear_varlen_prefill_backward(*map(_cu, (q, k, v, g, d_o)), cu, _cu(s0), _cu(dsT), **kw)
    ref = R.gradients(q, k, v, g, s0, scale, d_o, dsT, lens)
    for n in ("dq", "dk", "dv"):
        assert got[n].dtype == v.dtype
        R.close(n, got[n], ref[n], R.TOL[v.dtype])
    if s0 is not None:
        R.close("d_initial_state", got["d_initial_state"], ref["d_initial_state"], R.TOL[F32])
    if kind != "none":
        R.close("dlog_decay", got["dlog_decay"], ref["dlog_decay"], R.TOL_DECAY)
    else:
        assert got["dlog_decay"] is None
    return got, ref, d_o


@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 128, 255, 256, 257, 513])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_backward_lengths(kda, T, dtype):
    q, k, v, g, s0 = _inputs((1, T), 2, 128, 128, dtype, seed=20 + T)
    _check_backward(kda, q, k, v, g, s0, s0.flip(-1), "token")


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", ["token", "head", "none"])
def test_backward_sizes_types_and_decays(kda, dk, dv, dtype, kind):
    q, k, v, g, s0 = _inputs((2, 300), 2, dk, dv, dtype, kind, seed=21)
    _check_backward(kda, q, k, v, g, s0, None, kind)
    _check_backward(kda, q, k, v, g, None, s0, kind)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_backward_resets(kda, dtype):
    q, k, v, g, s0 = _inputs((1, 400), 2, 128, 128, dtype, seed=22, strength=0.02)
    resets = (0, 63, 64, 200, 201, 255, 256)
    for t in resets:
        g[0, t] = -math.inf
    got, _, _ = _check_backward(kda, q, k, v, g, s0, s0, "token")
    assert not got["dlog_decay"][0, list(resets)].any()


@pytest.mark.parametrize("dtype,dk,dv", [(BF, 128, 128), (F32, 128, 64)])
def test_backward_packed(kda, dtype, dk, dv):
    lens = [1, 0, 64, 129, 300, 257]
    q, k, v, g, s0 = _inputs((sum(lens),), 2, dk, dv, dtype, n_states=len(lens), seed=23)
    got, _, d_o = _check_backward(kda, q, k, v, g, s0, s0.flip(0), "token", lens)
    a, b = sum(lens[:4]), sum(lens[:5])
    one = kda.linear_prefill_backward(*(x[None, a:b].cuda() for x in (q, k, v, g, d_o)), s0[4:5].cuda(),
                                      s0.flip(0)[4:5].cuda(), scale=0.3)
    for n in ("dq", "dk", "dv", "dlog_decay"):
        assert torch.equal(got[n][a:b], one[n][0]), n
    assert torch.equal(got["d_initial_state"][4], one["d_initial_state"][0])


def test_backward_without_the_optional_gradients(kda):
    q, k, v, g, s0 = map(_cu, _inputs((1, 200), 2, 128, 128, F32, seed=24))
    full = kda.linear_prefill_backward(q, k, v, g, v, s0)
    some = kda.linear_prefill_backward(q, k, v, g, v, s0, want_decay_grad=False, want_initial_state_grad=False)
    assert some["dlog_decay"] is None and some["d_initial_state"] is None
    for n in ("dq", "dk", "dv"):
        R.close(n, some[n], full[n], R.TOL[F32])


def test_backward_no_tokens(kda):
    q, k, v, g, s0 = _inputs((2, 0), 2, 128, 128, BF, n_states=2)
    d = kda.linear_prefill_backward(*map(_cu, (q, k, v, g, v, None, s0)))
    assert torch.equal(d["d_initial_state"].cpu(), s0) and d["dq"].shape == (2, 0, 2, 128)
    d = kda.linear_prefill_backward(*map(_cu, (q, k, v, torch.zeros(2), v, None, s0)), decay="head")
    assert not d["dlog_decay"].any()


@pytest.mark.parametrize("kind", ["token", "head"])
def test_backward_against_differences(kda, kind):
    """Along a random direction of each input, the fp32 gradients against central differences of the 64-bit forward
    (step 1e-5: truncation and rounding below 1e-8), bound 1e-4 of the product of the norms' root mean square."""
    q, k, v, g, s0 = _inputs((1, 100), 2, 64, 64, F32, kind, seed=25)
    gen = torch.Generator().manual_seed(1)
    d_o, dsT = torch.randn(v.shape, generator=gen), torch.randn(s0.shape, generator=gen)
    got = kda.linear_prefill_backward(*map(_cu, (q, k, v, g, d_o, s0, dsT)), decay=kind, scale=0.5)
    x = {n: t.double() for n, t in zip(("dq", "dk", "dv", "dlog_decay", "d_initial_state"), (q, k, v, g, s0))}

    def loss(y):
        o, S = R.run64(y["dq"], y["dk"], y["dv"], y["dlog_decay"], y["d_initial_state"], 0.5)
        return float((o * d_o).sum() + (S * dsT).sum())

    for n in x:
        u = torch.randn(x[n].shape, generator=gen, dtype=torch.float64)
        h = 1e-5
        diff = (loss({**x, n: x[n] + h * u}) - loss({**x, n: x[n] - h * u})) / (2 * h)
        mine = float((got[n].cpu().double() * u).sum())
        size = float(got[n].cpu().double().norm() * u.norm()) / math.sqrt(u.numel())
        assert abs(mine - diff) <= 1e-4 * size, (n, mine, diff, size)
