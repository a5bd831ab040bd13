"""A NaN log decay: NaN from its token to the next reset, as in the recurrence
(0 where the decay is a reset, whatever the state held), in prefill and decode
alike; its neighbours keep their bits. Where the reference is a number, the
tolerances are those of the reference file."""
import math

import pytest
import torch

import _linear_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
T = 1300
# per head: the tokens with a NaN, those with a reset
EVENTS = [([100], []), ([0], [1]), ([63, 64], [65]), ([300], [300 + 7]), ([300], [700]), ([700], [300]),
          ([513, 1299], [600]), ([40, 520], [20, 44, 530]), ([], [128])]


def _inputs(dtype, d):
    gen = torch.Generator().manual_seed(1)
    H = len(EVENTS)
    q, v, d_o = (torch.randn(1, T, H, d, generator=gen).to(dtype) for _ in range(3))
    k = (torch.randn(1, T, H, d, generator=gen) * d ** -0.5).to(dtype)
    g = -torch.rand(1, T, H, generator=gen) * 0.1
    for h, (nans, resets) in enumerate(EVENTS):
        g[0, nans, h] = math.nan
        g[0, resets, h] = -math.inf
    s0, sT = (torch.randn(1, H, d, d, generator=gen) * 0.1 for _ in range(2))
    return q, k, v, g, d_o, s0, sT


def _same(name, x, ref, tol):
    x, ref = x.cpu().double(), ref.double()
    assert torch.equal(x.isnan(), ref.isnan()), name
    R.close(name, x[~ref.isnan()], ref[~ref.isnan()], tol)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 128), (BF, 64), (F32, 64)])
def test_forward(kda, dtype, d):
    q, k, v, g, _, s0, _ = _inputs(dtype, d)
    ro, rS = R.forward(q, k, v, g, s0, 0.3)
    o, S = kda.linear_prefill(*(x.cuda() for x in (q, k, v, g, s0)), scale=0.3)
    _same("o", o, ro, R.TOL[dtype])
    _same("S", S, rS, R.TOL[F32])
    n = 400  # in one segment, without a final state
    o, _ = kda.linear_prefill(*(x[:, :n].cuda() for x in (q, k, v, g)), scale=0.3, output_final_state=False)
    _same("o", o, R.forward(*(x[:, :n] for x in (q, k, v, g)), None, 0.3)[0], R.TOL[dtype])


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_one_decay_per_head(kda, dtype, d):
    q, k, v, g, _, s0, _ = _inputs(dtype, d)
    g = torch.full((len(EVENTS),), -0.01)
    g[2] = math.nan
    o, S = kda.linear_prefill(*(x.cuda() for x in (q, k, v, g, s0)), decay="head")
    assert o[:, :, 2].isnan().all() and S[:, 2].isnan().all()
    keep = [h for h in range(len(EVENTS)) if h != 2]
    assert o[:, :, keep].isfinite().all() and S[:, keep].isfinite().all()


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_prefill_as_decode(kda, dtype, d):
    q, k, v, g, _, s0, _ = (x.cuda() for x in _inputs(dtype, d))
    n = 70
    state, steps = s0.clone(), []
    for t in range(n):
        steps.append(kda.linear_decode_step(q[:, t], k[:, t], v[:, t], g[:, t].contiguous(), state, scale=0.3))
    o, S = kda.linear_prefill(*(x[:, :n].contiguous() for x in (q, k, v, g)), s0, scale=0.3)
    assert torch.equal(o.isnan(), torch.stack(steps, 1).isnan()) and torch.equal(S.isnan(), state.isnan())


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_packed_neighbours_keep_their_bits(kda, dtype, d):
    q, k, v, g, d_o, s0, _ = (x.cuda() for x in _inputs(dtype, d))
    H = len(EVENTS)
    clean = torch.nan_to_num(g, nan=-0.1, neginf=-math.inf)
    cu = torch.tensor([0, 290, 290, 800, T], dtype=torch.int32, device="cuda")
    states = s0.expand(4, H, d, d).contiguous()
    bad = clean.clone()
    bad[0, 400, :] = math.nan
    for grad in (True, False):
        out = []
        for x in (clean, bad):
            o, S = kda.linear_varlen_prefill(q[0], k[0], v[0], x[0], cu, states)
            r = kda.linear_varlen_prefill_backward(q[0], k[0], v[0], x[0], d_o[0], cu, states, want_decay_grad=grad)
            out.append({"o": o, "S": S, **{n: t for n, t in r.items() if t is not None}})
        for name, a in out[0].items():
            b = out[1][name]
            keep = [0, 1, 3] if a.dim() == 4 else list(range(290)) + list(range(800, T))
            assert torch.equal(a[keep], b[keep]), name


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 128), (BF, 64), (F32, 64)])
@pytest.mark.parametrize("decay_grad", [True, False])
def test_backward(kda, dtype, d, decay_grad):
    q, k, v, g, d_o, s0, sT = _inputs(dtype, d)
    ref = R.gradients(q, k, v, g, s0, 0.3, d_o, sT)
    got = kda.linear_prefill_backward(*(x.cuda() for x in (q, k, v, g, d_o, s0, sT)), scale=0.3,
                                      want_decay_grad=decay_grad)
    for n in ("dq", "dk", "dv"):
        _same(n, got[n], ref[n], R.TOL[dtype])
    _same("d_initial_state", got["d_initial_state"], ref["d_initial_state"], R.TOL[F32])
    if not decay_grad:
        return
    dg, resets = got["dlog_decay"].cpu(), g == -math.inf
    assert not dg[resets].any()
    # no number where the reference has none; around a NaN there may be more of them
    assert dg.isnan()[ref["dlog_decay"].isnan() & ~resets].all()
    h = len(EVENTS) - 1
    R.close("dlog_decay", dg[..., h], ref["dlog_decay"][..., h], R.TOL_DECAY)
