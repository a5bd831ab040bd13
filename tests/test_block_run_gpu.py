"""The operators around a block in a run, as a model calls them: positions of
several axes, window attention, the gated head norm and the residual norm, in
training over packed sequences and in serving token by token.

Tolerance of fp32 (relative 2-norm): every operator is held to 3e-6 or better by
tests of its own, a product with a 256-wide weight in fp32 to about 1e-6. Forward a
block is seven of these and backward as many again, two blocks so about thirty
errors of 3e-6 at most that add up, 1e-4; the gradients of weights are sums of rows
of these. bf16 is compared with itself: what one order of calls gives against
another's, bit for bit."""
import pytest
import torch

import _window_ref as W
from test_block_norm_gpu import close, gated_ref, normed
from test_rope_axes_gpu import rotated, sections

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
HQ, HK, D, MODEL, WINDOW, SINKS, EPS = 4, 2, 64, 256, 20, 3, 1e-6
AXIS = sections(8, 12, 12)
TOL = 1e-4


class Layer:
    """The weights of one block."""

    def __init__(self, dtype, seed):
        gen = torch.Generator().manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
        self.project = (rand(MODEL, (2 * HQ + 2 * HK) * D) / MODEL ** 0.5).to(dtype).cuda()
        self.back = (rand(HQ * D, MODEL) / (HQ * D) ** 0.5).to(dtype).cuda()
        self.wq, self.wk, self.head = (1 + 0.2 * rand(D).cuda() for _ in range(3))
        self.norm, self.post, self.channel = (1 + 0.2 * rand(MODEL).cuda() for _ in range(3))

    KEYS = ("project", "back", "wq", "wk", "head", "norm", "post", "channel")
    BRANCH = dict(branch_norm="rms", scale=0.7, eps=EPS)


def split(x):
    return x[..., :HQ, :], x[..., HQ:HQ + HK, :], x[..., HQ + HK:HQ + 2 * HK, :], x[..., HQ + 2 * HK:, :]


def forward(kda, w, y, x, pos, table, cu):
    """One block: y [T, MODEL] what it reads, x the stream; what the backward pass needs comes with the results."""
    p = (y @ w.project).view(len(y), -1, D)
    q, k, v, gate = split(p)
    qr, kr = kda.qk_norm_rope_axes(q, k, pos, table, AXIS, w.wq, w.wk, eps=EPS)
    o, lse = kda.window_varlen_attention(qr, kr, v, cu, window=WINDOW, sinks=SINKS)
    z = kda.gated_norm(o, gate, w.head, eps=EPS)
    b = z.view(len(y), -1) @ w.back
    h, out = kda.residual_norm(x, b, w.norm, branch_weight=w.post, channel_scale=w.channel, **w.BRANCH)
    return out, h, (y, p, qr, kr, o, lse, z, b, h)


def backward(kda, w, saved, d_out, d_h, pos, table, cu):
    y, p, qr, kr, o, lse, z, b, h = saved
    q, k, v, gate = split(p)
    g = kda.residual_norm_backward(h, b, d_out, d_h, w.norm, branch_weight=w.post, channel_scale=w.channel, **w.BRANCH)
    n = kda.gated_norm_backward(o, gate, (g["d_branch"] @ w.back.t()).view(z.shape), w.head, eps=EPS)
    a = kda.window_varlen_attention_backward(qr, kr, v, o, lse, n["dx"], cu, window=WINDOW, sinks=SINKS)
    r = kda.qk_norm_rope_axes_backward(q, k, a["dq"], a["dk"], pos, table, AXIS, w.wq, w.wk, eps=EPS)
    dp = torch.cat([r["dq"], r["dk"], a["dv"], n["dgate"]], 1).view(len(y), -1)
    grads = dict(project=y.t() @ dp, back=z.view(len(y), -1).t() @ g["d_branch"], wq=r["dq_weight"], wk=r["dk_weight"],
                 head=n["dweight"], norm=g["dweight"], post=g["dbranch_weight"], channel=g["dchannel_scale"])
    return dp @ w.project.t(), g["d_residual"], grads


def plain(w, y, x, pos, table, lens):
    p = (y @ w["project"]).view(len(y), -1, D)
    q, k, v, gate = split(p)
    q, k = (rotated(normed(a, "rms", EPS) * b, pos, table, AXIS, "half") for a, b in ((q, w["wq"]), (k, w["wk"])))
    o = torch.cat([W.attention(a, b, c, WINDOW, SINKS, D ** -0.5)[0]
                   for a, b, c in zip(q.split(lens), k.split(lens), v.split(lens))])
    z = gated_ref(o, gate, w["head"], "rms", "sigmoid", EPS)
    h = x + 0.7 * w["channel"] * w["post"] * normed(z.reshape(len(y), -1) @ w["back"], "rms", EPS)
    return normed(h, "rms", EPS) * w["norm"], h


def run_inputs(lens, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed)
    T = sum(lens)
    y, x, d_out, d_h = (torch.randn(T, MODEL, generator=gen) for _ in range(4))
    pos = torch.randint(0, 64, (3, T), generator=gen).int()
    cu = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32)
    return y.to(dtype).cuda(), x.cuda(), d_out.to(dtype).cuda(), d_h.cuda(), pos.cuda(), cu.cuda()


def train(kda, layers, y, x, d_out, d_h, pos, table, cu):
    saved = []
    for w in layers:
        y, x, s = forward(kda, w, y, x, pos, table, cu)
        saved.append(s)
    grads = []
    dy, dx = d_out, d_h
    for w, s in zip(reversed(layers), reversed(saved)):
        dy, dx, g = backward(kda, w, s, dy, dx, pos, table, cu)
        grads.append(g)
    return [y, x, dy, dx, *(t for g in grads for t in g.values())]


@pytest.mark.parametrize("lens", [[1], [70], [5, 0, 40, 1, 130]], ids=str)
def test_two_blocks_forward_and_back(kda, lens):
    layers = [Layer(F32, 1), Layer(F32, 2)]
    y, x, d_out, d_h, pos, cu = run_inputs(lens, F32)
    table = kda.rope_table(64, 2 * len(AXIS), device="cuda")
    got = train(kda, layers, y, x, d_out, d_h, pos, table, cu)
    y64, x64 = (t.double().cpu().requires_grad_() for t in (y, x))
    w64 = [{n: getattr(w, n).double().cpu().requires_grad_() for n in Layer.KEYS} for w in layers]
    a, b = y64, x64
    for w in w64:
        a, b = plain(w, a, b, pos.cpu(), table.double().cpu(), lens)
    torch.autograd.backward([a, b], [d_out.double().cpu(), d_h.double().cpu()])
    want = [a, b, y64.grad, x64.grad, *(w[n].grad for w in reversed(w64) for n in Layer.KEYS)]
    names = ["out", "stream", "d_in", "d_stream", *(f"{n} {i}" for i in (2, 1) for n in Layer.KEYS)]
    for n, g, r in zip(names, got, want):
        close(n, g, r.detach(), TOL)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_a_captured_step_of_training(kda, dtype):
    layers = [Layer(dtype, 1), Layer(dtype, 2)]
    y, x, d_out, d_h, pos, cu = run_inputs([90, 7, 200], dtype)
    table = kda.rope_table(64, 2 * len(AXIS), device="cuda")
    step = lambda: train(kda, layers, y, x, d_out, d_h, pos, table, cu)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for scale in (1.0, 0.5):
        y.mul_(scale)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip([t.clone() for t in out], step()))


def token(kda, w, y, x, pos, table, cache, slots, at):
    q, k, v, gate = split((y @ w.project).view(len(y), -1, D))
    q, k = kda.qk_norm_rope_axes(q, k, pos, table, AXIS, w.wq, w.wk, eps=EPS)
    o = kda.window_decode_step(q, k, v, *cache, slots, at, sinks=SINKS)
    b = kda.gated_norm(o, gate, w.head, eps=EPS).view(len(y), -1) @ w.back
    h, out = kda.residual_norm(x, b, w.norm, branch_weight=w.post, channel_scale=w.channel, **w.BRANCH)
    return out, h


def test_a_prompt_and_captured_tokens(kda):
    """Prompts through both blocks, then tokens one by one by a replayed graph: what all of it at once gives."""
    layers, more = [Layer(F32, 1), Layer(F32, 2)], 30
    lens = [4, 60]
    full = [n + more for n in lens]
    y, x, _, _, pos, cu = run_inputs(full, F32, 3)
    table = kda.rope_table(64, 2 * len(AXIS), device="cuda")
    a, b = y, x
    for w in layers:
        a, b, _ = forward(kda, w, a, b, pos, table, cu)
    starts = cu[:-1].tolist()
    pick = torch.cat([torch.arange(s, s + n) for s, n in zip(starts, lens)]).cuda()
    cu_p = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    slots = torch.tensor([2, 0], dtype=torch.int32, device="cuda")
    caches = [[torch.zeros(3, SINKS + WINDOW, HK, D, device="cuda") for _ in range(2)] for _ in layers]
    u, h, pos_p = y[pick], x[pick], pos[:, pick].contiguous()
    for w, cache in zip(layers, caches):
        u, h, (_, p, _, k, *_) = forward(kda, w, u, h, pos_p, table, cu_p)
        kda.window_cache_write(k, split(p)[2], cu_p, *cache, slots, sinks=SINKS)
    close("prompt", u, a[pick].double().cpu(), TOL)
    in_y, in_x, in_pos = y[:2].clone(), x[:2].clone(), pos[:, :2].contiguous()
    at = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def step():
        u, h = in_y, in_x
        for w, cache in zip(layers, caches):
            u, h = token(kda, w, u, h, in_pos, table, cache, slots, at)
        return u, h
    kept = [[c.clone() for c in cache] for cache in caches]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for cache, old in zip(caches, kept):
        for c, o in zip(cache, old):
            c.copy_(o)
    for i in range(more):
        now = torch.tensor([s + n + i for s, n in zip(starts, lens)], device="cuda")
        in_y.copy_(y[now]), in_x.copy_(x[now]), in_pos.copy_(pos[:, now])
        at.copy_(torch.tensor([n + i for n in lens], dtype=torch.int32))
        graph.replay()
        close("token", out[0], a[now].double().cpu(), TOL)
        close("stream", out[1], b[now].double().cpu(), TOL)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_two_calls_at_once(kda, dtype):
    """Two steps on two streams next to each other: the bits of each alone."""
    layers = [Layer(dtype, 1), Layer(dtype, 2)]
    table = kda.rope_table(64, 2 * len(AXIS), device="cuda")
    ins = [run_inputs(lens, dtype, i) for i, lens in enumerate([[900, 300], [40, 1000, 3]])]
    alone = [train(kda, layers, *i[:5], table, i[5]) for i in ins]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in ins], [None, None]
    for _ in range(3):
        for j, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[j] = train(kda, layers, *ins[j][:5], table, ins[j][5])
    torch.cuda.synchronize()
    for want, have in zip(alone, got):
        assert all(torch.equal(a, b) for a, b in zip(want, have))
