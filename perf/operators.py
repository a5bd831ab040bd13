"""Cases for the linear-attention operators and the query/key norm-and-rotation
that feeds them.

``run`` computes each operator in its plain form (elementary torch operations,
32 bits) or, where ``own`` is true, through the package's entry points. The
operators:

* ``norm_rope`` / ``norm_rope_bwd``: per-head norm of q and k and the rotary
  positions in one pass, and its gradients;
* ``prefill`` / ``packed``: linear attention with a decay,
  S_t = e^{g_t} S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t, on equal-length and
  on packed sequences;
* ``prefill_bwd``: its gradients;
* ``decode``: one token on a state, or on slots of a pool of states.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one token of one sequence in a served layer: launch latency
        {"name": "norm_rope_token", "op": "norm_rope", "tokens": 1, "hq": 32, "hk": 32, "d": 128, "dtype": "bf16",
         "norm": "l2", "weight": False, "layout": "half", "rot": 128, "max_pos": 4096, "fused": True},
        # the 4 x 4096 x 16 training batch: rms norm with a weight, half of each head rotated, q and k cut out of
        # one fused projection
        {"name": "norm_rope_batch", "op": "norm_rope", "tokens": 16384, "hq": 16, "hk": 16, "d": 128,
         "dtype": "bf16", "norm": "rms", "weight": True, "layout": "half", "rot": 64, "max_pos": 4096, "fused": True},
        # the same batch in the backward pass, whole heads rotated
        {"name": "norm_rope_bwd_batch", "op": "norm_rope_bwd", "tokens": 16384, "hq": 16, "hk": 16, "d": 128,
         "dtype": "bf16", "norm": "rms", "weight": True, "layout": "half", "rot": 128, "max_pos": 4096,
         "fused": False},
        # fp32 training of a small model: fewer key heads than query heads, an odd token count, interleaved pairs
        {"name": "norm_rope_bwd_fp32_odd", "op": "norm_rope_bwd", "tokens": 1021, "hq": 6, "hk": 2, "d": 64,
         "dtype": "fp32", "norm": "rms", "weight": True, "layout": "interleaved", "rot": 32, "max_pos": 1024,
         "fused": False},
        # fp32 of the small reference workload's size with an odd length: a check run, a small model
        {"name": "prefill_fp32_small", "op": "prefill", "B": 1, "T": 257, "H": 2, "dk": 64, "dv": 64,
         "dtype": "fp32", "decay": "token", "s0": True},
        # the benchmark's batch: 4 sequences of 4096 tokens, 16 heads, a decay per token
        {"name": "prefill_4x16x4096", "op": "prefill", "B": 4, "T": 4096, "H": 16, "dk": 128, "dv": 128,
         "dtype": "bf16", "decay": "token", "s0": False},
        # one long document, a fixed decay per head, continued from a state
        {"name": "prefill_1x32x131072", "op": "prefill", "B": 1, "T": 131072, "H": 32, "dk": 128, "dv": 128,
         "dtype": "bf16", "decay": "head", "s0": True},
        # prompts of one serving step packed along the token axis, ragged lengths
        {"name": "packed_16seq", "op": "packed", "N": 16, "tokens": 20011, "empty": False, "H": 16, "dk": 128, "dv": 128,
         "dtype": "bf16", "decay": "token", "s0": True},
        # the benchmark's batch in training: every gradient, the decay's too
        {"name": "prefill_bwd_4x16x4096", "op": "prefill_bwd", "B": 4, "T": 4096, "H": 16, "dk": 128, "dv": 128,
         "dtype": "bf16", "decay": "token", "s0": True},
        # fp32 training of a small model, odd length, different key and value widths
        {"name": "prefill_bwd_fp32_odd", "op": "prefill_bwd", "B": 2, "T": 999, "H": 4, "dk": 64, "dv": 128,
         "dtype": "fp32", "decay": "token", "s0": True},
        # one decode step of one sequence on a slot of a pool: latency
        {"name": "decode_1x32_slots", "op": "decode", "N": 1, "H": 32, "dk": 128, "dv": 128, "dtype": "bf16",
         "decay": "head", "slots": True},
        # the benchmark's decode step: 256 sequences, 32 heads
        {"name": "decode_256x32", "op": "decode", "N": 256, "H": 32, "dk": 128, "dv": 128, "dtype": "bf16",
         "decay": "token", "slots": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_bwd", "prefill", "prefill", "packed", "prefill_bwd", "prefill_bwd",
                     "decode"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("norm_rope", "norm_rope_bwd"):
        hk = rng.choice([1, 2, 4, 8, 16, 32])
        hq = hk * rng.choice([1, 1, 2, 3])
        d = rng.choice([64, 128])
        return {"op": op, "tokens": _log_int(rng, 1, 65536 * 16 // (hq + hk)), "hq": hq, "hk": hk, "d": d,
                "dtype": dtype, "norm": rng.choice(["l2", "rms", "rms", "none"]), "weight": rng.random() < 0.6,
                "layout": rng.choice(["half", "interleaved"]), "rot": rng.choice([16, 32, 48, 64, d]),
                "max_pos": _log_int(rng, 64, 1024 if dtype == "fp32" else 32768), "fused": rng.random() < 0.4}
    dk, dv = rng.choice([(128, 128), (128, 128), (64, 64), (64, 128), (128, 64)])
    decay = rng.choice(["token", "token", "head", "none"])
    H = _log_int(rng, 1, 32)
    if op == "prefill":
        B = rng.choice([1, 1, 2, 3, 8])
        return {"op": op, "B": B, "T": _log_int(rng, 1, min(65536, (1 << 21) // (B * H))), "H": H, "dk": dk,
                "dv": dv, "dtype": dtype, "decay": decay, "s0": rng.random() < 0.5}
    if op == "packed":
        return {"op": op, "N": _log_int(rng, 2, 48), "tokens": _log_int(rng, 100, min(65536, (1 << 20) // H)),
                "empty": rng.random() < 0.3, "H": H, "dk": dk, "dv": dv, "dtype": dtype,
                "decay": decay, "s0": rng.random() < 0.5}
    if op == "prefill_bwd":
        B = rng.choice([1, 2, 4])
        return {"op": op, "B": B, "T": _log_int(rng, 1, min(32768, (1 << 18) // (B * H))), "H": H, "dk": dk,
                "dv": dv, "dtype": dtype, "decay": decay, "s0": rng.random() < 0.5}
    return {"op": op, "N": _log_int(rng, 1, 256), "H": H, "dk": dk, "dv": dv, "dtype": dtype, "decay": decay,
            "slots": rng.random() < 0.5}


# ------------------------------------------------------------------ the inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _unit(g, *shape):
    x = _normal(g, *shape)
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + EPS)


def _table(max_pos, rot, base=10000.0):
    """cos | sin of position times frequency, in 64 bits, rounded once: [max_pos, rot] float32."""
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat([a.cos(), a.sin()], -1).float().contiguous()


def _log_decay(g, kind, lead, H):
    """Per token: -softplus(N(0, 1)) times a rate that differs by head (1e-3 to 0.2); per head: the slopes
    -2^(-8 (h + 1) / H)."""
    if kind == "none":
        return None
    h = torch.arange(H, dtype=torch.float32, device="cuda")
    if kind == "head":
        return -torch.exp2(-8.0 * (h + 1) / H)
    rate = 1e-3 * (200.0 ** (h / max(1, H - 1)))
    return -torch.nn.functional.softplus(_normal(g, *lead, H)) * rate


def _norm_rope_inputs(case, seed):
    g = _gen(seed)
    n, hq, hk, d, dt = case["tokens"], case["hq"], case["hk"], case["d"], DT[case["dtype"]]
    s = {"positions": torch.randint(0, case["max_pos"], (n,), generator=g, device="cuda", dtype=torch.int32),
         "table": _table(case["max_pos"], case["rot"])}
    if case["fused"]:  # q, k and v of a token lie side by side, as one projection writes them
        p = (_normal(g, n, hq + 2 * hk, d) * 1.5).to(dt)
        s["q"], s["k"] = p[:, :hq], p[:, hq:hq + hk]
    else:
        s["q"], s["k"] = (_normal(g, n, hq, d) * 1.5).to(dt), (_normal(g, n, hk, d) * 1.5).to(dt)
    s["wq"] = 1 + 0.1 * _normal(g, d) if case["weight"] else None
    s["wk"] = 1 + 0.1 * _normal(g, d) if case["weight"] else None
    if case["op"] == "norm_rope_bwd":
        s["dyq"], s["dyk"] = _normal(g, n, hq, d).to(dt), _normal(g, n, hk, d).to(dt)
    return s


def _lengths(case, seed):
    """Ragged lengths (log-uniform shares, a factor of 64 from shortest to longest) that make up the case's tokens;
    one sequence of no token where the case says so."""
    g = torch.Generator().manual_seed(int(seed) + 5)
    share = torch.exp(torch.rand(case["N"], generator=g, dtype=torch.float64) * math.log(64.0))
    if case["empty"]:
        share[case["N"] // 2] = 0
    ends = (share.cumsum(0) / share.sum() * case["tokens"]).round().long()
    return torch.diff(ends, prepend=torch.zeros(1, dtype=torch.long)).tolist()


def _linear_inputs(case, seed):
    g = _gen(seed)
    H, dk, dv, dt, op = case["H"], case["dk"], case["dv"], DT[case["dtype"]], case["op"]
    s = {"scale": dk ** -0.5}
    if op == "packed":
        s["lens"] = _lengths(case, seed)
        cu = [0]
        cu[1:] = torch.tensor(s["lens"]).cumsum(0).tolist()
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        lead, n = (cu[-1],), case["N"]
    elif op == "decode":
        lead, n = (case["N"],), case["N"]
    else:
        lead, n = (case["B"], case["T"]), case["B"]
    # rows of norm sqrt(d), as a norm by the root of the mean square leaves them
    s["q"] = (_unit(g, *lead, H, dk) * dk ** 0.5).to(dt)
    s["k"] = _unit(g, *lead, H, dk).to(dt)
    s["v"] = _normal(g, *lead, H, dv).to(dt)
    s["g"] = _log_decay(g, case["decay"], lead, H)
    if op == "decode":
        pool = n + 3 if case["slots"] else n
        s["state"] = _normal(g, pool, H, dk, dv) * 0.1
        s["slots"] = torch.randperm(pool, generator=g, device="cuda")[:n].int() if case["slots"] else None
        return s
    s["s0"] = _normal(g, n, H, dk, dv) * 0.1 if case["s0"] else None
    if op == "prefill_bwd":
        s["do"] = _normal(g, *lead, H, dv).to(dt)
        s["dsT"] = _normal(g, n, H, dk, dv) * 0.1 if case["s0"] else None
    return s


def prepare(case, seed):
    s = _norm_rope_inputs(case, seed) if case["op"].startswith("norm_rope") else _linear_inputs(case, seed)
    s["case"] = case
    return s


# ------------------------------------------------------------------ plain forms
def _rotate(x, cos, sin, layout, rot, sign):
    """The first ``rot`` channels of each head turned by the token's angles (sign = -1: turned back)."""
    a, rest = x[..., :rot], x[..., rot:]
    cos, sin = cos[:, None], sign * sin[:, None]
    if layout == "half":
        u, w = a[..., :rot // 2], a[..., rot // 2:]
        return torch.cat([u * cos - w * sin, w * cos + u * sin, rest], -1)
    u, w = a[..., 0::2], a[..., 1::2]
    return torch.cat([torch.stack([u * cos - w * sin, w * cos + u * sin], -1).flatten(-2), rest], -1)


def _rs(x, norm):
    ss = (x * x).sum(-1, keepdim=True)
    if norm == "none":
        return torch.ones_like(ss)
    return torch.rsqrt((ss / x.shape[-1] if norm == "rms" else ss) + EPS)


def _plain_norm_rope(s, x, w):
    c = s["case"]
    xf = x.float()
    n = xf * _rs(xf, c["norm"])
    row = s["table"][s["positions"].long()]
    h = c["rot"] // 2
    return _rotate(n if w is None else n * w, row[:, :h], row[:, h:], c["layout"], c["rot"], 1).to(x.dtype)


def _plain_norm_rope_bwd(s, x, w, dy):
    c = s["case"]
    xf = x.float()
    r = _rs(xf, c["norm"])
    row = s["table"][s["positions"].long()]
    h = c["rot"] // 2
    u = _rotate(dy.float(), row[:, :h], row[:, h:], c["layout"], c["rot"], -1)
    dw = None if w is None else (u * (xf * r)).sum((0, 1))
    dn = u if w is None else u * w
    dx = r * dn
    if c["norm"] != "none":
        t = (xf * dn).sum(-1, keepdim=True)
        dx = dx - xf * (r * r * r) * (t / c["d"] if c["norm"] == "rms" else t)
    return dx.to(x.dtype), dw


def _segment_sums(a):
    """[..., n] -> [..., n, n]: sum of a over (j, i] for i >= j, -inf above the diagonal."""
    n = a.shape[-1]
    low = torch.ones(n, n, dtype=torch.bool, device=a.device).tril()
    x = a[..., :, None].expand(*a.shape, n).masked_fill(~low.tril(-1), 0.0).cumsum(-2)
    return x.masked_fill(~low, -math.inf)


def _chunked(q, k, v, g):
    """[B, T, H, d] -> 32-bit [B, H, N, C, d], zero-padded to whole chunks; the log decay as [B, H, N, C]."""
    B, T, H, _ = q.shape
    C = 64 if T <= 4096 else 128 if T <= 16384 else 512
    N = max(1, -(-T // C))

    def cut(x):
        x = torch.nn.functional.pad(x.float(), (0, 0, 0, 0, 0, N * C - T))
        return x.view(B, N, C, H, -1).permute(0, 3, 1, 2, 4)

    if g is None:
        g = torch.zeros(B, T, H, device=q.device)
    elif g.dim() == 1:
        g = g.expand(B, T, H)
    return cut(q), cut(k), cut(v), cut(g[..., None])[..., 0], C, N


def _whole(x, T, dtype):
    B, H, N, C, d = x.shape
    return x.permute(0, 2, 3, 1, 4).reshape(B, N * C, H, d)[:, :T].to(dtype).contiguous()


def _states(k, v, g, s0):
    """The state before each chunk and after the last one: chunk sums joined by the decays between chunks."""
    L = g.cumsum(-1)
    A = L[..., -1]
    w = torch.exp(_segment_sums(g)[..., -1, :])  # decay from each token to the chunk's end
    local = (k * w[..., None]).transpose(-1, -2) @ v
    E = torch.exp(_segment_sums(torch.cat([torch.zeros_like(A[..., :1]), A], -1)))
    if s0 is None:
        s0 = torch.zeros_like(local[:, :, 0])
    every = torch.cat([s0[:, :, None], local], 2)
    S = (E @ every.flatten(-2)).view(*every.shape)
    return S[:, :, :-1], S[:, :, -1], L, w


def _plain_prefill(q0, k0, v0, g0, s0, scale):
    T = q0.shape[1]
    q, k, v, g, C, N = _chunked(q0, k0, v0, g0)
    S, last, L, _ = _states(k, v, g, s0)
    P = (q @ k.transpose(-1, -2)) * torch.exp(_segment_sums(g))
    o = scale * (P @ v + torch.exp(L)[..., None] * (q @ S))
    return _whole(o, T, v0.dtype), last.contiguous()


def _plain_prefill_bwd(s):
    T, dt, scale = s["q"].shape[1], s["q"].dtype, s["scale"]
    q, k, v, g, C, N = _chunked(s["q"], s["k"], s["v"], s["g"])
    do = _chunked(s["q"], s["k"], s["do"], s["g"])[2]
    S, _, L, w = _states(k, v, g, s["s0"])
    # the gradient of the state after each chunk: the same sums in reverse time
    A = L[..., -1]
    local = scale * ((q * torch.exp(L)[..., None]).transpose(-1, -2) @ do)
    E = torch.exp(_segment_sums(torch.cat([torch.zeros_like(A[..., :1]), A.flip(-1)], -1)))
    end = torch.zeros_like(local[:, :, 0]) if s["dsT"] is None else s["dsT"]
    G = (E @ torch.cat([end[:, :, None], local.flip(2)], 2).flatten(-2)).view(*local.shape[:2], N + 1, *local.shape[3:])
    ds0, G = G[:, :, -1], G[:, :, :-1].flip(2)
    D = torch.exp(_segment_sums(g))
    P, dP = (q @ k.transpose(-1, -2)) * D, (do @ v.transpose(-1, -2)) * D
    dq_in = scale * torch.exp(L)[..., None] * (do @ S.transpose(-1, -2))
    dk_in = w[..., None] * (v @ G.transpose(-1, -2))
    dq = dq_in + scale * (dP @ k)
    dk = dk_in + scale * (dP.transpose(-1, -2) @ q)
    dv = w[..., None] * (k @ G) + scale * (P.transpose(-1, -2) @ do)
    out = {"dq": _whole(dq, T, dt), "dk": _whole(dk, T, dt), "dv": _whole(dv, T, dt)}
    if s["g"] is not None:
        # what passes over the step into token t: pairs j < t <= i of the chunk, the state before it, the gradient after it
        M = scale * P * dP / D.masked_fill(D == 0, 1.0)
        row = M.sum(-1) - M.sum(-2) + (q * dq_in).sum(-1) - (k * dk_in).sum(-1)
        through = torch.exp(A) * (S * G).sum((-1, -2)) + (k * dk_in).sum((-1, -2))
        dg = row.flip(-1).cumsum(-1).flip(-1) + through[..., None]
        B, H = dg.shape[:2]
        dg = dg.permute(0, 2, 3, 1).reshape(B, N * C, H)[:, :T]
        out["dlog_decay"] = dg.sum((0, 1)) if s["g"].dim() == 1 else dg.contiguous()
    if s["s0"] is not None:
        out["d_initial_state"] = ds0.contiguous()
    return out


def _plain_packed(s):
    """Sequences set side by side, padded to the longest, and taken apart again."""
    lens, cu, H = s["lens"], s["cu"], s["q"].shape[1]
    N, T = len(lens), max(1, max(lens))
    n = torch.arange(T, device="cuda")
    inside = n[None, :] < (cu[1:] - cu[:-1])[:, None]
    at = torch.where(inside, cu[:-1, None] + n, 0).long()

    def spread(x):
        return x[at] * inside.view(N, T, *[1] * (x.dim() - 1))

    g = s["g"] if s["g"] is None or s["g"].dim() == 2 else s["g"].expand(s["q"].shape[0], H)
    g = None if g is None else spread(g)
    if g is None:
        g = torch.zeros(N, T, H, device="cuda")
    o, last = _plain_prefill(spread(s["q"]), spread(s["k"]), spread(s["v"]), g, s["s0"], s["scale"])
    return o[inside], last


def _plain_decode(s):
    q, k, v, S = s["q"].float(), s["k"].float(), s["v"].float(), s["state"]
    a = None if s["g"] is None else torch.exp(s["g"])[..., None, None]
    at = slice(None) if s["slots"] is None else s["slots"].long()
    new = S[at] * (1.0 if a is None else a) + k[..., :, None] * v[..., None, :]
    S[at] = new
    return (s["scale"] * (q[..., None, :] @ new)[..., 0, :]).to(s["v"].dtype), S


def _plain(s):
    op = s["case"]["op"]
    if op == "norm_rope":
        return _plain_norm_rope(s, s["q"], s["wq"]), _plain_norm_rope(s, s["k"], s["wk"])
    if op == "norm_rope_bwd":
        (dq, dwq), (dk, dwk) = (_plain_norm_rope_bwd(s, s["q"], s["wq"], s["dyq"]),
                                _plain_norm_rope_bwd(s, s["k"], s["wk"], s["dyk"]))
        return {"dq": dq, "dk": dk, "dq_weight": dwq, "dk_weight": dwk}
    if op == "prefill":
        return _plain_prefill(s["q"], s["k"], s["v"], s["g"], s["s0"], s["scale"])
    if op == "packed":
        return _plain_packed(s)
    if op == "prefill_bwd":
        return _plain_prefill_bwd(s)
    return _plain_decode(s)


# ------------------------------------------------------------------ the package's calls
def _own(s):
    import kda_gated_delta_chunkwise_gb300 as kda
    c = s["case"]
    op = c["op"]
    if op.startswith("norm_rope"):
        kw = dict(norm=c["norm"], layout=c["layout"], eps=EPS)
        if op == "norm_rope":
            return kda.qk_norm_rope(s["q"], s["k"], s["positions"], s["table"], s["wq"], s["wk"], **kw)
        return kda.qk_norm_rope_backward(s["q"], s["k"], s["dyq"], s["dyk"], s["positions"], s["table"], s["wq"],
                                         s["wk"], **kw)
    kw = dict(decay=c["decay"], scale=s["scale"])
    if op == "prefill":
        return kda.linear_prefill(s["q"], s["k"], s["v"], s["g"], s["s0"], **kw)
    if op == "packed":
        return kda.linear_varlen_prefill(s["q"], s["k"], s["v"], s["g"], s["cu"], s["s0"], **kw)
    if op == "prefill_bwd":
        out = kda.linear_prefill_backward(s["q"], s["k"], s["v"], s["g"], s["do"], s["s0"], s["dsT"],
                                          want_initial_state_grad=s["s0"] is not None, **kw)
        return {n: x for n, x in out.items() if x is not None}
    if s["slots"] is not None:
        o = kda.linear_decode_step_slots(s["q"], s["k"], s["v"], s["g"], s["state"], s["slots"], **kw)
    else:
        o = kda.linear_decode_step(s["q"], s["k"], s["v"], s["g"], s["state"], **kw)
    return o, s["state"]


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op.startswith("norm_rope"):
        n, rows = case["tokens"], case["tokens"] * (case["hq"] + case["hk"])
        table = min(n, case["max_pos"]) * case["rot"] * 4 + n * 4
        back = op == "norm_rope_bwd"
        return {"bytes": rows * case["d"] * es * (3 if back else 2) + table, "flops": rows * case["d"] * (16 if back else 8)}
    H, dk, dv = case["H"], case["dk"], case["dv"]
    if op == "packed":
        n, tokens = case["N"], case["tokens"]
    elif op == "decode":
        n = tokens = case["N"]
    else:
        n, tokens = case["B"], case["B"] * case["T"]
    th = tokens * H
    g = 4 * th if case["decay"] == "token" else 0
    state = n * H * dk * dv * 4
    if op == "decode":
        return {"bytes": 2 * state + th * (2 * dk + 2 * dv) * es + g, "flops": th * 4 * dk * dv}
    if op == "prefill_bwd":
        return {"bytes": th * (4 * dk + 3 * dv) * es + 2 * g + (3 * state if case["s0"] else 0),
                "flops": th * 10 * dk * dv}
    return {"bytes": th * (2 * dk + 2 * dv) * es + g + state * (2 if case["s0"] else 1), "flops": th * 4 * dk * dv}


# ------------------------------------------------------------------ 64 bits, from the definitions
def _exact_norm_rope(s, case):
    """Each pair of channels as a complex number times e^{i angle}; gradients by torch's reverse mode."""
    row = s["table"][s["positions"].long()].double()
    h, rot = case["rot"] // 2, case["rot"]
    turn = torch.complex(row[:, :h], row[:, h:])[:, None]

    def forward(x, w):
        y = x
        if case["norm"] != "none":
            den = x.pow(2).mean(-1, keepdim=True) if case["norm"] == "rms" else x.pow(2).sum(-1, keepdim=True)
            y = x / (den + EPS).sqrt()
        y = y if w is None else y * w
        a = y[..., :rot]
        if case["layout"] == "half":
            z = torch.complex(a[..., :h].contiguous(), a[..., h:].contiguous()) * turn
            a = torch.cat([z.real, z.imag], -1)
        else:
            z = torch.complex(a[..., 0::2].contiguous(), a[..., 1::2].contiguous()) * turn
            a = torch.view_as_real(z).flatten(-2)
        return torch.cat([a, y[..., rot:]], -1)

    res = []
    for x, w, dy in ((s["q"], s["wq"], s.get("dyq")), (s["k"], s["wk"], s.get("dyk"))):
        x = x.double().requires_grad_(dy is not None)
        w = None if w is None else w.double().requires_grad_(dy is not None)
        y = forward(x, w)
        if dy is not None:
            y.backward(dy.double())
            res.append((x.grad, None if w is None else w.grad))
        else:
            res.append(y)
    if case["op"] == "norm_rope":
        return tuple(res)
    return {"dq": res[0][0], "dk": res[1][0], "dq_weight": res[0][1], "dk_weight": res[1][1]}


def _rows(x, lens):
    """Token-major [n, T, H, ...] of a batch (lens None) or of a packed tensor, as time-major [T, n * H, ...] in 64 bits."""
    if lens is not None:
        x = torch.nn.utils.rnn.pad_sequence(list(torch.split(x, lens)), batch_first=True) if sum(lens) else x[None, :0].expand(len(lens), *x[:0].shape)
    x = x.double()
    return x.transpose(0, 1).flatten(1, 2).contiguous()


def _exact_linear(s, case):
    """The recurrence, token by token."""
    H, dk, dv, op, scale = case["H"], case["dk"], case["dv"], case["op"], s["scale"]
    if op == "decode":
        S = s["state"].double()
        at = torch.arange(case["N"], device="cuda") if s["slots"] is None else s["slots"].long()
        a = torch.ones(case["N"], H, device="cuda", dtype=torch.float64) if s["g"] is None else s["g"].double().exp().expand(case["N"], H)
        new = torch.einsum("nhkv,nh->nhkv", S[at], a) + torch.einsum("nhk,nhv->nhkv", s["k"].double(), s["v"].double())
        S[at] = new
        return scale * torch.einsum("nhkv,nhk->nhv", new, s["q"].double()), S
    lens = s.get("lens")
    n = case["N"] if op == "packed" else case["B"]
    q, k, v = (_rows(s[x], lens) for x in ("q", "k", "v"))
    T = q.shape[0]
    if s["g"] is None:
        g = torch.zeros(T, n * H, device="cuda", dtype=torch.float64)
    elif s["g"].dim() == 1:
        g = s["g"].double().repeat(n).expand(T, n * H)
    else:
        g = _rows(s["g"][..., None], lens)[..., 0]
    if lens is not None:  # after its end a sequence stands still
        alive = torch.arange(T, device="cuda")[:, None] < torch.tensor(lens, device="cuda").repeat_interleave(H)
        g = torch.where(alive, g, torch.zeros_like(g))
    a = g.exp()[..., None, None].contiguous()
    S = torch.zeros(n * H, dk, dv, device="cuda", dtype=torch.float64) if s["s0"] is None else s["s0"].double().flatten(0, 1).clone()
    if op == "prefill_bwd":
        do = _rows(s["do"], None)
        kept = torch.empty(T, n * H, dk, dv, device="cuda", dtype=torch.float64)
        dq, dkk, dvv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        dg = torch.empty(T, n * H, device="cuda", dtype=torch.float64)
        for t in range(T):
            torch.mul(S, a[t], out=kept[t])
            S = torch.baddbmm(kept[t], k[t][:, :, None], v[t][:, None, :])
            dq[t] = scale * torch.bmm(S, do[t][:, :, None])[..., 0]
        G = torch.zeros_like(S) if s["dsT"] is None else s["dsT"].double().flatten(0, 1).clone()
        for t in range(T - 1, -1, -1):
            G = torch.baddbmm(G, scale * q[t][:, :, None], do[t][:, None, :])
            dkk[t] = torch.bmm(G, v[t][:, :, None])[..., 0]
            dvv[t] = torch.bmm(k[t][:, None, :], G)[:, 0]
            dg[t] = (G * kept[t]).sum((-1, -2))
            G = G * a[t]

        def back(x):
            return x.view(T, n, H, *x.shape[2:]).transpose(0, 1).contiguous()

        out = {"dq": back(dq), "dk": back(dkk), "dv": back(dvv)}
        if s["g"] is not None:
            out["dlog_decay"] = back(dg) if s["g"].dim() > 1 else back(dg).sum((0, 1))
        if s["s0"] is not None:
            out["d_initial_state"] = G.view(n, H, dk, dv)
        return out
    o = torch.empty(T, n * H, 1, dv, device="cuda", dtype=torch.float64)
    q = q[:, :, None]
    kt, v = k[..., None], v[:, :, None]
    for t in range(T):
        S.mul_(a[t]).baddbmm_(kt[t], v[t])
        torch.bmm(q[t], S, out=o[t])
    o = (scale * o).view(T, n, H, dv).transpose(0, 1)
    if lens is not None:
        o = torch.cat([o[i, :m] for i, m in enumerate(lens)])
    return o.contiguous(), S.view(n, H, dk, dv)


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_norm_rope(s, case) if case["op"].startswith("norm_rope") else _exact_linear(s, case)
