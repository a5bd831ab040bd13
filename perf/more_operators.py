"""Cases for the operators around the recurrences of a hybrid layer stack.

``run`` computes each operator in its plain form (elementary torch operations,
32 bits) or, where ``own`` is true, through the package's entry points. The
operators:

* ``axes`` / ``axes_bwd``: the norm of q and k with rotary positions of several
  axes, and its gradients;
* ``gated`` / ``gated_bwd``: the norm of every head times a gate, behind a
  recurrence, and its gradients;
* ``residual`` / ``residual_bwd``: a branch (normed, scaled by channel) added to
  the residual stream and the sum's norm, and its gradients;
* ``window`` / ``packed``: attention with a sliding window and a few first
  tokens that stay visible, on equal lengths, and on packed prompts whose keys
  and values then go into the slots of a cache;
* ``window_bwd``: its gradients;
* ``decode``: one token per sequence on its slot of that cache.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one token of an image-and-text model in a served layer: launch latency
        {"name": "axes_token", "op": "axes", "tokens": 1, "hq": 32, "hk": 8, "d": 128, "dtype": "bf16", "norm": "rms",
         "weight": True, "layout": "half", "sections": "16,24,24", "cycle": False, "max_pos": 4096, "fused": True},
        # the 4 x 4096 x 16 training batch, time, height and width in turn over the channel pairs
        {"name": "axes_bwd_batch", "op": "axes_bwd", "tokens": 16384, "hq": 16, "hk": 16, "d": 128, "dtype": "bf16",
         "norm": "rms", "weight": True, "layout": "half", "sections": "24,20,20", "cycle": True, "max_pos": 4096,
         "fused": False},
        # the output of a recurrent layer over the same batch: head norm and sigmoid gate, the gate cut out of a
        # fused projection
        {"name": "gated_batch", "op": "gated", "tokens": 16384, "h": 16, "d": 128, "dtype": "bf16", "norm": "rms",
         "act": "sigmoid", "weight": True, "fused": True},
        # fp32 training of a small model, an odd token count, silu gate
        {"name": "gated_bwd_fp32_odd", "op": "gated_bwd", "tokens": 1021, "h": 6, "d": 64, "dtype": "fp32",
         "norm": "rms", "act": "silu", "weight": True, "fused": False},
        # one token's way from a block into the next, a stream of 32 heads of 128
        {"name": "residual_token", "op": "residual", "tokens": 1, "D": 4096, "dtype": "bf16", "stream": "bf16",
         "post": False, "channel": False},
        # the training batch on a stream of 16 heads of 128: branch norm, layer scale, residual stream in fp32
        {"name": "residual_bwd_batch", "op": "residual_bwd", "tokens": 16384, "D": 2048, "dtype": "bf16",
         "stream": "fp32", "post": True, "channel": True},
        # the benchmark's batch: 4 sequences of 4096 tokens, 16 heads
        {"name": "window_4x16x4096", "op": "window", "B": 4, "T": 4096, "hq": 16, "hk": 16, "d": 128, "dtype": "bf16",
         "window": 1024, "sinks": 4},
        # prompts of one serving step, ragged and long, four query heads to a key head, written into their cache slots
        {"name": "packed_65536x32", "op": "packed", "N": 16, "tokens": 65531, "hq": 32, "hk": 8, "d": 128,
         "dtype": "bf16", "window": 2048, "sinks": 4},
        # the benchmark's batch in training
        {"name": "window_bwd_4x16x4096", "op": "window_bwd", "B": 4, "T": 4096, "hq": 16, "hk": 16, "d": 128,
         "dtype": "bf16", "window": 1024, "sinks": 4},
        # fp32 training of a small model, odd lengths, a window that ends inside a tile
        {"name": "window_bwd_fp32_odd", "op": "window_bwd", "B": 2, "T": 999, "hq": 4, "hk": 2, "d": 64,
         "dtype": "fp32", "window": 100, "sinks": 3},
        # one decode step of one sequence: latency
        {"name": "decode_1x32", "op": "decode", "N": 1, "hq": 32, "hk": 8, "d": 128, "dtype": "bf16", "window": 2048,
         "sinks": 4, "pos_from": 2500, "pos_to": 2500},
        # the benchmark's decode batch: 256 sequences, 32 heads, some still filling their window
        {"name": "decode_256x32", "op": "decode", "N": 256, "hq": 32, "hk": 8, "d": 128, "dtype": "bf16",
         "window": 2048, "sinks": 4, "pos_from": 500, "pos_to": 100000},
    ]


def _log_int(rng, lo, hi):
    hi = max(lo, hi)
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["axes", "axes_bwd", "gated", "gated_bwd", "residual", "residual_bwd", "window", "window", "packed",
                     "window_bwd", "window_bwd", "decode", "decode"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    d = rng.choice([64, 128])
    if op in ("axes", "axes_bwd"):
        hk = rng.choice([1, 2, 4, 8, 16, 32])
        hq = hk * rng.choice([1, 1, 2, 3])
        rot = rng.choice([16, 32, 48, 64, d])
        axes = rng.choice([2, 3, 3, 4])
        cuts = sorted(rng.sample(range(1, rot // 2), axes - 1))
        sections = ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [rot // 2]))
        return {"op": op, "tokens": _log_int(rng, 1, 65536 * 16 // (hq + hk)), "hq": hq, "hk": hk, "d": d,
                "dtype": dtype, "norm": rng.choice(["l2", "rms", "rms", "none"]), "weight": rng.random() < 0.6,
                "layout": rng.choice(["half", "interleaved"]), "sections": sections, "cycle": rng.random() < 0.5,
                "max_pos": _log_int(rng, 64, 1024 if dtype == "fp32" else 32768), "fused": rng.random() < 0.4}
    if op in ("gated", "gated_bwd"):
        h = _log_int(rng, 1, 48)
        return {"op": op, "tokens": _log_int(rng, 1, (1 << 20) // h), "h": h, "d": d, "dtype": dtype,
                "norm": rng.choice(["rms", "rms", "l2", "none"]), "act": rng.choice(["sigmoid", "silu"]),
                "weight": rng.random() < 0.7, "fused": rng.random() < 0.4}
    if op in ("residual", "residual_bwd"):
        D = 8 * _log_int(rng, 2, 1024)
        return {"op": op, "tokens": _log_int(rng, 1, min(65536, (1 << 26) // D)), "D": D, "dtype": dtype,
                "stream": rng.choice(["bf16", "fp32"]) if dtype == "bf16" else "fp32", "post": rng.random() < 0.5,
                "channel": rng.random() < 0.4}
    hk = rng.choice([1, 1, 2, 3, 4, 8, 16])
    hq = hk * rng.choice([1, 1, 2, 4, 5, 8])
    window, sinks = _log_int(rng, 1, 4096), rng.choice([0, 1, 4, 4, 16, 100, 128])
    # as many query heads times tokens as the largest listed cases, fewer where fp32 or the backward costs more
    if op == "window":
        B = rng.choice([1, 1, 2, 3, 8])
        return {"op": op, "B": B, "T": _log_int(rng, 1, min(65536, (1 << (20 if dtype == "bf16" else 17)) // (B * hq))),
                "hq": hq, "hk": hk, "d": d, "dtype": dtype, "window": window, "sinks": sinks}
    if op == "packed":
        return {"op": op, "N": _log_int(rng, 2, 48), "tokens": _log_int(rng, 100, min(65536, (1 << (20 if dtype == "bf16" else 17)) // hq)),
                "hq": hq, "hk": hk, "d": d, "dtype": dtype, "window": window, "sinks": sinks}
    if op == "window_bwd":
        B = rng.choice([1, 2, 4])
        return {"op": op, "B": B, "T": _log_int(rng, 1, min(32768, (1 << (18 if dtype == "bf16" else 16)) // (B * hq))),
                "hq": hq, "hk": hk, "d": d, "dtype": dtype, "window": min(window, 2048), "sinks": sinks}
    N = _log_int(rng, 1, 256)
    lo = _log_int(rng, 1, 3000) - 1
    return {"op": op, "N": N, "hq": hq, "hk": hk, "d": d, "dtype": dtype,
            "window": min(window, max(1, (1 << 22) // (N * hk))), "sinks": sinks, "pos_from": lo, "pos_to": lo + _log_int(rng, 1, 200000)}


# ------------------------------------------------------------------ the inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 23)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _table(max_pos, rot, base=10000.0):
    """cos | sin of position times frequency, in 64 bits, rounded once: [max_pos, rot] float32."""
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat([a.cos(), a.sin()], -1).float().contiguous()


def _sections(case):
    return [int(n) for n in case["sections"].split(",")]


def _pair_axis(case):
    """The axis of every channel pair: the sections one after the other, or the axes in turn until each has its share."""
    left = _sections(case)
    if not case["cycle"]:
        return [a for a, n in enumerate(left) for _ in range(n)]
    out = []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                out.append(a)
                left[a] -= 1
    return out


def _lengths(case):
    """Ragged lengths (log-uniform shares, a factor of 64 from shortest to longest) that make up the case's tokens."""
    g = torch.Generator().manual_seed(case["tokens"] + 31 * case["N"])
    share = torch.exp(torch.rand(case["N"], generator=g, dtype=torch.float64) * math.log(64.0))
    ends = (share.cumsum(0) / share.sum() * case["tokens"]).round().long()
    return torch.diff(ends, prepend=torch.zeros(1, dtype=torch.long)).tolist()


def _positions(case):
    """Tokens that each sequence of a decode batch has behind it: spread over the case's range."""
    lo, hi = case["pos_from"], case["pos_to"]
    return [lo + (n * 7919 + 4099) % (hi - lo + 1) for n in range(case["N"])]


def _axes_inputs(case, g):
    n, hq, hk, d, dt = case["tokens"], case["hq"], case["hk"], case["d"], DT[case["dtype"]]
    axes = len(_sections(case))
    s = {"positions": torch.randint(0, case["max_pos"], (axes, n), generator=g, device="cuda", dtype=torch.int32),
         "table": _table(case["max_pos"], 2 * sum(_sections(case))), "pair_axis": _pair_axis(case)}
    if case["fused"]:  # q, k and v of a token lie side by side, as one projection writes them
        p = (_normal(g, n, hq + 2 * hk, d) * 1.5).to(dt)
        s["q"], s["k"] = p[:, :hq], p[:, hq:hq + hk]
    else:
        s["q"], s["k"] = (_normal(g, n, hq, d) * 1.5).to(dt), (_normal(g, n, hk, d) * 1.5).to(dt)
    s["wq"] = 1 + 0.1 * _normal(g, d) if case["weight"] else None
    s["wk"] = 1 + 0.1 * _normal(g, d) if case["weight"] else None
    if case["op"] == "axes_bwd":
        s["dyq"], s["dyk"] = _normal(g, n, hq, d).to(dt), _normal(g, n, hk, d).to(dt)
    return s


def _gated_inputs(case, g):
    n, h, d, dt = case["tokens"], case["h"], case["d"], DT[case["dtype"]]
    s = {"x": (_normal(g, n, h, d) * 0.3).to(dt)}
    s["gate"] = (_normal(g, n, 3 * h, d) * 2).to(dt)[:, 2 * h:] if case["fused"] else (_normal(g, n, h, d) * 2).to(dt)
    s["w"] = 1 + 0.1 * _normal(g, d) if case["weight"] else None
    if case["op"] == "gated_bwd":
        s["dy"] = _normal(g, n, h, d).to(dt)
    return s


def _residual_inputs(case, g):
    n, D, dt, ds = case["tokens"], case["D"], DT[case["dtype"]], DT[case["stream"]]
    s = {"branch": _normal(g, n, D).to(dt), "w": 1 + 0.1 * _normal(g, D), "scale": 0.5,
         "wb": 1 + 0.1 * _normal(g, D) if case["post"] else None,
         "c": 0.5 + 0.1 * _normal(g, D) if case["channel"] else None}
    s["h" if case["op"] == "residual_bwd" else "x"] = (_normal(g, n, D) * 3).to(ds)
    if case["op"] == "residual_bwd":
        s["dy"], s["dh"] = _normal(g, n, D).to(dt), _normal(g, n, D).to(ds)
    return s


def _window_inputs(case, g):
    hq, hk, d, dt, op = case["hq"], case["hk"], case["d"], DT[case["dtype"]], case["op"]
    entries = case["window"] + case["sinks"]
    s = {"scale": d ** -0.5}
    lead = (case["B"], case["T"]) if op in ("window", "window_bwd") else (case["tokens"],) if op == "packed" else (case["N"],)
    s["q"] = (_normal(g, *lead, hq, d) * 1.5).to(dt)
    s["k"], s["v"] = _normal(g, *lead, hk, d).to(dt), _normal(g, *lead, hk, d).to(dt)
    if op in ("packed", "decode"):
        pool = case["N"] + 2
        s["slots"] = torch.randperm(pool, generator=g, device="cuda")[:case["N"]].int()
        if op == "packed":
            s["lens"] = _lengths(case)
            cu = [0]
            cu[1:] = torch.tensor(s["lens"]).cumsum(0).tolist()
            s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
            s["k_cache"], s["v_cache"] = (torch.zeros(pool, entries, hk, d, dtype=dt, device="cuda") for _ in range(2))
        else:
            s["positions"] = torch.tensor(_positions(case), dtype=torch.int32, device="cuda")
            s["k_cache"], s["v_cache"] = (_normal(g, pool, entries, hk, d).to(dt) for _ in range(2))
    if op == "window_bwd":
        # o and lse as the forward pass left them
        s["do"] = _normal(g, *lead, hq, d).to(dt)
        s["o"], s["lse"] = _plain_window(s["q"], s["k"], s["v"], case, s["scale"])
    return s


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    make = (_axes_inputs if op.startswith("axes") else _gated_inputs if op.startswith("gated") else
            _residual_inputs if op.startswith("residual") else _window_inputs)
    s = make(case, g)
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


def _angles(s):
    """Every pair's cosine and sine, from the row of its own axis' position."""
    axis = torch.tensor(s["pair_axis"], device="cuda")
    pos = s["positions"].long()[axis].t()  # [tokens, pairs]
    pair = torch.arange(len(s["pair_axis"]), device="cuda")
    return s["table"][pos, pair], s["table"][pos, pair + len(s["pair_axis"])]


def _norm_back(x, r, dn, norm):
    dx = r * dn
    if norm == "none":
        return dx
    t = (x * dn).sum(-1, keepdim=True)
    return dx - x * (r * r * r) * (t / x.shape[-1] if norm == "rms" else t)


def _plain_axes(s):
    c = s["case"]
    cos, sin = _angles(s)
    out = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        n = x.float() * _rs(x.float(), c["norm"])
        out.append(_rotate(n if w is None else n * w, cos, sin, c["layout"], 2 * len(s["pair_axis"]), 1).to(x.dtype))
    return tuple(out)


def _plain_axes_bwd(s):
    c = s["case"]
    cos, sin = _angles(s)
    out = []
    for x, w, dy in ((s["q"], s["wq"], s["dyq"]), (s["k"], s["wk"], s["dyk"])):
        xf = x.float()
        r = _rs(xf, c["norm"])
        u = _rotate(dy.float(), cos, sin, c["layout"], 2 * len(s["pair_axis"]), -1)
        out.append((_norm_back(xf, r, u if w is None else u * w, c["norm"]).to(x.dtype),
                    None if w is None else (u * (xf * r)).sum((0, 1))))
    return {"dq": out[0][0], "dk": out[1][0], "dq_weight": out[0][1], "dk_weight": out[1][1]}


def _gate(g, act):
    """The gate's value and its derivative."""
    a = 1 / (1 + torch.exp(-g))
    return (a, a * (1 - a)) if act == "sigmoid" else (g * a, a * (1 + g * (1 - a)))


def _plain_gated(s):
    c = s["case"]
    x = s["x"].float()
    a, da = _gate(s["gate"].float(), c["act"])
    r = _rs(x, c["norm"])
    n = x * r
    if c["op"] == "gated":
        return ((n if s["w"] is None else n * s["w"]) * a).to(s["x"].dtype)
    dy, w = s["dy"].float(), 1.0 if s["w"] is None else s["w"]
    return {"dx": _norm_back(x, r, w * a * dy, c["norm"]).to(s["x"].dtype),
            "dgate": (w * n * da * dy).to(s["x"].dtype),
            "dweight": None if s["w"] is None else (n * a * dy).sum((0, 1))}


def _plain_residual(s):
    b = s["branch"].float()
    u = b if s["wb"] is None else s["wb"] * (b * _rs(b, "rms"))
    h = s["x"].float() + s["scale"] * (u if s["c"] is None else s["c"] * u)
    return h.to(s["x"].dtype), (s["w"] * (h * _rs(h, "rms"))).to(s["branch"].dtype)


def _plain_residual_bwd(s):
    h, dy, b = s["h"].float(), s["dy"].float(), s["branch"].float()
    r = _rs(h, "rms")
    g = s["dh"].float() + _norm_back(h, r, s["w"] * dy, "rms")
    out = {"d_residual": g.to(s["h"].dtype), "dweight": (h * r * dy).sum(0)}
    du = s["scale"] * (g if s["c"] is None else s["c"] * g)
    u = b
    if s["wb"] is None:
        out["d_branch"] = du.to(s["branch"].dtype)
    else:
        rb = _rs(b, "rms")
        u = s["wb"] * (b * rb)
        out["d_branch"] = _norm_back(b, rb, s["wb"] * du, "rms").to(s["branch"].dtype)
        out["dbranch_weight"] = (b * rb * du).sum(0)
    if s["c"] is not None:
        out["dchannel_scale"] = (s["scale"] * u * g).sum(0)
    return out


def _rows_per_block(heads, window):
    return max(64, min(1024, (1 << 27) // (heads * (min(window, 8192) + 1024)) // 64 * 64))


def _blocks(q, k, case):
    """Query blocks of a batch: (first, end, key positions, visible) with the sinks before the block's window."""
    T, W, S = q.shape[1], case["window"], case["sinks"]
    C = _rows_per_block(q.shape[0] * q.shape[2], W)
    for i0 in range(0, T, C):
        i1 = min(T, i0 + C)
        lo = max(0, i0 - W + 1)
        j = torch.cat([torch.arange(min(S, lo), device=q.device), torch.arange(lo, i1, device=q.device)])
        i = torch.arange(i0, i1, device=q.device)[:, None]
        yield i0, i1, j, (j <= i) & ((i - j < W) | (j < S))


def _scores(q, k, i0, i1, j, see, scale):
    """[B, Hk, G, rows, keys] 32-bit scores, -inf where not visible."""
    B, _, Hk, d = k.shape
    G = q.shape[2] // Hk
    qb = q[:, i0:i1].float().reshape(B, i1 - i0, Hk, G, d).permute(0, 2, 3, 1, 4)
    kb = k[:, j].float().permute(0, 2, 3, 1)[:, :, None]
    return qb, kb, (scale * (qb @ kb)).masked_fill(~see, -math.inf)


def _plain_window(q, k, v, case, scale):
    B, T, Hq, d = q.shape
    o, lse = torch.empty_like(q), torch.empty(B, T, Hq, device=q.device)
    for i0, i1, j, see in _blocks(q, k, case):
        _, _, s = _scores(q, k, i0, i1, j, see, scale)
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - m)
        l = p.sum(-1, keepdim=True)
        ob = (p @ v[:, j].float().permute(0, 2, 1, 3)[:, :, None]) / l
        o[:, i0:i1] = ob.permute(0, 3, 1, 2, 4).reshape(B, i1 - i0, Hq, d).to(q.dtype)
        lse[:, i0:i1] = (m + torch.log(l))[..., 0].permute(0, 3, 1, 2).reshape(B, i1 - i0, Hq)
    return o, lse


def _plain_packed(s):
    c, cu = s["case"], [0]
    o, lse = torch.empty_like(s["q"]), torch.empty(s["q"].shape[:2], device="cuda")
    W, S = c["window"], c["sinks"]
    slots = s["slots"].long()
    for n, m in enumerate(s["lens"]):
        a, b = cu[-1], cu[-1] + m
        cu.append(b)
        if m == 0:
            continue
        o[a:b], lse[a:b] = (x[0] for x in _plain_window(s["q"][None, a:b], s["k"][None, a:b], s["v"][None, a:b], c, s["scale"]))
        p = torch.cat([torch.arange(min(S, m), device="cuda"), torch.arange(max(min(S, m), m - W), m, device="cuda")])
        e = torch.where(p < S, p, S + (p - S) % W)
        s["k_cache"][slots[n], e] = s["k"][a:b][p]
        s["v_cache"][slots[n], e] = s["v"][a:b][p]
    return o, lse, s["k_cache"], s["v_cache"]


def _plain_window_bwd(s):
    c, q, k, v, scale = s["case"], s["q"], s["k"], s["v"], s["scale"]
    B, T, Hq, d = q.shape
    Hk = k.shape[2]
    G = Hq // Hk
    dq = torch.empty_like(q)
    dk, dv = (torch.zeros(B, Hk, T, d, device=q.device) for _ in range(2))

    def rows(x, i0, i1):  # [B, T, Hq, ...] -> [B, Hk, G, rows, ...]
        return x[:, i0:i1].float().reshape(B, i1 - i0, Hk, G, *x.shape[3:]).movedim(1, 3)

    for i0, i1, j, see in _blocks(q, k, c):
        qb, kb, sc = _scores(q, k, i0, i1, j, see, scale)
        p = torch.exp(sc - rows(s["lse"], i0, i1)[..., None])
        dob = rows(s["do"], i0, i1)
        dv[:, :, j] += (p.transpose(-1, -2) @ dob).sum(2)
        dp = dob @ v[:, j].float().permute(0, 2, 3, 1)[:, :, None]
        ds = p * (dp - (p * dp).sum(-1, keepdim=True))
        dq[:, i0:i1] = (scale * (ds @ kb.transpose(-1, -2))).permute(0, 3, 1, 2, 4).reshape(B, i1 - i0, Hq, d).to(q.dtype)
        dk[:, :, j] += scale * (ds.transpose(-1, -2) @ qb).sum(2)
    return {"dq": dq, "dk": dk.transpose(1, 2).to(q.dtype).contiguous(), "dv": dv.transpose(1, 2).to(q.dtype).contiguous()}


def _plain_decode(s):
    c = s["case"]
    N, hq, d = s["q"].shape
    hk, W, S = c["hk"], c["window"], c["sinks"]
    pos, slots = s["positions"].long(), s["slots"].long()
    e = torch.where(pos < S, pos, S + (pos - S) % W)
    s["k_cache"][slots, e] = s["k"]
    s["v_cache"][slots, e] = s["v"]
    out = torch.empty_like(s["q"])
    step = max(1, (1 << 27) // ((W + S) * hk * d))
    for a in range(0, N, step):
        at = slots[a:a + step]
        kc, vc = (s[x][at].float().permute(0, 2, 1, 3) for x in ("k_cache", "v_cache"))  # [n, hk, entries, d]
        see = torch.arange(W + S, device="cuda") <= pos[a:a + step, None]
        q = s["q"][a:a + step].float().view(-1, hk, hq // hk, d)
        sc = (s["scale"] * (q @ kc.transpose(-1, -2))).masked_fill(~see[:, None, None], -math.inf)
        p = torch.exp(sc - sc.amax(-1, keepdim=True))
        out[a:a + step] = ((p @ (vc * see[:, None, :, None])) / p.sum(-1, keepdim=True)).reshape(-1, hq, d).to(out.dtype)
    return out, s["k_cache"], s["v_cache"]


def _plain(s):
    op = s["case"]["op"]
    if op == "window":
        return _plain_window(s["q"], s["k"], s["v"], s["case"], s["scale"])
    return {"axes": _plain_axes, "axes_bwd": _plain_axes_bwd, "gated": _plain_gated, "gated_bwd": _plain_gated,
            "residual": _plain_residual, "residual_bwd": _plain_residual_bwd, "packed": _plain_packed,
            "window_bwd": _plain_window_bwd, "decode": _plain_decode}[op](s)


# ------------------------------------------------------------------ the package's calls
def _own(s):
    import kda_gated_delta_chunkwise_gb300 as kda
    c = s["case"]
    op = c["op"]
    if op.startswith("axes"):
        kw = dict(norm=c["norm"], layout=c["layout"], eps=EPS)
        if op == "axes":
            return kda.qk_norm_rope_axes(s["q"], s["k"], s["positions"], s["table"], s["pair_axis"], s["wq"], s["wk"], **kw)
        return kda.qk_norm_rope_axes_backward(s["q"], s["k"], s["dyq"], s["dyk"], s["positions"], s["table"],
                                              s["pair_axis"], s["wq"], s["wk"], **kw)
    if op.startswith("gated"):
        kw = dict(norm=c["norm"], activation=c["act"], eps=EPS)
        if op == "gated":
            return kda.gated_norm(s["x"], s["gate"], s["w"], **kw)
        return kda.gated_norm_backward(s["x"], s["gate"], s["dy"], s["w"], **kw)
    if op.startswith("residual"):
        kw = dict(branch_norm="rms" if c["post"] else "none", branch_weight=s["wb"], channel_scale=s["c"],
                  scale=s["scale"], eps=EPS)
        if op == "residual":
            return kda.residual_norm(s["x"], s["branch"], s["w"], **kw)
        out = kda.residual_norm_backward(s["h"], s["branch"], s["dy"], s["dh"], s["w"], **kw)
        return {n: x for n, x in out.items() if x is not None}
    if op == "decode":
        o = kda.window_decode_step(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], s["positions"],
                                   sinks=c["sinks"], scale=s["scale"])
        return o, s["k_cache"], s["v_cache"]
    kw = dict(window=c["window"], sinks=c["sinks"], scale=s["scale"])
    if op == "window":
        return kda.window_attention(s["q"], s["k"], s["v"], **kw)
    if op == "window_bwd":
        return kda.window_attention_backward(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], **kw)
    o, lse = kda.window_varlen_attention(s["q"], s["k"], s["v"], s["cu"], **kw)
    kda.window_cache_write(s["k"], s["v"], s["cu"], s["k_cache"], s["v_cache"], s["slots"], sinks=c["sinks"])
    return o, lse, s["k_cache"], s["v_cache"]


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def _pairs(T, W, S):
    """Visible pairs of a sequence of T tokens."""
    m = min(T, W)
    near = m * (m + 1) // 2 + (T - m) * W
    far = T - W  # token i sees min(S, i + 1 - W) sinks behind its window
    if far <= 0:
        return near
    n = min(far, S)
    return near + n * (n + 1) // 2 + (far - n) * S


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op.startswith("axes"):
        n, rows, back = case["tokens"], case["tokens"] * (case["hq"] + case["hk"]), op == "axes_bwd"
        table = min(n, case["max_pos"]) * 2 * sum(_sections(case)) * 4 + n * 4 * len(_sections(case))
        return {"bytes": rows * case["d"] * es * (3 if back else 2) + table, "flops": rows * case["d"] * (16 if back else 8)}
    if op.startswith("gated"):
        n = case["tokens"] * case["h"] * case["d"]
        return {"bytes": n * es * (5 if op == "gated_bwd" else 3), "flops": n * (20 if op == "gated_bwd" else 10)}
    if op.startswith("residual"):
        n, st = case["tokens"] * case["D"], DT[case["stream"]].itemsize
        if op == "residual":
            return {"bytes": n * 2 * (st + es), "flops": n * 8}
        reads_branch = case["post"] or case["channel"]
        return {"bytes": n * (3 * st + (3 if reads_branch else 2) * es), "flops": n * 20}
    hq, hk, d, W, S = case["hq"], case["hk"], case["d"], case["window"], case["sinks"]
    if op == "decode":
        n = sum(min(p + 1, W + S) for p in _positions(case))
        return {"bytes": 2 * n * hk * d * es + case["N"] * (2 * hq + 4 * hk) * d * es, "flops": 4 * n * hq * d}
    if op == "packed":
        lens = _lengths(case)
        tokens, pairs = case["tokens"], sum(_pairs(m, W, S) for m in lens)
        kept = sum(min(m, W + S) for m in lens)
        return {"bytes": tokens * ((2 * hq + 2 * hk) * d * es + 4 * hq) + 2 * kept * hk * d * es, "flops": 4 * pairs * hq * d}
    tokens, pairs = case["B"] * case["T"], case["B"] * _pairs(case["T"], W, S)
    if op == "window":
        return {"bytes": tokens * ((2 * hq + 2 * hk) * d * es + 4 * hq), "flops": 4 * pairs * hq * d}
    return {"bytes": tokens * ((4 * hq + 4 * hk) * d * es + 4 * hq), "flops": 10 * pairs * hq * d}


# ------------------------------------------------------------------ 64 bits, from the definitions
def _x_norm(x, norm):
    if norm == "none":
        return x
    den = x.pow(2).mean(-1, keepdim=True) if norm == "rms" else x.pow(2).sum(-1, keepdim=True)
    return x / (den + EPS).sqrt()


def _leaf(x):
    return None if x is None else x.double().requires_grad_()


def _grad(x):
    return None if x is None else x.grad


def _exact_axes(s, case):
    """Each pair of channels as a complex number times e^{i angle}; gradients by torch's reverse mode."""
    pairs = len(s["pair_axis"])
    turn = torch.empty(case["tokens"], pairs, dtype=torch.complex128, device="cuda")
    for i, a in enumerate(s["pair_axis"]):
        row = s["table"][s["positions"][a].long()].double()
        turn[:, i] = torch.complex(row[:, i], row[:, pairs + i])
    turn = turn[:, None]

    def forward(x, w):
        y = _x_norm(x, case["norm"])
        y = y if w is None else y * w
        a = y[..., :2 * pairs]
        if case["layout"] == "half":
            z = torch.complex(a[..., :pairs].contiguous(), a[..., pairs:].contiguous()) * turn
            a = torch.cat([z.real, z.imag], -1)
        else:
            a = torch.view_as_real(torch.complex(a[..., 0::2].contiguous(), a[..., 1::2].contiguous()) * turn).flatten(-2)
        return torch.cat([a, y[..., 2 * pairs:]], -1)

    if case["op"] == "axes":
        return tuple(forward(x.double(), None if w is None else w.double()) for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])))
    out = []
    for x, w, dy in ((s["q"], s["wq"], s["dyq"]), (s["k"], s["wk"], s["dyk"])):
        x, w = _leaf(x), _leaf(w)
        forward(x, w).backward(dy.double())
        out.append((x.grad, _grad(w)))
    return {"dq": out[0][0], "dk": out[1][0], "dq_weight": out[0][1], "dk_weight": out[1][1]}


def _exact_gated(s, case):
    x, g, w = _leaf(s["x"]), _leaf(s["gate"]), _leaf(s["w"])
    y = _x_norm(x, case["norm"]) * (torch.sigmoid(g) if case["act"] == "sigmoid" else torch.nn.functional.silu(g))
    y = y if w is None else y * w
    if case["op"] == "gated":
        return y.detach()
    y.backward(s["dy"].double())
    return {"dx": x.grad, "dgate": g.grad, "dweight": _grad(w)}


def _exact_residual(s, case):
    b, w, wb, c = (_leaf(s[n]) for n in ("branch", "w", "wb", "c"))
    u = b if wb is None else _x_norm(b, "rms") * wb
    add = s["scale"] * (u if c is None else u * c)
    if case["op"] == "residual":
        h = s["x"].double() + add
        return h.detach(), (_x_norm(h, "rms") * w).detach()
    # the stored sum is the input; what flows into it goes on to the residual and, through the sum, to the branch
    h = s["h"].double().requires_grad_()
    (_x_norm(h, "rms") * w).backward(s["dy"].double())
    g = h.grad + s["dh"].double()
    add.backward(g)
    out = {"d_residual": g, "dweight": w.grad, "d_branch": b.grad}
    if wb is not None:
        out["dbranch_weight"] = wb.grad
    if c is not None:
        out["dchannel_scale"] = c.grad
    return out


def _exact_rows(q, k, v, case, scale, i0, i1):
    """Rows i0 .. i1 of one sequence in 64 bits: softmax over the keys that any of them sees."""
    T, Hq, d = q.shape
    G = Hq // k.shape[1]
    keys = sorted(set(range(min(case["sinks"], i1))) | set(range(max(0, i0 - case["window"] + 1), i1)))
    j = torch.tensor(keys, device=q.device)
    i = torch.arange(i0, i1, device=q.device)
    hidden = (j[None] > i[:, None]) | ((i[:, None] - j[None] >= case["window"]) & (j[None] >= case["sinks"]))
    kk, vv = k[j].repeat_interleave(G, 1), v[j].repeat_interleave(G, 1)
    s = torch.einsum("ihd,jhd->hij", q[i0:i1], kk) * scale
    s = s.masked_fill(hidden, -math.inf)
    return torch.einsum("hij,jhd->ihd", torch.softmax(s, -1), vv), torch.logsumexp(s, -1).t()


def _exact_seq(q, k, v, case, scale):
    q, k, v = q.double(), k.double(), v.double()
    C = max(64, min(512, (1 << 26) // (q.shape[1] * (min(case["window"], q.shape[0]) + 512))))
    parts = [_exact_rows(q, k, v, case, scale, i, min(q.shape[0], i + C)) for i in range(0, q.shape[0], C)]
    return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])


def _exact_window_bwd(s, case):
    """The gradient of sum <do, o> through the softmax. o and lse came rounded; that is not part of the definition."""
    out = {n: torch.empty(s[n[1]].shape, dtype=torch.float64, device="cuda") for n in ("dq", "dk", "dv")}
    for b in range(case["B"]):
        q, k, v = (_leaf(s[n][b]) for n in ("q", "k", "v"))
        C = max(64, min(512, (1 << 26) // (case["hq"] * (min(case["window"], case["T"]) + 512))))
        for i in range(0, case["T"], C):
            o, _ = _exact_rows(q, k, v, case, s["scale"], i, min(case["T"], i + C))
            o.backward(s["do"][b, i:i + C].double())
        out["dq"][b], out["dk"][b], out["dv"][b] = q.grad, k.grad, v.grad
    return out


def _exact_decode(s, case):
    W, S, G = case["window"], case["sinks"], case["hq"] // case["hk"]
    kc, vc = s["k_cache"].clone(), s["v_cache"].clone()
    o = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    for n, (p, slot) in enumerate(zip(s["positions"].tolist(), s["slots"].tolist())):
        kc[slot, p if p < S else S + (p - S) % W] = s["k"][n]
        vc[slot, p if p < S else S + (p - S) % W] = s["v"][n]
        m = min(p + 1, W + S)
        kk, vv = (x[slot, :m].double().repeat_interleave(G, 1) for x in (kc, vc))
        a = torch.softmax(torch.einsum("hd,jhd->hj", s["q"][n].double(), kk) * s["scale"], -1)
        o[n] = torch.einsum("hj,jhd->hd", a, vv)
    return o, kc.double(), vc.double()


def _exact_cache(s, case):
    W, S = case["window"], case["sinks"]
    kc, vc, a = s["k_cache"].clone(), s["v_cache"].clone(), 0
    for m, slot in zip(s["lens"], s["slots"].tolist()):
        for e in (range(0, min(S, m)), range(max(min(S, m), m - W), m)):
            at = torch.tensor([p if p < S else S + (p - S) % W for p in e], dtype=torch.long, device="cuda")
            kc[slot, at], vc[slot, at] = s["k"][a + e.start:a + e.stop], s["v"][a + e.start:a + e.stop]
        a += m
    return kc.double(), vc.double()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("axes"):
        return _exact_axes(s, case)
    if op.startswith("gated"):
        return _exact_gated(s, case)
    if op.startswith("residual"):
        return _exact_residual(s, case)
    if op == "window_bwd":
        return _exact_window_bwd(s, case)
    if op == "decode":
        return _exact_decode(s, case)
    if op == "window":
        rows = [_exact_seq(s["q"][b], s["k"][b], s["v"][b], case, s["scale"]) for b in range(case["B"])]
        return torch.stack([r[0] for r in rows]), torch.stack([r[1] for r in rows])
    at = torch.tensor([0] + s["lens"]).cumsum(0).tolist()
    rows = [_exact_seq(s["q"][a:b], s["k"][a:b], s["v"][a:b], case, s["scale"]) for a, b in zip(at, at[1:]) if b > a]
    return (torch.cat([r[0] for r in rows]), torch.cat([r[1] for r in rows]), *_exact_cache(s, case))
