"""A linear-attention layer from the operators of this package: served (one
prefill, then token by token on a pool of states) and trained (one step of
gradient descent with the gradients of every operator).

    python examples/linear_attention_layer.py

x [B, T, C] -> q, k, v = x W (one product), norm and rotary positions of q and k,
linear attention with a decay per token and head, y = o W_o. The projections are
library products; the rest are qk_norm_rope, linear_prefill,
linear_decode_step_slots and their gradients.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import kda_gated_delta_chunkwise_gb300 as kda  # noqa: E402


class Layer:
    def __init__(self, channels: int = 256, heads: int = 4, d: int = 128, max_position: int = 4096, device="cuda",
                 dtype=torch.bfloat16, seed: int = 0):
        g = torch.Generator(device).manual_seed(seed)

        def weight(a, b):
            return (torch.randn(a, b, generator=g, device=device) * a ** -0.5).to(dtype)
        self.H, self.d = heads, d
        self.w = weight(channels, 3 * heads * d)
        self.w_o = weight(heads * d, channels)
        self.w_decay = weight(channels, heads).float()
        self.q_norm = torch.ones(d, device=device)
        self.k_norm = torch.ones(d, device=device)
        self.table = kda.rope_table(max_position, d, device=device)

    def project(self, x, positions):
        """q, k with norm and positions, v and the log decays, for x [.., C]."""
        qkv = (x @ self.w).unflatten(-1, (3, self.H, self.d))
        q, k, v = qkv.unbind(-3)  # slices: the operators take them as they are
        log_decay = -torch.nn.functional.softplus(x.float() @ self.w_decay) * 0.05
        qn, kn = kda.qk_norm_rope(q, k, positions, self.table, self.q_norm, self.k_norm, norm="rms")
        return q, k, v, qn, kn, log_decay.contiguous()

    @property
    def scale(self):
        return 1.0 / self.d

    def prefill(self, x):
        """(y, states) for the whole of x [B, T, C]."""
        B, T, _ = x.shape
        pos = torch.arange(T, dtype=torch.int32, device=x.device).expand(B, T).contiguous()
        _, _, v, qn, kn, g = self.project(x, pos)
        o, state = kda.linear_prefill(qn, kn, v, g, scale=self.scale)
        return o.flatten(-2) @ self.w_o, state

    def step(self, x, positions, pool, slots):
        """One token per sequence, x [N, C]; the states in pool[slots] move on in place."""
        _, _, v, qn, kn, g = self.project(x, positions)
        o = kda.linear_decode_step_slots(qn, kn, v, g, pool, slots, scale=self.scale)
        return o.flatten(-2) @ self.w_o

    def loss_and_gradients(self, x, target):
        """Mean square error and its gradients of w and the norms' weights."""
        B, T, _ = x.shape
        pos = torch.arange(T, dtype=torch.int32, device=x.device).expand(B, T).contiguous()
        q, k, v, qn, kn, g = self.project(x, pos)
        o, _ = kda.linear_prefill(qn, kn, v, g, scale=self.scale, output_final_state=False)
        err = (o.flatten(-2) @ self.w_o).float() - target
        d_y = (2.0 / err.numel() * err).to(o.dtype)
        d_o = (d_y @ self.w_o.T).view_as(o)
        a = kda.linear_prefill_backward(qn, kn, v, g, d_o, scale=self.scale, want_initial_state_grad=False)
        n = kda.qk_norm_rope_backward(q, k, a["dq"], a["dk"], pos, self.table, self.q_norm, self.k_norm, norm="rms")
        d_qkv = torch.stack((n["dq"], n["dk"], a["dv"]), -3).flatten(-3)
        d_w = x.flatten(0, 1).T @ d_qkv.flatten(0, 1)
        # the decay: g = -0.05 softplus(x W_g)
        d_pre = a["dlog_decay"] * -0.05 * torch.sigmoid(x.float() @ self.w_decay)
        d_wg = x.float().flatten(0, 1).T @ d_pre.flatten(0, 1)
        return err.square().mean(), {"w": d_w.float(), "w_decay": d_wg, "q_norm": n["dq_weight"],
                                     "k_norm": n["dk_weight"]}


def serve(layer: Layer, B: int = 2, T: int = 300, new: int = 5, seed: int = 1) -> float:
    """Prefill, then `new` tokens on a pool of states; how far their outputs are
    from those of one prefill over all of them (relative, 2-norm)."""
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(B, T + new, layer.w.shape[0], generator=g, device="cuda").to(layer.w.dtype)
    whole, _ = layer.prefill(x)
    _, state = layer.prefill(x[:, :T].contiguous())
    pool = torch.zeros(B + 3, *state.shape[1:], device="cuda")
    slots = torch.arange(B, 0, -1, dtype=torch.int32, device="cuda")  # any slots, in any order
    pool[slots.long()] = state
    got = [layer.step(x[:, t].contiguous(), torch.full((B,), t, dtype=torch.int32, device="cuda"), pool, slots)
           for t in range(T, T + new)]
    ref = whole[:, T:].float()
    return ((torch.stack(got, 1).float() - ref).norm() / ref.norm()).item()


def train(layer: Layer, B: int = 2, T: int = 300, rate: float = 0.05, seed: int = 2) -> tuple[float, float, float]:
    """One step against the gradient; (loss before, the change that the gradient promises, the change)."""
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(B, T, layer.w.shape[0], generator=g, device="cuda").to(layer.w.dtype)
    target = torch.randn(B, T, layer.w_o.shape[1], generator=g, device="cuda") * 0.1
    before, grads = layer.loss_and_gradients(x, target)
    promised = 0.0
    for name, d in grads.items():
        p = getattr(layer, name)
        new = (p.float() - rate * d / d.norm() * p.float().norm()).to(p.dtype)
        promised += ((new.float() - p.float()) * d).sum().item()  # of the step as rounded
        setattr(layer, name, new)
    after, _ = layer.loss_and_gradients(x, target)
    return before.item(), promised, after.item() - before.item()


def main():
    layer = Layer()
    print(f"decode against prefill: rel {serve(layer):.2e}")
    before, promised, change = train(layer, rate=0.005)
    print(f"loss {before:.5f}, a step: promised {promised:+.2e}, came to {change:+.2e}")


if __name__ == "__main__":
    main()
