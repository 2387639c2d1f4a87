"""Training steps of a residual block whose experts are bf16 matrices.

    python examples/train_experts.py [--tokens T] [--steps N]

The block:  x = norm(s0);  y = experts(x), routed by the fp32 logits of a router;  s1 = s0 + scale silu(gate) norm(y), which
moe_gated_norm computes with the next norm.  Its loss is the mean squared distance of s1's norm from a target.  Every step
runs the framework's forward and backward passes and updates the matrices in fp32; the router is fixed.  Synthetic tokens,
target and weights.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import quantised_moe_expert_gb300 as qm  # noqa: E402

EPS = 1e-6


class Block:
    """fp32 parameters of the block (names as in `params`) and their bf16 copies, which the kernels read."""

    def __init__(self, hidden, inter, n_experts, top_k, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        rnd = lambda *s, size=1.0: size * torch.randn(s, generator=g, device=device)
        G = n_experts + 1                                            # a shared expert, last
        self.shape = (hidden, inter, n_experts, top_k)
        self.params = {"gate": rnd(G, inter, hidden, size=hidden ** -0.5), "up": rnd(G, inter, hidden, size=hidden ** -0.5),
                       "down": rnd(G, hidden, inter, size=inter ** -0.5), "channel_gate": rnd(hidden),
                       "norm_in": 1 + rnd(hidden, size=0.1), "norm_post": 1 + rnd(hidden, size=0.1), "norm_out": 1 + rnd(hidden, size=0.1)}
        self.router = rnd(hidden, n_experts, size=hidden ** -0.5)
        self.shared_gate = rnd(hidden, size=hidden ** -0.5)
        self.scale = 0.5
        self.cast()

    def cast(self):
        self.w = {k: v.bfloat16() for k, v in self.params.items()}
        self.experts = qm.Experts16(self.w["gate"], self.w["up"], self.w["down"], self.shape[3], True)

    def route(self, x):
        """Picks of the tokens x: the arguments of Experts16 (a router of the user's own)."""
        T, (_, _, E, k) = x.shape[0], self.shape
        top = (x.float() @ self.router).topk(k, dim=1)
        order = torch.argsort(top.indices.reshape(-1), stable=True)
        inv = torch.empty_like(order)
        inv[order] = torch.arange(T * k, device=x.device)
        offsets = torch.zeros(E + 1, dtype=torch.int32, device=x.device)
        offsets[1:] = torch.bincount(top.indices.reshape(-1), minlength=E).cumsum(0)
        return inv.int(), offsets, torch.softmax(top.values, 1).bfloat16().contiguous(), torch.sigmoid(x.float() @ self.shared_gate).bfloat16()

    def forward(self, s0, ws):
        T, H = s0.shape
        w, new = self.w, lambda: torch.empty(T, H, dtype=torch.bfloat16, device=s0.device)
        x, s1, out = new(), new(), new()
        qm.moe_gated_norm(s0, None, None, qm.MOE_GATE_NONE, qm.MOE_ACT_NONE, 1.0, 0, None, w["norm_in"], 0.0, EPS, T, H, None, x)
        routing = self.route(x)
        y, kept = self.experts.forward(x, *routing, ws, keep=True)
        qm.moe_gated_norm(y, s0, w["channel_gate"], qm.MOE_GATE_CHANNEL, qm.MOE_ACT_SILU, self.scale, 1, w["norm_post"], w["norm_out"], 0.0,
                          EPS, T, H, s1, out)
        return out, (s0, y, s1, kept)

    def backward(self, dout, saved, ws):
        """Gradients of s0 (without the router's way) and of every parameter."""
        s0, y, s1, kept = saved
        T, H = s0.shape
        w, dev = self.w, s0.device
        f32, new = lambda n: torch.empty(n, device=dev), lambda: torch.empty(T, H, dtype=torch.bfloat16, device=dev)
        grads = {k: f32(H) for k in ("channel_gate", "norm_in", "norm_post", "norm_out")}
        grads |= {k: torch.empty_like(self.params[k]) for k in ("gate", "up", "down")}
        dy, ds = new(), new()
        qm.moe_gated_norm_grad(y, s1, w["channel_gate"], qm.MOE_GATE_CHANNEL, qm.MOE_ACT_SILU, self.scale, 1, w["norm_post"], w["norm_out"],
                               0.0, EPS, T, H, dout, None, dy, ds, grads["channel_gate"], grads["norm_post"], grads["norm_out"], ws)
        dx = self.experts.backward(dy, kept, ws, dgate=grads["gate"], dup=grads["up"], ddown=grads["down"])[0]
        ds0 = new()
        # the norm's way back to s0 and the residual's, in one sum
        qm.moe_gated_norm_grad(s0, s0, None, qm.MOE_GATE_NONE, qm.MOE_ACT_NONE, 1.0, 0, None, w["norm_in"], 0.0, EPS, T, H, dx, ds, ds0, None,
                               None, None, grads["norm_in"], ws)
        return ds0, grads


def workspace(tokens, hidden, device="cuda"):
    return torch.zeros(qm.moe_gated_norm_workspace_size(tokens, hidden), dtype=torch.uint8, device=device)


def run(tokens=512, steps=5, hidden=1024, inter=256, n_experts=32, top_k=4, lr=0.5, seed=0):
    """Losses of the steps."""
    block, ws = Block(hidden, inter, n_experts, top_k, seed), workspace(tokens, hidden)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    s0 = torch.randn(tokens, hidden, generator=g, device="cuda").bfloat16()
    target = torch.randn(tokens, hidden, generator=g, device="cuda")
    losses = []
    for _ in range(steps):
        out, saved = block.forward(s0, ws)
        d = out.float() - target
        losses.append(float(d.square().mean()))
        _, grads = block.backward((d * (2 / tokens)).bfloat16(), saved, ws)
        for k, v in grads.items():
            block.params[k] -= lr / hidden * v
        block.cast()
    assert qm.moe_get_device_status(ws) == 0
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--steps", type=int, default=5)
    a = ap.parse_args()
    for i, loss in enumerate(run(a.tokens, a.steps)):
        print(f"step {i}: mean squared distance {loss:.4f}")


if __name__ == "__main__":
    main()
