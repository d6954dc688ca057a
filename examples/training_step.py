"""One training step of a layer with routed experts and a shared one, from hidden states to clipped gradients:

  r = routed experts(x)                          MoETrain: router, top-k, SwiGLU experts, combine
  h = r + shared expert(x)                       GatedFFN, added in its own epilogue
  y = x + scale * h,  z = norm(y)                BlockNorm
  loss = mean cross entropy of z W_head^T        VocabularyLoss, without the logits
  gradients back the same way, then clipped to a norm together    GradientClip

Rows whose target is negative (padding) are left out of the loss.

  python examples/training_step.py [--tokens 4096 --hidden 1024 --inter 2048 --experts 8 --topk 2 --vocab 32000]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mixture_experts_grouped_moe_gb300 import moe  # noqa: E402


class Step:
    """Parameters, workspaces and one training step for a fixed number of tokens."""

    def __init__(self, T, H, I, E, k, V, shared=None, scale=0.5, max_norm=1.0, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        r = lambda *s, std=1.0: (torch.randn(*s, generator=g, device=device) * std).to(torch.bfloat16)  # noqa: E731
        S = shared or I
        self.T, self.V = T, V
        self.w = {"W_router": r(E, H, std=H ** -0.5), "W_gate_up": r(E, 2 * I, H, std=H ** -0.5),
                  "W_down": r(E, H, I, std=I ** -0.5)}
        self.S_gate_up, self.S_down = r(2 * S, H, std=H ** -0.5), r(H, S, std=S ** -0.5)
        self.w_pre, self.W_head = 1 + 0.1 * r(H), r(V, H, std=H ** -0.5)
        self.routed = moe.MoETrain(T, H, I, E, k, device=device)
        self.shared = moe.GatedFFN(T, H, S, moe.MOE_ACT_SILU, training=True, device=device)
        self.norm = moe.BlockNorm(T, H, scale=scale, device=device)
        self.head = moe.VocabularyLoss(T, H, V, training=True, device=device)
        self.clip = moe.GradientClip(max_norm, device=device)
        self.r = torch.empty(T, H, dtype=torch.bfloat16, device=device)

    def forward(self, x, targets):
        """The mean loss of the rows that count (fp32, on the GPU)."""
        self.x, self.targets = x, targets
        self.routed.forward(x, self.w, self.r)
        self.h = self.shared.forward(x, self.S_gate_up, self.S_down, add=self.r)
        _, self.z = self.norm.forward(self.h, x, w_pre=self.w_pre)
        counts = (targets >= 0) & (targets < self.V)
        self.dloss = counts.float() / counts.sum().clamp(min=1)
        return (self.head.forward(self.z, self.W_head, targets) * self.dloss).sum()

    def backward(self):
        """(gradients by name, clipped in place; their norm from before)."""
        g = {}
        head = self.head.backward(self.z, self.W_head, self.targets, self.dloss)
        norm = self.norm.backward(self.h, self.x, None, head["dx"], w_pre=self.w_pre)
        shared = self.shared.backward(self.x, self.S_gate_up, self.S_down, norm["dh"])
        routed = self.routed.backward(self.x, self.w, norm["dh"])
        g["W_head"], g["w_pre"] = head["dW"], norm["dw_pre"]
        g["S_gate_up"], g["S_down"] = shared["dW_gate_up"], shared["dW_down"]
        for n in ("W_router", "W_gate_up", "W_down"):
            g[n] = routed["d" + n]
        total = self.clip.clip(list(g.values()))
        self.dx = norm["d_residual"].float() + shared["dx"].float() + routed["dx"].float()
        return g, total

    def status(self):
        return [o.status() for o in (self.routed, self.shared, self.head)]


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, default in (("tokens", 4096), ("hidden", 1024), ("inter", 2048), ("experts", 8), ("topk", 2),
                          ("vocab", 32000)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    moe.load()
    step = Step(a.tokens, a.hidden, a.inter, a.experts, a.topk, a.vocab)
    x = torch.randn(a.tokens, a.hidden, device="cuda").to(torch.bfloat16)
    targets = torch.randint(0, a.vocab, (a.tokens,), device="cuda", dtype=torch.int32)
    for _ in range(3):
        step.forward(x, targets)
        step.backward()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    loss = step.forward(x, targets)
    g, norm = step.backward()
    end.record()
    torch.cuda.synchronize()
    assert all(s == moe.MOE_OK for s in step.status())
    print(f"one step of {a.tokens} tokens: {start.elapsed_time(end):.3f} ms, loss {loss.item():.4f}, "
          f"gradient norm {norm.item():.4f}")
    for name, v in g.items():
        print(f"  {name:10s} {str(tuple(v.shape)):20s} rms {v.float().square().mean().sqrt():.3e}")


if __name__ == "__main__":
    main()
