"""One MoE block trained in FP8 with experts of the caller's own: squared-ReLU MLPs, which the fused
layer (SwiGLU) does not cover, built from the operators around it.

  x --router--> ids, weights;  x --sort, permute to FP8--> W1 --relu^2--> W2 --unpermute with weights--> h
  y = residual + scale * gate * norm(h),  z = norm(y): the next block's input

The backward goes the same way back: the norms, the exchange (its gradient gives the router's), both
products' input gradients and, from transposed quantised rows, both weight gradients.  Every step is a
call of the library but the activation and the router's softmax, which are the caller's here.

  python examples/moe_block.py [--tokens 4096 --hidden 1024 --inter 2048 --experts 8 --topk 2]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mixture_experts_grouped_moe_gb300 import moe  # noqa: E402


class SquaredReluBlock:
    """Parameters, workspaces and one training step of the block for a fixed number of tokens."""

    def __init__(self, T, H, I, E, k, scale=0.5, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        r = lambda *s, std=1.0: (torch.randn(*s, generator=g, device=device) * std).to(torch.bfloat16)  # noqa: E731
        self.T, self.H, self.I, self.E, self.k = T, H, I, E, k
        self.W_router = r(E, H, std=H ** -0.5)
        self.W1, self.W2 = r(E, I, H, std=H ** -0.5), r(E, H, I, std=I ** -0.5)
        self.w_post, self.w_pre, self.gate = (1 + 0.1 * r(H) for _ in range(3))
        self.p1, self.p2 = moe.FP8Weights(self.W1, training=True), moe.FP8Weights(self.W2, training=True)
        self.norm = moe.BlockNorm(T, H, moe.MOE_GATE_CHANNEL, scale, device=device)
        # the weight gradients' 128-token blocks need whole blocks of 128 rows per expert
        self.ex = moe.TokenExchange(T, k, E, block_m=128, device=device)
        P = self.ex.P
        self.rows = -(-P // 128) * 128  # rows of the transposed operands
        zeros = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device=device)  # noqa: E731
        self.ids, self.wts = zeros(T, k, dt=torch.int32), zeros(T, k, dt=torch.float32)
        self.logits = zeros(T, E, dt=torch.float32)
        self.sorted_rows = torch.full((self.rows,), T * k, dtype=torch.int32, device=device)
        # sorted rows past the used ones are never written: zeros once, so that what the activation
        # makes of them stays finite
        self.up, self.ys = zeros(P, I), zeros(P, H)
        self.dact, self.dxs = zeros(P, I), zeros(P, H)

    def _by_rows(self, v):
        """Rows as FP8 codes with a scale per 1x128 group."""
        q = torch.empty(v.shape, dtype=torch.uint8, device=v.device)
        s = torch.empty(v.shape[0], v.shape[1] // 128, dtype=torch.float32, device=v.device)
        moe.moe_quantize_fp8_act(v, v.shape[0], v.shape[1], q, s)
        return q, s

    def _by_columns(self, v, gather=False):
        """Sorted rows (gather: tokens' rows in sorted order) as transposed FP8 codes, scales per 128 rows."""
        C = v.shape[1]
        q = torch.zeros(C, self.rows, dtype=torch.uint8, device=v.device)
        s = torch.zeros(self.rows // 128, C, dtype=torch.float32, device=v.device)
        ex = self.ex
        R = self.rows if gather else v.shape[0]
        moe.moe_quantize_fp8_act_t(v, C, R, C, self.sorted_rows if gather else None, self.T * self.k, self.k,
                                   ex.num_tokens_post_padded, q, self.rows, s)
        return q, s

    def forward(self, x, residual):
        ex = self.ex
        moe.moe_route_topk(x, self.W_router, None, self.T, self.H, self.E, self.k, self.ids, self.wts, self.logits)
        ex.sort(self.ids, self.wts)
        q, s = ex.permute_fp8(x)
        self.p1.product(q, s, by_block=True, exchange=ex, out=self.up)
        self.act = torch.relu(self.up).square()
        self.p2.product(*self._by_rows(self.act), exchange=ex, out=self.ys)
        self.h = ex.unpermute(self.ys)
        self.x, self.residual = x, residual
        return self.norm.forward(self.h, residual, self.w_post, self.w_pre, self.gate)

    def backward(self, dy, dz):
        """Gradients of loss = sum(dy * y) + sum(dz * z)."""
        ex = self.ex
        g = self.norm.backward(self.h, self.residual, dy, dz, self.w_post, self.w_pre, self.gate)
        dys, dw = ex.unpermute_backward(g.pop("dh"), self.ys)
        self.p2.input_gradient(*self._by_rows(dys), exchange=ex, out=self.dact)
        g["dW2"] = self.p2.weight_gradient(*self._by_columns(dys), *self._by_columns(self.act), exchange=ex)
        dup = self.dact * (2 * torch.relu(self.up))
        self.p1.input_gradient(*self._by_rows(dup), exchange=ex, out=self.dxs)
        self.sorted_rows[:ex.P] = ex.sorted_ids
        g["dW1"] = self.p1.weight_gradient(*self._by_columns(dup), *self._by_columns(self.x, gather=True), exchange=ex)
        dx = ex.permute_backward(self.dxs)
        # the router: softmax over the chosen logits, which the weights came from
        dl = self.wts * (dw - (self.wts * dw).sum(1, keepdim=True))
        dlogit = torch.zeros_like(self.logits).scatter_(1, self.ids.long(), dl)
        g["dW_router"] = dlogit.t() @ self.x.float()
        g["dx"] = (dx.float() + dlogit @ self.W_router.float()).to(dx.dtype)
        return g


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, default in (("tokens", 4096), ("hidden", 1024), ("inter", 2048), ("experts", 8), ("topk", 2)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    moe.load()
    b = SquaredReluBlock(a.tokens, a.hidden, a.inter, a.experts, a.topk)
    x, residual, dy, dz = (torch.randn(a.tokens, a.hidden, device="cuda").to(torch.bfloat16) for _ in range(4))
    for _ in range(3):
        b.forward(x, residual)
        b.backward(dy, dz)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    y, z = b.forward(x, residual)
    g = b.backward(dy, dz)
    end.record()
    torch.cuda.synchronize()
    assert b.p1.status() == moe.MOE_OK and b.p2.status() == moe.MOE_OK
    print(f"forward and backward of {a.tokens} tokens: {start.elapsed_time(end):.3f} ms")
    for name, v in {"y": y, "z": z, **g}.items():
        if v is not None:
            print(f"  {name:10s} {str(tuple(v.shape)):20s} rms {v.float().square().mean().sqrt():.4f}")


if __name__ == "__main__":
    main()
