"""The operators of a training step together (examples/training_step.py: routed and shared experts, norm, loss,
clipping) against the same step in 64 bits.

Tolerances, derived: between the inputs and a gradient lie about a dozen roundings to bf16 (h of the experts, their
rows, the sum, z; dl, dz, dh, gate | up, their gradients), each a relative 2^-9 at most, 2^-9 / sqrt(3) in the root mean
square, and independent: 4e-3.  A logit of size 2 that is off by 2^-8 of its size moves its probability by 0.8 %.
2e-2 of a gradient's 2-norm leaves a factor of two; a wrong layout, index or scale gives 100 %.  The loss is a mean of
logits' differences: 2^-7 absolutely."""
import os
import sys

import pytest
import torch

import ops_reference as ref

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_grouped_moe_gb300 import build
    build.build()
    from mixture_experts_grouped_moe_gb300 import moe as m
    m.load()
    return m


@pytest.mark.parametrize("T,H,I,E,k,V,S", [(200, 256, 256, 4, 2, 1001, 136), (40, 128, 256, 6, 3, 300, 512)])
def test_step(moe, T, H, I, E, k, V, S):
    from training_step import Step
    step = Step(T, H, I, E, k, V, shared=S, max_norm=0.25, seed=1)
    g = ref.gen(2)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    targets = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    targets[::5] = -100
    targets = targets.cuda()
    loss = step.forward(x, targets)
    grads, norm = step.backward()
    assert all(s == moe.MOE_OK for s in step.status())

    d = lambda t: t.detach().double().requires_grad_(True)  # noqa: E731
    X, leaves = d(x), {n: d(v) for n, v in list(step.w.items()) + [
        ("S_gate_up", step.S_gate_up), ("S_down", step.S_down), ("w_pre", step.w_pre), ("W_head", step.W_head)]}
    logits = X @ leaves["W_router"].t()
    # (the framework's own choice of experts: two nearly equal logits may fall either way in 64 bits)
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    moe.moe_route_topk(x, step.w["W_router"], None, T, H, E, k, ids, torch.empty(T, k, device="cuda"),
                       torch.empty(T, E, device="cuda"))
    ids = ids.long()
    wts = torch.softmax(logits.gather(1, ids), 1)
    h = 0
    for j in range(k):
        gu = torch.einsum("th,tih->ti", X, leaves["W_gate_up"][ids[:, j]])
        h = h + wts[:, j:j + 1] * torch.einsum("ti,thi->th", torch.nn.functional.silu(gu[:, :I]) * gu[:, I:],
                                               leaves["W_down"][ids[:, j]])
    gu = X @ leaves["S_gate_up"].t()
    h = h + (torch.nn.functional.silu(gu[:, :S]) * gu[:, S:]) @ leaves["S_down"].t()
    Y = X + 0.5 * h
    Z = Y * torch.rsqrt(Y.pow(2).mean(1, keepdim=True) + 1e-6) * leaves["w_pre"]
    kept = targets >= 0
    want = torch.nn.functional.cross_entropy(Z[kept] @ leaves["W_head"].t(), targets[kept].long())
    want.backward()
    assert abs(float(loss) - float(want.detach())) <= 2.0 ** -7
    total = torch.stack([v.grad.pow(2).sum() for v in leaves.values()]).sum().sqrt()
    assert abs(float(norm) / float(total) - 1) <= 2e-2
    factor = min(1.0, 0.25 / (float(total) + 1e-6))
    assert factor < 1
    for n, v in leaves.items():
        err = float((grads[n].double() - v.grad * factor).norm() / (v.grad * factor).norm())
        assert err <= 2e-2, (n, err)
    err = float((step.dx.double() - X.grad).norm() / X.grad.norm())
    assert err <= 2e-2, ("dx", err)


def test_captured_while_eager_objects_live(moe):
    """A whole step in a CUDA graph, next to another Step that runs eagerly between the replays."""
    from training_step import Step
    T, H, I, E, k, V = 150, 256, 256, 4, 2, 700
    a, b = (Step(T, H, I, E, k, V, seed=3) for _ in range(2))
    g = ref.gen(4)
    xs = [torch.randn(T, H, generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
    ts = [torch.randint(0, V, (T,), generator=g, dtype=torch.int32).cuda() for _ in range(2)]
    x, t = xs[0].clone(), ts[0].clone()
    a.forward(x, t)
    a.backward()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss = a.forward(x, t)
        grads, norm = a.backward()
    for i in (1, 0, 1):
        x.copy_(xs[i])
        t.copy_(ts[i])
        graph.replay()
        want = b.forward(xs[i], ts[i])
        wg, wn = b.backward()
        torch.cuda.synchronize()
        assert torch.equal(loss, want) and torch.equal(norm, wn)
        for n in wg:
            assert torch.equal(grads[n], wg[n]), n
