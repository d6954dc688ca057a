"""The example block (examples/moe_block.py: router, exchange, FP8 products, norms, and all gradients)
against the same block in 64 bits.

Tolerances, derived: an e4m3 code is off by at most 2^-4 of its value, about 2.6 % in the root mean
square; a product of two quantised factors by about 3.7 % of its own root mean square, errors of the
elements being independent.  The forward chains two such products (5.3 %) and halves by the gate and
scale; a gradient of the first weights chains three and one factor squared's slope (about 8 %).  15 %
relative L2 norm leaves a factor of two; a wrong layout, index or scale gives 100 %.
"""
import os
import sys

import pytest
import torch

import ops_reference as ref

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("T,H,I,E,k", [(300, 256, 384, 5, 2), (64, 128, 256, 16, 3)])
def test_block_forward_and_gradients(T, H, I, E, k):
    from mixture_experts_grouped_moe_gb300 import build
    build.build()
    from mixture_experts_grouped_moe_gb300 import moe
    moe.load()
    from moe_block import SquaredReluBlock
    b = SquaredReluBlock(T, H, I, E, k, scale=0.5, seed=1)
    x, res, dy, dz = ((torch.randn(T, H, generator=ref.gen(i))).to(torch.bfloat16).cuda() for i in range(4))
    y, z = b.forward(x, res)
    g = b.backward(dy, dz)
    assert b.p1.status() == moe.MOE_OK and b.p2.status() == moe.MOE_OK

    d = lambda t: t.detach().double().cpu().requires_grad_(True)  # noqa: E731
    X, R, W1, W2, Wr, wo, wi, ga = (d(t) for t in (x, res, b.W1, b.W2, b.W_router, b.w_post, b.w_pre, b.gate))
    ids = b.ids.cpu().long()
    wts = torch.softmax((X @ Wr.t()).gather(1, ids), 1)
    h = 0
    for j in range(k):
        up = torch.einsum("th,tih->ti", X, W1[ids[:, j]])
        h = h + wts[:, j:j + 1] * torch.einsum("ti,thi->th", torch.relu(up).square(), W2[ids[:, j]])
    Y, Z, _, _ = ref.block_norm(h, R, ga, wo, wi, 0.5, 0.0, 1e-6)
    ((Y * dy.double().cpu()).sum() + (Z * dz.double().cpu()).sum()).backward()
    pairs = {"y": (y, Y), "z": (z, Z), "d_residual": (g["d_residual"], R.grad), "dgate": (g["dgate"], ga.grad),
             "dw_post": (g["dw_post"], wo.grad), "dw_pre": (g["dw_pre"], wi.grad), "dW1": (g["dW1"], W1.grad),
             "dW2": (g["dW2"], W2.grad), "dx": (g["dx"], X.grad), "dW_router": (g["dW_router"], Wr.grad)}
    for name, (got, want) in pairs.items():
        got, want = got.double().cpu(), want.detach()
        err = float((got - want).norm() / want.norm())
        print(f"{name}: relL2 {err:.3f}")
        assert err <= 0.15, (name, err)
    for e in set(range(E)) - set(ids.reshape(-1).tolist()):
        assert not g["dW1"][e].any() and not g["dW2"][e].any()


def test_classes_refuse_wrong_shapes():
    from mixture_experts_grouped_moe_gb300 import moe
    moe.load()
    ex = moe.TokenExchange(8, 2, 4, 16)
    with pytest.raises(ValueError):
        ex.permute(torch.zeros(7, 64, device="cuda"))
    with pytest.raises(ValueError):
        ex.unpermute(torch.zeros(ex.P + 1, 64, device="cuda"))
    with pytest.raises(TypeError):
        ex.permute_fp8(torch.zeros(8, 128, device="cuda"))
    w = moe.FP8Weights(torch.zeros(2, 128, 128, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):  # two experts need the exchange
        w.product(torch.zeros(8, 128, dtype=torch.uint8, device="cuda"), torch.ones(8, 1, device="cuda"))
    n = moe.BlockNorm(4, 64)
    with pytest.raises(ValueError):
        n.forward(torch.zeros(4, 32, device="cuda"), torch.zeros(4, 32, device="cuda"))


def test_streams_given_to_the_classes():
    """Outputs that the classes make for a stream are that stream's own, and a strided or single row works."""
    from mixture_experts_grouped_moe_gb300 import moe
    moe.load()
    T, H, k, E = 333, 256, 2, 8
    ids, wts = ref.route(T, E, k, seed=7)
    x = torch.randn(T, 2 * H, device="cuda", generator=torch.Generator("cuda").manual_seed(1))[:, :H]
    st = torch.cuda.Stream()
    ex = moe.TokenExchange(T, k, E, 64)
    i, w = ids.cuda(), wts.cuda()
    st.wait_stream(torch.cuda.current_stream())
    for stream in (st, st.cuda_stream):
        ex.sort(i, w, stream=stream)
        back = ex.unpermute(ex.permute(x, stream=stream), stream=stream)
        n = moe.BlockNorm(T, H)
        y, _ = n.forward(back, back, stream=stream)
        st.synchronize()
        assert (back - x).abs().max() <= 4 * 2.0 ** -24 * x.abs().max()
        assert torch.equal(y, back + back)
    one = moe.TokenExchange(1, 1, 2, 16)
    one.sort(torch.ones(1, 1, dtype=torch.int32, device="cuda"), torch.ones(1, 1, device="cuda"))
    r = x[:1]
    assert torch.equal(one.unpermute(one.permute(r)), r)
