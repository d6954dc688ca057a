"""Batches without rows through the operator classes, with torch's empty tensors (null addresses)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_grouped_moe_gb300 import build
    build.build()
    from mixture_experts_grouped_moe_gb300 import moe as m
    m.load()
    return m


@pytest.mark.parametrize("E,block_m", [(4, 16), (4, 128), (40, 128)])
def test_no_tokens(moe, E, block_m):
    k, N, K = 2, 256, 128
    new = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    ex = moe.TokenExchange(0, k, E, block_m)
    ex.sort(new(0, k, dt=torch.int32), new(0, k, dt=torch.float32))
    assert int(ex.num_tokens_post_padded) == 0 and int(ex.num_left_out) == 0 and not ex.expert_counts.any()
    assert (ex.sorted_ids == 0).all() and (ex.expert_ids == -1).all()
    w = moe.FP8Weights(torch.ones(E, N, K, dtype=torch.bfloat16, device="cuda"), training=True)
    x = new(0, K)
    assert ex.permute(x).shape == (ex.P, K)
    q, s = ex.permute_fp8(x)
    ys = w.product(q, s, by_block=True, exchange=ex)
    assert ex.unpermute(ys).shape == (0, N)
    dys, dw = ex.unpermute_backward(new(0, N), ys)
    assert dys.shape == ys.shape and dw.shape == (0, k)
    assert ex.permute_backward(q.to(torch.float32)).shape == (0, K)
    if block_m % 128 == 0:
        R = -(-ex.P // 128) * 128
        sid = torch.full((R,), 0, dtype=torch.int32, device="cuda")
        ops = []
        for v in (new(0, N), x):
            C = v.shape[1]
            ops += [torch.full((C, R), 0x7F, dtype=torch.uint8, device="cuda"), new(R // 128, C, dt=torch.float32)]
            moe.moe_quantize_fp8_act_t(v, C, 0, C, sid, 0, k, ex.num_tokens_post_padded, ops[-2], R, ops[-1])
        dW = w.weight_gradient(*ops, exchange=ex, out=torch.full((E, N, K), float("nan"), device="cuda"))
        assert not dW.any()
    assert w.status() == moe.MOE_OK


def test_no_tokens_and_no_rows(moe):
    """Blocks of one and as many experts as slots a token: not even padding."""
    ex = moe.TokenExchange(0, 2, 2, 1)
    assert ex.P == 0
    ex.sort(torch.empty(0, 2, dtype=torch.int32, device="cuda"), torch.empty(0, 2, device="cuda"))
    assert int(ex.num_tokens_post_padded) == 0
    xs = ex.permute(torch.empty(0, 8, device="cuda"))
    assert xs.shape == (0, 8) and ex.unpermute(xs).shape == (0, 8)


def test_dense_product_without_rows(moe):
    N, K = 256, 128
    w = moe.FP8Weights(torch.ones(1, N, K, dtype=torch.bfloat16, device="cuda"))
    q = lambda *s: torch.empty(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    f = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    assert w.product(q(0, K), f(0, 1)).shape == (0, N)
    assert w.product(q(0, K), f(1, 0), by_block=True).shape == (0, N)
    out = torch.full((1, N, K), 2.0, device="cuda")
    w.weight_gradient(q(N, 0), f(0, N), q(K, 0), f(0, K), out=out, accumulate=True)
    assert (out == 2.0).all()
    w.weight_gradient(q(N, 0), f(0, N), q(K, 0), f(0, K), out=out)
    assert not out.any()


@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
def test_norms_without_rows(moe, gate):
    H = 64
    kind = ["none", "channel", "token", "full"].index(gate)
    n = moe.BlockNorm(0, H, kind)
    e = torch.empty(0, H, device="cuda")
    w = torch.ones(H, device="cuda")
    g = (None, torch.ones(H, device="cuda"), torch.empty(0, device="cuda"), e)[kind]
    y, z = n.forward(e, e, w, w, g)
    assert y.shape == z.shape == (0, H)
    out = n.backward(e, e, e, e, w, w, g)
    assert out["dh"].shape == out["d_residual"].shape == (0, H)
    assert not out["dw_post"].any() and not out["dw_pre"].any()
    if gate == "channel":
        assert not out["dgate"].any()
    elif gate != "none":
        assert out["dgate"].numel() == 0
