"""One expert behind an exchange (the others' slots are left out, as on a device that holds one of them):
product and both gradients against 64 bits from the same codes, each to 2^-16 of the sum of an element's
absolute terms and a unit in its last place (see test_gpu_gemm_block.py)."""
import pytest
import torch

import ops_reference as ref

pytestmark = pytest.mark.gpu


def nans(*shape):
    return torch.full(shape, float("nan"), device="cuda")


def bounded(got, want, mag, label):
    err = (got.double() - want).abs()
    assert (err <= 2.0 ** -16 * mag + 2.0 ** -23 * want.abs()).all(), (label, float(err.max()))


@pytest.mark.parametrize("T,block_m", [(200, 128), (300, 256), (9, 16)])
def test_product_and_gradients(T, block_m):
    from mixture_experts_grouped_moe_gb300 import build
    build.build()
    from mixture_experts_grouped_moe_gb300 import moe
    moe.load()
    N, K = 256, 128
    ids = torch.where(torch.rand(T, 1, generator=ref.gen(1)) < 0.6, 0, 1).to(torch.int32).cuda()
    rows = int((ids == 0).sum())
    assert 0 < rows < T
    W = torch.randn(1, N, K, generator=ref.gen(2)).to(torch.bfloat16).cuda()
    x, d = (torch.randn(T, c, generator=ref.gen(c)).to(torch.bfloat16).cuda() for c in (K, N))
    wts = torch.ones(T, 1, device="cuda")
    ex, w = moe.TokenExchange(T, 1, 1, block_m), moe.FP8Weights(W, training=True)
    ex.sort(ids, wts)
    assert int(ex.num_left_out) == T - rows
    used = -(-rows // block_m) * block_m
    wd = w.q[0].cpu().view(torch.float8_e4m3fn).double() * \
        w.s[0].cpu().double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    for v, run, weight, label in ((x, w.product, wd, "product"), (d, w.input_gradient, wd.t(), "input gradient")):
        q, s = ex.permute_fp8(v)
        got = run(q, s, by_block=True, exchange=ex, out=nans(ex.P, weight.shape[0])).cpu()
        a = q.cpu()[:used].view(torch.float8_e4m3fn).double() * s.cpu()[:, :used].t().double().repeat_interleave(128, 1)
        bounded(got[:used], a @ weight.t(), a.abs() @ weight.abs().t(), label)
        assert torch.isnan(got[used:]).all()
    if block_m % 128 == 0:
        R = -(-ex.P // 128) * 128
        sid = torch.full((R,), T, dtype=torch.int32, device="cuda")
        sid[:ex.P] = ex.sorted_ids
        ops = []
        for v in (d, x):
            ops += [torch.full((v.shape[1], R), 0x7F, dtype=torch.uint8, device="cuda"), nans(R // 128, v.shape[1])]
            moe.moe_quantize_fp8_act_t(v, v.shape[1], R, v.shape[1], sid, T, 1, ex.num_tokens_post_padded, ops[-2], R,
                                       ops[-1])
        got = w.weight_gradient(*ops, exchange=ex, out=nans(1, N, K)).cpu()[0]
        D, X = (q.cpu()[:, :used].view(torch.float8_e4m3fn).double() *
                s.cpu()[:used // 128].double().repeat_interleave(128, 0).t() for q, s in (ops[:2], ops[2:]))
        bounded(got, D @ X.t(), D.abs() @ X.abs().t(), "weight gradient")
    assert w.status() == moe.MOE_OK
