"""The weight gradient of rows that were sorted in blocks larger than 128: a segment's padding then holds
whole blocks of 128.  Against 64 bits from the same codes, to 2^-16 of the sum of an element's absolute
terms and a unit in its last place (see test_gpu_gemm_block.py)."""
import pytest
import torch

import ops_reference as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("block_m", [128, 256, 384])
def test_segments_of_larger_blocks(block_m):
    from mixture_experts_grouped_moe_gb300 import build
    build.build()
    from mixture_experts_grouped_moe_gb300 import moe
    moe.load()
    N, K = 128, 256
    counts = [100, 0, 129, 1, 300, 50]  # tokens of each expert
    E, T = len(counts), sum(counts)
    ids = torch.cat([torch.full((c,), e) for e, c in enumerate(counts)])[torch.randperm(T, generator=ref.gen(1))]
    ids = ids.to(torch.int32).view(T, 1)
    idd, wd = ids.cuda(), torch.ones(T, 1, device="cuda")
    x, d = (torch.randn(T, c, generator=ref.gen(c)).to(torch.bfloat16).cuda() for c in (K, N))
    w = moe.FP8Weights(torch.zeros(E, N, K, dtype=torch.bfloat16, device="cuda"))
    side = torch.cuda.Stream()
    for stream in (None, side):
        if stream is not None:
            side.wait_stream(torch.cuda.current_stream())
        ex = moe.TokenExchange(T, 1, E, block_m)
        side.wait_stream(torch.cuda.current_stream())
        ex.sort(idd, wd, stream=stream)
        R = -(-ex.P // 128) * 128
        p = ref.sort(ids, E, block_m)
        sid = torch.full((R,), T, dtype=torch.int32)
        sid[:p["P"]] = p["sorted_ids"]
        sidd = sid.cuda()
        side.wait_stream(torch.cuda.current_stream())
        ops = []
        for v in (d, x):
            q = torch.full((v.shape[1], R), 0x7F, dtype=torch.uint8, device="cuda")
            s = torch.full((R // 128, v.shape[1]), float("nan"), device="cuda")
            side.wait_stream(torch.cuda.current_stream())
            moe.moe_quantize_fp8_act_t(v, v.shape[1], R, v.shape[1], sidd, T, 1, ex.num_tokens_post_padded, q, R, s,
                                       stream)
            ops += [q, s]
        got = w.weight_gradient(*ops, exchange=ex, stream=stream)
        torch.cuda.synchronize()
        rows = p["rows"]
        deq = lambda q, s: (q[:, :rows].cpu().view(torch.float8_e4m3fn).double() *  # noqa: E731
                            s[:rows // 128].cpu().double().repeat_interleave(128, 0).t())
        D, X = deq(*ops[:2]), deq(*ops[2:])
        expert = p["expert_ids"].long().repeat_interleave(block_m)[:rows]
        for e in range(E):
            r = (expert == e).nonzero()[:, 0]
            want, mag = D[:, r] @ X[:, r].t(), D[:, r].abs() @ X[:, r].abs().t()
            err = (got[e].cpu().double() - want).abs()
            assert (err <= 2.0 ** -16 * mag + 2.0 ** -23 * want.abs()).all(), (e, float(err.max()))
            assert want.any() == (counts[e] > 0)
        assert w.status() == moe.MOE_OK
