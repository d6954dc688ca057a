"""Grouped products with a row count that ends inside a block: rows from it on stay as they are."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("block_m", [16, 64, 128, 256])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("N,K", [(128, 128), (129, 1024), (2048, 256), (20000, 128)])
def test_rows_past_the_count(block_m, out, N, K):
    from mixture_experts_grouped_moe_gb300 import build
    build.build()
    from mixture_experts_grouped_moe_gb300 import moe
    moe.load()
    M, used = 512, 300
    KB = K // 128
    a = torch.full((M, K), 0x38, dtype=torch.uint8, device="cuda")  # 1 in e4m3
    b = torch.full((N, K), 0x38, dtype=torch.uint8, device="cuda")
    sa, sb = torch.ones(M, KB, device="cuda"), torch.ones(-(-N // 128), KB, device="cuda")
    npp = torch.tensor([used], dtype=torch.int32, device="cuda")
    eid = torch.zeros(M // block_m, dtype=torch.int32, device="cuda")
    ws = torch.zeros(moe.MOE_GEMM_BLOCK_WS_BYTES, dtype=torch.uint8, device="cuda")
    dt, t = (torch.bfloat16, moe.MOE_ROW_BF16) if out == "bf16" else (torch.float32, moe.MOE_ROW_FP32)
    for ld in (N, N + 3):
        d = torch.full((M, ld), 3.0, dtype=dt, device="cuda")
        moe.moe_gemm_fp8_block(a, sa, 0, b, sb, M, N, K, 1, block_m, eid, npp, t, d, ld, ws, ws.numel())
        assert (d[:used, :N] == K).all()
        assert (d[used:] == 3.0).all() and (d[:, N:] == 3.0).all()
    assert moe.moe_workspace_status(ws) == moe.MOE_OK
