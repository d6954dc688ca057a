"""One workspace for batches of every size, and outputs that lie in a buffer with other rows."""
import pytest
import torch

import ops_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_grouped_moe_gb300 import build
    build.build()
    from mixture_experts_grouped_moe_gb300 import moe as m
    m.load()
    return m


@pytest.mark.parametrize("V", [300, 9000, 32000])
def test_workspace_of_the_largest_batch(moe, V):
    """The loss of smaller batches, and their gradients, in the workspace of the largest."""
    most, H, piece = 200, 256, 8192
    g = ref.gen(V)
    w = (torch.randn(V, H, generator=g) * 2 * H ** -0.5).bfloat16().cuda()
    size = moe.moe_vocab_loss_workspace_size(most, H, V, piece)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    for T in (1, 16, 32, 33, 128, 200, 7):
        x = torch.randn(T, H, generator=g).bfloat16().cuda()
        targets = torch.randint(0, V, (T,), generator=g, dtype=torch.int32).cuda()
        dloss = torch.rand(T, generator=g).cuda()
        loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        moe.moe_vocab_loss(moe.MOE_ROW_BF16, x, H, w, targets, T, H, V, loss, lse, ws, size)
        moe.moe_vocab_loss_backward(moe.MOE_ROW_BF16, x, H, w, targets, lse, dloss, T, H, V, piece, dx, H,
                                    moe.MOE_ROW_BF16, 0, dw, ws, size)
        f = moe.VocabularyLoss(T, H, V, training=True, piece=piece)
        assert torch.equal(loss, f.forward(x, w, targets)) and torch.equal(lse, f.lse)
        want = f.backward(x, w, targets, dloss, grad_dtype=torch.bfloat16)
        assert torch.equal(dx, want["dx"]) and torch.equal(dw, want["dW"])
        assert moe.moe_workspace_status(ws) == moe.MOE_OK
