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


@pytest.mark.parametrize("T", [1, 5, 300])
@pytest.mark.parametrize("ld_add,ld_out,start", [(256, 256, 128), (256, 256, 136), (256, 256, -128), (128, 128, 0),
                                                 (512, 256, 256), (136, 264, -1), (256, 256, 256 * 4 + 120)])
def test_ffn_output_beside_add(moe, T, ld_add, ld_out, start):
    """add and out as rows of one buffer, `start` elements apart: between each other's rows they are computed as if
    apart, the same rows too, and anything else in common is refused before a launch."""
    H, I = 120, 64
    start = -ld_out * T if start == -1 else start
    g = ref.gen(T)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).bfloat16().cuda()  # noqa: E731
    x, wgu, wd = r(T, H), r(2 * I, H, std=H ** -0.5), r(H, I, std=I ** -0.5)
    buf = r(max(0, -start) + T * (ld_add + ld_out) + max(0, start) + H)
    at = max(0, -start)
    add = torch.as_strided(buf, (T, H), (ld_add, 1), at)
    out = torch.as_strided(buf, (T, H), (ld_out, 1), at + start)
    places = lambda t, ld: {t.storage_offset() + i * ld + j for i in range(T) for j in range(H)}  # noqa: E731
    common = places(add, ld_add) & places(out, ld_out)
    f = moe.GatedFFN(T, H, I)
    if common and start != 0:
        before = buf.clone()
        with pytest.raises(moe.MoEError):
            f.forward(x, wgu, wd, add, out=out)
        torch.cuda.synchronize()
        assert torch.equal(buf, before)
        return
    want = f.forward(x, wgu, wd, add.clone())
    kept = torch.ones_like(buf, dtype=torch.bool)
    torch.as_strided(kept, (T, H), (ld_out, 1), at + start).fill_(False)
    before = buf.clone()
    f.forward(x, wgu, wd, add, out=out)
    assert torch.equal(out, want) and torch.equal(buf[kept], before[kept])
