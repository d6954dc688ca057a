"""Offsets that pass 32 bits in the operators of a training step: kept gate | up, the gradient of the logits and a
tensor to clip of more than 2^31 elements each.  The last rows (which lie behind that) against 64 bits."""
import pytest
import torch

import ops_reference as ref
import training_reference as tr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_grouped_moe_gb300 import build
    build.build()
    from mixture_experts_grouped_moe_gb300 import moe as m
    m.load()
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of free device memory")
    yield m
    torch.cuda.empty_cache()


def rand(*s, std=1.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*s, generator=g, device="cuda") * std).bfloat16()


def test_ffn(moe):
    T, H, I = 140000, 64, 8192
    assert T * 2 * I > 2 ** 31
    x, wgu, wd, dout = rand(T, H, seed=1), rand(2 * I, H, std=H ** -0.5), rand(H, I, std=I ** -0.5), rand(T, H, seed=2)
    f = moe.GatedFFN(T, H, I, training=True)
    out = f.forward(x, wgu, wd)
    n = 300
    d = x[-n:].double(), wgu.double(), wd.double()
    for got, want, bound in zip((f.gu[-n:], f.h[-n:], out[-n:]), tr.ffn(*d, "silu"), tr.ffn_bound(*d, "silu", "bf16")):
        tr.bounded(got, want, bound, "forward")
    g = f.backward(x, wgu, wd, dout)
    want, bound = tr.ffn_grads_bound(*d, "silu", f.gu[-n:].double(), f.h[-n:].double(), dout[-n:].double(), "bf16",
                                     "bf16")
    tr.bounded(g["dx"][-n:], want["dx"], bound["dx"], "dx")
    assert f.status() == moe.MOE_OK
    # the weights' gradients of rows without an output gradient but for the last ones
    dout[:-n] = 0
    g = f.backward(x, wgu, wd, dout)
    want, bound = tr.ffn_grads_bound(*d, "silu", f.gu[-n:].double(), f.h[-n:].double(), dout[-n:].double(), "bf16",
                                     "fp32")
    for name in ("dW_gate_up", "dW_down"):
        tr.bounded(g[name], want[name], bound[name], name)


def test_vocab_loss(moe):
    T, H, V = 140000, 64, 16384
    assert T * V > 2 ** 31
    x, w = rand(T, H, seed=3), rand(V, H, std=2 * H ** -0.5, seed=4)
    g = torch.Generator(device="cuda").manual_seed(5)
    y = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    dl = torch.rand(T, generator=g, device="cuda")
    f = moe.VocabularyLoss(T, H, V, training=True, piece=V)
    loss = f.forward(x, w, y)
    n = 300
    d = x[-n:].double(), w.double(), y[-n:]
    tr.bounded(loss[-n:], tr.loss(*d)[0], tr.loss_bound(*d)[0], "loss")
    y[:-n] = -1  # (only the last rows add to dW)
    f.forward(x, w, y)
    got = f.backward(x, w, y, dl)
    want, bound = tr.loss_grads_bound(*d, dl[-n:].double(), "bf16", "bf16")
    tr.bounded(got["dx"][-n:], want["dx"], bound["dx"], "dx")
    assert not got["dx"][:-n].any()
    want, bound = tr.loss_grads_bound(*d, dl[-n:].double(), "bf16", "fp32")
    tr.bounded(got["dW"], want["dW"], bound["dW"], "dW")
    assert f.status() == moe.MOE_OK


def test_clip(moe):
    n = 2 ** 31 + 4099
    t = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    t[:3] = 3.0
    t[-3:] = torch.tensor([4.0, -4.0, 4.0])
    clip = moe.GradientClip(1.0, eps=0.0)
    want = (3 * 9.0 + 3 * 16.0) ** 0.5
    norm = clip.clip([t])
    assert abs(float(norm) / want - 1) <= 2.0 ** -20
    w = torch.tensor([4.0, -4.0, 4.0], device="cuda", dtype=torch.float64) / want
    tr.bounded(t[-3:], w, w.abs() * (ref.HALF_ULP["bf16"] + 2.0 ** -18), "scaled")
    assert not t[3:-3].any()
