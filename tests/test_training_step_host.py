"""Refusals of the rest of a training step on the host (nothing is launched, no GPU needed), and the formulas of
its tests against differences in 64 bits."""
import ctypes

import pytest
import torch

import ops_reference as ref
import training_reference as tr
from mixture_experts_grouped_moe_gb300 import build as moe_build

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3
P = 1024  # a non-null, aligned stand-in for a device pointer
BF = torch.bfloat16


@pytest.fixture(scope="module")
def moe():
    moe_build.build()
    from mixture_experts_grouped_moe_gb300 import moe as m
    m.load()
    return m


def refused(fn, good, cases):
    """good: dict of a call that would be valid; each case changes some arguments."""
    for change, status in cases:
        assert not set(change) - set(good), change
        assert fn(*dict(good, **change).values()) == status, change


def test_ffn(moe):
    lib = moe.load()
    good = dict(t=0, act=0, x=P, ld=64, wgu=P, wd=P, add=P, ld_add=64, T=0, H=64, I=32, gu=P, h=P, out=P, ld_out=64,
                ws=P, wsb=1 << 30, st=None)
    assert lib.moe_ffn(*good.values()) == 0  # no tokens: nothing launched
    assert lib.moe_ffn(*dict(good, add=None, ld_add=0, gu=None, h=None).values()) == 0
    refused(lib.moe_ffn, good, [
        (dict(t=3), INVALID), (dict(t=-1), INVALID), (dict(t=2), UNSUPPORTED), (dict(act=3), INVALID),
        (dict(act=-1), INVALID), (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(I=0), INVALID),
        (dict(H=60, ld=60), UNSUPPORTED), (dict(I=12), UNSUPPORTED),
        (dict(H=1 << 21, ld=1 << 21, ld_out=1 << 21, ld_add=1 << 21), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED),
        (dict(ld=56), INVALID), (dict(ld=68), UNSUPPORTED), (dict(ld_out=68), UNSUPPORTED),
        (dict(ld_add=63), INVALID), (dict(ld_add=65), UNSUPPORTED), (dict(ld_out=8), INVALID), (dict(x=None), INVALID),
        (dict(wgu=None), INVALID), (dict(wd=None), INVALID), (dict(out=None), INVALID), (dict(ws=None), INVALID),
        (dict(x=P + 2), INVALID), (dict(wgu=P + 8), INVALID), (dict(add=P + 4), INVALID), (dict(out=P + 8), INVALID),
        (dict(h=None), INVALID), (dict(h=P + 8), INVALID), (dict(ws=P + 8), INVALID), (dict(wsb=64), WORKSPACE),
        (dict(ld=1 << 40), UNSUPPORTED)])
    need = moe.moe_ffn_workspace_size(100, 64, 32)
    assert lib.moe_ffn(*dict(good, T=100, h=None, gu=None, wsb=need - 1).values()) == WORKSPACE
    bwd = dict(t=0, act=0, x=P, ld=64, wgu=P, wd=P, gu=P, h=P, d=P, ld_d=64, T=0, H=64, I=32, dx=P, ld_dx=64, gt=0,
               acc=1, dwgu=P, dwd=P, ws=P, wsb=1 << 30, st=None)
    assert lib.moe_ffn_backward(*bwd.values()) == 0
    assert lib.moe_ffn_backward(*dict(bwd, gt=2, dx=None, ld_dx=0, dwgu=None, dwd=None).values()) == 0
    need = moe.moe_ffn_workspace_size(100, 64, 32, True)
    assert lib.moe_ffn_backward(*dict(bwd, T=100, wsb=need - 1).values()) == WORKSPACE
    refused(lib.moe_ffn_backward, bwd, [
        (dict(gt=1), INVALID), (dict(t=2, gt=2), UNSUPPORTED), (dict(acc=2), INVALID), (dict(gu=None), INVALID),
        (dict(h=None), INVALID), (dict(d=None), INVALID), (dict(ld_d=8), INVALID), (dict(ld_d=68), UNSUPPORTED),
        (dict(ld_dx=8), INVALID), (dict(ld_dx=68), UNSUPPORTED), (dict(dwd=P + 8), INVALID), (dict(dwgu=P + 4), INVALID),
        (dict(wsb=512), WORKSPACE), (dict(I=7), UNSUPPORTED), (dict(T=-1), INVALID)])
    assert moe.moe_ffn_workspace_size(8, 64, 32, True) > moe.moe_ffn_workspace_size(8, 64, 32) - 1 > 0
    for bad in ((-1, 64, 32), (8, 0, 32), (8, 60, 32), (8, 64, 33)):
        assert moe.moe_ffn_workspace_size(*bad) == 0


def test_vocab_loss(moe):
    lib = moe.load()
    good = dict(t=0, x=P, ld=64, W=P, y=P, T=0, H=64, V=1000, loss=P, lse=P, ws=P, wsb=1 << 30, st=None)
    assert lib.moe_vocab_loss(*good.values()) == 0
    refused(lib.moe_vocab_loss, good, [
        (dict(t=2), UNSUPPORTED), (dict(t=5), INVALID), (dict(T=-1), INVALID), (dict(H=0), INVALID),
        (dict(V=0), INVALID), (dict(V=1 << 25), UNSUPPORTED), (dict(H=60, ld=60), UNSUPPORTED), (dict(ld=60), INVALID),
        (dict(ld=66), UNSUPPORTED), (dict(x=P + 8), INVALID), (dict(W=P + 2), INVALID), (dict(y=P + 2), INVALID),
        (dict(y=None), INVALID), (dict(loss=None), INVALID), (dict(lse=None), INVALID), (dict(lse=P + 1), INVALID),
        (dict(wsb=100), WORKSPACE), (dict(ws=None), INVALID)])
    bwd = dict(t=0, x=P, ld=64, W=P, y=P, lse=P, dl=P, T=0, H=64, V=1000, piece=512, dx=P, ld_dx=64, gt=2, acc=1, dW=P,
               ws=P, wsb=1 << 30, st=None)
    assert lib.moe_vocab_loss_backward(*bwd.values()) == 0
    assert lib.moe_vocab_loss_backward(*dict(bwd, dx=None, ld_dx=0, dW=None).values()) == 0
    refused(lib.moe_vocab_loss_backward, bwd, [
        (dict(piece=0), INVALID), (dict(piece=-64), INVALID), (dict(piece=100), UNSUPPORTED), (dict(gt=1), INVALID),
        (dict(acc=-1), INVALID), (dict(dl=None), INVALID), (dict(lse=None), INVALID), (dict(ld_dx=63), INVALID),
        (dict(ld_dx=65), UNSUPPORTED), (dict(dx=P + 8), INVALID), (dict(dW=P + 8), INVALID), (dict(wsb=512), WORKSPACE)])
    need = moe.moe_vocab_loss_workspace_size(100, 64, 1000, 512)
    assert lib.moe_vocab_loss_backward(*dict(bwd, T=100, wsb=need - 1).values()) == WORKSPACE
    assert 0 < moe.moe_vocab_loss_workspace_size(8, 64, 100) < moe.moe_vocab_loss_workspace_size(8, 64, 100, 64)
    for bad in ((-1, 64, 100), (8, 65, 100), (8, 64, 0), (8, 64, 100, 65), (8, 64, 100, -64)):
        assert moe.moe_vocab_loss_workspace_size(*bad) == 0


def test_clip(moe):
    lib = moe.load()
    arr = lambda kind, *v: (kind * len(v))(*v)  # noqa: E731
    types, numel, at = arr(ctypes.c_int, 0, 2), arr(ctypes.c_int64, 3, 5), arr(ctypes.c_void_p, P, P + 4)
    good = dict(n=2, types=types, g=at, out=at, numel=numel, max_norm=1.0, eps=0.0, norm=P, ws=P, wsb=1 << 20, st=None)
    bad = [(dict(n=-1), INVALID), (dict(types=None), INVALID), (dict(g=None), INVALID), (dict(numel=None), INVALID),
           (dict(norm=None), INVALID), (dict(norm=P + 2), INVALID), (dict(ws=None), INVALID), (dict(ws=P + 4), INVALID),
           (dict(types=arr(ctypes.c_int, 0, 3)), INVALID), (dict(numel=arr(ctypes.c_int64, 3, -1)), INVALID),
           (dict(g=arr(ctypes.c_void_p, P, None)), INVALID), (dict(g=arr(ctypes.c_void_p, P + 1, P)), INVALID),
           (dict(g=arr(ctypes.c_void_p, P, P + 2)), INVALID), (dict(wsb=100), WORKSPACE),
           (dict(numel=arr(ctypes.c_int64, 3, 1 << 41)), UNSUPPORTED)]
    refused(lib.moe_clip_gradients, good, bad + [
        (dict(out=None), INVALID), (dict(out=arr(ctypes.c_void_p, P, None)), INVALID), (dict(max_norm=-1.0), INVALID),
        (dict(max_norm=float("nan")), INVALID), (dict(eps=-1.0), INVALID),
        (dict(out=arr(ctypes.c_void_p, P, P + 2)), INVALID)])
    norm = {k: v for k, v in good.items() if k not in ("out", "max_norm", "eps")}
    refused(lib.moe_grad_norm, norm, bad)


def test_objects(moe):
    """Shapes, types, strides, devices and the order of calls."""
    T, H, I, V = 4, 64, 32, 100
    for args in ((T, 60, I), (-1, H, I), (T, H, 0)):
        with pytest.raises(moe.MoEError):
            moe.GatedFFN(*args, device="cpu")
    for args, kw in (((T, 60, V), {}), ((T, H, V), dict(piece=100, training=True)), ((T, H, V), dict(piece=0))):
        with pytest.raises(moe.MoEError):
            moe.VocabularyLoss(*args, device="cpu", **kw)
    with pytest.raises(TypeError):
        moe.GatedFFN(T, H, I, dtype=torch.float32, device="cpu")
    with pytest.raises(TypeError):
        moe.VocabularyLoss(T, H, V, dtype=torch.float64, device="cpu")
    z = lambda *s, dt=BF: torch.zeros(*s, dtype=dt)  # noqa: E731
    f = moe.GatedFFN(T, H, I, training=True, device="cpu")
    x, wgu, wd = z(T, H), z(2 * I, H), z(H, I)
    for call in (lambda: f.forward(z(T + 1, H), wgu, wd), lambda: f.forward(z(H, T).t(), wgu, wd),
                 lambda: f.forward(x, z(I, H), wd), lambda: f.forward(x, z(H, 2 * I).t(), wd),
                 lambda: f.forward(x, wgu, wd, z(T, H + 8)), lambda: f.forward(x, wgu, wd, out=z(T, H - 8)),
                 lambda: f.forward(x, wgu, wd), lambda: f.backward(x, wgu, wd, x),
                 lambda: f.backward(x, wgu, wd, x, accumulate=True), lambda: f.backward(x, wgu, wd, z(T, I)),
                 lambda: moe.GatedFFN(T, H, I, device="cpu").backward(x, wgu, wd, x)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: f.forward(z(T, H, dt=torch.float16), wgu, wd), lambda: f.forward(x, wgu, wd.float()),
                 lambda: f.backward(x, wgu, wd, x, z(2 * I, H), z(H, I, dt=torch.float32)),
                 lambda: f.backward(x, wgu, wd, x, grad_dtype=torch.float16),
                 lambda: f.forward(x, wgu, wd, z(T, H, dt=torch.float32))):
        with pytest.raises(TypeError):
            call()
    v = moe.VocabularyLoss(T, H, V, training=True, device="cpu")
    w, y, d = z(V, H), z(T, dt=torch.int32), z(T, dt=torch.float32)
    for call in (lambda: v.forward(x, z(V, H + 8), y), lambda: v.forward(x, w, z(T + 1, dt=torch.int32)),
                 lambda: v.forward(x, w, y), lambda: v.backward(x, w, y, d),
                 lambda: v.backward(x, w, y, z(T - 1, dt=torch.float32)),
                 lambda: v.backward(x, w, y, d, accumulate=True),
                 lambda: moe.VocabularyLoss(T, H, V, device="cpu").backward(x, w, y, d)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: v.forward(x, w, y.long()), lambda: v.forward(x.half(), w, y),
                 lambda: v.backward(x, w, y, d.double())):
        with pytest.raises(TypeError):
            call()
    c = moe.GradientClip(1.0, n=2, device="cpu")
    for call in (lambda: c.clip([d, d]), lambda: c.clip([d[:3], d[2:]]), lambda: c.clip([d[:2], d[2:]], [d[2:], d[:2]]),
                 lambda: c.clip([d[:2], d[1:3]], [d[1:3], z(2, dt=torch.float32)])):
        with pytest.raises(ValueError, match="overlaps"):
            call()
    for call in (lambda: c.clip([d, d, d]), lambda: c.norm([z(4, 4).t()[:, :2]]), lambda: c.clip([d], [d, d]),
                 lambda: c.clip([d], [z(3, dt=torch.float32)]), lambda: c.norm([d]), lambda: c.clip([d]), lambda: moe.GradientClip(-1.0, device="cpu"),
                 lambda: moe.GradientClip(1.0, eps=float("nan"), device="cpu"),
                 lambda: moe.GradientClip(1.0, n=1 << 20, device="cpu")):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: c.norm([d.double()]), lambda: c.clip([d], [d.half()])):
        with pytest.raises(TypeError):
            call()


@pytest.mark.parametrize("kind", tr.ACTS)
def test_formulas_of_the_block_against_differences(kind):
    g = ref.gen(1)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    T, H, I = 5, 4, 3
    x, wgu, wd, dout = r(T, H), r(2 * I, H), r(H, I), r(T, H)
    gu, h, _ = tr.ffn(x, wgu, wd, kind)
    grads = tr.ffn_grads(x, wgu, wd, kind, gu, h, dout)
    eps = 1e-6
    for n, v in (("dx", x), ("dW_gate_up", wgu), ("dW_down", wd)):
        for i in range(v.numel()):
            keep, at = float(v.view(-1)[i]), []
            for s in (eps, -eps):
                v.view(-1)[i] = keep + s
                at.append(float((tr.ffn(x, wgu, wd, kind)[2] * dout).sum()))
            v.view(-1)[i] = keep
            assert abs((at[0] - at[1]) / (2 * eps) - float(grads[n].view(-1)[i])) < 1e-6, (n, i)


def test_formulas_of_the_loss_against_differences():
    g = ref.gen(2)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    T, H, V = 6, 4, 7
    x, w, dloss = r(T, H), r(V, H), r(T)
    targets = torch.tensor([0, 6, 3, -1, 7, 2], dtype=torch.int32)
    _, grads = tr.loss_grads(x, w, targets, dloss)
    eps = 1e-6
    for n, v in (("dx", x), ("dW", w)):
        for i in range(v.numel()):
            keep, at = float(v.view(-1)[i]), []
            for s in (eps, -eps):
                v.view(-1)[i] = keep + s
                at.append(float((tr.loss(x, w, targets)[0] * dloss).sum()))
            v.view(-1)[i] = keep
            assert abs((at[0] - at[1]) / (2 * eps) - float(grads[n].view(-1)[i])) < 1e-7, (n, i)
