"""The gated block's gradients in fp16 for output gradients far below one: [d gate | d up] is an operand of 16-bit
products and must not fall among fp16's subnormal steps (2^-24).

Bounds as in training_reference.py, but for the absolute step of [d gate | d up]: the largest |dout| is brought to
[1, 2) by a power of two, so that a step is 2^-24 of that scale.

dW_down has dout itself as an operand, here mostly subnormal.  An MMA brings its 16 products to the largest exponent
among them before it adds them, and what lies more than 2^-23 below that is dropped.  A product's exponent is the sum
of its operands' exponent fields, and a subnormal fp16 number's field is that of 2^-14.  So, for what is dropped, an
operand below 2^-14 counts as 2^-14: at most 2^-23 a product of up to 4 max(|dout|, 2^-14) max(|h|, 2^-14) (two
significands below 2)."""
import pytest
import torch

import ops_reference as ref
import training_reference as tr

pytestmark = pytest.mark.gpu
SIZES = [(3, 64, 520), (40, 136, 264), (257, 1000, 328), (700, 320, 1288)]


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_grouped_moe_gb300 import build
    build.build()
    from mixture_experts_grouped_moe_gb300 import moe as m
    m.load()
    return m


def inputs(T, H, I, steps, seed):
    """dout: multiples of 2^-24 up to steps of them, which fp16 holds exactly."""
    g = ref.gen(seed)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).half().cuda()  # noqa: E731
    dout = (torch.randint(-steps, steps + 1, (T, H), generator=g) * 2.0 ** -24).half().cuda()
    return r(T, H), r(2 * I, H, std=H ** -0.5), r(H, I, std=I ** -0.5), dout


def bounds(x, wgu, wd, kind, gu, h, dout):
    """tr.ffn_grads_bound with the scaled step, results in fp32."""
    I, e = wd.shape[1], ref.HALF_ULP["fp16"]
    most = float(dout.abs().max())
    tiny = ref.TINY["fp16"] * 2.0 ** torch.tensor(most).log2().floor().item() if 0 < most < 1 else ref.TINY["fp16"]
    a, da = tr.act(gu[:, :I], kind)
    u = gu[:, I:]
    dh, edh = dout @ wd, tr.ACC * (dout.abs() @ wd.abs())
    slope = da.abs() + 4.0 * (kind != "relu")
    dgu = torch.cat([dh * u * da, dh * a], 1)
    ed = torch.cat([edh * (u * da).abs() + (dh.abs() + edh) * u.abs() * slope * tr.FN,
                    edh * a.abs() + (dh.abs() + edh) * a.abs() * tr.FN], 1) * 1.01
    ed = ed + e * (dgu.abs() + ed) + tiny
    full = dgu.abs() + ed
    want = {"dx": dgu @ wgu, "dW_gate_up": dgu.t() @ x, "dW_down": dout.t() @ h}
    err = {"dx": (ed + tr.ACC * full) @ wgu.abs(), "dW_gate_up": (ed + tr.ACC * full).t() @ x.abs(),
           "dW_down": tr.ACC * (dout.abs().t() @ h.abs()) +
           2.0 ** -21 * (dout.abs().clamp(min=2.0 ** -14).t() @ h.abs().clamp(min=2.0 ** -14))}
    for n in err:
        t = "fp16" if n == "dx" else "fp32"
        err[n] = err[n] + ref.HALF_ULP[t] * 2 * (want[n].abs() + err[n]) + ref.TINY[t]
    return want, err


@pytest.mark.parametrize("steps", [4, 300, 60000])
@pytest.mark.parametrize("kind", tr.ACTS)
@pytest.mark.parametrize("T,H,I", SIZES)
def test_small_output_gradients(moe, T, H, I, kind, steps):
    x, wgu, wd, dout = inputs(T, H, I, steps, T + steps)
    code = {"silu": moe.MOE_ACT_SILU, "gelu": moe.MOE_ACT_GELU_TANH, "relu": moe.MOE_ACT_RELU}[kind]
    f = moe.GatedFFN(T, H, I, code, torch.float16, training=True)
    f.forward(x, wgu, wd)
    g = f.backward(x, wgu, wd, dout)
    want, err = bounds(*(v.double() for v in (x, wgu, wd)), kind, f.gu.double(), f.h.double(), dout.double())
    for n in want:
        tr.bounded(g[n], want[n], err[n], n)
    assert f.status() == moe.MOE_OK


def test_scale_of_the_output_gradient(moe):
    """An output gradient times a power of two gives the weights' gradients times it: bit for bit where dout stays a
    normal number (2^-14 and above; everything behind it is scaled), within the bounds where it does not.  Zeros give
    zeros, and an infinity or a NaN leaves the other rows' gradients as they were."""
    T, H, I = 300, 136, 264
    x, wgu, wd, _ = inputs(T, H, I, 1, 5)
    dout = (torch.randint(-8, 9, (T, H), generator=ref.gen(6)) * 2.0 ** -4).half().cuda()
    f = moe.GatedFFN(T, H, I, dtype=torch.float16, training=True)
    f.forward(x, wgu, wd)
    one = f.backward(x, wgu, wd, dout)
    for s in (2.0 ** -10, 2.0 ** -12, 2.0 ** -19):
        got = f.backward(x, wgu, wd, dout * s)
        want, err = bounds(*(v.double() for v in (x, wgu, wd)), "silu", f.gu.double(), f.h.double(),
                           (dout * s).double())
        for n in ("dW_gate_up", "dW_down"):
            assert s < 2.0 ** -10 or torch.equal(one[n] * s, got[n]), n
            tr.bounded(got[n], want[n], err[n], (n, s))
    g = f.backward(x, wgu, wd, dout * 0)
    assert not any(v.any() for v in g.values())
    for bad in (float("inf"), float("nan")):
        d = dout.clone() * 2.0 ** -12
        want = f.backward(x, wgu, wd, d)["dx"]
        d[17, 5] = bad
        dx = f.backward(x, wgu, wd, d)["dx"]
        rest = torch.arange(T, device="cuda") != 17
        assert torch.equal(dx[rest], want[rest]) and not dx[17].isfinite().any()


def test_scale_in_a_replayed_graph(moe):
    """The scale is found anew in every replay, next to an eager object at work on another stream."""
    T, H, I = 150, 136, 72
    x, wgu, wd, dout = inputs(T, H, I, 60000, 8)
    f, eager = (moe.GatedFFN(T, H, I, dtype=torch.float16, training=True) for _ in range(2))
    f.forward(x, wgu, wd)
    eager.forward(x, wgu, wd)
    d = dout.clone()
    f.backward(x, wgu, wd, d)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = f.backward(x, wgu, wd, d)
    for scale in (2.0 ** -8, 1.0, 2.0 ** 10, 2.0 ** -12):
        d.copy_(dout * scale)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        want = eager.backward(x, wgu, wd, d, stream=side)
        torch.cuda.synchronize()
        for n in got:
            assert torch.equal(got[n], want[n]), (n, scale)
