"""The gated block's activations over the range that 16 bits hold, by relative error."""
import pytest
import torch

import ops_reference as ref
import training_reference as tr

pytestmark = pytest.mark.gpu
TYPE = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_grouped_moe_gb300 import build
    build.build()
    from mixture_experts_grouped_moe_gb300 import moe as m
    m.load()
    return m


def act_code(moe, kind):
    return {"silu": moe.MOE_ACT_SILU, "gelu": moe.MOE_ACT_GELU_TANH, "relu": moe.MOE_ACT_RELU}[kind]


@pytest.mark.parametrize("T", [33, 200])
@pytest.mark.parametrize("t,kind,low", [("bf16", "silu", -85.0), ("bf16", "gelu", -9.5), ("fp16", "silu", -12.0),
                                        ("fp16", "gelu", -3.5)])
def test_gates_far_below_zero(moe, T, t, kind, low):
    """h where the activation is small, by its relative error.  The fast exponential's documented error is
    2 + 1.173 |q| steps, and q of the gelu takes four roundings and two rounded constants, each 2^-24 of it."""
    H, I = 8, 64
    x = torch.zeros(T, H, device="cuda", dtype=TYPE[t])
    x[:, 0] = torch.linspace(low, -0.5, T, device="cuda")
    x[:, 1] = 1
    wgu = torch.zeros(2 * I, H, device="cuda", dtype=TYPE[t])
    wgu[:I, 0] = 1
    wgu[I:, 1] = 1
    wd = torch.zeros(H, I, device="cuda", dtype=TYPE[t])
    f = moe.GatedFFN(T, H, I, act_code(moe, kind), TYPE[t], training=True)
    f.forward(x, wgu, wd)
    g = x[:, :1].double()
    want = tr.act(g, kind)[0].expand(T, I)
    q = g if kind == "silu" else 2 * (2 / torch.pi) ** 0.5 * (g + 0.044715 * g ** 3)
    off = (4 + 1.173 * q.abs()) * 2.0 ** -23 + q.abs() * (2.0 ** -21 if kind == "gelu" else 2.0 ** -23)
    bound = want.abs() * (ref.HALF_ULP[t] * (1 + off) + off + 2.0 ** -22) + ref.TINY[t]
    tr.bounded(f.h, want, bound, "h")
    assert float(want.abs().min()) > 0
