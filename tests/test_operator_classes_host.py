"""What the operator classes refuse on the host beyond shapes, strides and types: nothing here needs a GPU."""
import pytest
import torch

from mixture_experts_grouped_moe_gb300 import build as moe_build


@pytest.fixture(scope="module")
def moe():
    moe_build.build()
    from mixture_experts_grouped_moe_gb300 import moe as m
    m.load()
    return m


T, K_, E, H = 8, 2, 4, 128
BF = torch.bfloat16


def test_tensors_off_the_gpu(moe):
    """Right shapes and types, but addresses that a kernel must not be given."""
    ex = moe.TokenExchange(T, K_, E, 128, device="cpu")
    P = ex.P
    x, ys = torch.zeros(T, H, dtype=BF), torch.zeros(P, H, dtype=BF)
    w = moe.FP8Weights.__new__(moe.FP8Weights)  # (its constructor quantises on the GPU)
    w.E, w.N, w.K, w.training, w.ws = E, 256, H, True, torch.zeros(64, dtype=torch.uint8)
    w.q, w.s = torch.zeros(E, 256, H, dtype=torch.uint8), torch.ones(E, 2, 1)
    w.qt, w.st = torch.zeros(E, H, 256, dtype=torch.uint8), torch.ones(E, 1, 2)
    R = 128 * (-(-P // 128))
    q, s = torch.zeros(P, H, dtype=torch.uint8), torch.ones(P, 1)
    d, ds = torch.zeros(P, 256, dtype=torch.uint8), torch.ones(P, 2)
    dt, xt = torch.zeros(256, R, dtype=torch.uint8), torch.zeros(H, R, dtype=torch.uint8)
    dts, xts = torch.ones(R // 128, 256), torch.ones(R // 128, H)
    n = moe.BlockNorm(T, H, moe.MOE_GATE_CHANNEL, device="cpu")
    gate = torch.ones(H, dtype=BF)
    for call in (
        lambda: ex.sort(torch.zeros(T, K_, dtype=torch.int32), torch.zeros(T, K_), stream=0),
        lambda: ex.permute(x),
        lambda: ex.permute_fp8(x),
        lambda: ex.unpermute(ys),
        lambda: ex.unpermute_backward(x, ys),
        lambda: ex.permute_backward(ys),
        lambda: moe.FP8Weights(torch.zeros(1, 128, 128, dtype=BF)),
        lambda: w.update(torch.zeros(E, 256, H, dtype=BF)),
        lambda: w.product(q, s, exchange=ex),
        lambda: w.input_gradient(d, ds, exchange=ex),
        lambda: w.weight_gradient(dt, dts, xt, xts, exchange=ex),
        lambda: n.forward(x, x, gate=gate),
        lambda: n.backward(x, x, x, None, gate=gate),
    ):
        with pytest.raises(ValueError, match="on one GPU"):
            call()


def test_device_check_names_the_tensor(moe):
    a = torch.zeros(2)
    with pytest.raises(ValueError, match="x is on cpu"):
        moe._on_gpu(a, none=None, x=a)
    moe._on_gpu(a, none=None)

    class OnGpu:  # a stand-in for CUDA tensors of two devices
        def __init__(self, index):
            self.index, self.device = index, f"cuda:{index}"

        def get_device(self):
            return self.index

    moe._on_gpu(OnGpu(0), x=OnGpu(0))
    for owner, t in ((OnGpu(0), OnGpu(1)), (OnGpu(0), a), (a, OnGpu(0))):
        with pytest.raises(ValueError):
            moe._on_gpu(owner, x=t)


def test_exchange_before_its_sort(moe, monkeypatch):
    """The maps are unwritten until sort(): every use of them is refused, and allowed after it."""
    monkeypatch.setattr(moe, "_on_gpu", lambda *a, **k: None)
    launched = []
    for name in ("moe_align_sort_drop", "moe_permute", "moe_permute_fp8", "moe_unpermute", "moe_unpermute_backward",
                 "moe_permute_backward", "moe_gemm_fp8_block", "moe_wgrad_fp8_block"):
        monkeypatch.setattr(moe, name, lambda *a, name=name: launched.append(name))
    ex = moe.TokenExchange(T, K_, E, 128, device="cpu")
    P = ex.P
    R = 128 * (-(-P // 128))
    x, ys = torch.zeros(T, H, dtype=BF), torch.zeros(P, H, dtype=BF)
    w = moe.FP8Weights.__new__(moe.FP8Weights)
    w.E, w.N, w.K, w.training, w.ws = E, 256, H, True, torch.zeros(64, dtype=torch.uint8)
    w.q = w.s = w.qt = w.st = None
    uses = (
        lambda: ex.permute(x),
        lambda: ex.permute_fp8(x),
        lambda: ex.unpermute(ys),
        lambda: ex.unpermute_backward(x, ys),
        lambda: ex.permute_backward(ys),
        lambda: w.product(torch.zeros(P, H, dtype=torch.uint8), torch.ones(P, 1), exchange=ex),
        lambda: w.input_gradient(torch.zeros(P, 256, dtype=torch.uint8), torch.ones(P, 2), exchange=ex),
        lambda: w.weight_gradient(torch.zeros(256, R, dtype=torch.uint8), torch.ones(R // 128, 256),
                                  torch.zeros(H, R, dtype=torch.uint8), torch.ones(R // 128, H), exchange=ex),
    )
    for use in uses:
        with pytest.raises(ValueError, match="sort"):
            use()
    assert not launched
    ex.sort(torch.zeros(T, K_, dtype=torch.int32), torch.zeros(T, K_))
    for use in uses:
        use()
    assert len(launched) == 1 + len(uses)


def test_norm_backward_before_its_forward(moe, monkeypatch):
    """The statistics are unwritten until a forward() with that norm: a backward that reads them is refused."""
    monkeypatch.setattr(moe, "_on_gpu", lambda *a, **k: None)
    launched = []
    for name in ("moe_block_norm", "moe_block_norm_backward"):
        monkeypatch.setattr(moe, name, lambda *a, name=name: launched.append(name))
    n = moe.BlockNorm(T, H, device="cpu")
    x, w = torch.zeros(T, H, dtype=BF), torch.ones(H, dtype=BF)
    both = lambda: n.backward(x, x, x, x, w_post=w, w_pre=w)  # noqa: E731
    post = lambda: n.backward(x, x, x, None, w_post=w)  # noqa: E731
    for call in (both, post):
        with pytest.raises(ValueError, match="statistics"):
            call()
    n.backward(x, x, x, None)  # (no norm: no statistics)
    n.forward(x, x, w_post=w)
    post()
    with pytest.raises(ValueError, match="w_pre"):
        both()
    n.forward(x, x, w_post=w, w_pre=w)
    both()
    post()
    assert launched.count("moe_block_norm_backward") == 4


def test_empty_tensors(moe):
    """A batch without rows has null addresses: the calls that then launch nothing accept it."""
    none = lambda *s, dt=BF: torch.empty(*s, dtype=dt)  # noqa: E731
    i32, one = torch.int32, torch.zeros(1, dtype=torch.int32)
    assert none(0, H).data_ptr() == 0
    pos, wts, sid = none(0, dt=i32), none(0, K_, dt=torch.float32), torch.zeros(64, dtype=i32)
    xs, q, s = none(64, H), none(64, H, dt=torch.uint8), none(1, 64, dt=torch.float32)
    bf, f32 = moe.MOE_ROW_BF16, torch.float32
    moe.moe_permute(bf, none(0, H), H, pos, sid, one, 0, K_, H, 64, 1, xs, stream=0)
    moe.moe_permute(bf, none(0, H), H, pos, pos, one, 0, K_, H, 0, 1, none(0, H), stream=0)
    moe.moe_permute_fp8(none(0, H), H, pos, sid, one, 0, K_, H, 64, 1, q, s, stream=0)
    moe.moe_unpermute(bf, xs, pos, wts, 0, K_, H, 64, none(0, H), H, stream=0)
    moe.moe_unpermute_backward(bf, none(0, H), H, xs, pos, wts, sid, one, 0, K_, H, 64, 1, xs, wts, stream=0)
    moe.moe_permute_backward(bf, xs, pos, 0, K_, H, 64, none(0, H), H, stream=0)
    b, sb, ws = none(64, H, dt=torch.uint8), none(1, 1, dt=f32), torch.zeros(64, dtype=torch.uint8)
    codes, scales = none(0, H, dt=torch.uint8), none(0, 1, dt=f32)
    moe.moe_gemm_fp8_block(codes, scales, 0, b, sb, 0, 64, H, 1, 0, None, None, bf, none(0, 64), 64, ws, 64, stream=0)
    moe.moe_gemm_fp8_block(codes, scales, 0, b, sb, 0, 64, H, 1, 16, pos, one, bf, none(0, 64), 64, ws, 64, stream=0)
    moe.moe_quantize_fp8_act_t(none(0, H), H, 0, H, pos, 0, 1, one, none(H, 0, dt=torch.uint8), 0,
                               none(0, H, dt=f32), stream=0)
    for kind, gate in ((moe.MOE_GATE_NONE, None), (moe.MOE_GATE_TOKEN, none(0)), (moe.MOE_GATE_FULL, none(0, H))):
        moe.moe_block_norm(bf, none(0, H), none(0, H), gate, kind, one, one, 0, H, 1.0, 0.0, 1e-6, none(0, H),
                           none(0, H), none(0, dt=f32), none(0, dt=f32), stream=0)


def test_empty_tensors_where_rows_are_expected(moe):
    """With rows to move, a null address stays an error."""
    x, pos, xs = torch.zeros(T, H, dtype=BF), torch.zeros(T * K_, dtype=torch.int32), torch.zeros(64, H, dtype=BF)
    none, bf = torch.empty(0, dtype=BF), moe.MOE_ROW_BF16
    for args in ((none, pos, xs), (x, none, xs), (x, pos, none)):
        with pytest.raises(moe.MoEError):
            moe.moe_permute(bf, args[0], H, args[1], None, None, T, K_, H, 64, 0, args[2], stream=0)
    with pytest.raises(moe.MoEError):
        moe.moe_block_norm(bf, none, x, None, 0, None, None, T, H, 1.0, 0.0, 1e-6, x, None, None, None, stream=0)
    with pytest.raises(moe.MoEError):  # no tokens, but padding rows to write
        i32, n = torch.zeros(64, dtype=torch.int32), torch.empty(0, dtype=torch.int32)
        moe.moe_align_sort_drop(n, torch.empty(0), 0, 2, 4, 16, n, xs, i32, i32, i32, n, i32, i32, 1 << 20, stream=0)


@pytest.mark.parametrize("entry", ["map", "drop"])
def test_sorts_past_32_bits(moe, entry):
    """Sorted positions are int32: blocks so large that they could pass it are refused before a launch."""
    fn = getattr(moe, "moe_align_sort_" + entry)
    P = 1024  # a non-null, aligned stand-in for a device pointer
    args = (P,) * 6 + ((P,) if entry == "drop" else ())
    for T, k, E, block_m in ((1 << 20, 2, 1024, 1 << 21), (4, 1, 2, 1 << 30), (1 << 20, 4, 512, (1 << 22) - 1)):
        with pytest.raises(moe.MoEError) as err:
            fn(P, P, T, k, E, block_m, *args, P, 1 << 40, stream=0)
        assert err.value.status == moe.MOE_ERR_UNSUPPORTED
