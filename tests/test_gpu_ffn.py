"""The gated feed-forward block and its gradients against 64 bits: exactly on whole numbers, and within derived
bounds (training_reference.py) otherwise."""
import pytest
import torch

import ops_reference as ref
import training_reference as tr

pytestmark = pytest.mark.gpu

# (T, H, I): one token and the smallest matrices; sizes that end inside a tile, a half tile and a block of K; a
# tile and one more row; K split over pairs; several tiles each way
SIZES = [(1, 8, 8), (1, 264, 136), (3, 64, 520), (16, 1024, 256), (17, 72, 40), (33, 520, 1000), (100, 136, 264),
         (128, 2048, 128), (129, 256, 256), (256, 128, 384), (257, 1000, 328), (300, 64, 2056), (700, 320, 1288)]
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


def wide_rows(v, pad):
    """The rows of v in a wider buffer whose other elements are NaN."""
    b = torch.full((v.shape[0], v.shape[1] + pad), float("nan"), dtype=v.dtype, device=v.device)
    b[:, :v.shape[1]] = v
    return b[:, :v.shape[1]]


def whole(T, H, I, t, seed):
    """Small whole numbers whose products and sums fit: x, dout in {-1, 0, 1}, about 8 weights of a row not zero."""
    g = ref.gen(seed)

    def sparse(r, c):
        v = torch.randint(0, 2, (r, c), generator=g) * 2 - 1
        return (v * (torch.rand(r, c, generator=g) < min(1.0, 4.0 / c))).to(TYPE[t]).cuda()
    x = torch.randint(-1, 2, (T, H), generator=g).to(TYPE[t]).cuda()
    dout = torch.randint(-1, 2, (T, H), generator=g).to(TYPE[t]).cuda()
    add = torch.randint(-9, 10, (T, H), generator=g).to(TYPE[t]).cuda()
    return x, sparse(2 * I, H), sparse(H, I), add, dout


def real(T, H, I, t, seed):
    g = ref.gen(seed)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(TYPE[t]).cuda()  # noqa: E731
    return r(T, H, std=1.5), r(2 * I, H, std=H ** -0.5), r(H, I, std=I ** -0.5), r(T, H), r(T, H)


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("T,H,I", SIZES)
def test_whole_numbers(moe, T, H, I, t):
    """Every intermediate is a whole number that its type holds, so every output is the rounded exact one."""
    x, wgu, wd, add, dout = whole(T, H, I, t, T + H + I)
    f = moe.GatedFFN(T, H, I, moe.MOE_ACT_RELU, TYPE[t], training=True)
    out = f.forward(x, wgu, wd, add)
    d = [v.double() for v in (x, wgu, wd, add, dout)]
    gu, h, want = tr.ffn(*d[:3], "relu", d[3])
    assert h.abs().max() <= 256  # (what makes them exact)
    assert torch.equal(f.gu.double(), gu) and torch.equal(f.h.double(), h)
    assert torch.equal(out, want.to(TYPE[t]))
    g = f.backward(x, wgu, wd, dout)
    w = tr.ffn_grads(*d[:3], "relu", gu, h, d[4])
    dh = d[4] @ d[2]
    assert max((dh * gu[:, I:]).abs().max(), (dh * gu[:, :I]).abs().max()) <= 256
    for n in w:
        assert w[n].abs().max() <= 2 ** 24 and torch.equal(g[n], w[n].to(g[n].dtype)), n
    assert f.status() == moe.MOE_OK


@pytest.mark.parametrize("t,kind,pad,use_add", [("bf16", "silu", 0, True), ("fp16", "gelu", 8, False),
                                                 ("bf16", "gelu", 24, True), ("fp16", "silu", 0, True),
                                                 ("fp16", "relu", 64, False)])
@pytest.mark.parametrize("T,H,I", SIZES)
def test_against_64_bits(moe, T, H, I, t, kind, pad, use_add):
    x, wgu, wd, add, dout = real(T, H, I, t, T * 3 + H + I)
    xs, adds, douts = (wide_rows(v, pad) for v in (x, add, dout))
    out = wide_rows(torch.zeros_like(x), pad)
    d = [v.double() for v in (x, wgu, wd, add, dout)]
    a = d[3] if use_add else None
    f = moe.GatedFFN(T, H, I, act_code(moe, kind), TYPE[t], training=True)
    serve = moe.GatedFFN(T, H, I, act_code(moe, kind), TYPE[t])
    got = f.forward(xs, wgu, wd, adds if use_add else None, out)
    assert torch.equal(serve.forward(xs, wgu, wd, adds if use_add else None), got)
    if pad:  # nothing behind the rows is written
        behind = torch.as_strided(got, (T, pad), (H + pad, 1), got.storage_offset() + H)
        assert behind.isnan().all()
    for n, v, w, b in zip(("gu", "h", "out"), (f.gu, f.h, got), tr.ffn(*d[:3], kind, a),
                          tr.ffn_bound(*d[:3], kind, t, a)):
        tr.bounded(v, w, b, n)
    kept = f.gu.double(), f.h.double()
    for grad_t in (t, "fp32"):
        g = f.backward(xs, wgu, wd, douts, grad_dtype=ref.ROW[grad_t])
        want, bound = tr.ffn_grads_bound(*d[:3], kind, *kept, d[4], t, grad_t)
        for n in want:
            tr.bounded(g[n], want[n], bound[n], n)
        # added to what is there
        old = {n: torch.randn_like(g[n]) for n in ("dW_gate_up", "dW_down")}
        more = f.backward(xs, wgu, wd, douts, *(v.clone() for v in old.values()), accumulate=True)
        dold = {n: v.double() for n, v in old.items()}
        want, bound = tr.ffn_grads_bound(*d[:3], kind, *kept, d[4], t, grad_t, dold)
        for n in old:
            tr.bounded(more[n], want[n] + dold[n], bound[n], n + " accumulated")
    assert f.status() == moe.MOE_OK and serve.status() == moe.MOE_OK


def test_added_in_place(moe):
    """out may be add: the routed experts' output, to which the shared expert's is added."""
    T, H, I = 200, 256, 128
    x, wgu, wd, add, _ = real(T, H, I, "bf16", 1)
    f = moe.GatedFFN(T, H, I)
    want = f.forward(x, wgu, wd, add)
    assert torch.equal(f.forward(x, wgu, wd, add, out=add), want)


@pytest.mark.parametrize("T", [5, 300])
def test_some_gradients_only(moe, T):
    H, I = 136, 72
    x, wgu, wd, _, dout = real(T, H, I, "bf16", 2)
    f = moe.GatedFFN(T, H, I, training=True)
    f.forward(x, wgu, wd)
    g = f.backward(x, wgu, wd, dout)
    call = lambda dx, a, b: moe.moe_ffn_backward(  # noqa: E731
        f.row_type, f.act, x, H, wgu, wd, f.gu, f.h, dout, H, T, H, I, dx, H, moe.MOE_ROW_FP32, 0, a, b, f.ws,
        f.ws_bytes)
    new = {n: torch.full_like(v, float("nan")) for n, v in g.items()}
    call(new["dx"], None, None)
    assert torch.equal(new["dx"], g["dx"]) and new["dW_down"].isnan().all()
    call(None, new["dW_gate_up"], None)
    call(None, None, new["dW_down"])
    for n in g:
        assert torch.equal(new[n], g[n]), n
    call(None, None, None)
    # dx into rows of a wider buffer; a forward that keeps h alone
    wide = torch.full((T, H + 8), float("nan"), dtype=x.dtype, device="cuda")
    moe.moe_ffn_backward(f.row_type, f.act, x, H, wgu, wd, f.gu, f.h, dout, H, T, H, I, wide, H + 8, moe.MOE_ROW_FP32, 0,
                         None, None, f.ws, f.ws_bytes)
    assert torch.equal(wide[:, :H], g["dx"]) and wide[:, H:].isnan().all()
    h, out = torch.empty_like(f.h), torch.empty_like(x)
    moe.moe_ffn(f.row_type, f.act, x, H, wgu, wd, None, 0, T, H, I, None, h, out, H, f.ws, f.ws_bytes)
    assert torch.equal(h, f.h) and torch.equal(out, f.forward(x, wgu, wd))


def test_saturated_activations(moe):
    """Gates far out on both sides, where exp overflows: the activation's limits, no NaN."""
    T, H, I = 9, 8, 16
    x = torch.zeros(T, H, device="cuda", dtype=torch.bfloat16)
    x[:, 0] = torch.tensor([-1e18, -1e15, -1e5, -200, 0, 200, 1e5, 1e15, 1e18])
    wgu = torch.zeros(2 * I, H, device="cuda", dtype=torch.bfloat16)
    wgu[:I, 0] = 1
    wgu[I:, 1] = 1
    x[:, 1] = 2 ** -100
    wd = torch.ones(H, I, device="cuda", dtype=torch.bfloat16)
    dout = torch.ones(T, H, device="cuda", dtype=torch.bfloat16)
    for kind in ("silu", "gelu"):
        f = moe.GatedFFN(T, H, I, act_code(moe, kind), training=True)
        f.forward(x, wgu, wd)
        g = f.backward(x, wgu, wd, dout)
        want = torch.where(x[:, :1] > 0, x[:, :1].double(), torch.zeros(T, 1, device="cuda").double()) * 2.0 ** -100
        tr.bounded(f.h, want.expand(T, I), want.expand(T, I) * 2.0 ** -8 + 1e-30, kind)
        for n in g:
            assert g[n].isfinite().all(), (kind, n)


def test_replayed_graph_and_streams(moe):
    """Captured with its backward on one stream, replayed with other inputs; an eager call on another stream."""
    T, H, I = 150, 264, 136
    a = real(T, H, I, "bf16", 3)
    b = real(T, H, I, "bf16", 4)
    f, eager = (moe.GatedFFN(T, H, I, training=True) for _ in range(2))
    bufs = [v.clone() for v in a]
    x, wgu, wd, add, dout = bufs
    dw = [torch.empty_like(v, dtype=torch.float32) for v in (wgu, wd)]
    f.forward(x, wgu, wd, add)
    f.backward(x, wgu, wd, dout, *dw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = f.forward(x, wgu, wd, add)
        g = f.backward(x, wgu, wd, dout, *dw)
    for inputs in (b, a, b):
        for buf, v in zip(bufs, inputs):
            buf.copy_(v)
        graph.replay()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        o2 = eager.forward(*inputs[:4], stream=side)
        g2 = eager.backward(*inputs[:3], inputs[4], stream=side)
        torch.cuda.synchronize()
        assert torch.equal(out, o2)
        for n in g:
            assert torch.equal(g[n], g2[n]), n


def test_no_tokens(moe):
    H, I = 64, 32
    x = torch.empty(0, H, dtype=torch.bfloat16, device="cuda")
    wgu, wd = (torch.ones(*s, dtype=torch.bfloat16, device="cuda") for s in ((2 * I, H), (H, I)))
    f = moe.GatedFFN(0, H, I, training=True)
    assert f.forward(x, wgu, wd).shape == (0, H)
    g = f.backward(x, wgu, wd, x)
    assert not g["dW_gate_up"].any() and not g["dW_down"].any()
    old = torch.ones(2 * I, H, device="cuda"), torch.ones(H, I, device="cuda")
    g = f.backward(x, wgu, wd, x, *old, accumulate=True)
    assert (g["dW_gate_up"] == 1).all() and (g["dW_down"] == 1).all()


def test_two_at_once(moe):
    """Two objects at work on two streams at the same time, of sizes that take whole tiles, split ones and few tokens."""
    sizes = [(700, 320, 1288), (300, 1024, 512), (20, 512, 256), (257, 64, 2056)]
    objects, want = [], []
    for i, (T, H, I) in enumerate(sizes):
        a = real(T, H, I, "bf16", 20 + i)
        f = moe.GatedFFN(T, H, I, training=True)
        want.append((f.forward(*a[:4]).clone(), {n: v.clone() for n, v in f.backward(*a[:3], a[4]).items()}))
        objects.append((f, a))
    streams = [torch.cuda.Stream() for _ in sizes]
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for s, (f, a) in zip(streams, objects):
            got.append((f.forward(*a[:4], stream=s), f.backward(*a[:3], a[4], stream=s)))
        torch.cuda.synchronize()
        for (out, g), (o, w) in zip(got, want):
            assert torch.equal(out, o)
            for n in w:
                assert torch.equal(g[n], w[n]), n
    assert all(f.status() == moe.MOE_OK for f, _ in objects)
