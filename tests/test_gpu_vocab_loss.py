"""The cross entropy over a vocabulary and its gradients against 64 bits, within derived bounds
(training_reference.py), and against differences of the losses."""
import pytest
import torch

import ops_reference as ref
import training_reference as tr

pytestmark = pytest.mark.gpu

# (T, H, V): one row and one word; vocabularies that end inside a tile and a block; K long enough to be split over
# pairs, with few rows and with more
SIZES = [(1, 8, 1), (1, 64, 257), (3, 72, 1000), (16, 264, 4099), (127, 136, 255), (129, 64, 256), (256, 520, 513),
         (300, 1000, 777), (520, 64, 3001), (33, 2048, 300), (64, 4096, 1100), (40, 1024, 129)]
TYPE = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_grouped_moe_gb300 import build
    build.build()
    from mixture_experts_grouped_moe_gb300 import moe as m
    m.load()
    return m


def make(T, H, V, t, seed, left_out=0.2):
    g = ref.gen(seed)
    x = torch.randn(T, H, generator=g).to(TYPE[t]).cuda()
    w = (torch.randn(V, H, generator=g) * 2 * H ** -0.5).to(TYPE[t]).cuda()
    targets = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    drop = torch.rand(T, generator=g) < left_out
    bad = torch.tensor([-1, -100, V, 2 ** 31 - 1], dtype=torch.int32)[torch.randint(0, 4, (T,), generator=g)]
    dloss = torch.randn(T, generator=g) / T
    return x, w, torch.where(drop, bad, targets).cuda(), dloss.cuda()


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("T,H,V", SIZES)
def test_against_64_bits(moe, T, H, V, t):
    x, w, targets, dloss = make(T, H, V, t, T + H + V)
    xd, wd, dd = x.double(), w.double(), dloss.double()
    want, bound = tr.loss(xd, wd, targets), tr.loss_bound(xd, wd, targets)
    serve = moe.VocabularyLoss(T, H, V, TYPE[t])
    rows = torch.full((T, H + 8), float("nan"), dtype=TYPE[t], device="cuda")
    rows[:, :H] = x
    for piece in (64, 512, 8192):
        f = moe.VocabularyLoss(T, H, V, TYPE[t], training=True, piece=piece)
        loss = f.forward(rows[:, :H], w, targets)
        assert torch.equal(serve.forward(x, w, targets), loss)
        tr.bounded(loss, want[0], bound[0], "loss")
        tr.bounded(f.lse, want[1], bound[1], "lse")
        ok = (targets >= 0) & (targets < V)
        assert not loss[~ok].any()
        for grad_t in (t, "fp32"):
            g = f.backward(rows[:, :H], w, targets, dloss, grad_dtype=ref.ROW[grad_t])
            wg, bg = tr.loss_grads_bound(xd, wd, targets, dd, t, grad_t)
            for n in wg:
                tr.bounded(g[n], wg[n], bg[n], (n, piece))
            assert not g["dx"][~ok].any()
        old = torch.randn(V, H, device="cuda")
        more = f.backward(x, w, targets, dloss, old.clone(), accumulate=True)["dW"]
        wg, bg = tr.loss_grads_bound(xd, wd, targets, dd, t, "fp32", old.double())
        tr.bounded(more, wg["dW"] + old.double(), bg["dW"], "dW accumulated")
        assert f.status() == moe.MOE_OK
    assert serve.status() == moe.MOE_OK


@pytest.mark.parametrize("T,H,V", [(16, 8200, 40000), (32, 4104, 5000), (300, 4104, 10001), (300, 7176, 500)])
def test_long_rows(moe, T, H, V):
    """A logit of so many products is summed in parts (in one piece and split over CTAs, for few rows and for more)."""
    x, w, targets, dloss = make(T, H, V, "bf16", H + V)
    xd, wd = x.double(), w.double()
    f = moe.VocabularyLoss(T, H, V, training=True)
    loss = f.forward(x, w, targets)
    for got, want, bound, n in zip((loss, f.lse), tr.loss(xd, wd, targets), tr.loss_bound(xd, wd, targets),
                                   ("loss", "lse")):
        tr.bounded(got, want, bound, n)
    g = f.backward(x, w, targets, dloss)
    want, bound = tr.loss_grads_bound(xd, wd, targets, dloss.double(), "bf16", "fp32")
    tr.bounded(g["dx"], want["dx"], tr.loss_grads_bound(xd, wd, targets, dloss.double(), "bf16", "bf16")[1]["dx"], "dx")
    tr.bounded(g["dW"], want["dW"], bound["dW"], "dW")
    assert f.status() == moe.MOE_OK


def test_differences(moe):
    """The gradient along a direction against central differences of the losses.  x and the direction are multiples
    of 2^-4 below 4 and the step 2^-4, so that x +- step * direction are bf16 numbers; the third derivative of a
    log-sum-exp of logits that move by m along the direction is at most 2 m^3, and each loss is bounded as above."""
    T, H, V = 40, 64, 300
    g = ref.gen(7)
    x = (torch.randint(-16, 17, (T, H), generator=g) / 16).cuda()
    d = torch.randint(-1, 2, (T, H), generator=g).float().cuda()
    w = (torch.randn(V, H, generator=g) * 0.25).bfloat16().cuda()
    targets = torch.randint(0, V, (T,), generator=g, dtype=torch.int32).cuda()
    step = 2.0 ** -4
    f = moe.VocabularyLoss(T, H, V, training=True)
    up, down = ((x + s * step * d).bfloat16() for s in (1, -1))
    diff = (f.forward(up, w, targets).double() - f.forward(down, w, targets).double()) / (2 * step)
    f.forward(x.bfloat16(), w, targets)
    dx = f.backward(x.bfloat16(), w, targets, torch.ones(T, device="cuda"))["dx"].double()
    move = (d.double() @ w.double().t()).abs().amax(1)
    noise = sum(tr.loss_bound(v.double(), w.double(), targets)[0] for v in (up, down)) / (2 * step)
    _, b = tr.loss_grads_bound(x.double(), w.double(), targets, torch.ones(T, device="cuda").double(), "bf16", "bf16")
    bound = 2 * move ** 3 * step ** 2 / 6 + noise + (b["dx"] * d.abs()).sum(1)
    tr.bounded((dx * d).sum(1), diff, bound, "differences")


@pytest.mark.parametrize("T", [4, 300])
def test_rows_left_out_hold_anything(moe, T):
    """Padding rows of infinities and NaNs: their loss and gradient are zero, and they add nothing to dW."""
    H, V = 72, 500
    x, w, targets, dloss = make(T, H, V, "bf16", 3, 0.0)
    targets[::2] = -1
    f = moe.VocabularyLoss(T, H, V, training=True, piece=256)
    f.forward(x, w, targets)
    want = f.backward(x, w, targets, dloss)
    bad, badd = x.clone(), dloss.clone()
    bad[::2] = torch.tensor([float("nan"), float("inf")] * (H // 2), device="cuda", dtype=x.dtype)
    badd[::4] = float("nan")
    badd[2::4] = float("inf")
    loss = f.forward(bad, w, targets)
    assert not loss[::2].any() and loss.isfinite().all()
    g = f.backward(bad, w, targets, badd)
    for n in g:
        assert torch.equal(g[n], want[n]), n


def test_all_left_out_and_extreme_factors(moe):
    T, H, V = 130, 64, 300
    x, w, targets, dloss = make(T, H, V, "fp16", 5, 0.0)
    f = moe.VocabularyLoss(T, H, V, torch.float16, training=True)
    none = torch.full_like(targets, -1)
    assert not f.forward(x, w, none).any()
    g = f.backward(x, w, none, dloss)
    assert not g["dx"].any() and not g["dW"].any()
    f.forward(x, w, targets)
    for scale in (2.0 ** -60, 2.0 ** -15, 2.0 ** 40):  # dW in fp32 scales as the losses' gradients do
        a, b = (f.backward(x, w, targets, dloss * s)["dW"] for s in (1.0, scale))
        assert torch.equal(a * scale, b)
    assert not f.backward(x, w, targets, dloss * 0)["dW"].any()


def test_large_logits(moe):
    """Logits of hundreds: the maximum is taken off before any exponential."""
    T, H, V = 20, 64, 600
    x, w, targets, dloss = make(T, H, V, "bf16", 6, 0.0)
    x = x * 64
    f = moe.VocabularyLoss(T, H, V, training=True)
    loss = f.forward(x, w, targets)
    d = x.double(), w.double(), targets
    tr.bounded(loss, tr.loss(*d)[0], tr.loss_bound(*d)[0], "loss")
    g = f.backward(x, w, targets, dloss)
    assert all(v.isfinite().all() for v in g.values())


def test_replayed_graph(moe):
    T, H, V = 140, 72, 700
    a, b = (make(T, H, V, "bf16", s) for s in (8, 9))
    bufs = [v.clone() for v in a]
    f, eager = (moe.VocabularyLoss(T, H, V, training=True, piece=256) for _ in range(2))
    dW = torch.empty(V, H, device="cuda")
    f.forward(*bufs[:3])
    f.backward(*bufs, dW)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss = f.forward(*bufs[:3])
        g = f.backward(*bufs, dW)
    for inputs in (b, a):
        for buf, v in zip(bufs, inputs):
            buf.copy_(v)
        graph.replay()
        want = eager.forward(*inputs[:3])
        wg = eager.backward(*inputs)
        torch.cuda.synchronize()
        assert torch.equal(loss, want) and all(torch.equal(g[n], wg[n]) for n in g)


def test_no_rows(moe):
    H, V = 64, 100
    x = torch.empty(0, H, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(V, H, dtype=torch.bfloat16, device="cuda")
    none, f32 = torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty(0, device="cuda")
    f = moe.VocabularyLoss(0, H, V, training=True)
    assert f.forward(x, w, none).shape == (0,)
    assert not f.backward(x, w, none, f32)["dW"].any()


@pytest.mark.parametrize("T", [20, 300])
def test_some_gradients_only_and_strided(moe, T):
    """dx without dW and dW without dx, dx into rows of a wider buffer, dW added to in the rows' type."""
    H, V, piece = 72, 700, 256
    x, w, targets, dloss = make(T, H, V, "fp16", 11)
    f = moe.VocabularyLoss(T, H, V, torch.float16, training=True, piece=piece)
    f.forward(x, w, targets)
    want = f.backward(x, w, targets, dloss, grad_dtype=torch.float16)
    t = moe.MOE_ROW_FP16

    def call(dx, ld, dw, accumulate=0):
        moe.moe_vocab_loss_backward(t, x, H, w, targets, f.lse, dloss, T, H, V, piece, dx, ld, t, accumulate, dw, f.ws,
                                    f.ws_bytes)

    wide = torch.full((T, H + 16), float("nan"), dtype=x.dtype, device="cuda")
    call(wide, H + 16, None)
    assert torch.equal(wide[:, :H], want["dx"]) and wide[:, H:].isnan().all()
    dw = torch.full_like(w, float("nan"))
    call(None, 0, dw)
    assert torch.equal(dw, want["dW"])
    old = torch.randn(V, H, generator=ref.gen(12)).half().cuda()
    dw = old.clone()
    call(None, 0, dw, 1)
    xd, wd, dd = x.double(), w.double(), dloss.double()
    g, bound = tr.loss_grads_bound(xd, wd, targets, dd, "fp16", "fp16", old.double())
    tr.bounded(dw, g["dW"] + old.double(), bound["dW"], "dW accumulated")
    call(None, 0, None)
