"""Sums over a long K, against 64 bits, with positive terms: the tensor core's truncation then adds up instead of
averaging out, and a sum that should go in parts but does not is told apart.

Bounds.  An MMA adds 16 products to a sum of K at a time and may drop up to one step of it (2^-23 of its size): a sum
that grows evenly over n additions loses at most 2^-23 (n + 1) / 2 of itself.  Parts that are added with rounding lose
2^-24 (m + 1) / 2 more for m of them.  The terms here lie between 1/4 and 1 of the largest, which brings a running sum
from evenly growing by less than a tenth."""
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
    yield m
    torch.cuda.empty_cache()


def loss_of(K, part):
    """What a sum of K positive terms in parts of `part` loses at most, relative to it."""
    return 1.1 * 2.0 ** -23 * (part / 16 + 1) / 2 + 2.0 ** -24 * (-(-K // part) + 1) / 2


def positive(*shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return ((0.5 + 0.5 * torch.rand(*shape, generator=g, device="cuda")) * scale).bfloat16()


def logits_64(x, w):
    """x w^T in 64 bits, some words at a time."""
    xd = x.double()
    return torch.cat([xd @ v.double().t() for v in w.split(max(1, 2 ** 28 // w.shape[1]))], 1)


LOGIT = 2048  # of K at a time


# Few rows; few tiles, whose K 4 or 2 pairs of a cluster share; tiles enough that none is shared; and ordinary sizes
@pytest.mark.parametrize("T,K,V", [(16, 131072, 1000), (32, 65536, 300), (300, 262144, 500), (100, 131072, 5000),
                                   (300, 65536, 5120), (100, 7168, 8192), (100, 16384, 2000), (64, 4104, 300)])
def test_logits(moe, T, K, V):
    """The loss and lse of logits near 100."""
    x, w = positive(T, K, seed=1), positive(V, K, seed=2, scale=100 / (0.5625 * K))
    targets = torch.randint(0, V, (T,), generator=ref.gen(3), dtype=torch.int32).cuda()
    f = moe.VocabularyLoss(T, K, V)
    loss = f.forward(x, w, targets)
    assert f.status() == moe.MOE_OK
    l = logits_64(x, w)
    lse = torch.logsumexp(l, 1)
    top = l.amax(1)
    e = loss_of(K, LOGIT) * top + 2.0 ** -18 + 2.0 ** -21 * (top + 20)
    tr.bounded(f.lse, lse, e, "lse")
    tr.bounded(loss, lse - l.gather(1, targets.long()[:, None])[:, 0], 2 * e, "loss")


@pytest.mark.parametrize("T,K,V", [(20, 131072, 500), (300, 131072, 500), (300, 65536, 5120), (600, 131072, 2500)])
def test_gradient_of_sure_rows(moe, T, K, V):
    """Rows whose target has nearly all of the probability: 1 - p of the target is a small difference, in which the
    forward's and the backward's logits have to agree.  A logit that is off by e changes p by a factor exp(e); the
    forward's and the backward's sums each lose between nothing and loss_of."""
    x, w = positive(T, K, seed=4), positive(V, K, seed=5, scale=100 / (0.5625 * K))
    w[7] *= 1.15  # 15 above the others
    targets = torch.full((T,), 7, dtype=torch.int32, device="cuda")
    dloss = torch.ones(T, device="cuda")
    f = moe.VocabularyLoss(T, K, V, training=True)
    f.forward(x, w, targets)
    dx = f.backward(x, w, targets, dloss)["dx"]
    assert f.status() == moe.MOE_OK
    l = logits_64(x, w)
    p = torch.softmax(l, 1)
    top = l.amax(1, keepdim=True)
    assert 1e-5 < float((1 - p[:, 7]).max()) < 1e-2
    dl = p.clone()
    dl[:, 7] -= 1
    el = loss_of(K, LOGIT) * top + 2.0 ** -17 + 2.0 ** -20 * (top + 20)
    e = ref.HALF_ULP["bf16"]
    ed = p * (torch.expm1(el) + tr.FN) + 2.0 ** -23
    ed = ed + e * (dl.abs() + ed) + 2.0 ** -130
    full = dl.abs() + ed
    for i in range(0, K, 8192):
        wd = w[:, i:i + 8192].double()
        want, err = dl @ wd, ed @ wd + loss_of(V, max(V, 16)) * (full @ wd)
        tr.bounded(dx[:, i:i + 8192], want, err + e * (want.abs() + err) + ref.TINY["bf16"], "dx")


ROWS = 4096  # of a weight gradient in fp32 at a time


# One tile, whose rows four pairs share, and tiles enough that none is shared
@pytest.mark.parametrize("T,H,I", [(2 ** 21, 64, 64), (8192, 1792, 1792), (12000, 2048, 2056)])
def test_weight_gradient_of_many_rows(moe, T, H, I):
    """dW_down = dout^T h of rows that all add to it with the same sign."""
    x, dout = positive(T, H, seed=6), positive(T, H, seed=7)
    wgu, wd = positive(2 * I, H, seed=8, scale=1 / H), positive(H, I, seed=9, scale=1 / I)
    f = moe.GatedFFN(T, H, I, moe.MOE_ACT_RELU, training=True)
    f.forward(x, wgu, wd)
    g = f.backward(x, wgu, wd, dout)
    want = sum(a.double().t() @ b.double() for a, b in zip(dout.split(65536), f.h.split(65536)))
    e = want * (loss_of(T, ROWS) * 1.1 + 2.0 ** -22)
    tr.bounded(g["dW_down"], want, e, "dW_down")
    old = torch.full((H, I), 3.0, device="cuda")
    more = f.backward(x, wgu, wd, dout, torch.zeros(2 * I, H, device="cuda"), old, accumulate=True)
    tr.bounded(more["dW_down"], want + 3, e + 2.0 ** -23 * (want + 3), "accumulated")
    assert f.status() == moe.MOE_OK


def test_sixteen_bit_gradient_of_many_rows(moe):
    """The same in fp16: within a rounding of 64 bits."""
    T, H, I = 2 ** 21, 64, 64
    x, dout = positive(T, H, seed=6).half(), positive(T, H, seed=7, scale=2.0 ** -8).half()
    wgu, wd = positive(2 * I, H, seed=8, scale=1 / H).half(), positive(H, I, seed=9, scale=1 / I).half()
    f = moe.GatedFFN(T, H, I, moe.MOE_ACT_RELU, torch.float16, training=True)
    f.forward(x, wgu, wd)
    got = f.backward(x, wgu, wd, dout, grad_dtype=torch.float16)["dW_down"]
    want = dout.double().t() @ f.h.double()
    assert float(want.max()) < 60000
    e = want * (loss_of(T, ROWS) * 1.1 + 2.0 ** -22)
    tr.bounded(got, want, e + ref.HALF_ULP["fp16"] * (want + e), "dW_down")


@pytest.mark.parametrize("T", [4097, 40000])
def test_gradients_in_parts(moe, T):
    """More rows than one sum takes, the last part a single one: every gradient of both operators, written and added,
    within the bounds of fewer rows."""
    H, I, V, piece = 72, 136, 300, 192
    g = ref.gen(T)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).bfloat16().cuda()  # noqa: E731
    x, wgu, wd, dout = r(T, H), r(2 * I, H, std=H ** -0.5), r(H, I, std=I ** -0.5), r(T, H)
    f = moe.GatedFFN(T, H, I, training=True)
    f.forward(x, wgu, wd)
    d = [v.double() for v in (x, wgu, wd, f.gu, f.h, dout)]
    got = f.backward(x, wgu, wd, dout)
    want, bound = tr.ffn_grads_bound(*d[:3], "silu", *d[3:], "bf16", "fp32")
    for n in want:
        b = tr.ffn_grads_bound(*d[:3], "silu", *d[3:], "bf16", "bf16")[1][n] if n == "dx" else bound[n]
        tr.bounded(got[n], want[n], b, n)
    old = {n: torch.randn(got[n].shape, generator=g).cuda() for n in ("dW_gate_up", "dW_down")}
    more = f.backward(x, wgu, wd, dout, *(v.clone() for v in old.values()), accumulate=True)
    dold = {n: v.double() for n, v in old.items()}
    _, bound = tr.ffn_grads_bound(*d[:3], "silu", *d[3:], "bf16", "fp32", dold)
    for n in old:
        tr.bounded(more[n], want[n] + dold[n], bound[n], n + " accumulated")
    wv = r(V, H, std=2 * H ** -0.5)
    targets = torch.randint(-1, V, (T,), generator=g, dtype=torch.int32).cuda()
    dloss = (torch.randn(T, generator=g) / T).cuda()
    v = moe.VocabularyLoss(T, H, V, training=True, piece=piece)
    v.forward(x, wv, targets)
    got = v.backward(x, wv, targets, dloss)
    args = x.double(), wv.double(), targets, dloss.double(), "bf16"
    want, bound = tr.loss_grads_bound(*args, "fp32")
    tr.bounded(got["dW"], want["dW"], bound["dW"], "dW")
    tr.bounded(got["dx"], want["dx"], tr.loss_grads_bound(*args, "bf16")[1]["dx"], "dx")
    old = torch.randn(V, H, generator=g).cuda()
    more = v.backward(x, wv, targets, dloss, old.clone(), accumulate=True)["dW"]
    tr.bounded(more, want["dW"] + old.double(), tr.loss_grads_bound(*args, "fp32", old.double())[1]["dW"],
               "dW accumulated")
    assert f.status() == moe.MOE_OK and v.status() == moe.MOE_OK
