"""The norm of many gradients and their clipping against 64 bits.

Tolerances: a thread's 64 squares in fp32 err by at most 16 2^-24 of their sum in each of four chains and two more
additions, 2^-19 in all, halved by the square root; everything above is 64-bit, and the norm is rounded once to
fp32.  A scaled element has the factor's error (its division and sum, 2^-22, and the norm's 2^-20), one
multiplication and one rounding to its type."""
import math

import pytest
import torch

import ops_reference as ref
import training_reference as tr

pytestmark = pytest.mark.gpu
NORM = 2.0 ** -20


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_grouped_moe_gb300 import build
    build.build()
    from mixture_experts_grouped_moe_gb300 import moe as m
    m.load()
    return m


def tensors(sizes, types, seed, std=1.0):
    g = ref.gen(seed)
    return [(torch.randn(n, generator=g) * std).to(ref.ROW[types[i % len(types)]]).cuda() for i, n in enumerate(sizes)]


def check(moe, grads, max_norm, eps=1e-6):
    want = tr.norm(grads)
    k = min(1.0, max_norm / (float(want) + eps))
    clip = moe.GradientClip(max_norm, eps, n=len(grads))
    names = {v: n for n, v in ref.ROW.items()}
    tr.bounded(clip.norm(grads), want.reshape(1).cuda(), want.reshape(1).cuda() * NORM + 1e-300, "norm")
    before = [t.clone() for t in grads]
    out = [torch.full_like(t, float("nan")) for t in grads]
    norm = clip.clip(grads, out)
    assert torch.equal(norm, clip.norm(grads))
    for a, b in zip(grads, before):
        assert torch.equal(a, b)
    norm2 = clip.clip(grads)
    assert torch.equal(norm, norm2)
    for i, (a, o, b) in enumerate(zip(grads, out, before)):
        assert torch.equal(a, o), i
        if k == 1.0:
            assert torch.equal(a, b), i
        t = names[a.dtype]
        w = b.double() * k
        tr.bounded(a, w, w.abs() * (ref.HALF_ULP[t] + 2.0 ** -18) + ref.TINY[t], i)


@pytest.mark.parametrize("types", [["fp32"], ["bf16"], ["fp16"], ["fp32", "bf16", "fp16"]])
@pytest.mark.parametrize("sizes", [[1], [0, 3, 0], [7, 8, 9, 4095, 4096, 4097], [8192, 8193, 16384, 16385, 1],
                                   [300001, 5, 70000]])
def test_sizes_and_types(moe, sizes, types):
    for max_norm in (0.5, 1e9, 0.0):
        check(moe, tensors(sizes, types, sum(sizes) + 1), max_norm)


def test_many_tensors(moe):
    """More than one launch's worth, of every type."""
    check(moe, tensors([1 + i * 13 % 50 for i in range(1300)], ["fp32", "bf16", "fp16"], 3), 1.0)


def test_none(moe):
    clip = moe.GradientClip(1.0)
    assert clip.norm([]).item() == 0.0 and clip.clip([]).item() == 0.0


def test_unaligned_tensors(moe):
    """Views that start between 16-byte boundaries, and neighbours that must stay as they are."""
    for t in ("fp32", "bf16", "fp16"):
        for offset in (1, 2, 3, 5, 8):
            base = torch.randn(30000, generator=ref.gen(offset)).to(ref.ROW[t]).cuda()
            before = base.clone()
            g = base[offset:offset + 20001]
            want = tr.norm([g])
            clip = moe.GradientClip(1.0)
            tr.bounded(clip.clip([g]), want.reshape(1), want.reshape(1) * NORM, "norm")
            w = before[offset:offset + 20001].double() / float(want + 1e-6)
            tr.bounded(g, w, w.abs() * (ref.HALF_ULP[t] + 2.0 ** -18) + ref.TINY[t], "scaled")
            assert torch.equal(base[:offset], before[:offset])
            assert torch.equal(base[offset + 20001:], before[offset + 20001:])


@pytest.mark.parametrize("scale", [1e-30, 1e-18, 3e-16, 1e18, 1e30])
def test_squares_outside_fp32(moe, scale):
    """Elements whose squares fp32 cannot hold, next to ordinary and zero ones."""
    g = [t * scale for t in tensors([5000, 40000, 3], ["fp32"], 11)] + [torch.zeros(9000, device="cuda")]
    want = tr.norm(g)
    tr.bounded(moe.GradientClip(1.0).norm(g), want.reshape(1), want.reshape(1) * NORM, scale)
    check(moe, g, 1e-3 * float(want), eps=0.0)


def test_not_finite(moe):
    for bad in (float("inf"), float("nan")):
        g = tensors([5000, 300], ["fp32"], 12)
        g[1][7] = bad
        norm = moe.GradientClip(1.0).clip(g)
        assert math.isnan(norm.item()) if bad != bad else norm.item() == bad
        # as the formula says: a factor of 0 leaves zeros and one NaN, a NaN factor only NaNs
        assert g[1][7].isnan() and (not g[0].any() if bad == bad else g[0].isnan().all())


def test_replayed_graph(moe):
    g = tensors([5000, 77, 20000], ["fp32", "bf16"], 13)
    clip = moe.GradientClip(1.0)
    fresh = [t.clone() for t in g]
    clip.clip(g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = clip.clip(g)
    for f in (1.0, 3.0):
        for t, v in zip(g, fresh):
            t.copy_(v * f)
        want = [t.clone() for t in g]
        graph.replay()
        n2 = moe.GradientClip(1.0).clip(want)
        torch.cuda.synchronize()
        assert torch.equal(norm, n2) and all(torch.equal(a, b) for a, b in zip(g, want))


def test_a_gradient_listed_twice(moe):
    """Read twice and written to two places it counts twice in the norm; in place it is refused (on the host)."""
    g = tensors([5000], ["fp32"], 14)[0]
    out = [torch.empty_like(g) for _ in range(2)]
    norm = moe.GradientClip(1.0).clip([g, g], out)
    want = tr.norm([g, g])
    tr.bounded(norm, want.reshape(1), want.reshape(1) * NORM, "norm")
    assert torch.equal(out[0], out[1])
    with pytest.raises(ValueError):
        moe.GradientClip(1.0).clip([g, g])
