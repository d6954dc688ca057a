"""Refusals of the operators around the layer: bad arguments are turned down on the host before
anything touches CUDA (no GPU needed)."""
import pytest

from mixture_experts_grouped_moe_gb300 import build as moe_build


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    from mixture_experts_grouped_moe_gb300 import moe as m
    return m.load()


INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3
P = 1024  # a non-null, aligned stand-in for a device pointer: nothing is launched


def refused(fn, good, cases):
    """good: dict of a call that would be valid; each case changes some arguments."""
    names = list(good)
    for change, status in cases:
        args = [dict(good, **change)[n] for n in names]
        assert fn(*args) == status, change


def test_sort_map(lib):
    good = dict(ids=P, w=P, T=4, k=2, E=4, bm=16, si=P, sw=P, se=P, npp=P, cnt=None, pos=P, ws=P, wsb=1 << 20, st=None)
    refused(lib.moe_align_sort_map, good, [
        (dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(bm=0), INVALID), (dict(k=5), UNSUPPORTED),
        (dict(E=2000), UNSUPPORTED), (dict(pos=None), INVALID), (dict(ws=None), INVALID), (dict(wsb=8), WORKSPACE),
        (dict(T=1 << 30), UNSUPPORTED)])


def test_permute(lib):
    good = dict(t=0, x=P, ld=64, pos=P, si=P, npp=P, T=0, k=2, H=64, P=16, z=1, xs=P, st=None)
    assert lib.moe_permute(*good.values()) == 0  # no tokens: nothing launched
    refused(lib.moe_permute, good, [
        (dict(t=3), INVALID), (dict(t=-1), INVALID), (dict(T=-1), INVALID), (dict(k=0), INVALID),
        (dict(H=0), INVALID), (dict(P=-1), INVALID), (dict(ld=63), INVALID), (dict(z=2), INVALID),
        (dict(x=None), INVALID), (dict(xs=None), INVALID), (dict(pos=None), INVALID), (dict(si=None), INVALID),
        (dict(npp=None), INVALID), (dict(x=P + 1), INVALID), (dict(t=2, xs=P + 2), INVALID),
        (dict(k=33), UNSUPPORTED), (dict(T=1 << 30), UNSUPPORTED), (dict(P=1 << 31), UNSUPPORTED)])
    assert lib.moe_permute(*dict(good, z=0, si=None, npp=None).values()) == 0


def test_permute_fp8(lib):
    good = dict(x=P, ld=128, pos=P, si=P, npp=P, T=0, k=2, H=128, P=16, z=1, q=P, s=P, st=None)
    assert lib.moe_permute_fp8(*good.values()) == 0
    refused(lib.moe_permute_fp8, good, [
        (dict(H=64), UNSUPPORTED), (dict(ld=130), UNSUPPORTED), (dict(ld=100), INVALID), (dict(x=P + 2), INVALID),
        (dict(q=P + 8), INVALID), (dict(s=P + 1), INVALID), (dict(q=None), INVALID), (dict(npp=None), INVALID)])


def test_unpermute(lib):
    good = dict(t=0, ys=P, pos=P, w=P, T=0, k=2, H=64, P=16, out=P, ld=64, st=None)
    assert lib.moe_unpermute(*good.values()) == 0
    refused(lib.moe_unpermute, good, [
        (dict(t=9), INVALID), (dict(ys=None), INVALID), (dict(out=None), INVALID), (dict(ld=63), INVALID),
        (dict(k=40), UNSUPPORTED), (dict(out=P + 1), INVALID)])
    back = dict(t=0, d=P, pos=P, T=0, k=2, H=64, P=16, dx=P, ld=64, st=None)
    refused(lib.moe_permute_backward, back, [(dict(d=None), INVALID), (dict(ld=1), INVALID), (dict(H=-2), INVALID)])
    bwd = dict(t=0, d=P, ld=64, ys=P, pos=P, w=P, si=P, npp=P, T=0, k=2, H=64, P=16, z=1, dys=P, dw=P, st=None)
    assert lib.moe_unpermute_backward(*bwd.values()) == 0
    refused(lib.moe_unpermute_backward, bwd, [
        (dict(dw=None), INVALID), (dict(dys=None), INVALID), (dict(si=None), INVALID), (dict(ld=5), INVALID),
        (dict(d=P + 1), INVALID), (dict(P=1 << 40), UNSUPPORTED)])


def test_product(lib):
    good = dict(A=P, sa=P, by=0, B=P, sb=P, M=8, N=64, K=128, E=1, bm=0, eid=None, npp=None, t=0, D=P, ld=64, ws=P,
                wsb=64, st=None)
    grouped = dict(good, E=4, bm=16, eid=P, npp=P)
    assert lib.moe_gemm_fp8_block(*dict(good, M=0).values()) == 0
    refused(lib.moe_gemm_fp8_block, good, [
        (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(A=None), INVALID),
        (dict(D=None), INVALID), (dict(ws=None), INVALID), (dict(ld=63), INVALID), (dict(by=2), INVALID),
        (dict(t=1), INVALID), (dict(E=2), INVALID), (dict(bm=16), INVALID), (dict(eid=P), INVALID),
        (dict(A=P + 8), INVALID), (dict(B=P + 1), INVALID), (dict(sa=P + 2), INVALID), (dict(D=P + 1), INVALID),
        (dict(t=2, D=P + 2), INVALID), (dict(K=120), UNSUPPORTED), (dict(K=1 << 21), UNSUPPORTED),
        (dict(wsb=32), WORKSPACE)])
    refused(lib.moe_gemm_fp8_block, grouped, [
        (dict(bm=24), UNSUPPORTED), (dict(bm=0), UNSUPPORTED), (dict(bm=192), UNSUPPORTED), (dict(npp=None), INVALID)])


def test_weight_gradient(lib):
    good = dict(A=P, sa=P, B=P, sb=P, P=256, M=64, N=64, E=2, cnt=P, D=P, acc=0, ws=P, wsb=64, st=None)
    refused(lib.moe_wgrad_fp8_block, good, [
        (dict(P=-128), INVALID), (dict(M=0), INVALID), (dict(N=-4), INVALID), (dict(E=0), INVALID),
        (dict(cnt=None), INVALID), (dict(D=None), INVALID), (dict(acc=2), INVALID), (dict(sb=P + 4), INVALID),
        (dict(P=200), UNSUPPORTED), (dict(N=66), UNSUPPORTED), (dict(E=1025), UNSUPPORTED), (dict(wsb=0), WORKSPACE)])


def test_transposing_quantiser(lib):
    good = dict(X=P, ld=64, R=0, C=64, si=None, S=0, k=1, n=None, q=P, ldq=128, s=P, st=None)
    assert lib.moe_quantize_fp8_act_t(*good.values()) == 0
    refused(lib.moe_quantize_fp8_act_t, good, [
        (dict(R=-1), INVALID), (dict(C=0), INVALID), (dict(ld=56), INVALID), (dict(X=None), INVALID),
        (dict(R=129, ldq=128), INVALID), (dict(si=P, k=0), INVALID), (dict(X=P + 2), INVALID), (dict(q=P + 4), INVALID),
        (dict(C=60), UNSUPPORTED), (dict(ld=65), UNSUPPORTED), (dict(ldq=136), UNSUPPORTED)])


def test_block_norm(lib):
    good = dict(t=0, h=P, r=P, g=P, gk=1, wo=P, wi=P, T=0, H=64, sc=1.0, off=0.0, eps=1e-6, y=P, z=P, rh=None, ry=None,
                st=None)
    assert lib.moe_block_norm(*good.values()) == 0
    refused(lib.moe_block_norm, good, [
        (dict(t=5), INVALID), (dict(h=None), INVALID), (dict(r=None), INVALID), (dict(y=None), INVALID),
        (dict(z=None), INVALID), (dict(wi=None), INVALID), (dict(gk=4), INVALID), (dict(gk=0), INVALID),
        (dict(g=None), INVALID), (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(h=P + 1), INVALID),
        (dict(H=16385), UNSUPPORTED)])
    bwd = dict(t=0, h=P, r=P, g=P, gk=1, wo=P, wi=P, rh=P, ry=P, dy=P, dz=P, T=4, H=64, sc=1.0, off=0.0, dr=P, dh=P,
               dg=P, dwo=P, dwi=P, ws=P, wsb=1 << 20, st=None)
    refused(lib.moe_block_norm_backward, bwd, [
        (dict(rh=None), INVALID), (dict(ry=None), INVALID), (dict(dz=None), INVALID), (dict(dwo=None), INVALID),
        (dict(dwi=None), INVALID), (dict(dg=None), INVALID), (dict(ws=None), INVALID), (dict(dh=None), INVALID),
        (dict(wi=None), INVALID), (dict(wi=None, dz=None, dy=None), INVALID), (dict(g=None, gk=0), INVALID),
        (dict(r=P + 1), INVALID), (dict(r=None), INVALID), (dict(dwo=P + 2), INVALID), (dict(H=20000), UNSUPPORTED), (dict(wsb=16), WORKSPACE)])
    assert lib.moe_block_norm_workspace_size(-1, 64) == 0 and lib.moe_block_norm_workspace_size(4, 1 << 20) == 0


def test_classes_refuse_on_the_host(lib):
    """What the entry points cannot see (shapes, strides and types of tensors) the classes refuse before any
    launch: nothing here needs a GPU."""
    import torch
    from mixture_experts_grouped_moe_gb300 import moe
    T, k, E, H = 8, 2, 4, 128
    ex = moe.TokenExchange(T, k, E, 16, device="cpu")
    P, bf = ex.P, torch.bfloat16
    x, ys = torch.zeros(T, H, dtype=bf), torch.zeros(P, H, dtype=bf)
    refused = [
        (TypeError, lambda: ex.sort(torch.zeros(T, k, dtype=torch.int64), torch.zeros(T, k))),
        (ValueError, lambda: ex.sort(torch.zeros(T, k + 1, dtype=torch.int32), torch.zeros(T, k))),
        (ValueError, lambda: ex.permute(x, xs=torch.zeros(P, H - 1, dtype=bf))),
        (TypeError, lambda: ex.permute(x, xs=torch.zeros(P, H))),
        (ValueError, lambda: ex.permute(torch.zeros(H, T, dtype=bf).t())),
        (TypeError, lambda: ex.permute(torch.zeros(T, H, dtype=torch.float64))),
        (ValueError, lambda: ex.permute_fp8(x, q=torch.zeros(P, H // 2, dtype=torch.uint8))),
        (ValueError, lambda: ex.permute_fp8(x, s=torch.zeros(P, H // 128))),
        (ValueError, lambda: ex.unpermute(ys, out=torch.zeros(T, H // 2, dtype=bf))),
        (ValueError, lambda: ex.unpermute(ys, out=torch.zeros(T, H))),
        (ValueError, lambda: ex.unpermute_backward(x, ys[:, :64].contiguous())),
        (TypeError, lambda: ex.unpermute_backward(x, ys.float())),
        (ValueError, lambda: ex.permute_backward(ys, dx=torch.zeros(T, H // 2, dtype=bf))),
    ]
    w = moe.FP8Weights.__new__(moe.FP8Weights)  # (its constructor quantises on the GPU)
    w.E, w.N, w.K, w.training, w.ws = E, 256, H, False, torch.zeros(64, dtype=torch.uint8)
    w.q, w.s = torch.zeros(E, 256, H, dtype=torch.uint8), torch.ones(E, 2, 1)
    q, s = torch.zeros(P, H, dtype=torch.uint8), torch.ones(P, 1)
    dt, xt = torch.zeros(256, 128, dtype=torch.uint8), torch.zeros(H, 128, dtype=torch.uint8)
    refused += [
        (ValueError, lambda: w.product(q, s)),
        (ValueError, lambda: w.product(q, s[:1], exchange=ex)),
        (ValueError, lambda: w.product(q, s, by_block=True, exchange=ex)),
        (TypeError, lambda: w.product(q.int(), s, exchange=ex)),
        (ValueError, lambda: w.product(q, s, exchange=ex, out=torch.zeros(P, 128, dtype=bf))),
        (TypeError, lambda: w.product(q, s, exchange=ex, out_dtype=torch.float16)),
        (ValueError, lambda: w.product(q, s, exchange=moe.TokenExchange(T, k, 2 * E, 16, device="cpu"))),
        (ValueError, lambda: w.input_gradient(q, s, exchange=ex)),
        (ValueError, lambda: w.weight_gradient(dt, torch.ones(1, 256), xt, torch.ones(1, H), exchange=ex)),  # blocks of 16
    ]
    n = moe.BlockNorm(T, H, moe.MOE_GATE_CHANNEL, device="cpu")
    gate = torch.ones(H, dtype=bf)
    refused += [
        (ValueError, lambda: n.forward(x, x, gate=torch.ones(T, dtype=bf))),
        (TypeError, lambda: n.forward(x, x, gate=gate.float())),
        (TypeError, lambda: n.forward(x, x.float(), gate=gate)),
        (ValueError, lambda: n.forward(x, x, gate=gate, w_post=torch.ones(H - 8, dtype=bf))),
        (ValueError, lambda: n.forward(x, x, gate=gate, y=torch.zeros(T, 2 * H, dtype=bf)[:, :H])),
        (TypeError, lambda: n.backward(x, x, x.half(), x, gate=gate)),
    ]
    for error, call in refused:
        with pytest.raises(error):
            call()
