"""Slots left out of the exchange (ids outside [0, E)): sort, FP8 permute, grouped products, unpermute and
every gradient against 64 bits, on buffers that start as NaN.

Tolerances, derived: codes, scales and maps are exact.  A block-scaled product in fp32 is off by at most
2^-16 of the sum of its absolute terms and half a unit of its result (see test_gpu_gemm_block.py); the
weighted sum of k of them adds 2 (k + 1) 2^-24 of the sum of its absolute terms, together below 2^-15.  A
dot product over N elements in fp32 errs by at most (N + 8) 2^-24 of the sum of its absolute terms.
"""
import pytest
import torch

import ops_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_grouped_moe_gb300 import build
    build.build()
    from mixture_experts_grouped_moe_gb300 import moe as m
    m.load()
    return m


def drop(ids, E):
    """About a slot in five left out, all of token 3's and all of expert 1's, by ids below and above the range."""
    T, k = ids.shape
    gone = torch.rand(T, k, generator=ref.gen(21)) < 0.2
    gone[3] = True
    gone |= ids == 1
    bad = torch.where(torch.rand(T, k, generator=ref.gen(22)) < 0.5, -1, E).to(torch.int32)
    return torch.where(gone, bad, ids), int(gone.sum())


def nans(*shape, dt=torch.float32):
    return torch.full(shape, float("nan"), dtype=dt, device="cuda")


def deq_rows(q, s):
    return q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, 1)


def deq_weights(q, s):
    return (q.view(torch.float8_e4m3fn).double() *
            s.double().repeat_interleave(128, 1).repeat_interleave(128, 2)[:, :q.shape[1], :q.shape[2]])


def bounded(got, want, lim, label):
    err = (got.double() - want).abs()
    assert torch.isfinite(got).all(), label
    assert (err <= lim).all(), (label, float((err - lim).max()))


# the sorts of few and of many experts, and the one of many slots; blocks of 16 go to the few-row kernel
@pytest.mark.parametrize("T,E,k,block_m", [(40, 8, 2, 128), (30, 40, 3, 128), (900, 8, 2, 128), (20, 6, 2, 16)])
def test_chain(moe, T, E, k, block_m):
    N, K = 256, 384
    ids, wts = ref.route(T, E, k, seed=T)
    ids, gone = drop(ids, E)
    p = ref.sort(ids, E, block_m)
    P, S, rows, pos = p["P"], T * k, p["rows"], p["slot_pos"].long()
    assert 0 < gone < S and (pos < 0).sum() == gone
    x = torch.randn(T, K, generator=ref.gen(1)).to(torch.bfloat16)
    W = torch.randn(E, N, K, generator=ref.gen(2)).to(torch.bfloat16)
    ids_d, wts_d, xd, Wd = ids.cuda(), wts.cuda(), x.cuda(), W.cuda()
    ex, w = moe.TokenExchange(T, k, E, block_m), moe.FP8Weights(Wd, training=True)
    ex.sort(ids_d, wts_d)
    assert int(ex.num_left_out) == gone and int(ex.num_tokens_post_padded) == rows
    for name, got in (("sorted_ids", ex.sorted_ids), ("slot_pos", ex.slot_pos), ("expert_ids", ex.expert_ids),
                      ("counts", ex.expert_counts)):
        assert torch.equal(got.cpu(), p[name]), name

    # dispatch: the slots' rows, zero rows with scale 1 for padding, the rest untouched
    q, s = torch.full((P, K), 0x7F, dtype=torch.uint8, device="cuda"), nans(K // 128, P)
    ex.permute_fp8(xd, q, s)
    xs = torch.zeros(P, K, dtype=torch.bfloat16)
    token = torch.arange(S) // k
    kept = pos >= 0
    xs[pos[kept]] = x[token[kept]]
    wq, ws = ref.quantize_groups(xs)
    gq, gs = q.cpu()[:rows], s.cpu()[:, :rows]
    zero = lambda c: torch.where(c == 0x80, 0, c)  # noqa: E731  (a zero's sign aside)
    assert torch.equal(zero(gq), zero(wq.view(torch.uint8)[:rows])) and torch.equal(gs, ws.t()[:, :rows])
    assert (q.cpu()[rows:] == 0x7F).all() and torch.isnan(s.cpu()[:, rows:]).all()
    xs2 = nans(P, K, dt=torch.bfloat16)
    ex.permute(xd, xs2)
    assert torch.equal(xs2.cpu()[:rows], xs[:rows])

    # grouped product on the exchange's scales by block, and back with the weights
    ys = nans(P, N)
    w.product(q, s, by_block=True, exchange=ex, out=ys)
    A, B = deq_rows(gq, gs.t()), deq_weights(w.q.cpu(), w.s.cpu())
    expert = p["expert_ids"].long().repeat_interleave(block_m)[:rows]
    want, mag = torch.zeros(P, N, dtype=torch.float64), torch.zeros(P, N, dtype=torch.float64)
    for e in range(E):
        r = (expert == e).nonzero()[:, 0]
        want[r], mag[r] = A[r] @ B[e].t(), A[r].abs() @ B[e].abs().t()
    bounded(ys.cpu()[:rows], want[:rows], 2.0 ** -16 * mag[:rows] + 2.0 ** -23 * want[:rows].abs(), "product")
    h = ex.unpermute(ys, out=nans(T, N))
    hw, _ = ref.unpermute(want, p["slot_pos"], wts, T, k)
    _, hm = ref.unpermute(mag, p["slot_pos"], wts, T, k)
    bounded(h.cpu(), hw, 2.0 ** -15 * hm, "unpermute")
    assert not h[3].any()

    # the exchange's gradients
    dout = torch.randn(T, N, generator=ref.gen(3))
    ysr = ys.cpu().double()
    dys, dw = ex.unpermute_backward(dout.cuda(), ys)
    dys_c, dw_c = dys.cpu(), dw.cpu().reshape(-1)
    exact = torch.zeros(P, N, dtype=torch.float64)
    exact[pos[kept]] = wts.reshape(-1)[kept].double()[:, None] * dout.double()[token[kept]]
    bounded(dys_c[:rows], exact[:rows], 2.0 ** -23 * exact[:rows].abs(), "dys")
    terms = dout.double()[token[kept]] * ysr[pos[kept]]
    bounded(dw_c[kept], terms.sum(1), (N + 8) * 2.0 ** -24 * terms.abs().sum(1), "dweights")
    assert not dw_c[~kept].any()
    dxs = torch.randn(P, K, generator=ref.gen(4))
    named = torch.zeros(P, dtype=torch.bool)
    named[pos[kept]] = True
    dxs[~named] = float("nan")
    dx = ex.permute_backward(dxs.cuda()).cpu()
    dx_w, dx_m = ref.unpermute(dxs, p["slot_pos"], None, T, k)
    bounded(dx, dx_w, 2 * (k + 1) * 2.0 ** -24 * dx_m + 2.0 ** -24 * dx_w.abs(), "dx")
    assert not dx[3].any()

    # the product's input gradient, from the output gradient's rows in FP8
    G = dys.to(torch.bfloat16)
    qg, sg = torch.full((P, N), 0x7F, dtype=torch.uint8, device="cuda"), nans(P, N // 128)
    moe.moe_quantize_fp8_act(G, P, N, qg, sg)
    din = w.input_gradient(qg, sg, exchange=ex, out=nans(P, K)).cpu()
    Gd = deq_rows(qg.cpu()[:rows], sg.cpu()[:rows])
    for e in range(E):
        r = (expert == e).nonzero()[:, 0]
        di, dm = Gd[r] @ B[e], Gd[r].abs() @ B[e].abs()
        bounded(din[r], di, 2.0 ** -16 * dm + 2.0 ** -23 * di.abs(), "input gradient")
    if block_m % 128:
        return

    # the weight gradient, from transposed operands
    R = -(-P // 128) * 128
    sid = torch.full((R,), S, dtype=torch.int32, device="cuda")
    sid[:P] = ex.sorted_ids
    qx, sx = torch.full((K, R), 0x7F, dtype=torch.uint8, device="cuda"), nans(R // 128, K)
    qt, st = torch.full((N, R), 0x7F, dtype=torch.uint8, device="cuda"), nans(R // 128, N)
    moe.moe_quantize_fp8_act_t(xd, K, R, K, sid, S, k, ex.num_tokens_post_padded, qx, R, sx)
    moe.moe_quantize_fp8_act_t(G, N, P, N, None, 0, 1, ex.num_tokens_post_padded, qt, R, st)
    xt, xts = ref.quantize_groups(xs[:rows].t().contiguous())
    assert torch.equal(zero(qx.cpu()[:, :rows]), zero(xt.view(torch.uint8)))
    assert torch.equal(sx.cpu()[:rows // 128], xts.t())
    dW = w.weight_gradient(qt, st, qx, sx, exchange=ex, out=nans(E, N, K)).cpu()
    Xd = deq_rows(qx.cpu()[:, :rows], sx.cpu()[:rows // 128].t())
    Gd = deq_rows(qt.cpu()[:, :rows], st.cpu()[:rows // 128].t())
    for e in range(E):
        r = (expert == e).nonzero()[:, 0]
        we, me = Gd[:, r] @ Xd[:, r].t(), Gd[:, r].abs() @ Xd[:, r].abs().t()
        bounded(dW[e], we, 2.0 ** -16 * me + 2.0 ** -23 * we.abs(), "weight gradient")
    assert not dW[1].any()
    assert w.status() == moe.MOE_OK


@pytest.mark.parametrize("T,E", [(1, 4), (5, 40), (600, 8)])
def test_every_slot_left_out(moe, T, E):
    """No row at all: no padding either, zero rows back, and gradients of zero."""
    k, N, K = 2, 128, 128
    ids = torch.full((T, k), E, dtype=torch.int32, device="cuda")
    wts = torch.ones(T, k, device="cuda")
    ex = moe.TokenExchange(T, k, E, 128)
    ex.sort(ids, wts)
    assert int(ex.num_left_out) == T * k and int(ex.num_tokens_post_padded) == 0
    assert not ex.expert_counts.any() and (ex.slot_pos == -1).all() and (ex.sorted_ids == T * k).all()
    w = moe.FP8Weights(torch.ones(E, N, K, dtype=torch.bfloat16, device="cuda"))
    q, s = ex.permute_fp8(torch.ones(T, K, dtype=torch.bfloat16, device="cuda"))
    ys = w.product(q, s, by_block=True, exchange=ex, out=nans(ex.P, N))
    assert torch.isnan(ys).all()
    assert not ex.unpermute(ys, out=nans(T, N)).any()
    _, dw = ex.unpermute_backward(torch.ones(T, N, device="cuda"), ys)
    assert not dw.any()


def test_refusing_sort_still_refuses(moe):
    """moe_align_sort_map keeps -1 for a routing with such an id; the sort that drops them needs its count."""
    T, k, E = 8, 2, 4
    ex = moe.TokenExchange(T, k, E, 16)
    ids = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    ids[2, 1] = E
    args = (ids, torch.ones(T, k, device="cuda"), T, k, E, 16, ex.sorted_ids, ex.sorted_weights, ex.expert_ids,
            ex.num_tokens_post_padded, ex.expert_counts, ex.slot_pos)
    moe.moe_align_sort_map(*args, ex.ws, ex.ws_bytes)
    assert int(ex.num_tokens_post_padded) == -1
    moe.moe_align_sort_drop(*args, ex.num_left_out, ex.ws, ex.ws_bytes)
    assert int(ex.num_tokens_post_padded) == 16 and int(ex.num_left_out) == 1
    with pytest.raises(moe.MoEError):
        moe.moe_align_sort_drop(*args, None, ex.ws, ex.ws_bytes)
