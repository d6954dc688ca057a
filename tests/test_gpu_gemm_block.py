"""The block-scaled FP8 product (dense and grouped by expert), its weight gradient and the transposing
quantiser against plain 64-bit forms.

Tolerances, derived.  Products of e4m3 codes are exact in fp32 (8 significant bits); the tensor core
adds the 128 products of a block in fp32, at worst cutting each addend to 2^-21 of the block's
largest, and the block sums are scaled and added in fp32.  So an element differs from the 64-bit
value by at most 2^-16 of the sum of its absolute terms, plus half a unit of the output type.
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


def codes(shape, seed):
    return (torch.randn(shape, generator=ref.gen(seed)) * 120).clamp(-448, 448).to(torch.float8_e4m3fn)


def scales(shape, seed):
    return torch.exp(torch.randn(shape, generator=ref.gen(seed))) * 1e-2


def workspace(moe):
    return torch.zeros(moe.MOE_GEMM_BLOCK_WS_BYTES, dtype=torch.uint8, device="cuda")


def close(got, want, mag, out):
    err = (got.double() - want).abs()
    lim = 2.0 ** -16 * mag + ref.HALF_ULP[out] * 1.001 * want.abs()
    assert torch.isfinite(got).all()
    assert (err <= lim).all(), float((err - lim).max())


def out_type(moe, out):
    return moe.MOE_ROW_FP32 if out == "fp32" else moe.MOE_ROW_BF16


@pytest.mark.parametrize("by_block", [0, 1])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 16), (1, 4096, 1024), (3, 130, 144), (16, 128, 128), (17, 256, 2048), (33, 777, 400), (64, 1000, 4096),
    (65, 64, 128), (128, 256, 384), (200, 1001, 272), (1000, 513, 640), (129, 8200, 512), (2500, 2304, 256),
])
def test_dense(moe, M, N, K, out, by_block):
    KB, NB = -(-K // 128), -(-N // 128)
    a, b, sa, sb = codes((M, K), 1), codes((N, K), 2), scales((M, KB), 3), scales((NB, KB), 4)
    want, mag = ref.product(a, sa, b, sb)
    ld = N + 5
    d = torch.full((M, ld), 3.0, dtype=ref.ROW[out], device="cuda")
    ad, bd, sbd = a.cuda(), b.cuda(), sb.cuda()
    sad = (sa.t().contiguous() if by_block else sa).cuda()
    ws = workspace(moe)
    moe.moe_gemm_fp8_block(ad, sad, by_block, bd, sbd, M, N, K, 1, 0, None, None, out_type(moe, out), d, ld, ws,
                           ws.numel())
    close(d[:, :N].cpu(), want, mag, out)
    assert (d[:, N:] == 3.0).all()
    assert moe.moe_workspace_status(ws) == moe.MOE_OK
    # a row pitch that the wide stores take
    if N % 8 == 0:
        d2 = torch.empty(M, N, dtype=ref.ROW[out], device="cuda")
        moe.moe_gemm_fp8_block(ad, sad, by_block, bd, sbd, M, N, K, 1, 0, None, None, out_type(moe, out), d2, N, ws,
                               ws.numel())
        assert torch.equal(d2, d[:, :N])


@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("T,E,k,block_m,N,K", [
    (1, 4, 2, 16, 256, 512), (32, 8, 2, 16, 384, 1024), (60, 5, 3, 32, 200, 256), (100, 6, 2, 64, 1000, 144),
    (300, 8, 2, 128, 640, 512), (20, 40, 4, 128, 136, 256), (500, 3, 1, 256, 3001, 128), (900, 8, 2, 128, 2048, 256),
])
def test_grouped(moe, T, E, k, block_m, N, K, out):
    ids, _ = ref.route(T, E, k, seed=5)
    ids[ids == E - 1] = 0  # an expert without tokens (a token may repeat an expert here)
    p = ref.sort(ids, E, block_m)
    P, KB, NB = p["P"], -(-K // 128), -(-N // 128)
    a, b, sa, sb = codes((P, K), 1), codes((E, N, K), 2), scales((P, KB), 3), scales((E, NB, KB), 4)
    sa[p["rows"]:] = float("nan")  # rows past the sorted ones are never part of a result
    d = torch.full((P, N), 3.0, dtype=ref.ROW[out], device="cuda")
    ad, sad, bd, sbd, eid, npp = a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), p["expert_ids"].cuda(), p["npp"].cuda()
    ws = workspace(moe)
    moe.moe_gemm_fp8_block(ad, sad, 0, bd, sbd, P, N, K, E, block_m, eid, npp, out_type(moe, out), d, N, ws,
                           ws.numel())
    got = d.cpu()
    for i in range(p["rows"] // block_m):
        e, r = int(p["expert_ids"][i]), slice(i * block_m, (i + 1) * block_m)
        want, mag = ref.product(a[r], sa[r], b[e], sb[e])
        close(got[r], want, mag, out)
    assert (got[p["rows"]:] == 3.0).all()
    assert moe.moe_workspace_status(ws) == moe.MOE_OK


def test_rejected_sort_computes_nothing(moe):
    """num_tokens_post_padded = -1 (a bad id): no row of D is written."""
    P, N, K = 256, 256, 256
    a, b = codes((P, K), 1).cuda(), codes((2, N, K), 2).cuda()
    sa, sb = torch.ones(P, 2, device="cuda"), torch.ones(2, 2, 2, device="cuda")
    npp = torch.tensor([-1], dtype=torch.int32, device="cuda")
    for block_m in (16, 128):
        eid = torch.zeros(P // block_m, dtype=torch.int32, device="cuda")
        d = torch.full((P, N), 3.0, device="cuda")
        ws = workspace(moe)
        moe.moe_gemm_fp8_block(a, sa, 0, b, sb, P, N, K, 2, block_m, eid, npp, moe.MOE_ROW_FP32, d, N, ws, ws.numel())
        assert (d == 3.0).all()


def test_nan_code_stays_in_its_row(moe):
    M, N, K = 150, 300, 256
    a, b, sa, sb = codes((M, K), 1), codes((N, K), 2), scales((M, 2), 3), scales((3, 2), 4)
    a.view(torch.uint8)[7, 130] = 0x7F  # e4m3 NaN
    for m in (M, 20):
        d = torch.empty(m, N, device="cuda")
        ad, sad, bd, sbd, ws = a[:m].contiguous().cuda(), sa[:m].contiguous().cuda(), b.cuda(), sb.cuda(), workspace(moe)
        moe.moe_gemm_fp8_block(ad, sad, 0, bd, sbd, m, N, K, 1, 0, None, None, moe.MOE_ROW_FP32, d, N, ws, ws.numel())
        nan = torch.isnan(d).cpu()
        assert nan[7].all() and nan.sum() == N


@pytest.mark.parametrize("rows,C", [(1, 8), (128, 64), (300, 200), (1000, 1096)])
def test_transposing_quantiser(moe, rows, C):
    x = (torch.randn(rows, C + 8, generator=ref.gen(6)) * 3).to(torch.bfloat16)
    x[:min(rows, 128), 3] = 0
    R = -(-rows // 128) * 128
    xt = torch.zeros(C, R, dtype=torch.bfloat16)
    xt[:, :rows] = x[:, :C].t()
    q, s = ref.quantize_groups(xt)
    gq = torch.full((C, R + 16), 9, dtype=torch.uint8, device="cuda")
    gs = torch.empty(R // 128, C, device="cuda")
    xd = x.cuda()
    moe.moe_quantize_fp8_act_t(xd, C + 8, rows, C, None, 0, 1, None, gq, R + 16, gs)
    assert torch.equal(gs.cpu(), s.t())
    a, b = gq[:, :R].cpu(), q.view(torch.uint8)
    assert torch.equal(torch.where(a == 128, 0, a), torch.where(b == 128, 0, b))
    assert (gq[:, R:] == 9).all()


def test_transposing_quantiser_gathers_in_sorted_order(moe):
    T, E, k, C = 150, 4, 2, 72
    ids, _ = ref.route(T, E, k, seed=5)
    p = ref.sort(ids, E, 128)
    R = -(-p["P"] // 128) * 128
    x = torch.randn(T, C, generator=ref.gen(7)).to(torch.bfloat16)
    xs = torch.zeros(R, C, dtype=torch.bfloat16)
    xs[p["slot_pos"].long()] = x.repeat_interleave(k, 0)
    q, s = ref.quantize_groups(xs.t().contiguous())
    sid = torch.full((R,), T * k, dtype=torch.int32)
    sid[:p["P"]] = p["sorted_ids"]
    xd, sidd, npp = x.cuda(), sid.cuda(), p["npp"].cuda()
    gq, gs = torch.full((C, R), 9, dtype=torch.uint8, device="cuda"), torch.full((R // 128, C), 9.0, device="cuda")
    moe.moe_quantize_fp8_act_t(xd, C, R, C, sidd, T * k, k, npp, gq, R, gs)
    n = p["rows"]
    a, b = gq[:, :n].cpu(), q.view(torch.uint8)[:, :n]
    assert torch.equal(torch.where(a == 128, 0, a), torch.where(b == 128, 0, b))
    assert torch.equal(gs[:n // 128].cpu(), s.t()[:n // 128])
    assert (gq[:, n:] == 9).all() and (gs[n // 128:] == 9).all()


def wgrad_operands(M, N, P, seed):
    a, b = codes((M, P), seed), codes((N, P), seed + 1)
    return a, scales((P // 128, M), seed + 2), b, scales((P // 128, N), seed + 3)


@pytest.mark.parametrize("M,N,counts", [
    (5, 4, [128]), (128, 256, [300, 0, 5]), (200, 136, [1, 1, 1, 260]), (640, 1024, [0, 0, 700, 129, 0, 64, 3, 1]),
    (1500, 2052, [400, 90]), (256, 512, [0]),
])
@pytest.mark.parametrize("accumulate", [0, 1])
def test_weight_gradient(moe, M, N, counts, accumulate):
    E = len(counts)
    blocks = [-(-c // 128) for c in counts]
    P = 128 * (sum(blocks) + 1)  # one unused block at the end
    a, sa, b, sb = wgrad_operands(M, N, P, 1)
    D0 = torch.randn(E, M, N, generator=ref.gen(9))
    D = D0.cuda() if accumulate else torch.full((E, M, N), float("nan"), device="cuda")
    ad, sad, bd, sbd, c, ws = (*(v.cuda() for v in (a, sa, b, sb, torch.tensor(counts, dtype=torch.int32))),
                               workspace(moe))
    moe.moe_wgrad_fp8_block(ad, sad, bd, sbd, P, M, N, E, c, D, accumulate, ws, ws.numel())
    af = a.double() * sa.double().repeat_interleave(128, 0).t()
    bf = b.double() * sb.double().repeat_interleave(128, 0).t()
    at = 0
    for e, nb in enumerate(blocks):
        r = slice(128 * at, 128 * (at + nb))
        at += nb
        want, mag = af[:, r] @ bf[:, r].t(), af[:, r].abs() @ bf[:, r].abs().t()
        if accumulate:
            want, mag = want + D0[e].double(), mag + D0[e].double().abs()
        close(D[e].cpu(), want, mag, "fp32")
        if nb == 0 and not accumulate:
            assert not D[e].any()
    assert moe.moe_workspace_status(ws) == moe.MOE_OK


def test_weight_gradient_of_the_product(moe):
    """loss = sum(G * (X W^T)) over each expert's rows: the operators' gradient from transposed,
    quantised X and G equals a difference of the loss in 64 bits along a direction of W, and the
    formula G^T X, to the quantisation's error (each factor is off by at most 2^-4 of itself)."""
    T, E, k, N, K = 200, 3, 2, 96, 136
    ids, _ = ref.route(T, E, k, seed=5)
    p = ref.sort(ids, E, 128)
    R = -(-p["P"] // 128) * 128
    sid = torch.full((R,), T * k, dtype=torch.int32)
    sid[:p["P"]] = p["sorted_ids"]
    x = torch.randn(T, K, generator=ref.gen(1)).to(torch.bfloat16)
    G = torch.zeros(R, N, dtype=torch.bfloat16)
    G[p["slot_pos"].long()] = torch.randn(T * k, N, generator=ref.gen(2)).to(torch.bfloat16)
    xd, Gd, sidd, npp, cnt, ws = (*(v.cuda() for v in (x, G, sid, p["npp"], p["counts"])), workspace(moe))
    qx, sx = torch.zeros(K, R, dtype=torch.uint8, device="cuda"), torch.zeros(R // 128, K, device="cuda")
    qg, sg = torch.zeros(N, R, dtype=torch.uint8, device="cuda"), torch.zeros(R // 128, N, device="cuda")
    moe.moe_quantize_fp8_act_t(xd, K, R, K, sidd, T * k, k, npp, qx, R, sx)
    moe.moe_quantize_fp8_act_t(Gd, N, R, N, None, 0, 1, npp, qg, R, sg)
    D = torch.empty(E, N, K, device="cuda")
    moe.moe_wgrad_fp8_block(qg, sg, qx, sx, R, N, K, E, cnt, D, 0, ws, ws.numel())
    xs = torch.zeros(R, K, dtype=torch.float64)
    xs[p["slot_pos"].long()] = x.double().repeat_interleave(k, 0)
    W = torch.randn(E, N, K, generator=ref.gen(3), dtype=torch.float64)
    V = torch.randn(E, N, K, generator=ref.gen(4), dtype=torch.float64)

    def loss(w):
        at, total = 0, 0.0
        for e, c in enumerate(p["counts"].tolist()):
            r = slice(at, at + -(-c // 128) * 128)
            at = r.stop
            total += float((G[r].double() * (xs[r] @ w[e].t())).sum())
        return total

    diff = (loss(W + 1e-3 * V) - loss(W - 1e-3 * V)) / 2e-3
    # quantisation errors of the elements are independent: the inner product of about
    # E*N*K*T*k/E terms errs by 2^-4.. of the root of the sum of squares, well inside 5 % of it
    at = 0
    sq = 0.0
    for e, c in enumerate(p["counts"].tolist()):
        r = slice(at, at + -(-c // 128) * 128)
        at = r.stop
        want = G[r].double().t() @ xs[r]
        mag = G[r].double().abs().t() @ xs[r].abs()
        assert ((D[e].cpu().double() - want).abs() <= 0.13 * mag).all()
        sq += float((V[e].pow(2) * (G[r].double().pow(2).t() @ xs[r].pow(2))).sum())
    assert abs(float((D.cpu().double() * V).sum()) - diff) <= 0.2 * sq ** 0.5 + 1e-6 * abs(diff)


def test_reproducible(moe):
    for M, N, K in ((1, 2048, 8192), (700, 1024, 1024)):
        a, b, sa, sb = codes((M, K), 1).cuda(), codes((N, K), 2).cuda(), scales((M, K // 128), 3).cuda(), \
            scales((N // 128, K // 128), 4).cuda()
        ws = workspace(moe)
        got = []
        for _ in range(2):
            d = torch.empty(M, N, device="cuda")
            moe.moe_gemm_fp8_block(a, sa, 0, b, sb, M, N, K, 1, 0, None, None, moe.MOE_ROW_FP32, d, N, ws, ws.numel())
            got.append(d)
        assert torch.equal(*got)
