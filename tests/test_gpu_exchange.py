"""The token exchange operators (sort with its inverse map, permute, unpermute and their gradients)
against plain 64-bit forms.

Tolerances, derived: permute moves bits and is compared exactly; so are the sort's maps and the FP8
codes and scales (an IEEE division and a rounding each).  A sum over k <= 32 slots in fp32 has an
error of at most k 2^-24 of the sum of its absolute terms (plus as much again for the products),
and one rounding to the row type; a dot product over H elements summed in fp32 has one of at most
(H + 8) 2^-24 of the sum of its absolute terms.
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


def row_type(moe, t):
    return {"bf16": moe.MOE_ROW_BF16, "fp16": moe.MOE_ROW_FP16, "fp32": moe.MOE_ROW_FP32}[t]


def gpu_plan(p):
    return {n: (v.cuda() if isinstance(v, torch.Tensor) else v) for n, v in p.items()}


def rows(shape, t, seed):
    return (torch.randn(shape, generator=ref.gen(seed)) * 2).to(ref.ROW[t])


@pytest.mark.parametrize("T,E,k,block_m", [(1, 1, 1, 1), (5, 4, 2, 16), (300, 33, 3, 16), (1025, 40, 8, 128),
                                           (700, 8, 2, 1)])
def test_sort_map(moe, T, E, k, block_m):
    ids, wts = ref.route(T, E, k, seed=T)
    if T > 1:  # a slot whose id is out of range is left out and gets position -1
        ids[T // 2, 0] = E
        ids[T - 1, k - 1] = -3
    want = ref.sort(ids, E, block_m)
    got = {n: torch.full_like(want[n], -77).cuda() for n in ("sorted_ids", "slot_pos", "expert_ids", "counts", "npp")}
    sw = torch.empty(want["P"], device="cuda")
    need = moe.moe_align_sort_workspace_size(T, k, E)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    ids_d, wts_d = ids.cuda(), wts.cuda()  # (kept alive over the call)
    moe.moe_align_sort_map(ids_d, wts_d, T, k, E, block_m, got["sorted_ids"], sw, got["expert_ids"], got["npp"],
                           got["counts"], got["slot_pos"], ws, need)
    for n, v in got.items():
        assert torch.equal(v.cpu(), want[n]), n
    pos = want["slot_pos"].long()
    full = torch.zeros(want["P"])
    full[pos[pos >= 0]] = wts.reshape(-1)[pos >= 0]
    assert torch.equal(sw.cpu(), full)


SHAPES = [  # T, H, E, k, block_m
    (1, 1, 1, 1, 1), (3, 7, 4, 2, 16), (37, 129, 8, 3, 16), (64, 128, 16, 8, 64), (130, 1000, 6, 2, 128),
    (9, 5000, 40, 32, 1), (33, 9001, 5, 4, 8), (260, 4096, 8, 2, 128),
]


@pytest.mark.parametrize("t", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,H,E,k,block_m", SHAPES)
def test_permute(moe, T, H, E, k, block_m, t):
    ids, _ = ref.route(T, E, k, seed=1)
    p = ref.sort(ids, E, block_m)
    pos = p["slot_pos"].clone()
    if T > 2:
        pos[0] = -1           # left out
        pos[1] = p["P"] + 5   # outside the rows: skipped
    ld = H + (3 if H % 2 else 8)  # a row pitch of its own, odd and even
    x = rows((T, ld), t, 2)
    for zero in (0, 1):
        want = torch.full((p["P"], H), 5.0, dtype=ref.ROW[t])
        if zero:
            real = p["sorted_ids"][:p["rows"]] < T * k
            want[:p["rows"]][~real] = 0
        for s in range(T * k):
            if 0 <= int(pos[s]) < p["P"]:
                want[int(pos[s])] = x[s // k, :H]
        xs = torch.full((p["P"], H), 5.0, dtype=ref.ROW[t], device="cuda")
        xd, g = x.cuda(), gpu_plan(p)
        moe.moe_permute(row_type(moe, t), xd, ld, pos.cuda(), g["sorted_ids"], g["npp"], T, k, H, p["P"], zero, xs)
        assert torch.equal(xs.cpu(), want), zero


def test_permute_keeps_nan_and_inf_bits(moe):
    ids, _ = ref.route(8, 4, 2, seed=5)
    p = gpu_plan(ref.sort(ids, 4, 16))
    x = torch.randint(-32768, 32767, (8, 64), generator=ref.gen(3), dtype=torch.int16).cuda()
    x[0, 0], x[1, 3] = 0x7F80, 0x7FC1  # bf16 infinity and a NaN
    xs = torch.zeros(p["P"], 64, dtype=torch.int16, device="cuda")
    moe.moe_permute(moe.MOE_ROW_BF16, x, 64, p["slot_pos"], None, None, 8, 2, 64, p["P"], 0, xs)
    assert torch.equal(xs[p["slot_pos"].long()], x.repeat_interleave(2, 0))


@pytest.mark.parametrize("T,H,E,k,block_m", [(1, 128, 1, 1, 1), (37, 384, 8, 3, 16), (300, 4096, 8, 2, 128),
                                             (50, 7168, 16, 8, 64)])
def test_permute_fp8(moe, T, H, E, k, block_m):
    ids, _ = ref.route(T, E, k, seed=1)
    p = ref.sort(ids, E, block_m)
    ld = H + 8
    x = rows((T, ld), "bf16", 2) * torch.exp2(torch.randint(-20, 20, (T, 1), generator=ref.gen(4))).to(torch.bfloat16)
    x[T // 2, :128] = 0  # an all-zero group: scale 1
    x[T // 3, 5] = 3e38  # one outlier in its group
    q, s = ref.quantize_groups(x[:, :H])
    wq = torch.full((p["P"], H), 7, dtype=torch.uint8)
    ws = torch.full((H // 128, p["P"]), 9.0)
    pad = torch.zeros(p["P"], dtype=torch.bool)
    pad[:p["rows"]] = p["sorted_ids"][:p["rows"]] >= T * k
    wq[pad], ws[:, pad] = 0, 1.0
    pos = p["slot_pos"].long()
    wq[pos] = q.view(torch.uint8).repeat_interleave(k, 0)
    ws[:, pos] = s.repeat_interleave(k, 0).t()
    gq = torch.full((p["P"], H), 7, dtype=torch.uint8, device="cuda")
    gs = torch.full((H // 128, p["P"]), 9.0, device="cuda")
    xd, g = x.cuda(), gpu_plan(p)
    moe.moe_permute_fp8(xd, ld, g["slot_pos"], g["sorted_ids"], g["npp"], T, k, H, p["P"], 1, gq, gs)
    assert torch.equal(gs.cpu(), ws)
    # a zero's sign aside, every code is the same
    a, b = gq.cpu(), wq
    assert torch.equal(torch.where(a == 128, 0, a), torch.where(b == 128, 0, b))


@pytest.mark.parametrize("t", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,H,E,k,block_m", SHAPES)
def test_unpermute_and_gradients(moe, T, H, E, k, block_m, t):
    ids, wts = ref.route(T, E, k, seed=1)
    p = ref.sort(ids, E, block_m)
    pos = p["slot_pos"].clone()
    if T > 2:
        pos[0] = -1
        pos[k:2 * k] = -1  # token 1 has no row at all
        wts[2, 0] = 0.0
    rt, g = row_type(moe, t), gpu_plan(p)
    pd, wd = pos.cuda(), wts.cuda()
    ys, dout = rows((p["P"], H), t, 7), rows((T, H + 4), t, 8)
    skipped = torch.ones(p["P"], dtype=torch.bool)
    skipped[pos[pos >= 0].long()] = False
    ys[skipped] = float("nan")  # rows that no slot names are never read
    ysd, doutd = ys.cuda(), dout.cuda()
    half, tiny = ref.HALF_ULP[t], ref.TINY[t]

    for w in (wts, None):
        ld = H + 2
        out = torch.full((T, ld), 3.0, dtype=ref.ROW[t], device="cuda")
        if w is None:
            moe.moe_permute_backward(rt, ysd, pd, T, k, H, p["P"], out, ld)
        else:
            moe.moe_unpermute(rt, ysd, pd, wd, T, k, H, p["P"], out, ld)
        want, mag = ref.unpermute(ys, pos, w, T, k)
        err = (out[:, :H].cpu().double() - want).abs()
        assert (err <= 2 * (k + 1) * 2.0 ** -24 * mag + half * 1.001 * want.abs() + tiny).all()
        assert (out[:, H:] == 3.0).all()
        if T > 2:
            assert not out[1, :H].any()

    for in_place in (False, True):
        dys = ysd.clone() if in_place else torch.full((p["P"], H), 5.0, dtype=ref.ROW[t], device="cuda")
        dw = torch.full((T, k), 9.0, device="cuda")
        moe.moe_unpermute_backward(rt, doutd, H + 4, dys if in_place else ysd, pd, wd, g["sorted_ids"], g["npp"], T, k,
                                   H, p["P"], 1, dys, dw)
        d64 = dout[:, :H].double()
        for s in range(T * k):
            q, tt, j = int(pos[s]), s // k, s % k
            if q < 0:
                assert dw[tt, j] == 0
                continue
            prod = d64[tt] * ys[q].double()
            assert abs(float(dw[tt, j]) - float(prod.sum())) <= (H + 8) * 2.0 ** -24 * float(prod.abs().sum())
            exact = float(wts[tt, j]) * d64[tt]
            err = (dys[q].cpu().double() - exact).abs()
            assert (err <= (half * 1.001 + 2.0 ** -24) * exact.abs() + tiny).all()
        pad = p["sorted_ids"][:p["rows"]] >= T * k
        assert not dys.cpu()[:p["rows"]][pad].any()


def test_gradients_against_differences(moe):
    """The combine is linear in ys and in the weights: a central difference of it along a direction
    equals the gradient's inner product with that direction (fp32 rows)."""
    T, H, E, k = 40, 96, 6, 2
    ids, wts = ref.route(T, E, k, seed=3)
    p = ref.sort(ids, E, 16)
    g = gpu_plan(p)
    real = torch.zeros(p["P"], 1)
    real[p["slot_pos"].long()] = 1
    ys, dirs, dout = (torch.randn(p["P"], H, generator=ref.gen(4)) * real,
                      torch.randn(p["P"], H, generator=ref.gen(5)) * real, torch.randn(T, H, generator=ref.gen(6)))
    dirw = torch.randn(T, k, generator=ref.gen(7))

    def f(y, w):
        return float((ref.unpermute(y, p["slot_pos"], w, T, k)[0] * dout.double()).sum())

    ysd, dd, wd = ys.cuda(), dout.cuda(), wts.cuda()
    dys, dw = torch.zeros(p["P"], H, device="cuda"), torch.empty(T, k, device="cuda")
    moe.moe_unpermute_backward(moe.MOE_ROW_FP32, dd, H, ysd, g["slot_pos"], wd, None, None, T, k, H, p["P"], 0, dys,
                               dw)
    h = 2.0 ** -6
    for grad, diff in ((dys.cpu().double() * dirs, f(ys.double() + h * dirs, wts) - f(ys.double() - h * dirs, wts)),
                       (dw.cpu().double() * dirw, f(ys, wts.double() + h * dirw) - f(ys, wts.double() - h * dirw))):
        # linear: the difference is exact up to fp64; the gradient carries fp32 sums of H terms
        assert abs(float(grad.sum()) - diff / (2 * h)) <= (H + 8) * 2.0 ** -24 * float(grad.abs().sum()) * 4 + 1e-6


def test_round_trip_and_other_stream(moe):
    """Permute then unpermute with weights that sum to 1 gives x back, on a stream of its own."""
    T, H, E, k = 777, 512, 8, 2
    ids, wts = ref.route(T, E, k, seed=3)
    x = rows((T, H), "fp32", 4).cuda()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        plan = moe.TokenExchange(T, k, E, 128)
        plan.sort(ids.cuda(), wts.cuda())
        back = plan.unpermute(plan.permute(x))
    st.synchronize()
    assert (back - x).abs().max() <= 4 * 2.0 ** -24 * x.abs().max()


def test_reproducible(moe):
    T, H, E, k = 500, 1024, 8, 4
    ids, wts = ref.route(T, E, k, seed=3)
    p, wd = gpu_plan(ref.sort(ids, E, 128)), wts.cuda()
    ys, dout = rows((p["P"], H), "bf16", 1).cuda(), rows((T, H), "bf16", 2).cuda()
    got = []
    for _ in range(2):
        out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
        dys, dw = torch.zeros_like(ys), torch.empty(T, k, device="cuda")
        moe.moe_unpermute(moe.MOE_ROW_BF16, ys, p["slot_pos"], wd, T, k, H, p["P"], out, H)
        moe.moe_unpermute_backward(moe.MOE_ROW_BF16, dout, H, ys, p["slot_pos"], wd, None, None, T, k, H, p["P"], 0,
                                   dys, dw)
        got.append((out, dys, dw))
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_zero_tokens(moe):
    one = torch.zeros(64, device="cuda")
    moe.moe_permute(moe.MOE_ROW_FP32, one, 8, one, one, one, 0, 2, 8, 4, 1, one)
    moe.moe_unpermute(moe.MOE_ROW_FP32, one, one, one, 0, 2, 8, 4, one, 8)
    moe.moe_unpermute_backward(moe.MOE_ROW_FP32, one, 8, one, one, one, one, one, 0, 2, 8, 4, 1, one, one)
    torch.cuda.synchronize()
    assert not one.any()
