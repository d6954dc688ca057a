"""The norms around a block, with gate and residual scale, against their 64-bit formulas.

Tolerances, derived.  Sums over H elements in fp32 err by at most (H / 256 + 16) 2^-24 relative to
their absolute terms with the kernel's tree (a thread adds at most H / threads values in turn, then
a tree); 16384 elements give below 2^-17.  Every result is a short chain of fp32 operations on such
a sum and then one rounding to the row type, so an element may differ from the 64-bit value by half
a unit of the row type plus 2^-16 of the magnitudes it is formed from.  The backward's reference
starts from the kernel's own rounded y, as the operator does.
"""
import pytest
import torch

import ops_reference as ref

pytestmark = pytest.mark.gpu
GATES = ["none", "channel", "token", "full"]


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_grouped_moe_gb300 import build
    build.build()
    from mixture_experts_grouped_moe_gb300 import moe as m
    m.load()
    return m


def make(T, H, t, gate, seed, post=True, pre=True):
    g = ref.gen(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    dt = ref.ROW[t]
    d = {"h": (r(T, H) * torch.exp(r(T, 1))).to(dt), "res": (2 * r(T, H)).to(dt),
         "w_post": (1 + 0.3 * r(H)).to(dt) if post else None, "w_pre": (1 + 0.3 * r(H)).to(dt) if pre else None,
         "dy": r(T, H).to(dt), "dz": r(T, H).to(dt) if pre else None}
    shape = {"none": None, "channel": (1, H), "token": (T, 1), "full": (T, H)}[gate]
    d["gate"] = None if shape is None else torch.sigmoid(r(*shape)).to(dt)
    return d


def run(moe, d, t, gate, scale, offset, eps, use_dy=True):
    rt = {"bf16": moe.MOE_ROW_BF16, "fp16": moe.MOE_ROW_FP16, "fp32": moe.MOE_ROW_FP32}[t]
    gk = GATES.index(gate)
    T, H = d["h"].shape
    c = {n: None if v is None else v.cuda() for n, v in d.items()}
    new = lambda *s, dt=torch.float32: torch.full(s, float("nan"), dtype=dt, device="cuda")  # noqa: E731
    o = {"y": new(T, H, dt=ref.ROW[t]), "z": new(T, H, dt=ref.ROW[t]) if d["w_pre"] is not None else None,
         "rh": new(T), "ry": new(T)}
    moe.moe_block_norm(rt, c["h"], c["res"], c["gate"], gk, c["w_post"], c["w_pre"], T, H, scale, offset, eps, o["y"],
                       o["z"], o["rh"], o["ry"])
    o["d_residual"], o["dh"] = new(T, H, dt=ref.ROW[t]), new(T, H, dt=ref.ROW[t])
    o["dgate"] = None if c["gate"] is None else new(*c["gate"].shape, dt=ref.ROW[t] if gate == "full" else torch.float32)
    o["dw_post"] = new(H) if d["w_post"] is not None else None
    o["dw_pre"] = new(H) if d["w_pre"] is not None else None
    need = moe.moe_block_norm_workspace_size(T, H)
    ws = new(need // 4)
    moe.moe_block_norm_backward(rt, c["h"], c["res"], c["gate"], gk, c["w_post"], c["w_pre"], o["rh"], o["ry"],
                                c["dy"] if use_dy else None, c["dz"], T, H, scale, offset, o["d_residual"], o["dh"],
                                o["dgate"], o["dw_post"], o["dw_pre"], ws, need)
    return {n: None if v is None else v.cpu() for n, v in o.items()}


def close(got, want, mag, half, tiny, label, rel=2.0 ** -16):
    err = (got.double() - want).abs()
    lim = rel * mag + half * 1.001 * want.abs() + tiny
    assert torch.isfinite(got).all(), label
    assert (err <= lim).all(), (label, float((err - lim).max()), float(err.max()))


def check(moe, T, H, t, gate, seed, post=True, pre=True, scale=0.3, offset=0.0, eps=1e-6, use_dy=True):
    d = make(T, H, t, gate, seed, post, pre)
    o = run(moe, d, t, gate, scale, offset, eps, use_dy)
    f = {n: None if v is None else v.double() for n, v in d.items()}
    half, tiny = ref.HALF_ULP[t], ref.TINY[t]
    y, z, rh, ry = ref.block_norm(f["h"], f["res"], f["gate"], f["w_post"], f["w_pre"], scale, offset, eps)
    close(o["y"], y, f["res"].abs() + (y - f["res"]).abs(), half, tiny, "y")
    if pre:
        # z's magnitude follows y's own terms
        zm = (f["res"].abs() + (y - f["res"]).abs()) * ry * (f["w_pre"] + offset).abs()
        close(o["z"], z, zm, half, tiny, "z")
        assert ((o["ry"].double() - ry[:, 0]).abs() <= 2.0 ** -16 * ry[:, 0]).all()
    if post:
        assert ((o["rh"].double() - rh[:, 0]).abs() <= 2.0 ** -16 * rh[:, 0]).all()
    g = ref.block_norm_grads(f["h"], y, f["gate"], f["w_post"], f["w_pre"], rh, ry, f["dy"] if use_dy else None,
                             f["dz"], scale, offset)
    # magnitudes: every term of D with the row mean's largest contribution
    D = torch.zeros_like(y) if not use_dy else f["dy"].abs()
    if pre:
        u = (f["dz"] * (f["w_pre"] + offset)).abs()
        yh = (f["res"].abs() + (y - f["res"]).abs()) * ry
        D = D + ry * (u + yh * (u * yh).mean(1, keepdim=True))
        close(o["dw_pre"], g["dw_pre"], (f["dz"].abs() * yh).sum(0), 2.0 ** -24, 0.0, "dw_pre")
    close(o["d_residual"], g["d_residual"], D, half, tiny, "d_residual")
    hh = (f["h"] * (rh if post else 1.0)).abs()
    w = torch.ones(1, dtype=torch.float64) if not post else (f["w_post"] + offset).abs()
    dn = abs(scale) * D * (1.0 if f["gate"] is None else f["gate"].abs())
    v = dn * w
    if post:
        close(o["dh"], g["dh"], rh * (v + hh * (v * hh).mean(1, keepdim=True)), half, tiny, "dh")
        close(o["dw_post"], g["dw_post"], (dn * hh).sum(0), 2.0 ** -24, 0.0, "dw_post")
    else:
        close(o["dh"], g["dh"], v, half, tiny, "dh")
    gm = abs(scale) * hh * w * D
    if gate == "full":
        close(o["dgate"], g["dgate_el"], gm, half, tiny, "dgate")
    elif gate == "channel":
        close(o["dgate"], g["dgate_el"].sum(0, keepdim=True), gm.sum(0, keepdim=True), 2.0 ** -24, 0.0, "dgate")
    elif gate == "token":
        close(o["dgate"], g["dgate_el"].sum(1, keepdim=True), gm.sum(1, keepdim=True), 2.0 ** -24, 0.0, "dgate")


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("t", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,H", [(1, 1), (1, 128), (5, 97), (33, 1000), (700, 257), (310, 4096)])
def test_shapes(moe, T, H, t, gate):
    check(moe, T, H, t, gate, seed=T + H)


@pytest.mark.parametrize("t,H", [("bf16", 2056), ("bf16", 7168), ("bf16", 16384), ("bf16", 3001), ("bf16", 9001),
                                 ("fp32", 1500), ("fp32", 5000), ("fp32", 12292), ("fp32", 16383), ("fp16", 4100)])
def test_widths(moe, t, H):
    """Every number of pieces a thread holds, aligned and odd widths."""
    check(moe, 7, H, t, "channel", seed=H)


@pytest.mark.parametrize("post,pre,use_dy", [(False, True, True), (True, False, True), (True, True, False),
                                             (False, False, True)])
@pytest.mark.parametrize("gate", ["none", "token"])
def test_one_norm_only(moe, post, pre, use_dy, gate):
    check(moe, 400, 640, "bf16", gate, seed=9, post=post, pre=pre, use_dy=use_dy, offset=1.0, scale=-0.7)


def test_weight_offset_and_eps(moe):
    check(moe, 20, 512, "fp32", "full", seed=10, offset=1.0, eps=0.1)


def test_zero_rows(moe):
    """A row of zeros: rstd = eps^-1/2, nothing becomes NaN."""
    d = make(4, 256, "bf16", "channel", 11)
    d["h"][1], d["res"][1] = 0, 0
    o = run(moe, d, "bf16", "channel", 1.0, 0.0, 1e-6)
    assert not o["y"][1].any() and not o["z"][1].any()
    assert abs(float(o["rh"][1]) - 1000.0) < 0.1
    assert all(torch.isfinite(v).all() for v in o.values() if v is not None)


def test_nan_stays_in_its_row(moe):
    d = make(6, 300, "fp32", "token", 12)
    d["h"][2, 7], d["res"][4, 9] = float("nan"), float("inf")
    o = run(moe, d, "fp32", "token", 1.0, 0.0, 1e-6)
    for r in range(6):
        assert torch.isfinite(o["y"][r]).all() == (r not in (2, 4))
        assert torch.isfinite(o["d_residual"][r]).all() == (r not in (2, 4))


def test_in_place(moe):
    T, H = 50, 1024
    d = make(T, H, "bf16", "channel", 13)
    want = run(moe, d, "bf16", "channel", 0.5, 0.0, 1e-6)
    c = {n: v.cuda() for n, v in d.items()}
    rh, ry = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    h2, res2 = c["h"].clone(), c["res"].clone()
    moe.moe_block_norm(moe.MOE_ROW_BF16, h2, res2, c["gate"], 1, c["w_post"], c["w_pre"], T, H, 0.5, 0.0, 1e-6,
                       res2, h2, rh, ry)  # y over the residual, z over h
    assert torch.equal(res2.cpu(), want["y"]) and torch.equal(h2.cpu(), want["z"])
    need = moe.moe_block_norm_workspace_size(T, H)
    ws, dwo, dwi, dg = (torch.empty(n, device="cuda") for n in (need // 4, H, H, H))
    moe.moe_block_norm_backward(moe.MOE_ROW_BF16, c["h"], c["res"], c["gate"], 1, c["w_post"], c["w_pre"], rh, ry,
                                c["dy"], c["dz"], T, H, 0.5, 0.0, c["dy"], c["h"], dg, dwo, dwi, ws, need)
    assert torch.equal(c["dy"].cpu(), want["d_residual"]) and torch.equal(c["h"].cpu(), want["dh"])
    assert torch.equal(dg.cpu(), want["dgate"][0]) and torch.equal(dwo.cpu(), want["dw_post"])


def test_gradients_against_differences(moe):
    """Central differences of the 64-bit forward along random directions equal the gradients' inner
    products with them: truncation of order step^2, fp32 gradients of relative error 2^-16."""
    T, H, scale, offset, eps = 12, 160, 0.4, 1.0, 1e-5
    for gate in GATES:
        d = make(T, H, "fp32", gate, 14)
        o = run(moe, d, "fp32", gate, scale, offset, eps)
        f = {n: None if v is None else v.double() for n, v in d.items()}

        def loss(p):
            y, z, _, _ = ref.block_norm(p["h"], p["res"], p["gate"], p["w_post"], p["w_pre"], scale, offset, eps)
            return float((y * f["dy"]).sum() + (z * f["dz"]).sum())

        grads = {"h": o["dh"], "res": o["d_residual"], "w_post": o["dw_post"], "w_pre": o["dw_pre"]}
        if gate != "none":
            grads["gate"] = o["dgate"]
        for n, grad in grads.items():
            direction = torch.randn(f[n].shape, generator=ref.gen(15), dtype=torch.float64)
            step = 1e-5
            up, down = dict(f), dict(f)
            up[n], down[n] = f[n] + step * direction, f[n] - step * direction
            diff = (loss(up) - loss(down)) / (2 * step)
            terms = grad.double().view(direction.shape) * direction
            assert abs(float(terms.sum()) - diff) <= 2.0 ** -14 * float(terms.abs().sum()) + 1e-6, (gate, n)


def test_reproducible_and_no_rows(moe):
    d = make(1000, 384, "bf16", "channel", 16)
    a, b = (run(moe, d, "bf16", "channel", 0.5, 0.0, 1e-6) for _ in range(2))
    assert all(torch.equal(a[n], b[n]) for n in a)
    # no rows: the column sums are zero
    e = torch.empty(8, device="cuda")
    dwo, dwi = torch.full((8,), 3.0, device="cuda"), torch.full((8,), 3.0, device="cuda")
    need = moe.moe_block_norm_workspace_size(0, 8)
    ws = torch.empty(need // 4, device="cuda")
    moe.moe_block_norm_backward(2, e, e, None, 0, e, e, e, e, e, e, 0, 8, 1.0, 0.0, e, e, None, dwo, dwi, ws, need)
    assert not dwo.any() and not dwi.any()
