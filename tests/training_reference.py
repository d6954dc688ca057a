"""Plain 64-bit forms of the rest of a training step (gated feed-forward block, cross entropy over a vocabulary,
gradient norm and clipping), on whatever device their tensors are, and the bounds that its tests hold results to.

Bounds.  A product of 16-bit numbers is exact in fp32; the tensor core's fp32 sums of K of them err by at most
ACC = 2^-16 of the sum of the absolute terms: an MMA adds 16 products at a time, so K = 2^12, the most used
here, takes 2^8 additions, each off by at most one step (2^-23, should it truncate) of a partial sum that grows
from nothing to the whole, half of it on average: 2^8 2^-23 / 2.
Functions: exp and the reciprocal err by a few 2^-22, FN = 2^-19 covers one activation or one softmax term.
A rounding to the row type is half a step, ref.HALF_ULP.  The rest propagates these absolutely."""
import torch

import ops_reference as ref

ACC, FN = 2.0 ** -16, 2.0 ** -19
ACTS = ("silu", "gelu", "relu")


def act(g, kind):
    """(act(g), act'(g))"""
    if kind == "relu":
        on = (g > 0).to(g.dtype)
        return g * on, on
    if kind == "silu":
        q, dq = g, torch.ones_like(g)
    else:
        c = 2 * (2 / torch.pi) ** 0.5
        q, dq = c * (g + 0.044715 * g ** 3), c * (1 + 3 * 0.044715 * g ** 2)
    s = torch.sigmoid(q)
    return g * s, s + g * s * (1 - s) * dq


def ffn(x, wgu, wd, kind, add=None):
    I = wd.shape[1]
    gu = x @ wgu.t()
    h = act(gu[:, :I], kind)[0] * gu[:, I:]
    out = h @ wd.t()
    return gu, h, out if add is None else out + add


def ffn_bound(x, wgu, wd, kind, t, add=None):
    """Largest error of (gu, h, out) of the operator for rows of type t; slopes of the activations are below 1.2."""
    I, e = wd.shape[1], ref.HALF_ULP[t]
    gu, h, out = ffn(x, wgu, wd, kind, add)
    mag = x.abs() @ wgu.abs().t()
    g, u = gu[:, :I], gu[:, I:]
    a = act(g, kind)[0]
    eh = 1.2 * ACC * mag[:, :I] * (u.abs() + ACC * mag[:, I:]) + a.abs() * ACC * mag[:, I:] + (e + FN) * h.abs()
    eh = 1.01 * eh + ref.TINY[t]
    eo = eh @ wd.abs().t() + ACC * ((h.abs() + eh) @ wd.abs().t())
    return (ACC * mag + e * (gu.abs() + ACC * mag) + ref.TINY[t], eh, eo + e * (out.abs() + eo) + ref.TINY[t])


def ffn_grads(x, wgu, wd, kind, gu, h, dout):
    """Formulas of the backward from the kept gate | up and h."""
    I = wd.shape[1]
    a, da = act(gu[:, :I], kind)
    dh = dout @ wd
    dgu = torch.cat([dh * gu[:, I:] * da, dh * a], 1)
    return {"dx": dgu @ wgu, "dW_gate_up": dgu.t() @ x, "dW_down": dout.t() @ h}


def ffn_grads_bound(x, wgu, wd, kind, gu, h, dout, t, grad_t, old=None):
    """Largest errors of the operator's gradients, from the same kept values."""
    I, e = wd.shape[1], ref.HALF_ULP[t]
    a, da = act(gu[:, :I], kind)
    g, u = gu[:, :I], gu[:, I:]
    dh, edh = dout @ wd, ACC * (dout.abs() @ wd.abs())
    # the slope's terms g s (1 - s) q' and s, each to FN of its size; |g s (1 - s) q'| < 1
    slope = da.abs() + 4.0 * (kind != "relu")
    dgu = torch.cat([dh * u * da, dh * a], 1)
    ed = torch.cat([edh * (u * da).abs() + (dh.abs() + edh) * u.abs() * slope * FN,
                    edh * a.abs() + (dh.abs() + edh) * a.abs() * FN], 1) * 1.01
    ed = ed + e * (dgu.abs() + ed) + ref.TINY[t]
    w = ffn_grads(x, wgu, wd, kind, gu, h, dout)
    full = dgu.abs() + ed
    err = {"dx": (ed + ACC * full) @ wgu.abs(), "dW_gate_up": (ed + ACC * full).t() @ x.abs(),
           "dW_down": ACC * (dout.abs().t() @ h.abs())}
    out = {}
    for n, v in err.items():
        tt = t if n == "dx" else grad_t
        o = 0.0 if n == "dx" or old is None else old[n].abs()
        out[n] = v + ref.HALF_ULP[tt] * 2 * (w[n].abs() + v + o) + ref.TINY[tt]
    return w, out


def loss(x, w, targets):
    """(loss, lse)"""
    l = x @ w.t()
    lse = torch.logsumexp(l, 1)
    ok = (targets >= 0) & (targets < w.shape[0])
    at = torch.where(ok, targets, torch.zeros_like(targets)).long()
    own = l.gather(1, at[:, None])[:, 0]
    return torch.where(ok, lse - own, torch.zeros_like(lse)), lse


def loss_bound(x, w, targets):
    """Largest errors of (loss, lse): of a logit ACC of its absolute terms; the sum of V exponentials in parts, 2^-18;
    the last subtractions and the logarithm, 2^-22 of their operands."""
    el = ACC * (x.abs() @ w.abs().t()).amax(1)
    top = (x @ w.t()).abs().amax(1)
    e = el + 2.0 ** -18 + 2.0 ** -21 * (top + 20)
    return 2 * e, e


def loss_grads(x, w, targets, dloss):
    V = w.shape[0]
    ok = (targets >= 0) & (targets < V)
    p = torch.softmax(x @ w.t(), 1)
    at = torch.where(ok, targets, torch.zeros_like(targets)).long()
    p = p.scatter_add(1, at[:, None], -torch.ones_like(p[:, :1]))
    dl = torch.where(ok[:, None], p * dloss[:, None], torch.zeros_like(p))
    return dl, {"dx": dl @ w, "dW": dl.t() @ x}


def loss_grads_bound(x, w, targets, dloss, t, grad_t, old=None):
    e = ref.HALF_ULP[t]
    dl, g = loss_grads(x, w, targets, dloss)
    p = torch.softmax(x @ w.t(), 1)
    mag = x.abs() @ w.abs().t()
    top = (x @ w.t()).abs().amax(1, keepdim=True)
    el = ACC * (mag + mag.amax(1, keepdim=True)) + 2.0 ** -17 + 2.0 ** -20 * (top + 20)
    ok = ((targets >= 0) & (targets < w.shape[0]))[:, None]
    # a power of two brings the largest factor to [2^14, 2^15): below, 16-bit steps are TINY of that scale
    most = dloss[ok[:, 0]].abs().max() if ok.any() else dloss.new_ones(())
    tiny = ref.TINY[t] * float(most) * 2.0 ** -14 * 2
    ed = torch.where(ok, dloss.abs()[:, None] * (p * (torch.expm1(el) + FN) + 2.0 ** -23), torch.zeros_like(p))
    ed = ed + e * (dl.abs() + ed) + torch.where(ok, torch.full_like(p, tiny), torch.zeros_like(p))
    err = {"dx": ed @ w.abs() + ACC * ((dl.abs() + ed) @ w.abs()),
           "dW": ed.t() @ x.abs() + ACC * ((dl.abs() + ed).t() @ x.abs())}
    out = {}
    for n, v in err.items():
        tt = t if n == "dx" else grad_t
        o = 0.0 if n == "dx" or old is None else old.abs()
        out[n] = v + ref.HALF_ULP[tt] * 2 * (g[n].abs() + v + o) + ref.TINY[tt]
    return g, out


def norm(tensors):
    s = sum((t.double() ** 2).sum() for t in tensors) if tensors else torch.zeros((), dtype=torch.float64)
    return torch.as_tensor(s, dtype=torch.float64).sqrt()


def bounded(got, want, bound, label):
    """Every element within its bound, and none a NaN."""
    err = (got.double() - want).abs()
    worst = (err / bound).nan_to_num(nan=float("inf")).max() if err.numel() else torch.zeros(())
    off = int((~(err <= bound)).sum())
    assert not off, (label, f"worst error / bound {float(worst):.3g}", f"{off} of {err.numel()}")
