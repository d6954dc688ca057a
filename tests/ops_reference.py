"""Plain 64-bit forms of the operators around the layer, for their tests (CPU tensors)."""
import torch

ROW = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# half a unit in the last place of a rounded result, relative to it
HALF_ULP = {n: torch.finfo(t).eps / 2 for n, t in ROW.items()}
# the smallest positive step of the type (results below the normal range round absolutely)
TINY = {"bf16": 2.0 ** -133, "fp16": 2.0 ** -25, "fp32": 2.0 ** -149}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def route(T, E, k, seed):
    """Distinct experts per token, and weights that sum to 1."""
    val, ids = torch.randn(T, E, generator=gen(seed)).topk(k, dim=1)
    return ids.to(torch.int32), torch.softmax(val, 1)


def sort(ids, E, block_m):
    """Slot order by expert, whole blocks per expert: dict of CPU int tensors (bad ids left out)."""
    T, k = ids.shape
    S = T * k
    P = S + E * block_m - k
    flat = ids.reshape(-1).tolist()
    sorted_ids, slot_pos, eids, counts = [S] * P, [-1] * S, [-1] * (-(-P // block_m)), [0] * E
    at = 0
    for e in range(E):
        mine = [s for s, v in enumerate(flat) if v == e]
        counts[e] = len(mine)
        for i, s in enumerate(mine):
            sorted_ids[at + i] = s
            slot_pos[s] = at + i
        pad = -(-len(mine) // block_m) * block_m
        for b in range(at // block_m, (at + pad) // block_m):
            eids[b] = e
        at += pad
    bad = any(not 0 <= v < E for v in flat)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return {"sorted_ids": i32(sorted_ids), "slot_pos": i32(slot_pos), "expert_ids": i32(eids), "counts": i32(counts),
            "npp": i32([-1 if bad else at]), "rows": at, "P": P}


def unpermute(ys, slot_pos, wts, T, k):
    """(sum, sum of absolute terms) over each token's slots, skipping positions outside the rows."""
    out = torch.zeros(T, ys.shape[1], dtype=torch.float64)
    mag = torch.zeros_like(out)
    for t in range(T):
        for j in range(k):
            p = int(slot_pos[t * k + j])
            if 0 <= p < ys.shape[0]:
                w = 1.0 if wts is None else float(wts[t, j])
                out[t] += w * ys[p].double()
                mag[t] += abs(w) * ys[p].double().abs()
    return out, mag


def quantize_groups(x):
    """e4m3 codes (as float64 values) and fp32 scales per 1x128 group of each row."""
    g = x.float().view(x.shape[0], -1, 128)
    amax = g.abs().amax(2)
    s = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    q = (g / s[:, :, None]).to(torch.float8_e4m3fn)
    return q.view(x.shape), s


def product(a, sa, b, sb):
    """Dequantised product of one expert: (D, sum of absolute terms), a [M][K], sa [M][KB], b [N][K], sb [NB][KB]."""
    K = a.shape[1]
    ad = a.double() * sa.double().repeat_interleave(128, 1)[:, :K]
    bd = b.double() * sb.double().repeat_interleave(128, 0)[:b.shape[0]].repeat_interleave(128, 1)[:, :K]
    return ad @ bd.t(), ad.abs() @ bd.abs().t()


def block_norm(h, res, gate, w_post, w_pre, scale, offset, eps):
    """y, z, rstd_h, rstd_y in float64; gate broadcastable or None, w_post / w_pre or None."""
    rh = (h.pow(2).mean(1, keepdim=True) + eps).rsqrt()
    n = h if w_post is None else h * rh * (w_post + offset)
    y = res + scale * (n if gate is None else gate * n)
    ry = (y.pow(2).mean(1, keepdim=True) + eps).rsqrt()
    z = None if w_pre is None else y * ry * (w_pre + offset)
    return y, z, rh, ry


def block_norm_grads(h, y, gate, w_post, w_pre, rh, ry, dy, dz, scale, offset):
    """The formulas of the backward, in float64, from a given y."""
    D = torch.zeros_like(h) if dy is None else dy.clone()
    out = {}
    if w_pre is not None:
        u = dz * (w_pre + offset)
        yh = y * ry
        D = D + ry * (u - yh * (u * yh).mean(1, keepdim=True))
        out["dw_pre"] = (dz * yh).sum(0)
    hh = h * (rh if w_post is not None else torch.ones_like(rh))
    w = 1.0 if w_post is None else w_post + offset
    dn = scale * D * (1.0 if gate is None else gate)
    v = dn * w
    if w_post is None:
        out["dh"] = v
    else:
        out["dh"] = rh * (v - hh * (v * hh).mean(1, keepdim=True))
        out["dw_post"] = (dn * hh).sum(0)
    out["d_residual"] = D
    out["dgate_el"] = scale * hh * w * D
    return out
