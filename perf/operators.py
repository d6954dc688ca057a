"""Cases of the operators around the fused MoE layer: the token exchange (sort by expert, permute,
unpermute and their gradients), the block-scaled FP8 product (dense, grouped by expert, weight
gradient) and the norms before and after a block with its gate and residual scale.

`run` computes a case in its plain form (elementary torch operations in 32 bits) or, with `own`
set, through the package's entry points; `exact` gives the same results from the definitions in
64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
E4M3_MAX = 448.0


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # a handful of tokens of a small layer: the exchange's latency
        {"name": "dispatch_tiny", "op": "dispatch", "T": 16, "H": 128, "E": 4, "k": 2, "block_m": 16, "type": "bf16",
         "zipf": 0.0},
        # FP8 prefill: the rows leave as e4m3 codes with their 1x128 scales, ready for the grouped product
        {"name": "dispatch_fp8_prefill", "op": "dispatch_fp8", "T": 8192, "H": 4096, "E": 8, "k": 2, "block_m": 128,
         "type": "bf16", "zipf": 0.3},
        # an odd width and token count in full precision, three experts a token
        {"name": "combine_odd_fp32", "op": "combine", "T": 1023, "H": 1001, "E": 24, "k": 3, "block_m": 1,
         "type": "fp32", "zipf": 0.5},
        # training on many small experts: both gradients of the exchange
        {"name": "exchange_bwd_finegrained", "op": "exchange_bwd", "T": 4096, "H": 7168, "E": 256, "k": 8,
         "block_m": 128, "type": "bf16", "zipf": 1.2},
        # one token through one expert's down projection: streaming the weights
        {"name": "product_single", "op": "product", "T": 1, "N": 4096, "K": 14336, "E": 0, "k": 1, "block_m": 1,
         "out": "bf16", "zipf": 0.0},
        # 32 tokens decoded, two of eight experts each, gate and up projections together
        {"name": "product_decode_grouped", "op": "product", "T": 32, "N": 28672, "K": 4096, "E": 8, "k": 2,
         "block_m": 16, "out": "bf16", "zipf": 0.0},
        # prefill: 8192 sorted rows over eight experts
        {"name": "product_prefill_grouped", "op": "product", "T": 4096, "N": 14336, "K": 4096, "E": 8, "k": 2,
         "block_m": 128, "out": "bf16", "zipf": 0.3},
        # a dense layer whose sizes end inside a tile, a scale block and a column block
        {"name": "product_odd_dense", "op": "product", "T": 1000, "N": 1416, "K": 2000, "E": 0, "k": 1, "block_m": 1,
         "out": "fp32", "zipf": 0.0},
        # training: the weight gradient of eight experts' down projections
        {"name": "wgrad_grouped", "op": "wgrad", "T": 4096, "N": 4096, "K": 14336, "E": 8, "k": 2, "block_m": 128,
         "zipf": 0.3},
        # decoding: both norms around a block, 32 tokens
        {"name": "norm_decode", "op": "norm", "T": 32, "H": 4096, "type": "bf16", "gate": "channel"},
        # training on a long batch: forward and every gradient
        {"name": "norm_train_prefill", "op": "norm_train", "T": 8192, "H": 4096, "type": "bf16", "gate": "channel"},
        # an odd width, a gate per token
        {"name": "norm_train_odd", "op": "norm_train", "T": 1023, "H": 1001, "type": "fp16", "gate": "token"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _odd(rng, n):
    """n, or near n and odd, one time in two."""
    return n if rng.random() < 0.5 else max(1, n | 1)


def draw(rng):
    op = rng.choice(["dispatch", "dispatch_fp8", "combine", "exchange_bwd", "product", "product", "product_dense",
                     "wgrad", "norm", "norm_train"])
    if op in ("norm", "norm_train"):
        return {"op": op, "T": _odd(rng, _log(rng, 1, 8000)), "H": _odd(rng, _log(rng, 64, 4000)),
                "type": rng.choice(["bf16", "fp16", "fp32"]) if rng.random() < 0.5 else "bf16",
                "gate": rng.choice(["none", "channel", "token", "full"])}
    E = rng.choice([4, 8, 16, 24, 61, 128, 256])
    k = rng.choice([1, 2, 2, 4, 8])
    k = min(k, E)
    zipf = rng.choice([0.0, 0.3, 1.2])
    if op in ("dispatch", "combine", "exchange_bwd"):
        return {"op": op, "T": _odd(rng, _log(rng, 1, 4000)), "H": _odd(rng, _log(rng, 64, 7000)), "E": E, "k": k,
                "block_m": rng.choice([1, 16, 64, 128]), "type": rng.choice(["bf16", "fp16", "fp32"]), "zipf": zipf}
    if op == "dispatch_fp8":
        return {"op": op, "T": _odd(rng, _log(rng, 1, 8000)), "H": 128 * _log(rng, 1, 32), "E": E, "k": min(k, 4),
                "block_m": rng.choice([16, 64, 128]), "type": "bf16", "zipf": zipf}
    if op == "product_dense":
        return {"op": "product", "T": _odd(rng, _log(rng, 1, 4000)), "N": _odd(rng, _log(rng, 64, 14000)),
                "K": 16 * _log(rng, 4, 450), "E": 0, "k": 1, "block_m": 1, "out": rng.choice(["bf16", "fp32"]),
                "zipf": 0.0}
    E = min(E, 61)
    if op == "product":
        block_m = rng.choice([16, 32, 64, 128])
        return {"op": op, "T": _odd(rng, _log(rng, 1, 4000 if block_m == 128 else 256)), "N": 8 * _log(rng, 8, 512),
                "K": 128 * _log(rng, 1, 32), "E": E, "k": min(k, 4), "block_m": block_m,
                "out": rng.choice(["bf16", "fp32"]), "zipf": zipf}
    return {"op": op, "T": _odd(rng, _log(rng, 16, 4000)), "N": 16 * _log(rng, 8, 128), "K": 16 * _log(rng, 8, 128),
            "E": min(E, 24), "k": min(k, 2), "block_m": 128, "zipf": zipf}


# ------------------------------------------------------------------- inputs

def _route(c, g):
    """Distinct experts for each token and weights that sum to 1, as a router gives them."""
    T, E, k = c["T"], c["E"], c["k"]
    logit = torch.randn(T, E, generator=g, device=DEV)
    rank = torch.randperm(E, generator=g, device=DEV).float() + 1.0
    val, ids = (logit - c["zipf"] * rank.log()).topk(k, dim=1)
    return ids.to(torch.int32), torch.softmax(val, 1)


def _plan(ids, E, block_m):
    """The sort's outputs by elementary operations: slots of each expert in ascending order, each
    expert padded to whole blocks."""
    T, k = ids.shape
    S = T * k
    P = S + E * block_m - k
    flat = ids.reshape(-1).long()
    counts = torch.zeros(E, dtype=torch.int64, device=DEV).scatter_add_(0, flat, torch.ones_like(flat))
    padded = (counts + block_m - 1) // block_m * block_m
    ends = padded.cumsum(0)
    order = torch.sort(flat, stable=True).indices
    e_of = flat[order]
    first = counts.cumsum(0) - counts
    place = (ends - padded)[e_of] + torch.arange(S, device=DEV) - first[e_of]
    slot_pos = torch.empty(S, dtype=torch.int64, device=DEV)
    slot_pos[order] = place
    sorted_ids = torch.full((P,), S, dtype=torch.int64, device=DEV)
    sorted_ids[place] = order
    nb = (P + block_m - 1) // block_m
    start = torch.arange(nb, device=DEV) * block_m
    block_e = torch.searchsorted(ends, start, right=True)
    block_e = torch.where(start < ends[-1], block_e, torch.full_like(block_e, -1))
    return {"slot_pos": slot_pos.int(), "sorted_ids": sorted_ids.int(), "expert_ids": block_e.int(),
            "npp": ends[-1:].int(), "counts": counts.int(), "P": P, "nb": nb}


def _rand(shape, g, dt, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dt)


def _codes(rows, cols, g):
    """e4m3 codes of a quantised normal matrix (each 1x128 group's largest near 448)."""
    out = torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device=DEV)
    step = max(1, (1 << 28) // max(1, cols))
    for r in range(0, rows, step):
        n = min(step, rows - r)
        out[r:r + n] = (torch.randn(n, cols, generator=g, device=DEV) * 150.0).clamp_(-E4M3_MAX, E4M3_MAX).to(
            torch.float8_e4m3fn)
    return out


def _scales(shape, g, std):
    """Scales of groups whose largest value is std-distributed."""
    return std / 150.0 * torch.exp(0.3 * torch.randn(shape, generator=g, device=DEV))


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = {"c": c, "ws": torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)}
    op, T = c["op"], c["T"]
    if op in ("norm", "norm_train"):
        H, dt = c["H"], TYPES[c["type"]]
        s["h"] = _rand((T, H), g, dt, 0.5)
        s["residual"] = _rand((T, H), g, dt, 2.0)
        s["w_post"] = (1 + 0.2 * torch.randn(H, generator=g, device=DEV)).to(dt)
        s["w_pre"] = (1 + 0.2 * torch.randn(H, generator=g, device=DEV)).to(dt)
        shape = {"none": None, "channel": (1, H), "token": (T, 1), "full": (T, H)}[c["gate"]]
        s["gate"] = None if shape is None else torch.sigmoid(torch.randn(shape, generator=g, device=DEV)).to(dt)
        s["eps"], s["scale"] = 1e-6, 0.22
        for n in ("y", "z"):
            s[n] = torch.empty(T, H, dtype=dt, device=DEV)
        s["rstd"] = torch.empty(2, T, device=DEV)
        if op == "norm_train":
            s["dy"], s["dz"] = _rand((T, H), g, dt, 0.1), _rand((T, H), g, dt, 0.1)
            s["dres"], s["dh"] = torch.empty_like(s["y"]), torch.empty_like(s["y"])
            # summed gradients stay in 32 bits
            s["dgate"] = None if shape is None else torch.empty(
                shape, device=DEV, dtype=dt if c["gate"] == "full" else torch.float32)
            s["dw_post"], s["dw_pre"] = torch.empty(H, device=DEV), torch.empty(H, device=DEV)
            s["ws"] = torch.zeros(32 << 20, dtype=torch.uint8, device=DEV)
        return s
    if op in ("dispatch", "dispatch_fp8", "combine", "exchange_bwd"):
        H, dt = c["H"], TYPES[c["type"]]
        s["ids"], s["wts"] = _route(c, g)
        p = _plan(s["ids"], c["E"], c["block_m"])
        P = p["P"]
        if op in ("dispatch", "dispatch_fp8"):
            # each token with its own magnitude, as activations have
            mag = torch.exp(torch.randn(T, 1, generator=g, device=DEV))
            s["x"] = (torch.randn(T, H, generator=g, device=DEV) * mag).to(dt)
            for n in ("sorted_ids", "expert_ids", "npp", "counts", "slot_pos"):
                s[n] = torch.empty_like(p[n])
            s["sorted_w"] = torch.empty(P, device=DEV)
            if op == "dispatch":
                s["xs"] = torch.zeros(P, H, dtype=dt, device=DEV)
            else:
                s["q"] = torch.zeros(P, H, dtype=torch.float8_e4m3fn, device=DEV)
                s["s"] = torch.ones(H // 128, P, device=DEV)
            s["P"] = P
            return s
        s["p"] = p
        s["ys"] = _rand((P, H), g, dt)
        s["out"] = torch.empty(T, H, dtype=dt, device=DEV)
        if op == "exchange_bwd":
            s["dout"] = _rand((T, H), g, dt)
            s["dys"] = torch.zeros(P, H, dtype=dt, device=DEV)
            s["dw"] = torch.empty(T, c["k"], device=DEV)
            s["dxs"] = _rand((P, H), g, dt)
        return s
    N, K, E = c["N"], c["K"], c["E"]
    p = None
    rows = T
    if E:
        ids, _ = _route(c, g)
        p = _plan(ids, E, c["block_m"])
        rows = p["P"]
        p["host_counts"] = p["counts"].tolist()
    s["p"] = p
    if op == "product":
        KB = (K + 127) // 128
        s["a"] = _codes(rows, K, g)
        s["sa"] = _scales((rows, KB), g, 1.0)
        s["b"] = _codes(max(E, 1) * N, K, g)
        s["sb"] = _scales((max(E, 1), (N + 127) // 128, KB), g, 1.0 / math.sqrt(K))
        s["d"] = torch.zeros(rows, N, dtype=TYPES[c["out"]], device=DEV)
        return s
    # weight gradient: both operands with the tokens along K, padding rows zero
    pad = (p["sorted_ids"] >= T * c["k"])
    KB = (rows + 127) // 128
    rows = KB * 128
    pad = torch.cat([pad, pad.new_ones(rows - pad.numel())])
    s["rows"] = rows
    for n, width in (("a", N), ("b", K)):
        codes = _codes(width, rows, g)
        codes.view(torch.uint8).masked_fill_(pad[None, :], 0)
        s[n] = codes
        s["s" + n] = _scales((KB, width), g, 1.0)
    s["d"] = torch.empty(E, N, K, device=DEV)
    return s


# --------------------------------------------------------------- plain form

def _plain_norm(s, backward):
    c = s["c"]
    dt = TYPES[c["type"]]
    h, res = s["h"].float(), s["residual"].float()
    wo, wi = s["w_post"].float(), s["w_pre"].float()
    gate = 1.0 if s["gate"] is None else s["gate"].float()
    r1 = torch.rsqrt((h * h).mean(1, keepdim=True) + s["eps"])
    hh = h * r1
    y = res + s["scale"] * gate * (hh * wo)
    r2 = torch.rsqrt((y * y).mean(1, keepdim=True) + s["eps"])
    yh = y * r2
    out = {"y": y.to(dt), "z": (yh * wi).to(dt)}
    if not backward:
        return out
    dy, dz = s["dy"].float(), s["dz"].float()
    dyn = dz * wi
    dt_ = dy + r2 * (dyn - yh * (dyn * yh).mean(1, keepdim=True))
    dn = s["scale"] * gate * dt_
    dnw = dn * wo
    dh = r1 * (dnw - hh * (dnw * hh).mean(1, keepdim=True))
    out.update(dres=dt_.to(dt), dh=dh.to(dt), dw_post=(dn * hh).sum(0), dw_pre=(dz * yh).sum(0))
    if s["gate"] is not None:
        dg = s["scale"] * (hh * wo) * dt_
        out["dgate"] = {"channel": lambda: dg.sum(0, keepdim=True), "token": lambda: dg.sum(1, keepdim=True),
                        "full": lambda: dg.to(dt)}[c["gate"]]()
    return out


def _plain_dispatch(s):
    c = s["c"]
    p = _plan(s["ids"], c["E"], c["block_m"])
    S = c["T"] * c["k"]
    pos = p["slot_pos"].long()
    token = torch.arange(S, device=DEV) // c["k"]
    out = {n: p[n] for n in ("sorted_ids", "expert_ids", "npp", "counts", "slot_pos")}
    out["sorted_w"] = torch.zeros(p["P"], device=DEV).index_copy_(0, pos, s["wts"].reshape(-1))
    if c["op"] == "dispatch":
        out["xs"] = torch.zeros(p["P"], c["H"], dtype=s["x"].dtype, device=DEV).index_copy_(0, pos, s["x"][token])
        return out
    x = s["x"].float().view(c["T"], -1, 128)
    amax = x.abs().amax(2)
    sc = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
    q = (x / sc[:, :, None]).to(torch.float8_e4m3fn).view(c["T"], -1).view(torch.uint8)
    out["q"] = torch.zeros(p["P"], c["H"], dtype=torch.uint8, device=DEV).index_copy_(0, pos, q[token]).view(
        torch.float8_e4m3fn)
    out["s"] = torch.ones(p["P"], c["H"] // 128, device=DEV).index_copy_(0, pos, sc[token]).t().contiguous()
    return out


def _plain_combine(s):
    c = s["c"]
    pos = s["p"]["slot_pos"].long()
    rows = s["ys"][pos].float().view(c["T"], c["k"], c["H"])
    return (rows * s["wts"][:, :, None]).sum(1).to(s["ys"].dtype)


def _plain_exchange_bwd(s):
    c = s["c"]
    pos = s["p"]["slot_pos"].long()
    dt = s["ys"].dtype
    rows = s["ys"][pos].float().view(c["T"], c["k"], c["H"])
    dout = s["dout"].float()[:, None, :]
    dw = (rows * dout).sum(2)
    d = (s["wts"][:, :, None] * dout).to(dt).view(-1, c["H"])
    dys = torch.zeros_like(s["dys"]).index_copy_(0, pos, d)
    dx = s["dxs"][pos].float().view(c["T"], c["k"], c["H"]).sum(1).to(dt)
    return {"dys": dys, "dw": dw, "dx": dx}


def _segments(s):
    """Each expert's rows [first, last) in sorted order, whole blocks (known to the program that sorted)."""
    c = s["c"]
    if s["p"] is None:
        return [(0, c["T"])]
    out, at = [], 0
    for n in s["p"]["host_counts"]:
        m = -(-n // c["block_m"]) * c["block_m"]
        out.append((at, at + m))
        at += m
    return out


def _wide(sb, N, K):
    """A [n][k] block scale for each element."""
    return sb.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]


def _plain_product(s):
    c = s["c"]
    N, K = c["N"], c["K"]
    d = torch.zeros_like(s["d"])
    for e, (lo, hi) in enumerate(_segments(s)):
        if hi > lo:
            a = s["a"][lo:hi].float() * s["sa"][lo:hi].repeat_interleave(128, 1)[:, :K]
            b = s["b"][e * N:(e + 1) * N].float() * _wide(s["sb"][e], N, K)
            d[lo:hi] = (a @ b.t()).to(d.dtype)
    return d


def _plain_wgrad(s):
    d = torch.zeros_like(s["d"])
    for e, (lo, hi) in enumerate(_segments(s)):
        if hi > lo:
            a = s["a"][:, lo:hi].float() * s["sa"][lo // 128:hi // 128].repeat_interleave(128, 0).t()
            b = s["b"][:, lo:hi].float() * s["sb"][lo // 128:hi // 128].repeat_interleave(128, 0).t()
            d[e] = a @ b.t()
    return d


# ------------------------------------------------------- the package's calls

def _own_norm(s, moe, backward):
    c = s["c"]
    T, H = c["T"], c["H"]
    t = {"bf16": moe.MOE_ROW_BF16, "fp16": moe.MOE_ROW_FP16, "fp32": moe.MOE_ROW_FP32}[c["type"]]
    gate = {"none": moe.MOE_GATE_NONE, "channel": moe.MOE_GATE_CHANNEL, "token": moe.MOE_GATE_TOKEN,
            "full": moe.MOE_GATE_FULL}[c["gate"]]
    moe.moe_block_norm(t, s["h"], s["residual"], s["gate"], gate, s["w_post"], s["w_pre"], T, H, s["scale"], 0.0,
                       s["eps"], s["y"], s["z"], s["rstd"][0], s["rstd"][1])
    out = {"y": s["y"], "z": s["z"]}
    if not backward:
        return out
    moe.moe_block_norm_backward(t, s["h"], s["residual"], s["gate"], gate, s["w_post"], s["w_pre"], s["rstd"][0],
                                s["rstd"][1], s["dy"], s["dz"], T, H, s["scale"], 0.0, s["dres"], s["dh"],
                                s["dgate"], s["dw_post"], s["dw_pre"], s["ws"], s["ws"].numel())
    out.update(dres=s["dres"], dh=s["dh"], dw_post=s["dw_post"], dw_pre=s["dw_pre"])
    if s["gate"] is not None:
        out["dgate"] = s["dgate"]
    return out


def _own_exchange(s, moe):
    c = s["c"]
    T, H, E, k = c["T"], c["H"], c["E"], c["k"]
    t = {"bf16": moe.MOE_ROW_BF16, "fp16": moe.MOE_ROW_FP16, "fp32": moe.MOE_ROW_FP32}[c["type"]]
    if c["op"] in ("dispatch", "dispatch_fp8"):
        moe.moe_align_sort_map(s["ids"], s["wts"], T, k, E, c["block_m"], s["sorted_ids"], s["sorted_w"],
                               s["expert_ids"], s["npp"], s["counts"], s["slot_pos"], s["ws"], s["ws"].numel())
        out = {n: s[n] for n in ("sorted_ids", "expert_ids", "npp", "counts", "slot_pos", "sorted_w")}
        if c["op"] == "dispatch":
            moe.moe_permute(t, s["x"], H, s["slot_pos"], s["sorted_ids"], s["npp"], T, k, H, s["P"], 1, s["xs"])
            out["xs"] = s["xs"]
        else:
            moe.moe_permute_fp8(s["x"], H, s["slot_pos"], s["sorted_ids"], s["npp"], T, k, H, s["P"], 1, s["q"],
                                s["s"])
            out["q"], out["s"] = s["q"], s["s"]
        return out
    p = s["p"]
    if c["op"] == "combine":
        moe.moe_unpermute(t, s["ys"], p["slot_pos"], s["wts"], T, k, H, p["P"], s["out"], H)
        return s["out"]
    moe.moe_unpermute_backward(t, s["dout"], H, s["ys"], p["slot_pos"], s["wts"], p["sorted_ids"], p["npp"], T, k, H,
                               p["P"], 1, s["dys"], s["dw"])
    moe.moe_permute_backward(t, s["dxs"], p["slot_pos"], T, k, H, p["P"], s["out"], H)
    return {"dys": s["dys"], "dw": s["dw"], "dx": s["out"]}


def _own_product(s, moe):
    c = s["c"]
    p = s["p"]
    if c["op"] == "wgrad":
        moe.moe_wgrad_fp8_block(s["a"], s["sa"], s["b"], s["sb"], s["rows"], c["N"], c["K"], c["E"], p["counts"],
                                s["d"], 0, s["ws"], s["ws"].numel())
        return s["d"]
    t = {"bf16": moe.MOE_ROW_BF16, "fp32": moe.MOE_ROW_FP32}[c["out"]]
    if p is None:
        moe.moe_gemm_fp8_block(s["a"], s["sa"], 0, s["b"], s["sb"], c["T"], c["N"], c["K"], 1, 0, None, None, t,
                               s["d"], c["N"], s["ws"], s["ws"].numel())
    else:
        moe.moe_gemm_fp8_block(s["a"], s["sa"], 0, s["b"], s["sb"], p["P"], c["N"], c["K"], c["E"], c["block_m"],
                               p["expert_ids"], p["npp"], t, s["d"], c["N"], s["ws"], s["ws"].numel())
    return s["d"]


def run(state):
    op = state["c"]["op"]
    if own:
        from mixture_experts_grouped_moe_gb300 import moe
        if op in ("norm", "norm_train"):
            return _own_norm(state, moe, op == "norm_train")
        return _own_product(state, moe) if op in ("product", "wgrad") else _own_exchange(state, moe)
    if op in ("norm", "norm_train"):
        return _plain_norm(state, op == "norm_train")
    return {"dispatch": _plain_dispatch, "dispatch_fp8": _plain_dispatch, "combine": _plain_combine,
            "exchange_bwd": _plain_exchange_bwd, "product": _plain_product, "wgrad": _plain_wgrad}[op](state)


# --------------------------------------------------------------------- work

def _distinct(E, S):
    """Experts that at least one of S evenly drawn slots chooses, on average."""
    return E * (1.0 - (1.0 - 1.0 / E) ** S)


def work(case):
    c = case
    op, T = c["op"], c["T"]
    if op in ("norm", "norm_train"):
        n, e = T * c["H"], SIZE[c["type"]]
        gate = {"none": 0, "channel": c["H"], "token": T, "full": n}[c["gate"]]
        fwd = 4 * n * e + (gate + 2 * c["H"]) * e
        if op == "norm":
            return {"bytes": fwd, "flops": 10 * n}
        dgate = gate * (e if c["gate"] == "full" else 4)
        return {"bytes": fwd + 6 * n * e + (gate + 2 * c["H"]) * e + dgate + 8 * c["H"], "flops": 35 * n}
    S = T * c["k"]
    if op in ("dispatch", "dispatch_fp8", "combine", "exchange_bwd"):
        H, e = c["H"], SIZE[c["type"]]
        if op == "dispatch":
            return {"bytes": (T + S) * H * e + 24 * S, "flops": 0}
        if op == "dispatch_fp8":
            return {"bytes": T * H * e + S * H + S * H // 128 * 4 + 24 * S, "flops": 2 * T * H}
        if op == "combine":
            return {"bytes": (T + S) * H * e + 8 * S, "flops": 2 * S * H}
        return {"bytes": (T + 2 * S) * H * e + (T + S) * H * e + 16 * S, "flops": 4 * S * H}
    N, K, E = c["N"], c["K"], c["E"]
    if op == "wgrad":
        return {"bytes": S * (N + K) * (1 + 4 / 128) + E * N * K * 4, "flops": 2 * S * N * K}
    used = _distinct(E, S) if E else 1
    return {"bytes": S * K * (1 + 4 / 128) + used * N * K * (1 + 4 / 16384) + S * N * SIZE[c["out"]],
            "flops": 2 * S * N * K}


# ------------------------------------------------------------------ 64 bits

def _exact_norm(s, backward):
    """Row by row definitions; the gradients from the derivative of the two norms' quotients."""
    d = {n: v.double() for n, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    H = s["c"]["H"]
    gate = torch.ones(1, 1, dtype=torch.float64, device=DEV) if s["gate"] is None else d["gate"]
    m1 = (d["h"].pow(2).sum(1, keepdim=True) / H + s["eps"]).sqrt()
    n = d["h"] / m1 * d["w_post"]
    y = d["residual"] + s["scale"] * gate * n
    m2 = (y.pow(2).sum(1, keepdim=True) / H + s["eps"]).sqrt()
    out = {"y": y, "z": y / m2 * d["w_pre"]}
    if not backward:
        return out

    def through(u, v, m):  # gradient of sum(u * v / m(v)), m = sqrt(mean(v^2) + eps), with respect to v
        return u / m - v * (u * v).sum(1, keepdim=True) / (H * m.pow(3))

    tot = d["dy"] + through(d["dz"] * d["w_pre"], y, m2)
    branch = s["scale"] * gate * tot
    out["dres"] = tot
    out["dh"] = through(branch * d["w_post"], d["h"], m1)
    out["dw_post"] = (branch * d["h"] / m1).sum(0)
    out["dw_pre"] = (d["dz"] * y / m2).sum(0)
    if s["gate"] is not None:
        dg = s["scale"] * tot * n
        out["dgate"] = dg.sum(0, keepdim=True) if gate.shape[0] == 1 else dg.sum(1, keepdim=True) \
            if gate.shape[1] == 1 else dg
    return out


def exact(case, seed):
    c = dict(case)
    s = prepare(c, seed)
    op, T = c["op"], c["T"]
    if op in ("norm", "norm_train"):
        return _exact_norm(s, op == "norm_train")
    if op in ("dispatch", "dispatch_fp8"):
        pos = _plan(s["ids"], c["E"], c["block_m"])["slot_pos"].long()
        P = s["P"]
        w = torch.zeros(P, dtype=torch.float64, device=DEV)
        w[pos] = s["wts"].double().reshape(-1)
        if op == "dispatch":
            xs = torch.zeros(P, c["H"], dtype=torch.float64, device=DEV)
            for j in range(c["k"]):
                xs[pos[j::c["k"]]] = s["x"].double()
            return {"sorted_w": w, "xs": xs}
        return {"sorted_w": w, "q": None, "s": None}
    if op in ("combine", "exchange_bwd"):
        k, pos = c["k"], s["p"]["slot_pos"].long().view(T, -1)
        if op == "combine":
            out = torch.zeros(T, c["H"], dtype=torch.float64, device=DEV)
            for j in range(k):
                out += s["wts"][:, j:j + 1].double() * s["ys"][pos[:, j]].double()
            return out
        dys = torch.zeros(s["dys"].shape, dtype=torch.float64, device=DEV)
        dw = torch.empty(T, k, dtype=torch.float64, device=DEV)
        dx = torch.zeros(T, c["H"], dtype=torch.float64, device=DEV)
        for j in range(k):
            dys[pos[:, j]] = s["wts"][:, j:j + 1].double() * s["dout"].double()
            dw[:, j] = torch.einsum("th,th->t", s["dout"].double(), s["ys"][pos[:, j]].double())
            dx += s["dxs"][pos[:, j]].double()
        return {"dys": dys, "dw": dw, "dx": dx}
    N, K = c["N"], c["K"]
    d = torch.zeros(s["d"].shape, dtype=torch.float64, device=DEV)
    at = 0
    for e, n in enumerate(s["p"]["host_counts"] if s["p"] is not None else [T]):
        m = n if s["p"] is None else -(-n // c["block_m"]) * c["block_m"]
        if op == "wgrad":
            for b in range(at // 128, (at + m) // 128):  # one block of 128 tokens after the other
                sl = slice(128 * b, 128 * b + 128)
                d[e] += (s["a"][:, sl].double() * s["sa"][b].double()[:, None]) @ (
                    s["b"][:, sl].double() * s["sb"][b].double()[:, None]).t()
        elif m:
            for b in range((K + 127) // 128):  # one scale block of K after the other
                sl = slice(128 * b, min(K, 128 * b + 128))
                col = s["sb"][e, :, b].double().repeat_interleave(128)[:N]
                part = s["a"][at:at + m, sl].double() @ s["b"][e * N:(e + 1) * N, sl].double().t()
                d[at:at + m] += part * s["sa"][at:at + m, b].double()[:, None] * col[None, :]
        at += m
    return d
