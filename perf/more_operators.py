"""Cases of the operators of a training step around the experts: the gated feed-forward block that every
token passes (a shared expert or a dense layer; forward, and forward with all gradients), the cross entropy
over a large vocabulary straight from the hidden states (forward, and with its gradients), and the norm of
all gradients with their clipping.

`run` computes a case in its plain form (elementary torch operations in 32 bits) or, with `own` set, through
the package's entry points; `exact` gives the same results from the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one token through a shared expert of a fine-grained layer: the latency of decoding
        {"name": "ffn_single", "op": "ffn", "T": 1, "H": 7168, "I": 2048, "type": "bf16", "act": "silu", "add": True,
         "pad": 0},
        # 32 sequences decoded, a wide dense layer: streaming the weights
        {"name": "ffn_decode", "op": "ffn", "T": 32, "H": 4096, "I": 14336, "type": "bf16", "act": "silu",
         "add": True, "pad": 0},
        # sizes that end inside every tile, another activation and type, rows apart in a wider buffer
        {"name": "ffn_odd", "op": "ffn", "T": 1001, "H": 1000, "I": 1416, "type": "fp16", "act": "gelu", "add": False,
         "pad": 24},
        # prefill of 8192 tokens through a wide dense layer
        {"name": "ffn_prefill", "op": "ffn", "T": 8192, "H": 4096, "I": 14336, "type": "bf16", "act": "silu",
         "add": False, "pad": 0},
        # training a shared expert next to routed ones, whose output it is added to
        {"name": "ffn_train", "op": "ffn_train", "T": 4096, "H": 7168, "I": 2048, "type": "bf16", "act": "silu",
         "add": True, "pad": 0},
        # training at a small odd size
        {"name": "ffn_train_odd", "op": "ffn_train", "T": 515, "H": 520, "I": 1000, "type": "fp16", "act": "relu",
         "add": False, "pad": 8},
        # scoring the next token of 16 sequences
        {"name": "loss_score", "op": "loss", "T": 16, "H": 4096, "V": 32000, "type": "bf16", "left_out": 0.0},
        # training: the loss of 4096 tokens and its gradients
        {"name": "loss_train", "op": "loss_train", "T": 4096, "H": 4096, "V": 32000, "type": "bf16", "left_out": 0.0},
        # training on a padded batch, an odd vocabulary
        {"name": "loss_train_odd", "op": "loss_train", "T": 777, "H": 1000, "V": 10007, "type": "fp16",
         "left_out": 0.3},
        # many small parameters of odd sizes (norms, biases, adapters)
        {"name": "clip_small", "op": "clip", "count": 60, "low": 1, "high": 6000, "type": "mixed", "max_norm": 1.0},
        # the weights of a block of eight experts and its router
        {"name": "clip_block", "op": "clip", "count": 16, "low": 2097152, "high": 2097152, "type": "fp32",
         "max_norm": 1.0},
        # every gradient of a wide layer of eight experts
        {"name": "clip_layer", "op": "clip", "count": 24, "low": 58720256, "high": 58720256, "type": "fp32",
         "max_norm": 1.0},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _odd(rng, n):
    """n, or near n and odd, one time in two."""
    return n if rng.random() < 0.5 else max(1, n | 1)


def draw(rng):
    op = rng.choice(["ffn", "ffn", "ffn_train", "loss", "loss_train", "clip"])
    if op in ("ffn", "ffn_train"):
        H, I = 8 * _log(rng, 8, 900), 8 * _log(rng, 8, 1800)
        most = int(2e12 / ((6 if op == "ffn" else 18) * H * I))
        return {"op": op, "T": min(most, _odd(rng, _log(rng, 1, 8000))), "H": H, "I": I,
                "type": rng.choice(["bf16", "bf16", "fp16"]), "act": rng.choice(["silu", "silu", "gelu", "relu"]),
                "add": rng.random() < 0.5, "pad": rng.choice([0, 0, 8, 64])}
    if op in ("loss", "loss_train"):
        H, V = 8 * _log(rng, 8, 900), _odd(rng, _log(rng, 50, 130000))
        most = int(2e12 / ((2 if op == "loss" else 6) * H * V))
        return {"op": op, "T": min(most, _odd(rng, _log(rng, 1, 8000))), "H": H, "V": V,
                "type": rng.choice(["bf16", "bf16", "fp16"]), "left_out": rng.choice([0.0, 0.1, 0.9])}
    count = _log(rng, 1, 60)
    high = _log(rng, 10, min(20000000, 400000000 // count))
    return {"op": op, "count": count, "low": _log(rng, 1, high), "high": high,
            "type": rng.choice(["bf16", "fp16", "fp32", "mixed"]), "max_norm": rng.choice([1.0, 1.0, 1e6])}


# ------------------------------------------------------------------- inputs

def _rand(shape, g, dt, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dt)


def _rows(T, H, pad, g, dt, std=1.0):
    """Rows that stand H + pad elements apart."""
    return _rand((T, H + pad), g, dt, std)[:, :H]


def _sizes(c):
    """Sizes of a clip case's tensors, spread over [low, high]."""
    lo, hi, n = c["low"], c["high"], c["count"]
    return [round(lo * (hi / lo) ** ((i * 37 % n) / max(1, n - 1))) for i in range(n)]


def _kinds(c):
    return [("fp32", "bf16", "fp16")[i % 3] if c["type"] == "mixed" else c["type"] for i in range(c["count"])]


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = {"c": c}
    op = c["op"]
    if op == "clip":
        sizes, kinds = _sizes(c), _kinds(c)
        std = 4.0 / math.sqrt(sum(sizes))  # a norm near 4
        s["grads"] = [_rand((n,), g, TYPES[k], std) for n, k in zip(sizes, kinds)]
        s["clipped"] = [torch.empty_like(t) for t in s["grads"]]
        s["norm"] = torch.empty(1, device=DEV)
        s["eps"] = 1e-6
        s["ws"] = torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)
        return s
    T, H, dt = c["T"], c["H"], TYPES[c["type"]]
    if op in ("ffn", "ffn_train"):
        I, pad = c["I"], c["pad"]
        s["x"] = _rows(T, H, pad, g, dt)
        s["w_gate_up"] = _rand((2 * I, H), g, dt, H ** -0.5)  # gate rows first
        s["w_down"] = _rand((H, I), g, dt, I ** -0.5)
        s["add"] = _rows(T, H, pad, g, dt) if c["add"] else None
        s["out"] = torch.empty(T, H, dtype=dt, device=DEV)
        bytes_ = 64 << 20
        if op == "ffn_train":
            s["gu"], s["h"] = torch.empty(T, 2 * I, dtype=dt, device=DEV), torch.empty(T, I, dtype=dt, device=DEV)
            s["dout"] = _rows(T, H, pad, g, dt, 0.1)
            s["dx"] = torch.empty(T, H, dtype=dt, device=DEV)
            s["dw_gate_up"], s["dw_down"] = torch.empty_like(s["w_gate_up"]), torch.empty_like(s["w_down"])
            bytes_ += T * 2 * I * 2
        else:
            bytes_ += T * I * 2
        s["ws"] = torch.zeros(bytes_, dtype=torch.uint8, device=DEV)
        return s
    V = c["V"]
    s["x"] = _rand((T, H), g, dt)
    s["w"] = _rand((V, H), g, dt, 2.0 * H ** -0.5)  # logits with a deviation of 2
    t = torch.randint(0, V, (T,), generator=g, device=DEV)
    drop = torch.rand(T, generator=g, device=DEV) < c["left_out"]
    s["targets"] = torch.where(drop, torch.full_like(t, -100), t).int()
    s["loss"], s["lse"] = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    s["piece"] = 8192
    bytes_ = (64 << 20) + T * 8 * (V // 128 + 2)
    if op == "loss_train":
        # the mean over the rows that count, each with a weight of its own
        wts = 0.5 + torch.rand(T, generator=g, device=DEV)
        s["dloss"] = wts / max(1, T)
        s["dx"], s["dw"] = torch.empty(T, H, dtype=dt, device=DEV), torch.empty_like(s["w"])
        bytes_ += T * H * 6 + T * s["piece"] * 2
    s["ws"] = torch.zeros(bytes_, dtype=torch.uint8, device=DEV)
    return s


# --------------------------------------------------------------- plain form

def _act(g, kind):
    """The activation and its derivative."""
    if kind == "silu":
        sg = 1.0 / (1.0 + torch.exp(-g))
        return g * sg, sg * (1.0 + g * (1.0 - sg))
    if kind == "relu":
        on = (g > 0).float()
        return g * on, on
    a = math.sqrt(2.0 / math.pi)
    t = torch.tanh(a * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * a * (1.0 + 3 * 0.044715 * g * g)


def _plain_ffn(s, backward):
    c = s["c"]
    dt, I = TYPES[c["type"]], c["I"]
    x, wgu, wd = s["x"].float(), s["w_gate_up"].float(), s["w_down"].float()
    gu = x @ wgu.t()
    a, da = _act(gu[:, :I], c["act"])
    u = gu[:, I:]
    h = a * u
    out = h @ wd.t()
    if s["add"] is not None:
        out = out + s["add"].float()
    if not backward:
        return {"out": out.to(dt)}
    d = s["dout"].float()
    dh = d @ wd
    dgu = torch.cat([dh * u * da, dh * a], 1)
    return {"out": out.to(dt), "dx": (dgu @ wgu).to(dt), "dw_gate_up": (dgu.t() @ x).to(dt),
            "dw_down": (d.t() @ h).to(dt)}


def _plain_loss(s, backward):
    c = s["c"]
    dt = TYPES[c["type"]]
    x, w, t = s["x"].float(), s["w"].float(), s["targets"].long()
    counts = (t >= 0) & (t < c["V"])
    at = torch.where(counts, t, torch.zeros_like(t))[:, None]
    logits = x @ w.t()
    top = logits.amax(1, keepdim=True)
    lse = top + torch.exp(logits - top).sum(1, keepdim=True).log()
    loss = torch.where(counts, (lse - logits.gather(1, at))[:, 0], torch.zeros_like(top[:, 0]))
    out = {"loss": loss, "lse": lse[:, 0]}
    if not backward:
        return out
    p = torch.exp(logits - lse)
    p.scatter_add_(1, at, -torch.ones_like(lse))
    p = p * torch.where(counts, s["dloss"], torch.zeros_like(loss))[:, None]
    out.update(dx=(p @ w).to(dt), dw=(p.t() @ x).to(dt))
    return out


def _plain_clip(s):
    norm = torch.stack([t.float().pow(2).sum(dtype=torch.float64) for t in s["grads"]]).sum().sqrt().float()
    k = torch.clamp(s["c"]["max_norm"] / (norm + s["eps"]), max=1.0)
    return {"norm": norm.reshape(1), "clipped": [(t.float() * k).to(t.dtype) for t in s["grads"]]}


# ------------------------------------------------------- the package's calls

def _own_ffn(s, moe, backward):
    c = s["c"]
    T, H, I = c["T"], c["H"], c["I"]
    t = {"bf16": moe.MOE_ROW_BF16, "fp16": moe.MOE_ROW_FP16}[c["type"]]
    act = {"silu": moe.MOE_ACT_SILU, "gelu": moe.MOE_ACT_GELU_TANH, "relu": moe.MOE_ACT_RELU}[c["act"]]
    ws, ld = s["ws"], H + c["pad"]
    moe.moe_ffn(t, act, s["x"], ld, s["w_gate_up"], s["w_down"], s["add"], ld, T, H, I, s.get("gu"), s.get("h"),
                s["out"], H, ws, ws.numel())
    if not backward:
        return {"out": s["out"]}
    moe.moe_ffn_backward(t, act, s["x"], ld, s["w_gate_up"], s["w_down"], s["gu"], s["h"], s["dout"], ld, T, H, I,
                         s["dx"], H, t, 0, s["dw_gate_up"], s["dw_down"], ws, ws.numel())
    return {n: s[n] for n in ("out", "dx", "dw_gate_up", "dw_down")}


def _own_loss(s, moe, backward):
    c = s["c"]
    T, H, V = c["T"], c["H"], c["V"]
    t = {"bf16": moe.MOE_ROW_BF16, "fp16": moe.MOE_ROW_FP16}[c["type"]]
    ws = s["ws"]
    moe.moe_vocab_loss(t, s["x"], H, s["w"], s["targets"], T, H, V, s["loss"], s["lse"], ws, ws.numel())
    if not backward:
        return {"loss": s["loss"], "lse": s["lse"]}
    moe.moe_vocab_loss_backward(t, s["x"], H, s["w"], s["targets"], s["lse"], s["dloss"], T, H, V, s["piece"],
                                s["dx"], H, t, 0, s["dw"], ws, ws.numel())
    return {n: s[n] for n in ("loss", "lse", "dx", "dw")}


def _own_clip(s, moe):
    moe.moe_clip_gradients(s["grads"], s["clipped"], s["c"]["max_norm"], s["eps"], s["norm"], s["ws"],
                           s["ws"].numel())
    return {"norm": s["norm"], "clipped": s["clipped"]}


def run(state):
    op = state["c"]["op"]
    if own:
        from mixture_experts_grouped_moe_gb300 import moe
        if op == "clip":
            return _own_clip(state, moe)
        return (_own_ffn if op in ("ffn", "ffn_train") else _own_loss)(state, moe, op.endswith("_train"))
    if op == "clip":
        return _plain_clip(state)
    return (_plain_ffn if op in ("ffn", "ffn_train") else _plain_loss)(state, op.endswith("_train"))


# --------------------------------------------------------------------- work

def work(case):
    c = case
    op = c["op"]
    if op == "clip":
        # all are read for the norm, and read and written for the scaling
        n = sum(k * SIZE[t] for k, t in zip(_sizes(c), _kinds(c)))
        return {"bytes": 3 * n, "flops": 3 * sum(_sizes(c))}
    T, H, e = c["T"], c["H"], SIZE[c["type"]]
    if op in ("ffn", "ffn_train"):
        w, rows = 3 * H * c["I"] * e, T * H * e
        n = w + (3 if c["add"] else 2) * rows
        if op == "ffn":
            return {"bytes": n, "flops": 6 * T * H * c["I"]}
        return {"bytes": n + w + 2 * rows, "flops": 18 * T * H * c["I"]}
    n = (T + c["V"]) * H * e + 12 * T
    if op == "loss":
        return {"bytes": n, "flops": 2 * T * H * c["V"]}
    return {"bytes": 2 * n - 8 * T, "flops": 6 * T * H * c["V"]}


# ------------------------------------------------------------------ 64 bits

def _exact_ffn(s, backward):
    """Gradients by differentiation of the definition."""
    c = s["c"]
    leaves = [s[n].double().requires_grad_(backward) for n in ("x", "w_gate_up", "w_down")]
    x, wgu, wd = leaves
    gate, up = (torch.nn.functional.linear(x, w) for w in wgu.split(c["I"]))
    act = {"silu": torch.nn.functional.silu, "relu": torch.nn.functional.relu,
           "gelu": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[c["act"]]
    out = torch.nn.functional.linear(act(gate) * up, wd)
    if s["add"] is not None:
        out = out + s["add"].double()
    r = {"out": out.detach()}
    if backward:
        r.update(zip(("dx", "dw_gate_up", "dw_down"), torch.autograd.grad(out, leaves, s["dout"].double())))
    return r


def _exact_loss(s, backward):
    """Gradients by differentiation of the weighted sum of the losses."""
    V = s["c"]["V"]
    x, w = (s[n].double().requires_grad_(backward) for n in ("x", "w"))
    lse = torch.logsumexp(torch.nn.functional.linear(x, w), 1)
    kept = ((s["targets"] >= 0) & (s["targets"] < V)).nonzero()[:, 0]
    own_logit = (x[kept] * w[s["targets"][kept].long()]).sum(1)
    loss = torch.zeros_like(lse).index_copy(0, kept, lse[kept] - own_logit)
    r = {"loss": loss.detach(), "lse": lse.detach()}
    if backward:
        r.update(zip(("dx", "dw"), torch.autograd.grad(loss, (x, w), s["dloss"].double())))
    return r


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(t, dtype=torch.float64)) ** 2 for t in s["grads"]))
        k = min(1.0, case["max_norm"] / (norm + s["eps"]))
        return {"norm": torch.tensor([norm], dtype=torch.float64, device=DEV),
                "clipped": [t.double() * k for t in s["grads"]]}
    return (_exact_ffn if op in ("ffn", "ffn_train") else _exact_loss)(s, op.endswith("_train"))
