"""Workloads of the operators around the expert forward: routing, RMS norm and the int8 product.

Each case is one call (or, for ``norm_matmul``, the two calls of a quantised projection) as a
serving program makes it.  ``run`` has two forms: elementary torch operations, and, where the
module's ``own`` is true, the framework's operators.  ``exact`` gives the same results from the
definitions in 64 bits.

Shapes are those of the expert-forward workloads (hidden 2048 / 4096 / 7168, 128 or 256 experts,
top-8, 1 to 8192 tokens) and generic ones around them.
"""

import math

import numpy as np
import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
INT8_MAX = 127.0
MOST_FLOPS = 2 * 8192 * 4096 * 8192     # the largest listed product
MOST_ROUTE = 8191 * 256                 # the largest listed router's logits
MOST_NORM = 8192 * 4096                 # the largest listed norm's values


# --------------------------------------------------------------------------- #
# Cases
# --------------------------------------------------------------------------- #
def _route(tokens, experts, topk, dtype, score, bias, groups, keep, top, renorm, scale):
    return {"op": "route", "tokens": tokens, "experts": experts, "topk": topk, "dtype": dtype,
            "score": score, "bias": bias, "groups": groups, "keep": keep, "top": top,
            "renorm": renorm, "scale": scale}


def _norm(rows, hidden, dtype, residual, weight, quant):
    return {"op": "norm", "rows": rows, "hidden": hidden, "dtype": dtype, "residual": residual,
            "weight": weight, "quant": quant}


def _matmul(tokens, k, n, out, bias):
    return {"op": "matmul", "tokens": tokens, "k": k, "n": n, "out": out, "bias": bias}


def _norm_matmul(rows, hidden, n):
    return {"op": "norm_matmul", "rows": rows, "hidden": hidden, "n": n}


def listed():
    cases = {
        # One decoded token of the 128-expert layer: the call's latency is all there is.
        "route 1 token, 128 softmax": _route(1, 128, 8, "f32", "softmax", False, 1, 1, 1, True, 1.0),
        # A decode batch of the 256-expert layer, sigmoid scores, balance bias, 4 of 8 groups.
        "route 256 tokens, 256 grouped": _route(256, 256, 8, "f32", "sigmoid", True, 8, 4, 2, True, 2.5),
        # A prefill of the 128-expert layer, logits as the BF16 product leaves them.
        "route 8192 tokens, 128 bf16": _route(8192, 128, 8, "bf16", "softmax", False, 1, 1, 1, True, 1.0),
        # The largest router: an odd prefill batch, 256 experts, groups and bias.
        "route 8191 tokens, 256 grouped": _route(8191, 256, 8, "f32", "sigmoid", True, 8, 4, 2, True, 2.5),
        # One decoded token's norm before router and experts.
        "norm 1 x 2048": _norm(1, 2048, "bf16", "bf16", "bf16", "none"),
        # A decode batch behind the experts: the blend's FP32 output joins the residual stream,
        # and the next projection wants E4M3 beside the BF16.
        "norm 256 x 7168 to e4m3": _norm(256, 7168, "f32", "bf16", "bf16", "e4m3"),
        # A prefill's norm.
        "norm 8192 x 4096": _norm(8192, 4096, "bf16", "bf16", "bf16", "none"),
        # A decode batch through norm, int8 codes and a projection.
        "norm and product 32 x 4096": _norm_matmul(32, 4096, 5120),
        # One decoded token's projection: the weights' bytes.
        "product 1 x 2048 x 4096": _matmul(1, 2048, 4096, "bf16", False),
        # A decode batch's projection.
        "product 256 x 7168 x 2048": _matmul(256, 7168, 2048, "bf16", False),
        # A ragged batch into an odd width (a vocabulary slice), FP32 out with a bias.
        "product 1000 x 2048 x 4099": _matmul(1000, 2048, 4099, "f32", True),
        # The largest: a prefill's projection.
        "product 8192 x 4096 x 8192": _matmul(8192, 4096, 8192, "bf16", False),
    }
    return [dict(c, name=name) for name, c in cases.items()]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "norm", "matmul", "matmul", "norm_matmul"])
    if op == "route":
        tokens = _log_int(rng, 1, 8192)
        groups = rng.choice([1, 1, 4, 8])
        experts = groups * _log_int(rng, 8 if groups == 1 else 4, 512 // groups)
        experts = max(groups * 4, min(experts, MOST_ROUTE // tokens // groups * groups))
        keep = rng.randint(1, groups)
        topk = rng.randint(1, min(16, keep * (experts // groups)))
        return _route(tokens, experts, topk, rng.choice(["f32", "bf16"]),
                      rng.choice(["softmax", "sigmoid"]), rng.random() < 0.5, groups, keep,
                      rng.choice([1, 2]) if groups > 1 else 1, rng.random() < 0.7,
                      rng.choice([1.0, 2.5]))
    if op == "norm":
        hidden = _log_int(rng, 64, 8192)
        rows = _log_int(rng, 1, min(8192, MOST_NORM // hidden))
        return _norm(rows, hidden, rng.choice(["bf16", "f32"]), rng.choice(["none", "bf16", "f32"]),
                     rng.choice(["bf16", "f32"]), rng.choice(["none", "e4m3"]))
    k = 16 * _log_int(rng, 8, 512)
    n = _log_int(rng, 64, 8192)
    tokens = _log_int(rng, 1, min(8192, MOST_FLOPS // (2 * k * n)))
    if op == "norm_matmul":
        return _norm_matmul(tokens, k, n)
    return _matmul(tokens, k, n, rng.choice(["bf16", "f32"]), rng.random() < 0.5)


_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _codes(g, rows, cols):
    """int8 codes of a normal row quantised to its maximum, about four deviations."""
    t = torch.empty(rows, cols, dtype=torch.int8, device="cuda")
    step = max(1, (1 << 26) // cols)
    for at in range(0, rows, step):
        part = torch.randn(min(step, rows - at), cols, generator=g, device="cuda")
        t[at:at + step] = (part * 31.0).round_().clamp_(-127, 127).to(torch.int8)
    return t


def prepare(case, seed):
    g = _generator(seed)
    c = dict(case)
    rand = lambda *shape: torch.rand(*shape, generator=g, device="cuda")    # noqa: E731
    randn = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    if c["op"] == "route":
        m, e = c["tokens"], c["experts"]
        # Logits of a trained router: unit-scale noise over a per-expert offset.
        logits = randn(m, e) * 1.5 + randn(e)
        c["logits"] = logits.to(_TYPES[c["dtype"]])
        c["balance"] = randn(e) * 0.05 if c["bias"] else None
        c["ids"] = torch.empty(m, c["topk"], dtype=torch.int32, device="cuda")
        c["weights"] = torch.empty(m, c["topk"], dtype=torch.float32, device="cuda")
        return c
    if c["op"] in ("norm", "norm_matmul"):
        rows, hidden = c["rows"], c["hidden"]
        kind = c["op"] == "norm"
        # A few channels carry values far above the rest, as hidden states do.
        loud = 1.0 + 15.0 * (rand(hidden) < 0.005)
        c["x"] = (randn(rows, hidden) * loud).to(_TYPES[c["dtype"] if kind else "bf16"])
        residual = c["residual"] if kind else "bf16"
        c["res"] = None if residual == "none" else (randn(rows, hidden) * 2 * loud).to(_TYPES[residual])
        c["res_out"] = None if c["res"] is None else torch.empty_like(c["res"])
        c["gain"] = (1.0 + 0.1 * randn(hidden)).to(_TYPES[c["weight"] if kind else "bf16"])
        quant = c["quant"] if kind else "int8"
        c["y"] = torch.empty(rows, hidden, dtype=torch.bfloat16, device="cuda") if kind else None
        kinds = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
        c["q"] = None if quant == "none" else torch.empty(rows, hidden, dtype=kinds[quant], device="cuda")
        c["q_scale"] = None if quant == "none" else torch.empty(rows, device="cuda")
        if kind:
            return c
    tokens, k = (c["rows"], c["hidden"]) if c["op"] == "norm_matmul" else (c["tokens"], c["k"])
    if c["op"] == "matmul":
        c["x_q"] = _codes(g, tokens, k)
        c["x_scale"] = 0.01 + 0.05 * rand(tokens)
    c["w_q"] = _codes(g, c["n"], k)
    c["w_scale"] = 0.0002 + 0.001 * rand(c["n"])
    c["b"] = randn(c["n"]) if c.get("bias") else None
    c["out_t"] = torch.empty(tokens, c["n"], dtype=_TYPES[c.get("out", "bf16")], device="cuda")
    return c


# --------------------------------------------------------------------------- #
# The plain forms
# --------------------------------------------------------------------------- #
def _plain_route(s):
    m, e, k = s["tokens"], s["experts"], s["topk"]
    logits = s["logits"].double()  # a choice is a comparison of near values: 64 bits
    if s["score"] == "softmax":
        p = (logits - logits.amax(dim=1, keepdim=True)).exp()
        p = p / p.sum(dim=1, keepdim=True)
    else:
        p = 1.0 / (1.0 + (-logits).exp())
    choice = logits if s["balance"] is None else p + s["balance"].double()
    if s["groups"] > 1:
        by_group = (p if s["balance"] is None and s["top"] > 1 else choice).view(m, s["groups"], -1)
        best = by_group.sort(dim=2, descending=True, stable=True).values[:, :, :s["top"]].sum(dim=2)
        order = best.sort(dim=1, descending=True, stable=True).indices[:, :s["keep"]]
        kept = torch.zeros(m, s["groups"], dtype=torch.bool, device="cuda").scatter_(1, order, True)
        choice = choice.masked_fill(~kept.repeat_interleave(e // s["groups"], dim=1), -math.inf)
    ids = choice.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, ids)
    if s["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return [ids.to(torch.int32), (w * s["scale"]).float()]


def _plain_norm(x, res, gain, quant):
    """(x + res in the residual's type, the norm in 32 bits, codes, scales)."""
    r = x.float() if res is None else x.float() + res.float()
    y = r * torch.rsqrt(r.square().mean(dim=1, keepdim=True) + EPS) * gain.float()
    q = scale = None
    if quant != "none":
        most = INT8_MAX if quant == "int8" else E4M3_MAX
        scale = y.abs().amax(dim=1, keepdim=True) / most
        q = y / scale
        q = q.round().clamp(-most, most) if quant == "int8" else q.clamp(-most, most).to(torch.float8_e4m3fn)
        scale = scale[:, 0]
    return None if res is None else r.to(res.dtype), y, q, scale


def _plain_matmul(x_q, x_scale, w_q, w_scale, bias, dtype):
    # Sums of up to 8192 products of 127 * 127 pass 24 bits: 64 hold them exactly.
    out = (x_q.double() @ w_q.double().T) * x_scale.double()[:, None] * w_scale.double()
    return (out if bias is None else out + bias.double()).to(dtype)


def _plain(s):
    if s["op"] == "route":
        return _plain_route(s)
    if s["op"] == "norm":
        r, y, q, scale = _plain_norm(s["x"], s["res"], s["gain"], s["quant"])
        return {"y": y.to(torch.bfloat16), "residual": r, "q": q, "scale": scale}
    if s["op"] == "norm_matmul":
        r, _, q, scale = _plain_norm(s["x"], s["res"], s["gain"], "int8")
        out = _plain_matmul(q, scale, s["w_q"], s["w_scale"], None, torch.bfloat16)
        return {"out": out, "residual": r, "scale": scale}
    return _plain_matmul(s["x_q"], s["x_scale"], s["w_q"], s["w_scale"], s["b"], s["out_t"].dtype)


# --------------------------------------------------------------------------- #
# The framework's operators
# --------------------------------------------------------------------------- #
def _own(s):
    import nvfp4_weight_quantized_moe_b200 as nvm

    if s["op"] == "route":
        nvm.route_topk(s["logits"], s["ids"], s["weights"], score=s["score"], bias=s["balance"],
                       num_groups=s["groups"], topk_groups=s["keep"], group_top=s["top"],
                       renormalize=s["renorm"], scale=s["scale"])
        return [s["ids"], s["weights"]]
    if s["op"] == "norm":
        nvm.add_rms_norm(s["x"], s["gain"], EPS, out=s["y"], residual=s["res"],
                         residual_out=s["res_out"], q=s["q"], q_scale=s["q_scale"])
        return {"y": s["y"], "residual": s["res_out"], "q": s["q"], "scale": s["q_scale"]}
    if s["op"] == "norm_matmul":
        nvm.add_rms_norm(s["x"], s["gain"], EPS, residual=s["res"], residual_out=s["res_out"],
                         q=s["q"], q_scale=s["q_scale"])
        nvm.int8_matmul(s["q"], s["q_scale"], s["w_q"], s["w_scale"], s["out_t"])
        return {"out": s["out_t"], "residual": s["res_out"], "scale": s["q_scale"]}
    nvm.int8_matmul(s["x_q"], s["x_scale"], s["w_q"], s["w_scale"], s["out_t"], bias=s["b"])
    return s["out_t"]


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------- #
# What a pass cannot do without
# --------------------------------------------------------------------------- #
_BYTES = {"bf16": 2, "f32": 4, "none": 0, "e4m3": 1, "int8": 1}


def work(case):
    c = case
    if c["op"] == "route":
        m, e, k = c["tokens"], c["experts"], c["topk"]
        return {"bytes": m * e * _BYTES[c["dtype"]] + m * k * 8 + (4 * e if c["bias"] else 0),
                "flops": 4 * m * e}
    if c["op"] == "norm":
        rows, hidden = c["rows"], c["hidden"]
        per = _BYTES[c["dtype"]] + 2 * _BYTES[c["residual"]] + 2 + _BYTES[c["quant"]]
        return {"bytes": rows * hidden * per + hidden * _BYTES[c["weight"]]
                + (4 * rows if c["quant"] != "none" else 0), "flops": 5 * rows * hidden}
    if c["op"] == "norm_matmul":
        rows, k, n = c["rows"], c["hidden"], c["n"]
        return {"bytes": rows * k * 6 + 2 * k + 4 * rows + n * k + 4 * n + 2 * rows * n,
                "flops": 2 * rows * n * k + 6 * rows * k}
    m, k, n = c["tokens"], c["k"], c["n"]
    return {"bytes": m * k + n * k + 4 * (m + n) + m * n * _BYTES[c["out"]] + (4 * n if c["bias"] else 0),
            "flops": 2 * m * n * k}


# --------------------------------------------------------------------------- #
# The definitions in 64 bits
# --------------------------------------------------------------------------- #
def _exact_route(s):
    """Experts ranked one choice at a time, on the host."""
    l = s["logits"].double().cpu().numpy()
    m, e = l.shape
    if s["score"] == "softmax":
        z = np.exp(l - l.max(axis=1)[:, None])
        p = z / z.sum(axis=1)[:, None]
    else:
        p = np.where(l >= 0, 1 / (1 + np.exp(-np.abs(l))), np.exp(-np.abs(l)) / (1 + np.exp(-np.abs(l))))
    b = None if s["balance"] is None else s["balance"].double().cpu().numpy()
    choice = l.copy() if b is None else p + b
    rows = np.arange(m)
    if s["groups"] > 1:
        width = e // s["groups"]
        base = p if b is None and s["top"] > 1 else choice
        best = -np.partition(-base.reshape(m, s["groups"], width), s["top"] - 1, axis=2)[:, :, :s["top"]].sum(axis=2)
        closed = np.ones((m, s["groups"]), dtype=bool)
        for _ in range(s["keep"]):
            at = best.argmax(axis=1)
            closed[rows, at] = False
            best[rows, at] = -np.inf
        choice[np.repeat(closed, width, axis=1)] = -np.inf
    ids = np.empty((m, s["topk"]), dtype=np.int32)
    for j in range(s["topk"]):
        ids[:, j] = choice.argmax(axis=1)
        choice[rows, ids[:, j]] = -np.inf
    w = p[rows[:, None], ids]
    if s["renorm"]:
        w = w / w.sum(axis=1)[:, None]
    return [ids, w * s["scale"]]


def _exact_norm(s, quant):
    """Row blocks in float64; a code's value is the nearest of the type's to y / scale."""
    x, res, gain = s["x"], s["res"], s["gain"].double()
    y = torch.empty(x.shape, dtype=torch.float64, device="cuda")
    total = None if res is None else torch.empty_like(y)
    for at in range(0, x.shape[0], 1024):
        r = x[at:at + 1024].double()
        if res is not None:
            r = r + res[at:at + 1024].double()
            total[at:at + 1024] = r
        norm = (r * r).sum(dim=1) / r.shape[1] + EPS
        y[at:at + 1024] = r * gain / norm.sqrt()[:, None]
    if quant == "none":
        return total, y, None, None
    most = INT8_MAX if quant == "int8" else E4M3_MAX
    scale = torch.maximum(y.amax(dim=1), -y.amin(dim=1)) / most
    t = y / scale[:, None]
    if quant == "int8":
        return total, y, torch.round(t), scale
    # E4M3 keeps 4 significant bits, and steps of 2^-9 below 2^-6.
    exponent = torch.frexp(t).exponent.clamp(min=-5) - 4
    step = torch.ldexp(torch.ones_like(t), exponent)
    return total, y, (torch.round(t / step) * step).clamp(-most, most), scale


def _exact_product(x_q, x_scale, w_q, w_scale, bias):
    """Whole-number sums: slices of 1024 products stay under 2^24, their sums in int64."""
    total = torch.zeros(x_q.shape[0], w_q.shape[0], dtype=torch.int64, device="cuda")
    for at in range(0, x_q.shape[1], 1024):
        total += (x_q[:, at:at + 1024].float() @ w_q[:, at:at + 1024].float().T).to(torch.int64)
    out = total.double() * (x_scale.double()[:, None] * w_scale.double()[None, :])
    return out if bias is None else out + bias.double()[None, :]


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "route":
        return _exact_route(s)
    if s["op"] == "norm":
        total, y, q, scale = _exact_norm(s, s["quant"])
        return {"y": y, "residual": total, "q": q, "scale": scale}
    if s["op"] == "norm_matmul":
        total, _, q, scale = _exact_norm(s, "int8")
        return {"out": _exact_product(q, scale, s["w_q"], s["w_scale"], None), "residual": total,
                "scale": scale}
    return _exact_product(s["x_q"], s["x_scale"], s["w_q"], s["w_scale"], s["b"])
