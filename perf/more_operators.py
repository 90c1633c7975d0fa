"""Timed cases of the operators between the FP8 products of a layer of experts.

The operators, and what a pass of each computes:

* ``norm``: s = x + residual in the residual's type (s = x where there is no
  residual), y = s / sqrt(mean(s^2) + eps) * weight over each row, and y in FP8
  with one E8M0 code for each group of 128: along the rows and, in training,
  along the columns too.  ``norm_backward``: the gradients of s and of weight for
  the gradient of y, the gradient that reaches s past the norm added.
* ``activate``: a = act(gate) * up of the two halves of an up projection's
  result (a = act(gate) where there is no second half), in FP8 as above.  With
  experts, the column groups begin anew with each expert's rows.
  ``activate_backward``: the gradients of both halves for the gradient of a, in
  FP8 along rows and columns, the operands of the up projection's own gradients.
* ``route``: each token's experts and their weights from a router's logits:
  scores (softmax or sigmoid), a bias that takes part in the choice alone,
  groups of experts of which the best are kept, the best experts in those, their
  scores as weights, made to sum to 1 if asked.  ``route_backward``: the
  gradient of the logits for that of the weights.

A group's scale is 2^S with S = max(ceil(log2(amax / 448)), -127), its code S +
127, its payload RTNE_E4M3(y / 2^S).  With ``own`` unset a pass computes these
with elementary torch operations in 32 bits (scores and choices of ``route`` in
64, where two may lie next to each other), with ``own`` set it makes the calls
that a program makes of this repository's package.  Payloads and codes come back
as the E4M3 and E8M0 values that they are.
"""
import math

import torch

own = False

GROUP = 128
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
INF = float("inf")


# ---- the cases -------------------------------------------------------------------------

def listed():
    return [
        # one token's step before a projection: latency alone
        {"name": "norm_token", "kind": "norm", "rows": 1, "k": 8192, "dtype": "bf16", "stream": "bf16",
         "residual": True, "y": False, "cols": False},
        # a short prompt in fp32 through a layer whose sizes are multiples of nothing
        {"name": "norm_odd", "kind": "norm", "rows": 333, "k": 2857, "dtype": "fp32", "stream": "fp32",
         "residual": True, "y": True, "cols": False},
        # a long prompt before a layer of experts: y for the router and the experts' rows, FP8 for a shared one
        {"name": "norm_prompt", "kind": "norm", "rows": 8192, "k": 8192, "dtype": "bf16", "stream": "bf16",
         "residual": True, "y": True, "cols": False},
        # a training step with the residual held in fp32, for the forward and the weight-gradient product
        {"name": "norm_train", "kind": "norm", "rows": 4096, "k": 8192, "dtype": "bf16", "stream": "fp32",
         "residual": True, "y": False, "cols": True},
        # the way back through the norm of a training step
        {"name": "norm_backward", "kind": "norm_backward", "rows": 8192, "k": 8192, "dtype": "bf16", "stream": "bf16",
         "residual": True},
        # a few sequences' next tokens between the products of 48 experts
        {"name": "activate_token", "kind": "activate", "tokens": 9, "top_k": 6, "experts": 48, "f": 1024, "drop": 0.0,
         "dtype": "bf16", "act": "silu", "gated": True, "cols": False},
        # a prompt between the projections of a large MLP
        {"name": "activate_prompt", "kind": "activate", "rows": 2048, "f": 28672, "dtype": "bf16", "act": "silu",
         "gated": True, "cols": False},
        # a training step's rows between the products of 48 experts, some slots dropped at capacity
        {"name": "activate_train", "kind": "activate", "tokens": 8192, "top_k": 6, "experts": 48, "f": 1024,
         "drop": 0.02, "dtype": "bf16", "act": "silu", "gated": True, "cols": True},
        # the way back between the same products
        {"name": "activate_backward", "kind": "activate_backward", "tokens": 8192, "top_k": 6, "experts": 48, "f": 1024,
         "drop": 0.02, "dtype": "bf16", "act": "silu", "gated": True},
        # a few sequences' next tokens
        {"name": "route_token", "kind": "route", "tokens": 9, "experts": 48, "top_k": 6, "dtype": "bf16",
         "score": "softmax", "renormalize": True, "bias": False, "groups": 1, "top_groups": 1, "group_top": 1,
         "padding": 0.0, "closed": 0},
        # a long prompt's tokens to many experts, balanced by a bias, each token kept to half of the groups
        {"name": "route_prompt", "kind": "route", "tokens": 16384, "experts": 256, "top_k": 8, "dtype": "fp32",
         "score": "sigmoid", "renormalize": True, "bias": True, "groups": 8, "top_groups": 4, "group_top": 2,
         "padding": 0.05, "closed": 0},
        # a training step's way back to the router
        {"name": "route_backward", "kind": "route_backward", "tokens": 16384, "experts": 128, "top_k": 8,
         "dtype": "fp32", "score": "softmax", "renormalize": False, "bias": False, "groups": 1, "top_groups": 1,
         "group_top": 1, "padding": 0.05, "closed": 0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """A layer's size: mostly a multiple of 128 or of 16, sometimes of nothing."""
    v = _log_int(rng, lo, hi)
    step = rng.choice((128, 128, 16, 16, 1))
    return max(step, v // step * step)


def draw(rng):
    kind = rng.choice(("norm", "norm", "norm_backward", "activate", "activate", "activate_backward", "route", "route",
                       "route_backward"))
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    if kind.startswith("norm"):
        k = _size(rng, 64, 16384)
        rows = _log_int(rng, 1, min(16384, (1 << 25) // k))
        residual = rng.random() < 0.75
        stream = rng.choice((dtype, "fp32")) if residual else dtype
        case = {"kind": kind, "rows": rows, "k": k, "dtype": dtype, "stream": stream, "residual": residual}
        if kind == "norm":
            case["cols"] = rng.random() < 0.4
            case["y"] = rng.random() < 0.5
        return case
    if kind.startswith("activate"):
        f = _size(rng, 64, 28672)
        most = min(16384, (1 << 24) // f)
        case = {"kind": kind, "f": f, "dtype": dtype, "act": rng.choice(("silu", "silu", "gelu_tanh", "relu2")),
                "gated": rng.random() < 0.75}
        if rng.random() < 0.6:
            case["experts"] = _log_int(rng, 4, 160)
            case["top_k"] = rng.randint(1, min(8, case["experts"]))
            case["tokens"] = _log_int(rng, 1, max(1, most // case["top_k"]))
            case["drop"] = rng.choice((0.0, 0.0, 0.05))
        else:
            case["rows"] = _log_int(rng, 1, most)
        if kind == "activate":
            case["cols"] = rng.random() < 0.5
        return case
    groups = rng.choice((1, 1, 4, 8))
    experts = _log_int(rng, max(4, 2 * groups), 512) // groups * groups
    top_groups = rng.randint(1, groups)
    most = experts // groups * top_groups
    renormalize = rng.random() < 0.6
    least = 2 if kind == "route_backward" and renormalize else 1    # a single weight of 1 has no gradient
    return {"kind": kind, "tokens": _log_int(rng, 1, 32768), "experts": experts,
            "top_k": rng.randint(least, min(10, most)), "dtype": dtype, "score": rng.choice(("softmax", "sigmoid")),
            "renormalize": renormalize,
            "bias": rng.random() < 0.5, "groups": groups, "top_groups": top_groups, "group_top": rng.choice((1, 2)),
            "padding": rng.choice((0.0, 0.1)), "closed": rng.choice((0, 0, 3))}


# ---- inputs ----------------------------------------------------------------------------

def _activations(g, rows, cols, dtype):
    """Rows of unlike magnitude with a few channels far above the rest."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= torch.exp2(torch.randint(-3, 3, (rows, 1), generator=g, device="cuda").float())
    x *= torch.where(torch.rand(cols, generator=g, device="cuda") < 0.01, 16.0, 1.0)
    return x.to(dtype)


def _ceil(n, step=GROUP):
    return -(-n // step)


def _routing(case, g):
    """Offsets [experts + 1] of the slots of a router with favourites, sorted by expert; some are dropped."""
    t, k, n = case["tokens"], case["top_k"], case["experts"]
    logits = torch.randn(t, n, generator=g, device="cuda") + 0.7 * torch.randn(n, generator=g, device="cuda")
    ids = logits.topk(k, dim=1).indices
    ids = torch.where(torch.rand(t, k, generator=g, device="cuda") < case["drop"], n, ids).reshape(-1)
    return torch.searchsorted(ids.sort().values, torch.arange(n + 1, device="cuda")).int()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kind, s = case["kind"], {"case": case}
    dtype = DTYPES[case["dtype"]]
    if kind.startswith("norm"):
        rows, k, stream = case["rows"], case["k"], DTYPES[case["stream"]]
        s["weight"] = (1 + 0.1 * torch.randn(k, generator=g, device="cuda")).to(dtype)
        s["x"] = _activations(g, rows, k, dtype if kind == "norm" else stream)
        if rows > 4:
            s["x"][rows // 3] = 0    # the row of a padded place
        if kind == "norm":
            s["residual"] = _activations(g, rows, k, stream) if case["residual"] else None
            if rows > 4 and case["residual"]:
                s["residual"][rows // 3] = 0
            return s
        s["dy"] = _activations(g, rows, k, dtype)
        if rows > 4:
            s["dy"][rows // 3] = 0
        s["dresidual"] = _activations(g, rows, k, stream) if case["residual"] else None
        return s
    if kind.startswith("activate"):
        f, experts = case["f"], case.get("experts", 0)
        rows = case["tokens"] * case["top_k"] if experts else case["rows"]
        s["offsets"] = _routing(case, g) if experts else None
        h = _activations(g, rows, 2 * f if case["gated"] else f, torch.float32)
        if experts:
            h *= (torch.arange(rows, device="cuda") < s["offsets"][-1])[:, None]
        s["h"] = h.to(dtype)
        if kind == "activate_backward":
            s["da"] = _activations(g, rows, f, dtype)
        return s
    t, n = case["tokens"], case["experts"]
    logits = 1.5 * torch.randn(t, n, generator=g, device="cuda") + 0.7 * torch.randn(n, generator=g, device="cuda")
    if case["closed"]:    # experts that take no tokens at present, and a token that none may take
        logits[:, torch.randperm(n, generator=g, device="cuda")[:min(case["closed"], n - 1)]] = -INF
        logits[t // 2] = -INF
    s["logits"] = logits.to(dtype)
    s["bias"] = 0.1 * torch.randn(n, generator=g, device="cuda") if case["bias"] else None
    s["mask"] = torch.rand(t, generator=g, device="cuda") >= case["padding"] if case["padding"] else None
    if kind == "route_backward":
        s["ids"] = _plain_route(s)["ids"]
        s["dweights"] = torch.randn(t, case["top_k"], generator=g, device="cuda")
    return s


# ---- the plain forms -------------------------------------------------------------------

def _codes(amax):
    """E8M0 codes of groups with these largest magnitudes: amax = m 2^e with m in [0.5, 1), 448 = 0.875 * 2^9."""
    m, e = torch.frexp(amax)
    s = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-127)
    return torch.where(amax == 0, 0, s + 127).to(torch.uint8)


def _scales(codes):
    return torch.exp2(codes.double() - 127).float()


def _quantize_rows(v):
    rows, k = v.shape
    v = torch.nn.functional.pad(v, (0, _ceil(k) * GROUP - k)).view(rows, -1, GROUP)
    codes = _codes(v.abs().amax(-1))
    q = (v / _scales(codes)[..., None]).to(torch.float8_e4m3fn)
    return q.view(rows, -1)[:, :k].contiguous(), codes.view(torch.float8_e8m0fnu)


def _quantize_cols(v, offsets):
    """Payload [rows, K] and codes of groups of 128 rows, begun anew with each expert's rows.  Rows of no expert
    have payload 0, code rows that no group needs are 0."""
    rows, k = v.shape
    at = torch.arange(rows, device=v.device)
    if offsets is None:
        group, last, taken = at // GROUP, _ceil(rows), None
    else:
        ends = offsets.long()
        expert = torch.searchsorted(ends[1:], at, right=True)
        first = torch.nn.functional.pad(((ends.diff() + GROUP - 1) // GROUP).cumsum(0), (1, 0))
        last = rows // GROUP + ends.numel() - 1
        taken = (at < ends[-1])[:, None]
        group = torch.where(taken[:, 0], first[expert] + (at - ends[expert]) // GROUP, last)
    amax = v.new_zeros((last + 1, k)).scatter_reduce_(0, group[:, None].expand(rows, k), v.abs(), "amax")
    codes = _codes(amax)
    q = v / _scales(codes)[group]
    if taken is not None:
        q = torch.where(taken, q, 0.0)
    return q.to(torch.float8_e4m3fn), codes[:last].view(torch.float8_e8m0fnu)


def _plain_norm(s):
    case = s["case"]
    x = s["x"].float()
    out = {}
    if case["residual"]:
        out["residual"] = (x + s["residual"].float()).to(s["residual"].dtype)
        x = out["residual"].float()
    y = x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * s["weight"].float()
    out["row"], out["row_scale"] = _quantize_rows(y)
    if case["cols"]:
        out["col"], out["col_scale"] = _quantize_cols(y, None)
    if case["y"]:
        out["y"] = y.to(s["x"].dtype)
    return out


def _plain_norm_backward(s):
    x, dy = s["x"].float(), s["dy"].float()
    r = torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)
    u, g = x * r, dy * s["weight"].float()
    dx = r * (g - u * (g * u).mean(1, keepdim=True))
    if s["dresidual"] is not None:
        dx = dx + s["dresidual"].float()
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * u).sum(0)}


def _halves(s):
    f, h = s["case"]["f"], s["h"].float()
    return (h[:, :f], h[:, f:]) if s["case"]["gated"] else (h, None)


def _logistic(z):
    e = torch.exp(-z.abs())    # no overflow, and no cancellation where z is far below 0
    return torch.where(z < 0, e, 1.0) / (1 + e)


def _act(name, g):
    """act(g) and its derivative."""
    if name == "silu":
        p = _logistic(g)
        return g * p, p * (1 + g * (1 - p))
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        p = _logistic(2 * c * (g + 0.044715 * g ** 3))    # (1 + tanh(z)) / 2 = 1 / (1 + exp(-2 z))
        return g * p, p + g * p * (1 - p) * 2 * c * (1 + 3 * 0.044715 * g * g)
    r = g.clamp(min=0)
    return r * r, 2 * r


def _plain_activate(s):
    case = s["case"]
    gate, up = _halves(s)
    a = _act(case["act"], gate)[0]
    if up is not None:
        a = a * up
    out = {}
    out["row"], out["row_scale"] = _quantize_rows(a)
    if case["cols"]:
        out["col"], out["col_scale"] = _quantize_cols(a, s["offsets"])
    return out


def _plain_activate_backward(s):
    gate, up = _halves(s)
    a, d = _act(s["case"]["act"], gate)
    da = s["da"].float()
    dh = da * d if up is None else torch.cat((da * up * d, da * a), 1)
    row, row_scale = _quantize_rows(dh)
    col, col_scale = _quantize_cols(dh, s["offsets"])
    return {"row": row, "row_scale": row_scale, "col": col, "col_scale": col_scale}


def _scores(logits, kind):
    """Scores in 64 bits; an expert whose logit is -inf is closed and scores 0."""
    l = logits.double()
    if kind == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    e = torch.exp(l - l.amax(1, keepdim=True).clamp(min=-1e300))
    return e / e.sum(1, keepdim=True).clamp(min=1e-300)


def _plain_route(s):
    case, logits = s["case"], s["logits"]
    tokens, experts = logits.shape
    score = _scores(logits, case["score"])
    key = logits.double() if s["bias"] is None else score + s["bias"].double()
    value = score if s["bias"] is None else key
    open_ = logits > -INF
    if s["mask"] is not None:
        open_ = open_ & s["mask"][:, None]
    key = torch.where(open_, key, -INF)
    if case["groups"] > 1:
        best, at = key.view(tokens, case["groups"], -1).sort(dim=2, descending=True, stable=True)
        best, at = best[..., :case["group_top"]], at[..., :case["group_top"]]
        if case["group_top"] == 1:
            rank = best[..., 0]
        else:
            v = value.view(tokens, case["groups"], -1).gather(2, at)
            rank = torch.where(best[..., 0] > -INF, torch.where(best > -INF, v, 0.0).sum(2), -INF)
        order = rank.sort(dim=1, descending=True, stable=True).indices[:, :case["top_groups"]]
        kept = torch.zeros_like(rank, dtype=torch.bool).scatter_(1, order, True)
        key = torch.where(kept.repeat_interleave(experts // case["groups"], 1), key, -INF)
    best, ids = key.sort(dim=1, descending=True, stable=True)
    best, ids = best[:, :case["top_k"]], ids[:, :case["top_k"]]
    w = torch.where(best > -INF, score.gather(1, ids), 0.0)
    if case["renormalize"]:
        w = w / torch.where(w.sum(1, keepdim=True) > 0, w.sum(1, keepdim=True), 1.0)
    return {"ids": torch.where(best > -INF, ids, -1).int(), "weights": w.float()}


def _plain_route_backward(s):
    case, ids = s["case"], s["ids"].long()
    score = _scores(s["logits"], case["score"])
    rest = (1 - score).gather(1, ids.clamp(min=0)).float()    # in 64 bits, where scores next to 1 cancel
    score = score.float()
    kept = ids >= 0
    p = torch.where(kept, score.gather(1, ids.clamp(min=0)), 0.0)
    g = torch.where(kept, s["dweights"], 0.0)
    if case["renormalize"]:    # the weights are p / sum(p)
        total = p.sum(1, keepdim=True)
        w = p / torch.where(total > 0, total, 1.0)
        d = w * (g - (g * w).sum(1, keepdim=True))    # p times the gradient of p
    else:
        d = p * g
    if case["score"] == "sigmoid":
        d = d * rest
    out = torch.zeros_like(score).scatter_add_(1, ids.clamp(min=0), torch.where(kept, d, 0.0))
    if case["score"] == "softmax" and not case["renormalize"]:    # where they sum to 1 the gradients sum to 0 by themselves
        out = out - score * d.sum(1, keepdim=True)
    return {"dlogits": out.to(s["logits"].dtype)}


def _plain(s):
    return {"norm": _plain_norm, "norm_backward": _plain_norm_backward, "activate": _plain_activate,
            "activate_backward": _plain_activate_backward, "route": _plain_route,
            "route_backward": _plain_route_backward}[s["case"]["kind"]](s)


# ---- the package's calls ---------------------------------------------------------------

def _fp8(row, row_scale, col=None, col_scale=None):
    out = {"row": row.view(torch.float8_e4m3fn), "row_scale": row_scale.view(torch.float8_e8m0fnu)}
    if col is not None:
        out["col"], out["col_scale"] = col.view(torch.float8_e4m3fn), col_scale.view(torch.float8_e8m0fnu)
    return out


def _own(s):
    import microscaling_weight_quantization_amd as mxq
    case = s["case"]
    kind = case["kind"]
    if kind == "norm":
        if case["cols"]:
            *q, residual, y = mxq.mxq_rms_norm_fp8_group128_row_col(s["x"], s["weight"], EPS, residual=s["residual"],
                                                                    with_y=case["y"])
        else:
            *q, residual, y = mxq.mxq_rms_norm_fp8_group128(s["x"], s["weight"], EPS, residual=s["residual"],
                                                            with_y=case["y"])
        out = _fp8(*q)
        if case["residual"]:
            out["residual"] = residual
        if case["y"]:
            out["y"] = y
        return out
    if kind == "norm_backward":
        dx, dweight = mxq.mxq_rms_norm_backward(s["dy"], s["x"], s["weight"], EPS, dresidual=s["dresidual"])
        return {"dx": dx, "dweight": dweight}
    if kind.startswith("activate"):
        f, h = case["f"], s["h"]
        gate, up = (h[:, :f], h[:, f:]) if case["gated"] else (h, None)
        if kind == "activate_backward":
            return _fp8(*mxq.mxq_activate_fp8_group128_backward(s["da"], gate, up, case["act"], offsets=s["offsets"]))
        if case["cols"]:
            return _fp8(*mxq.mxq_activate_fp8_group128_row_col(gate, up, case["act"], offsets=s["offsets"]))
        return _fp8(*mxq.mxq_activate_fp8_group128(gate, up, case["act"]))
    how = {"score": case["score"], "renormalize": case["renormalize"]}
    if kind == "route":
        ids, weights = mxq.mxq_route_experts(s["logits"], case["top_k"], bias=s["bias"], mask=s["mask"],
                                             n_groups=case["groups"], top_groups=case["top_groups"],
                                             group_top=case["group_top"], **how)
        return {"ids": ids, "weights": weights}
    return {"dlogits": mxq.mxq_route_experts_backward(s["dweights"], s["logits"], s["ids"], **how)}


def run(state):
    return _own(state) if own else _plain(state)


# ---- the least that a pass moves and computes ------------------------------------------

def work(case):
    kind = case["kind"]
    size = {"bf16": 2, "fp32": 4}[case["dtype"]]
    if kind.startswith("norm"):
        rows, k = case["rows"], case["k"]
        stream = {"bf16": 2, "fp32": 4}[case["stream"]]
        n = rows * k
        if kind == "norm_backward":
            return {"bytes": n * (size + stream * (3 if case["residual"] else 2)) + k * (size + 4), "flops": 12 * n}
        moved = n * (size + (2 * stream if case["residual"] else 0) + (size if case["y"] else 0) + 1) + k * size
        moved += rows * _ceil(k) + (n + _ceil(rows) * k if case["cols"] else 0)
        return {"bytes": moved, "flops": n * (8 if case["cols"] else 7)}
    if kind.startswith("activate"):
        f, experts = case["f"], case.get("experts", 0)
        rows = case["tokens"] * case["top_k"] if experts else case["rows"]
        h = 2 * f if case["gated"] else f
        if kind == "activate_backward":
            code_rows = rows // GROUP + experts if experts else _ceil(rows)
            return {"bytes": rows * (h + f) * size + 2 * rows * h + rows * _ceil(h) + code_rows * h,
                    "flops": 16 * rows * h}
        moved = rows * (h * size + f + _ceil(f))
        if case["cols"]:
            moved += rows * f + (rows // GROUP + experts if experts else _ceil(rows)) * f
        return {"bytes": moved, "flops": 10 * rows * f}
    t, n, k = case["tokens"], case["experts"], case["top_k"]
    if kind == "route":
        return {"bytes": t * (n * size + 8 * k) + 4 * n, "flops": 8 * t * n}
    return {"bytes": t * (2 * n * size + 8 * k), "flops": 8 * t * n}


# ---- the definitions in 64 bits --------------------------------------------------------

def _exact_groups(v):
    """v / 2^S of groups along the last axis, before the rounding to 8 bits."""
    amax = v.abs().amax(-1, keepdim=True)
    s = torch.floor(torch.log2(torch.where(amax == 0, 1.0, amax))) - 8
    s = s + (amax > 448 * torch.exp2(s)).double()
    return v * torch.exp2(-torch.where(amax == 0, 0.0, s.clamp(min=-127)))


def _exact_rows(v):
    rows, k = v.shape
    full = v.new_zeros(rows, _ceil(k) * GROUP)
    full[:, :k] = v
    return _exact_groups(full.view(rows, -1, GROUP)).view(rows, -1)[:, :k]


def _exact_cols(v, offsets):
    rows = v.shape[0]
    ends = [0, rows] if offsets is None else offsets.tolist()
    out = torch.zeros_like(v)
    for lo, hi in zip(ends, ends[1:]):
        if hi > lo:
            out[lo:hi] = _exact_rows(v[lo:hi].t().contiguous()).t()
    return out


def _exact_fp8(v, cols, offsets=None):
    """A code next to a border may fall on either side of it; the payload tells whether it is the right one."""
    out = {"row": _exact_rows(v), "row_scale": None}
    if cols:
        out["col"], out["col_scale"] = _exact_cols(v, offsets), None
    return out


def _exact_norm(case, s):
    x, w = s["x"].double(), s["weight"].double()
    k = case["k"]
    out = {}
    if s.get("residual") is not None:
        out["residual"] = x + s["residual"].double()
        x = out["residual"].to(s["residual"].dtype).double()    # the norm is that of the sum as it is stored
    root = torch.sqrt((x * x).sum(1) / k + EPS)[:, None]
    if case["kind"] == "norm":
        y = x / root * w
        out.update(_exact_fp8(y, case["cols"]))
        if case["y"]:
            out["y"] = y
        return out
    dy = s["dy"].double()
    inner = (dy * w * x).sum(1, keepdim=True)
    dx = dy * w / root - x * inner / (k * root ** 3)
    if s["dresidual"] is not None:
        dx += s["dresidual"].double()
    return {"dx": dx, "dweight": (dy * x / root).sum(0)}


def _exact_act(name, g):
    """With h = (1 + tanh(z)) / 2, and 1 - tanh(z)^2 = 4 h (1 - h), without their cancellation."""
    half = lambda z: torch.exp(-torch.logaddexp(torch.zeros_like(z), -2 * z))  # noqa: E731
    if name == "silu":
        return g * half(g / 2), half(g / 2) + g * half(g / 2) * half(-g / 2)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        z = c * (g + 0.044715 * g * g * g)
        return g * half(z), half(z) + 2 * g * half(z) * half(-z) * c * (1 + 0.134145 * g * g)
    return torch.where(g > 0, g * g, 0.0), torch.where(g > 0, 2 * g, 0.0)


def _exact_activate(case, s):
    f, h = case["f"], s["h"].double()
    a, d = _exact_act(case["act"], h[:, :f])
    up = h[:, f:] if case["gated"] else 1.0
    if case["kind"] == "activate":
        return _exact_fp8(a * up, case["cols"], s["offsets"])
    da = s["da"].double()
    dh = da * up * d
    if case["gated"]:
        dh = torch.cat((dh, da * a), 1)
    return _exact_fp8(dh, True, s["offsets"])


def _exact_scores(logits, kind):
    l = logits.double()
    if kind == "sigmoid":
        return torch.where(l > 0, 1 / (1 + torch.exp(-l)), torch.exp(l) / (1 + torch.exp(l)))
    return torch.nan_to_num(torch.exp(l - torch.logsumexp(l, 1, keepdim=True)), nan=0.0)


def _exact_route(case, s):
    t, n = s["logits"].shape
    score = _exact_scores(s["logits"], case["score"])
    left = s["logits"].double() if s["bias"] is None else score + s["bias"].double()
    value = score if s["bias"] is None else left.clone()
    left = torch.where(s["logits"].double() == -INF, -INF, left)
    if s["mask"] is not None:
        left[~s["mask"]] = -INF
    if case["groups"] > 1:    # group by group, the first of those that rank alike
        size = n // case["groups"]
        rank = []
        for j in range(case["groups"]):
            part, v = left[:, j * size:(j + 1) * size].clone(), value[:, j * size:(j + 1) * size]
            total = torch.full((t,), -INF, dtype=torch.float64, device=left.device)
            for i in range(min(case["group_top"], size)):
                best = part.amax(1)
                at = (part == best[:, None]).double().argmax(1, keepdim=True)
                more = v.gather(1, at)[:, 0] if case["group_top"] > 1 else best
                total = torch.where(best == -INF, total, more if i == 0 else total + more)
                part.scatter_(1, at, -INF)
            rank.append(total)
        rank = torch.stack(rank, 1)
        before = torch.zeros_like(rank)
        for j in range(case["groups"]):
            ahead = (rank > rank[:, j:j + 1]).double()
            ahead[:, :j] += (rank[:, :j] == rank[:, j:j + 1]).double()
            before[:, j] = ahead.sum(1)
        for j in range(case["groups"]):
            left[:, j * size:(j + 1) * size][before[:, j] >= case["top_groups"]] = -INF
    weights = torch.zeros((t, case["top_k"]), dtype=torch.float64, device=left.device)
    for j in range(case["top_k"]):
        best = left.amax(1)
        at = (left == best[:, None]).double().argmax(1, keepdim=True)
        weights[:, j] = torch.where(best == -INF, 0.0, score.gather(1, at)[:, 0])
        left.scatter_(1, at, -INF)
    if case["renormalize"]:
        weights = torch.nan_to_num(weights / weights.sum(1, keepdim=True), nan=0.0)
    return {"ids": None, "weights": weights}


def _exact_route_backward(case, s):
    """The chain rule with the scores' whole Jacobian, token by token of the choices."""
    ids, score = s["ids"].long(), _exact_scores(s["logits"], case["score"])
    t, n = score.shape
    chosen = torch.zeros((t, n), dtype=torch.float64, device=score.device)
    g = torch.zeros_like(chosen)
    for j in range(case["top_k"]):
        at = torch.nonzero(ids[:, j] >= 0).squeeze(1)
        chosen[at, ids[at, j]] = 1
        g[at, ids[at, j]] = s["dweights"][at, j].double()
    if case["renormalize"]:
        total = (chosen * score).sum(1, keepdim=True)
        total = torch.where(total > 0, total, 1.0)
        g = chosen * (g - (g * (score / total)).sum(1, keepdim=True)) / total
    if case["score"] == "sigmoid":
        return {"dlogits": g * score * (1 - score)}
    return {"dlogits": score * (g - (g * score).sum(1, keepdim=True))}


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind.startswith("norm"):
        return _exact_norm(case, s)
    if kind.startswith("activate"):
        return _exact_activate(case, s)
    return _exact_route(case, s) if kind == "route" else _exact_route_backward(case, s)
