"""Timed cases of the FP8 products and of the expert routing around them.

The operators, and what a pass of each computes:

* ``quantize``: activations or gradients in FP8 with one E8M0 code for each
  group of 128 -- along the row (the operand of a forward or an input-gradient
  product), and in training along the column as well (the operand of a
  weight-gradient product).
* ``matmul``: y = x w^T, ``dgrad``: dx = dy w, ``wgrad``: dw = dy^T x, of FP8
  payloads whose codes stand for groups of 128 (activations, gradients) and for
  128 x 128 tiles (weights).  With experts, rows are sorted by expert and each
  expert has a weight of its own.
* ``route``: token slots sorted by expert, and the tokens' rows brought into
  that order, quantized on the way or as they are.
* ``combine``: the experts' rows brought back to their tokens, weighted and
  added up; with ``backward`` also the gradients of rows and weights.

A group's scale is 2^S with S = max(ceil(log2(amax / 448)), -127), its code S +
127, its payload RTNE_E4M3(x / 2^S).  With ``own`` unset a pass computes these
with elementary torch operations in 32 bits, with ``own`` set it makes the calls
that a program makes of this repository's package.
"""
import math

import torch

own = False

GROUP = 128
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---- the cases -------------------------------------------------------------------------

def listed():
    return [
        # one token's activations before a projection: latency alone
        {"name": "quantize_token", "kind": "quantize", "rows": 1, "k": 8192, "dtype": "bf16", "cols": False},
        # a training step's activations, for the forward and the weight-gradient product
        {"name": "quantize_train", "kind": "quantize", "rows": 8192, "k": 8192, "dtype": "bf16", "cols": True},
        # one token through the up projection of a large MLP: the weight's bytes are the work
        {"name": "matmul_token", "kind": "matmul", "m": 1, "n": 28672, "k": 8192, "out": "bf16"},
        # a short prompt through a layer whose sizes are multiples of nothing
        {"name": "matmul_odd", "kind": "matmul", "m": 333, "n": 5003, "k": 2857, "out": "fp32"},
        # a long prompt or a training step's tokens through a square projection
        {"name": "matmul_prompt", "kind": "matmul", "m": 8192, "n": 8192, "k": 8192, "out": "bf16"},
        # the gradient of the up projection's input
        {"name": "dgrad_train", "kind": "dgrad", "m": 4096, "n": 28672, "k": 8192, "out": "bf16"},
        # the gradients of 48 experts' weights, summed in fp32 for the optimizer
        {"name": "wgrad_experts", "kind": "wgrad", "tokens": 4096, "top_k": 6, "experts": 48, "n": 1024, "k": 2048,
         "drop": 0.0, "out": "fp32"},
        # a few sequences' next tokens through 48 experts: each weight is read for a row or two
        {"name": "experts_token", "kind": "matmul", "tokens": 9, "top_k": 6, "experts": 48, "n": 1024, "k": 2048,
         "drop": 0.0, "out": "bf16"},
        # a prompt through the same experts, some slots dropped at capacity
        {"name": "experts_prompt", "kind": "matmul", "tokens": 8192, "top_k": 6, "experts": 48, "n": 1024, "k": 2048,
         "drop": 0.02, "out": "bf16"},
        # routing a few sequences' next tokens, rows quantized on their way to the experts
        {"name": "route_token", "kind": "route", "tokens": 9, "top_k": 6, "experts": 48, "k": 2048, "drop": 0.0,
         "dtype": "bf16", "fp8": True},
        # routing a prompt's tokens, rows as they are
        {"name": "route_prompt", "kind": "route", "tokens": 16384, "top_k": 8, "experts": 128, "k": 2048,
         "drop": 0.02, "dtype": "bf16", "fp8": False},
        # a training step's way back: the layer's output, then the gradients of rows and weights
        {"name": "combine_train", "kind": "combine", "tokens": 8192, "top_k": 6, "experts": 48, "k": 2048,
         "drop": 0.02, "dtype": "bf16", "backward": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """A layer's size: mostly a multiple of 128 or of 16, sometimes of nothing."""
    v = _log_int(rng, lo, hi)
    step = rng.choice((128, 128, 16, 16, 1))
    return max(step, v // step * step)


def draw(rng):
    kind = rng.choice(("quantize", "matmul", "matmul", "dgrad", "wgrad", "experts", "experts", "route", "combine"))
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    if kind == "quantize":
        k = _size(rng, 128, 16384)
        rows = _log_int(rng, 1, min(16384, (1 << 26) // k))
        return {"kind": kind, "rows": rows, "k": k, "dtype": dtype, "cols": rng.random() < 0.5}
    if kind in ("matmul", "dgrad", "wgrad"):
        n, k = _size(rng, 256, 16384), _size(rng, 256, 16384)
        n = min(n, (1 << 28) // k)
        m = _log_int(rng, 1, max(1, min(16384, (1 << 38) // (n * k))))
        return {"kind": kind, "m": m, "n": n, "k": k, "out": rng.choice(("bf16", "bf16", "fp32"))}
    experts = _log_int(rng, 4, 160)
    top_k = rng.randint(1, min(8, experts))
    drop = rng.choice((0.0, 0.0, 0.05))
    if kind == "experts":
        n, k = _size(rng, 256, 4096), _size(rng, 256, 4096)
        experts = max(4, min(experts, (1 << 28) // (n * k)))
        top_k = min(top_k, experts)
        tokens = _log_int(rng, 1, max(1, min(16384, (1 << 37) // (n * k * top_k))))
        return {"kind": rng.choice(("matmul", "matmul", "dgrad", "wgrad")), "tokens": tokens, "top_k": top_k,
                "experts": experts, "n": n, "k": k, "drop": drop, "out": rng.choice(("bf16", "bf16", "fp32"))}
    k = _size(rng, 256, 8192)
    tokens = _log_int(rng, 1, max(1, min(32768, (1 << 27) // (k * top_k))))
    case = {"kind": kind, "tokens": tokens, "top_k": top_k, "experts": experts, "k": k, "drop": drop, "dtype": dtype}
    case["fp8" if kind == "route" else "backward"] = rng.random() < 0.5
    return case


# ---- inputs ----------------------------------------------------------------------------

def _activations(g, rows, cols, dtype):
    """Rows of unlike magnitude with a few channels far above the rest."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= torch.exp2(torch.randint(-3, 3, (rows, 1), generator=g, device="cuda").float())
    x *= torch.where(torch.rand(cols, generator=g, device="cuda") < 0.01, 16.0, 1.0)
    return x.to(dtype)


def _codes(amax):
    """E8M0 codes of groups with these largest magnitudes: amax = m 2^e with m in [0.5, 1), 448 = 0.875 * 2^9."""
    m, e = torch.frexp(amax)
    s = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-127)
    return torch.where(amax == 0, 0, s + 127).to(torch.uint8)


def _scales(codes):
    return torch.exp2(codes.double() - 127).float()


def _pad(x, rows, cols):
    return torch.nn.functional.pad(x, (0, cols - x.shape[-1], 0, rows - x.shape[-2]))


def _ceil(n, step=GROUP):
    return -(-n // step)


def _quantize_rows(x):
    rows, k = x.shape
    v = _pad(x.float(), rows, _ceil(k) * GROUP).view(rows, -1, GROUP)
    codes = _codes(v.abs().amax(-1))
    q = (v / _scales(codes)[..., None]).to(torch.float8_e4m3fn)
    return q.view(rows, -1)[:, :k].contiguous(), codes


def _weight(g, experts, n, k):
    """FP8 weights with a code for each 128 x 128 tile."""
    q = torch.empty((experts, n, k), dtype=torch.float8_e4m3fn, device="cuda")
    codes = torch.empty((experts, _ceil(n), _ceil(k)), dtype=torch.uint8, device="cuda")
    for e in range(experts):
        w = torch.randn(n, k, generator=g, device="cuda") * 0.02
        w = _pad(w, _ceil(n) * GROUP, _ceil(k) * GROUP).view(_ceil(n), GROUP, _ceil(k), GROUP)
        codes[e] = _codes(w.abs().amax((1, 3)))
        w = (w / _scales(codes[e])[:, None, :, None]).view(_ceil(n) * GROUP, _ceil(k) * GROUP)[:n, :k]
        q[e] = w.to(torch.float8_e4m3fn)
    return q, codes


def _routing(case, g):
    """Expert ids [tokens, top_k] of a router with favourites (-1: a dropped slot) and the slots' weights."""
    t, k, n = case["tokens"], case["top_k"], case["experts"]
    logits = torch.randn(t, n, generator=g, device="cuda") + 0.7 * torch.randn(n, generator=g, device="cuda")
    top = logits.topk(k, dim=1)
    ids = torch.where(torch.rand(t, k, generator=g, device="cuda") < case["drop"], -1, top.indices).int()
    if case["drop"]:
        ids[t // 2] = -1    # a token that no expert takes
    return ids, torch.softmax(top.values, dim=1)


def _sort(ids, experts):
    """(offsets [experts + 1], slots, positions): slots in the order of their experts, dropped ones last and
    complemented, and the same the other way round."""
    flat = ids.reshape(-1).long()
    dropped = (flat < 0) | (flat >= experts)
    key, order = torch.where(dropped, experts, flat).sort(stable=True)
    offsets = torch.searchsorted(key, torch.arange(experts + 1, device=key.device))
    position = torch.empty_like(order)
    position[order] = torch.arange(order.numel(), device=order.device)
    slots = torch.where(key == experts, ~order, order)
    position = torch.where(dropped, ~position, position)
    return offsets.int(), slots.int(), position.int().view(ids.shape)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kind, s = case["kind"], {"case": case}
    if kind == "quantize":
        s["x"] = _activations(g, case["rows"], case["k"], DTYPES[case["dtype"]])
        return s
    if kind in ("matmul", "dgrad", "wgrad"):
        n, k, experts = case["n"], case["k"], case.get("experts", 0)
        m = case["tokens"] * case["top_k"] if experts else case["m"]
        s["offsets"], s["most"] = None, m
        if experts:
            s["offsets"] = _sort(_routing(case, g)[0], experts)[0]
            s["most"] = max(1, int(s["offsets"].diff().max()))
        if kind == "wgrad":
            segments = s["offsets"] if experts else torch.tensor([0, m], dtype=torch.int32, device="cuda")
            s["dy"] = _quantize_cols(_activations(g, m, n, torch.float32), segments, s["most"])
            s["x"] = _quantize_cols(_activations(g, m, k, torch.float32), segments, s["most"])
            return s
        s["a"] = _quantize_rows(_activations(g, m, n if kind == "dgrad" else k, torch.float32))
        w, codes = _weight(g, max(1, experts), n, k)
        s["w"] = (w, codes) if experts else (w[0], codes[0])
        return s
    s["ids"], s["weights"] = _routing(case, g)
    dtype = DTYPES[case["dtype"]]
    if kind == "route":
        s["x"] = _activations(g, case["tokens"], case["k"], dtype)
        return s
    s["offsets"], s["slots"], s["position"] = _sort(s["ids"], case["experts"])
    s["rows"] = _activations(g, case["tokens"] * case["top_k"], case["k"], dtype)
    s["dy"] = _activations(g, case["tokens"], case["k"], dtype)
    return s


# ---- the plain forms -------------------------------------------------------------------

def _places(offsets, rows, most):
    """Where each sorted row stands in a [experts * most + 1] layout that gives every expert `most` rows (the last
    place takes the rows of no expert), and its expert."""
    at = torch.arange(rows, device=offsets.device)
    expert = torch.searchsorted(offsets[1:].long(), at, right=True)
    experts = offsets.numel() - 1
    place = expert * most + at - offsets.long()[expert]
    return torch.where(expert == experts, experts * most, place), expert


def _spread(x, places, experts, most):
    out = x.new_zeros((experts * most + 1, x.shape[1]))
    out[places] = x
    out[-1] = 0
    return out[:-1].view(experts, most, -1)


def _first_groups(offsets):
    """The first group of 128 of each segment: groups begin anew with every segment."""
    return torch.nn.functional.pad(((offsets.diff() + GROUP - 1) // GROUP).cumsum(0), (1, 0))


def _group_of_row(offsets, rows):
    at = torch.arange(rows, device=offsets.device)
    expert = torch.searchsorted(offsets[1:].long(), at, right=True)
    first = _first_groups(offsets)
    return torch.where(at < offsets[-1], first[expert] + (at - offsets.long()[expert]) // GROUP, -1)


def _quantize_cols(x, offsets, most):
    """Payload [rows, K] and codes [rows // 128 + segments, K] of groups of 128 rows, begun anew with each segment.
    Rows of no segment have payload 0, groups that hold no row code 0."""
    rows, k = x.shape
    experts, slots = offsets.numel() - 1, _ceil(most)
    places, expert = _places(offsets, rows, slots * GROUP)
    v = _spread(x.float(), places, experts, slots * GROUP).view(experts * slots, GROUP, k)
    codes = _codes(v.abs().amax(1))
    q = (v / _scales(codes)[:, None]).view(-1, k)
    q = torch.where((expert < experts)[:, None], q[places.clamp(max=experts * slots * GROUP - 1)], 0.0)
    out = torch.zeros((rows // GROUP + experts + 1, k), dtype=torch.uint8, device=x.device)
    group = torch.arange(slots, device=x.device)[None, :].expand(experts, slots)
    first = _first_groups(offsets)
    to = torch.where(group < first.diff()[:, None], first[:-1, None] + group, out.shape[0] - 1)
    out[to.reshape(-1)] = codes
    return q.to(torch.float8_e4m3fn), out[:-1]


def _rows32(q, codes):
    return q.float() * _scales(codes).repeat_interleave(GROUP, 1)[:, :q.shape[1]]


def _cols32(q, codes, offsets):
    if offsets is None:
        return q.float() * _scales(codes).repeat_interleave(GROUP, 0)[:q.shape[0]]
    group = _group_of_row(offsets, q.shape[0])
    return torch.where((group >= 0)[:, None], q.float() * _scales(codes)[group.clamp(min=0)], 0.0)


def _tiles32(q, codes):
    n, k = q.shape[-2:]
    s = _scales(codes).repeat_interleave(GROUP, -1).repeat_interleave(GROUP, -2)
    return q.float() * s[..., :n, :k]


def _plain_product(s):
    case, out, offsets = s["case"], DTYPES[s["case"]["out"]], s["offsets"]
    if case["kind"] == "wgrad":
        dy, x = _cols32(*s["dy"], offsets), _cols32(*s["x"], offsets)
        if offsets is None:
            return (dy.t().contiguous() @ x).to(out)
        experts, most = offsets.numel() - 1, s["most"]
        places, _ = _places(offsets, dy.shape[0], most)
        dy, x = _spread(dy, places, experts, most), _spread(x, places, experts, most)
        return torch.bmm(dy.transpose(1, 2).contiguous(), x).to(out)
    a, w = _rows32(*s["a"]), _tiles32(*s["w"])
    if offsets is None:
        return (a @ (w if case["kind"] == "dgrad" else w.t())).to(out)
    experts, most = offsets.numel() - 1, s["most"]
    places, expert = _places(offsets, a.shape[0], most)
    a = _spread(a, places, experts, most)
    if case["kind"] == "dgrad":
        y = torch.bmm(a, w)
    else:
        y = torch.bmm(w, a.transpose(1, 2).contiguous()).transpose(1, 2)
    y = y.reshape(experts * most, -1)[places.clamp(max=experts * most - 1)]
    return torch.where((expert < experts)[:, None], y, 0.0).to(out)


def _gather(x, slots, top_k):
    """Each sorted slot's token row; a dropped slot's row is 0."""
    rows = x[torch.where(slots < 0, 0, slots).long() // top_k]
    return torch.where((slots >= 0)[:, None], rows, torch.zeros((), dtype=x.dtype, device=x.device))


def _plain_combine(s):
    case, position, w = s["case"], s["position"].long(), s["weights"]
    kept = position >= 0
    rows = s["rows"][position.clamp(min=0)].float() * kept[..., None]
    out = {"y": (rows * w[..., None]).sum(1).to(s["rows"].dtype)}
    if case["backward"]:
        dy = s["dy"].float()
        out["dweights"] = (rows * dy[:, None]).sum(-1)
        slots = s["slots"].long()
        at = slots.clamp(min=0)
        drows = dy[at // case["top_k"]] * w.reshape(-1)[at][:, None]
        out["drows"] = torch.where((slots >= 0)[:, None], drows, 0.0).to(s["rows"].dtype)
    return out


def _plain(s):
    case = s["case"]
    kind = case["kind"]
    if kind == "quantize":
        q, codes = _quantize_rows(s["x"])
        out = {"row": q, "row_codes": codes}
        if case["cols"]:
            offsets = torch.arange(0, 2 * case["rows"], case["rows"], dtype=torch.int32, device="cuda")
            out["col"], out["col_codes"] = _quantize_cols(s["x"], offsets, case["rows"])
            out["col_codes"] = out["col_codes"][:_ceil(case["rows"])]
        return out
    if kind == "route":
        offsets, slots, position = _sort(s["ids"], case["experts"])
        rows = _gather(s["x"], slots, case["top_k"])
        out = {"offsets": offsets, "slots": slots, "position": position}
        if case["fp8"]:
            out["rows"], out["codes"] = _quantize_rows(rows)
        else:
            out["rows"] = rows
        return out
    if kind == "combine":
        return _plain_combine(s)
    return _plain_product(s)


# ---- the package's calls ---------------------------------------------------------------

def _own(s):
    import microscaling_weight_quantization_amd as mxq
    case = s["case"]
    kind, fp8 = case["kind"], torch.float8_e4m3fn
    out = {}
    if "out" in case:    # activations and their gradients in bf16 take the matrix cores' own FP8 sums, others sums in fp32
        out = {"out_dtype": DTYPES[case["out"]], "fast_accum": case["out"] == "bf16"}
    if kind == "quantize":
        if case["cols"]:
            q, codes, col, col_codes = mxq.mxq_quantize_fp8_group128_row_col(s["x"])
            return {"row": q.view(fp8), "row_codes": codes, "col": col.view(fp8), "col_codes": col_codes}
        q, codes = mxq.mxq_quantize_fp8_group128(s["x"])
        return {"row": q.view(fp8), "row_codes": codes}
    if kind == "matmul":
        return mxq.mxq_matmul_fp8_block128(*s["a"], *s["w"], offsets=s["offsets"], **out)
    if kind == "dgrad":
        return mxq.mxq_matmul_fp8_block128_dgrad(*s["a"], *s["w"], offsets=s["offsets"], **out)
    if kind == "wgrad":
        return mxq.mxq_matmul_fp8_group128_wgrad(*s["dy"], *s["x"], offsets=s["offsets"],
                                                 out_dtype=DTYPES[case["out"]])
    if kind == "route":
        offsets, slots, position = mxq.mxq_sort_experts(s["ids"], case["experts"])
        out = {"offsets": offsets, "slots": slots, "position": position}
        if case["fp8"]:
            q, out["codes"] = mxq.mxq_quantize_fp8_group128(s["x"], slots=slots, top_k=case["top_k"])
            out["rows"] = q.view(fp8)
        else:
            out["rows"] = mxq.mxq_dispatch_rows(s["x"], slots, case["top_k"])
        return out
    out = {"y": mxq.mxq_combine_rows(s["rows"], s["position"], s["weights"])}
    if case["backward"]:
        out["drows"], out["dweights"] = mxq.mxq_combine_rows_backward(s["dy"], s["rows"], s["position"], s["weights"])
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ---- the least that a pass moves and computes ------------------------------------------

def work(case):
    kind = case["kind"]
    if kind == "quantize":
        rows, k = case["rows"], case["k"]
        size = 2 if case["dtype"] == "bf16" else 4
        outs = rows * k + rows * _ceil(k) + (rows * k + _ceil(rows) * k if case["cols"] else 0)
        return {"bytes": rows * k * size + outs, "flops": 2 * rows * k * (2 if case["cols"] else 1)}
    if kind in ("matmul", "dgrad", "wgrad"):
        n, k, experts = case["n"], case["k"], case.get("experts", 0)
        m = case["tokens"] * case["top_k"] if experts else case["m"]
        taken = experts * (1 - (1 - 1 / experts) ** m) if experts else 1    # the experts that get a row, for an even router
        size = 2 if case["out"] == "bf16" else 4
        if kind == "wgrad":
            moved = m * (n + k) * (1 + 1 / GROUP) + max(1, experts) * n * k * size
        else:
            inner, outer = (n, k) if kind == "dgrad" else (k, n)
            moved = m * inner * (1 + 1 / GROUP) + taken * n * k + m * outer * size
        return {"bytes": moved, "flops": 2 * m * n * k}
    rows, k = case["tokens"] * case["top_k"], case["k"]
    size = 2 if case["dtype"] == "bf16" else 4
    if kind == "route":
        out = k + _ceil(k) if case["fp8"] else k * size
        return {"bytes": case["tokens"] * k * size + rows * (out + 12) + 4 * case["experts"], "flops": 2 * rows * k if case["fp8"] else 0}
    moved = rows * (k * size + 8) + case["tokens"] * k * size
    flops = 2 * rows * k
    if case["backward"]:    # the rows are read for the layer's output and again for the weights' gradient
        moved += rows * (2 * k * size + 12) + case["tokens"] * k * size
        flops += 3 * rows * k
    return {"bytes": moved, "flops": flops}


# ---- the definitions in 64 bits --------------------------------------------------------

def _e4m3_64(v):
    """v rounded to nearest, ties to even, on the E4M3 grid: steps of 2^(e - 3) for |v| in [2^e, 2^(e + 1)), e >= -6."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.round(v / step) * step


def _exact_groups(v):
    """(payload values, codes) of groups along the last axis."""
    amax = v.abs().amax(-1, keepdim=True)
    s = torch.floor(torch.log2(torch.where(amax == 0, 1.0, amax))) - 8
    s = s + (amax > 448 * torch.exp2(s)).double()
    s = torch.where(amax == 0, -127.0, s.clamp(min=-127))
    return _e4m3_64(v * torch.exp2(-s)), (s + 127).squeeze(-1).to(torch.uint8)


def _exact_quantize(x):
    x, (rows, k) = x.double(), x.shape
    full = x.new_zeros(rows, _ceil(k) * GROUP)
    full[:, :k] = x
    q, codes = _exact_groups(full.view(rows, -1, GROUP))
    return q.view(rows, -1)[:, :k], codes


def _value64(code):
    return torch.ldexp(torch.ones((), dtype=torch.float64, device=code.device), code.to(torch.int32) - 127)


def _segment64(q, codes, lo, hi, group):
    """Rows lo to hi of a column-wise operand, whose first group is `group`."""
    at = group + torch.arange(hi - lo, device=q.device) // GROUP
    return q[lo:hi].double() * _value64(codes)[at]


def exact(case, seed):
    kind = case["kind"]
    s = prepare(case, seed)
    if kind == "quantize":
        q, codes = _exact_quantize(s["x"])
        out = {"row": q, "row_codes": codes}
        if case["cols"]:
            q, codes = _exact_quantize(s["x"].t())
            out["col"], out["col_codes"] = q.t(), codes.t().contiguous()
        return out
    if kind in ("matmul", "dgrad", "wgrad"):
        experts = case.get("experts", 0)
        m = case["tokens"] * case["top_k"] if experts else case["m"]
        ends = s["offsets"].tolist() if experts else [0, m]
        parts, group = [], 0
        for e, (lo, hi) in enumerate(zip(ends, ends[1:])):
            if kind == "wgrad":
                parts.append(_segment64(*s["dy"], lo, hi, group).t() @ _segment64(*s["x"], lo, hi, group))
                group += _ceil(hi - lo)
                continue
            q, codes = s["a"][0][lo:hi], s["a"][1][lo:hi]
            at = torch.arange(q.shape[1], device=q.device) // GROUP
            a = q.double() * _value64(codes)[:, at]
            w, tiles = (s["w"][0][e], s["w"][1][e]) if experts else s["w"]
            rows = torch.arange(case["n"], device=q.device) // GROUP
            cols = torch.arange(case["k"], device=q.device) // GROUP
            w = w.double() * _value64(tiles)[rows][:, cols]
            parts.append(a @ w if kind == "dgrad" else a @ w.t())
        if kind == "wgrad":
            return torch.stack(parts) if experts else parts[0]
        parts.append(torch.zeros((m - ends[-1], parts[0].shape[1]), dtype=torch.float64, device="cuda"))
        return torch.cat(parts)
    tokens, top_k = case["tokens"], case["top_k"]
    if kind == "route":
        ids = s["ids"].reshape(-1).tolist()
        slots = sorted(range(len(ids)), key=lambda i: ids[i] if ids[i] >= 0 else case["experts"])
        kept = sum(i >= 0 for i in ids)
        rows = torch.zeros((len(ids), case["k"]), dtype=torch.float64, device="cuda")
        rows[:kept] = s["x"].double()[torch.tensor(slots[:kept], dtype=torch.long, device="cuda") // top_k]
        if case["fp8"]:
            rows, codes = _exact_quantize(rows)
            return {"offsets": None, "slots": None, "position": None, "rows": rows, "codes": codes}
        return {"offsets": None, "slots": None, "position": None, "rows": rows}
    position, w = s["position"].long(), s["weights"].double()
    rows, dy = s["rows"].double(), s["dy"].double()
    y = torch.zeros((tokens, case["k"]), dtype=torch.float64, device="cuda")
    dw, drows = torch.zeros_like(w), torch.zeros_like(rows)
    for j in range(top_k):
        at = torch.nonzero(position[:, j] >= 0).squeeze(1)
        p = position[at, j]
        y[at] += w[at, j, None] * rows[p]
        dw[at, j] = (dy[at] * rows[p]).sum(1)
        drows[p] = w[at, j, None] * dy[at]
    return {"y": y, "dweights": dw, "drows": drows} if case["backward"] else {"y": y}
