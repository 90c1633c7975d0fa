"""Plain 64-bit forms of what stands between the FP8 products -- the norm, the
activation, the routing -- on the CPU, for the tests, and how far a kernel may be from them.

A rounding to a type is off by at most half a step, eps / 2 of the value: HALF for
fp32, 2^-8 for bf16, 2^-4 of the value or 2^-10 of the scale for E4M3.  Kernels work in
fp32; `rel` below counts the steps 2 HALF of what is computed.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from tests import fp8_ref as ref

HALF = 2.0 ** -24
INF = float("inf")


def host(t):
    return t.detach().cpu()


def f64(t):
    return host(t).to(torch.float64)


# ---- FP8 outputs -------------------------------------------------------------------------

def code_of(amax):
    """E8M0 codes of groups with these largest magnitudes (64 bits)."""
    m, e = np.frexp(amax.numpy())
    s = np.where(m > 0.875, e - 8, e - 9)
    return torch.from_numpy(np.where(amax.numpy() == 0, 0, np.maximum(s, -127) + 127).astype(np.int64))


def _group_amax(v, which, n):
    out = torch.zeros((n, v.shape[1]), dtype=torch.float64)
    return out.scatter_reduce_(0, which[:, None].expand_as(v), v.abs(), "amax")


def _check(q, codes, want, off, which, n, what):
    """Payload rows whose codes stand in codes[which[row], column]; `off` is how far the value before the rounding may be."""
    finite = torch.isfinite(want)
    low = _group_amax((want.abs() - off).clamp(min=0), which, n)
    high = _group_amax(want.abs() + off, which, n)
    c = host(codes).long()
    bad = _group_amax((~finite).double(), which, n) > 0
    assert torch.equal(c == 255, bad), f"{what}: poisoned groups differ"
    fine = (c >= code_of(torch.where(bad, 0.0, low))) & (c <= code_of(torch.where(bad, 0.0, high)))
    assert bool((fine | bad).all()), f"{what}: codes {c[~(fine | bad)][:5].tolist()}"
    scale = torch.exp2(c.double() - 127)[which]
    payload = ref.payload_values(q)
    poisoned = bad[which]
    assert bool((host(q).view(torch.uint8)[poisoned] == 0x7F).all()), f"{what}: payload of a poisoned group"
    got = torch.where(poisoned, 0.0, payload * scale)
    want = torch.where(poisoned, 0.0, want)
    half = torch.maximum(2.0 ** -4 * (want.abs() + off), 2.0 ** -10 * scale)
    wrong = (got - want).abs() > torch.where(poisoned, 0.0, half + off)
    assert not bool(wrong.any()), (f"{what}: off by {float((got - want).abs()[wrong][0]):.3g} at "
                                   f"{torch.nonzero(wrong)[0].tolist()}, wanted {float(want[wrong][0]):.6g}")


def check_rows(q, codes, want, off, what="rows"):
    """Row groups of `want` (64 bits): every code that of a largest magnitude within `off`, every payload the rounding."""
    rows, K = want.shape
    n = ref.ceil_div(K)
    assert q.shape == (rows, K) and codes.shape == (rows, n), (what, q.shape, codes.shape)
    if want.numel() == 0:
        return
    _check(host(q).t().contiguous(), host(codes).t().contiguous(), want.t().contiguous(), off.t().contiguous(),
           torch.arange(K) // ref.GROUP, n, what)


def check_cols(q, codes, want, off, offsets=None, what="columns"):
    """Column groups, begun anew with each expert; rows of no expert have payload 0, unneeded codes are 0."""
    rows, K = want.shape
    segs = ref.segments(None if offsets is None else offsets.tolist(), rows)
    n = ref.ceil_div(rows) if offsets is None else rows // ref.GROUP + len(segs)
    assert q.shape == (rows, K) and codes.shape == (n, K), (what, q.shape, codes.shape)
    which = torch.full((rows,), -1, dtype=torch.long)
    first = 0
    for lo, hi in segs:
        which[lo:hi] = first + torch.arange(hi - lo) // ref.GROUP
        first += ref.ceil_div(hi - lo)
    assert bool((host(codes)[first:] == 0).all()), f"{what}: code rows that no group needs"
    owned = which >= 0
    assert bool((host(q).view(torch.uint8)[~owned] == 0).all()), f"{what}: rows of no expert"
    if bool(owned.any()) and K:
        _check(host(q)[owned], codes, want[owned], off[owned], which[owned], n, what)


def check_values(got, want, off, what):
    """A floating output: `off` plus the rounding to its type: eps / 2 of the value, and of the smallest normal value
    below that (values below 2^-126 lie 2^-126 eps apart: 2^-133 in bf16, 2^-149 in fp32)."""
    g = f64(got)
    assert g.shape == want.shape, f"{what}: {list(g.shape)} for {list(want.shape)}"
    odd = ~torch.isfinite(want)
    assert torch.equal(torch.isnan(g), torch.isnan(want)), f"{what}: NaN in other places"
    assert torch.equal(g[odd & ~torch.isnan(want)], want[odd & ~torch.isnan(want)]), f"{what}: infinities"
    info = torch.finfo(got.dtype)
    allowed = off + info.eps / 2 * torch.clamp(want.abs() + off, min=info.smallest_normal) + 2.0 ** -149
    d = torch.where(odd, 0.0, (g - want).abs())
    wrong = d > torch.where(odd, 0.0, allowed)
    assert not bool(wrong.any()), (f"{what}: off by {float(d[wrong][0]):.3g}, allowed {float(allowed[wrong][0]):.3g}, at "
                                   f"{torch.nonzero(wrong)[0].tolist()}")


# ---- the norm ----------------------------------------------------------------------------

def norm_steps(K):
    """Additions on the way of one value into a row's sum: a lane's pieces of eight (at least 256 lanes share a row of
    more than 512), the eight, the lanes of a wave, the waves."""
    return ref.ceil_div(K, 2048) + 3 + 6 + 16


def stored_sum(x, residual):
    """s in 64 bits.  The sum of two fp32 values, rounded to fp32 and then to the residual's type."""
    if residual is None:
        return f64(x)
    return (host(x).float() + host(residual).float()).to(residual.dtype).double()


def norm(s, weight, eps):
    """(y, how far fp32 may be): the sum of squares is off by a half step for each addition, the root halves that,
    and the root, the quotient, eps and two products add up to eight half steps."""
    K = s.shape[1]
    w = torch.ones(K, dtype=torch.float64) if weight is None else f64(weight)
    y = s / torch.sqrt((s * s).sum(1, keepdim=True) / K + eps) * w
    y = torch.where(torch.isinf((s * s).sum(1, keepdim=True)) & torch.isinf(s), torch.nan, y)
    return y, torch.nan_to_num(y.abs()) * (norm_steps(K) / 2 + 8) * HALF


def norm_backward(dy, s, weight, eps, dres):
    """((dx, how far), (dweight, how far)).  A dot product of K terms is off by a half step of the sum of magnitudes for
    each addition, and its terms by as many as the root (above) and three products."""
    K, rows = s.shape[1], s.shape[0]
    w = torch.ones(K, dtype=torch.float64) if weight is None else f64(weight)
    dy = f64(dy)
    r = 1 / torch.sqrt((s * s).sum(1, keepdim=True) / K + eps)
    u, g = s * r, dy * w
    m = (g * u).mean(1, keepdim=True)
    dx = r * (g - u * m)
    size = r * (g.abs() + u.abs() * (g * u).abs().mean(1, keepdim=True))
    steps = 2 * norm_steps(K) + 24
    off = size * steps * HALF
    if dres is not None:
        dx = dx + f64(dres)
        off = off + (f64(dres).abs() + size) * HALF
    dw = (dy * u).sum(0)
    return (dx, off), (dw, (dy * u).abs().sum(0) * (rows + steps) * HALF)


# ---- the activation ------------------------------------------------------------------------

def _logistic(z):
    e = torch.exp(-z.abs())
    return torch.where(z < 0, e, 1.0) / (1 + e), torch.where(z < 0, 1.0, e) / (1 + e)


KGELU = 2 * math.sqrt(2 / math.pi)


def act(name, g):
    """(act(g), act'(g), the sum of magnitudes of act'(g)'s terms, steps of either).  exp(-z) in fp32 is off by a few half
    steps and by z times those of z: three roundings in z (six where z is a cubic), one in z log2(e)."""
    if name == "silu":
        p, q = _logistic(g)
        return g * p, p * (1 + g * q), p * (1 + g.abs() * q), 4 * g.abs() + 24
    if name == "gelu_tanh":
        z = KGELU * (g + 0.044715 * g ** 3)
        p, q = _logistic(z)
        t = g * p * q * KGELU * (1 + 3 * 0.044715 * g * g)
        return g * p, p + t, p + t.abs(), 10 * z.abs() + 32
    r = g.clamp(min=0)
    r = torch.where(torch.isnan(g), g, r)
    return r * r, 2 * r, 2 * r, torch.full_like(g, 4.0)


def activate(name, gate, up):
    g = f64(gate)
    a, _, _, steps = act(name, g)
    if up is not None:
        a = a * f64(up)
    # results below the smallest normal fp32 value lose places: 2^-148 times what multiplies them
    tiny = 2.0 ** -148 * (1 + g.abs()) * (1 if up is None else 1 + f64(up).abs())
    return a, torch.nan_to_num(a.abs() * (steps + 2) * HALF + tiny, nan=0.0, posinf=0.0)


def activate_backward(name, da, gate, up):
    g, da = f64(gate), f64(da)
    a, d, size, steps = act(name, g)
    u = torch.ones_like(g) if up is None else f64(up)
    dg, off = da * u * d, (da * u).abs() * size * (steps + 4) * HALF
    if up is not None:
        dg, off = torch.cat((dg, da * a), 1), torch.cat((off, (da * a).abs() * (steps + 4) * HALF), 1)
    tiny = 2.0 ** -148 * (1 + g.abs()) ** 3 * (1 + u.abs()) * (1 + da.abs())
    tiny = tiny if up is None else torch.cat((tiny, tiny), 1)
    return dg, torch.nan_to_num(off + tiny, nan=0.0, posinf=0.0)


# ---- the routing -----------------------------------------------------------------------------

def scores(logits, kind):
    out = []
    for l in f64(logits).tolist():
        if kind == "sigmoid":
            out.append([0.0 if v == -INF else 1 / (1 + math.exp(-v)) if v > 0 else math.exp(v) / (1 + math.exp(v)) for v in l])
            continue
        top = max(l)
        e = [0.0 if v == -INF else math.exp(v - top) for v in l]
        total = math.fsum(e)
        out.append([v / total if total else 0.0 for v in e])
    return out


def route(logits, top_k, bias=None, score="softmax", renormalize=True, scale=1.0, n_groups=1, top_groups=1, group_top=1,
          mask=None):
    """(ids, weights), token by token from the definition."""
    l64 = f64(logits).tolist()
    b = None if bias is None else f64(bias).tolist()
    all_ids, all_w = [], []
    for t, p in enumerate(scores(logits, score)):
        key = list(l64[t]) if b is None else [-INF if v == -INF else s + c for v, s, c in zip(l64[t], p, b)]
        if mask is not None and not bool(host(mask)[t]):
            key = [-INF] * len(key)
        value = p if b is None else key
        order = lambda es: sorted((e for e in es if key[e] > -INF), key=lambda e: (-key[e], e))
        taken = range(len(key))
        if n_groups > 1:
            size = len(key) // n_groups
            ranks = []
            for g in range(n_groups):
                best = order(range(g * size, (g + 1) * size))[:group_top]
                if best:
                    ranks.append((-(key[best[0]] if group_top == 1 else sum(value[e] for e in best)), g))
            taken = [g * size + i for _, g in sorted(ranks)[:top_groups] for i in range(size)]
        ids = order(taken)[:top_k]
        total = math.fsum(p[e] for e in ids)
        w = [scale * p[e] / (total if renormalize and total else 1.0) for e in ids]
        all_ids.append(ids + [-1] * (top_k - len(ids)))
        all_w.append(w + [0.0] * (top_k - len(ids)))
    return torch.tensor(all_ids, dtype=torch.int32).view(-1, top_k), torch.tensor(all_w, dtype=torch.float64).view(-1, top_k)


def route_backward(dweights, logits, ids, score="softmax", renormalize=True, scale=1.0):
    """(dlogits, sums of magnitudes) by the chain rule, token by token."""
    g64 = f64(dweights).tolist()
    out, size = [], []
    for t, p in enumerate(scores(logits, score)):
        chosen = [(e, g) for e, g in zip(host(ids)[t].tolist(), g64[t]) if 0 <= e < len(p)]
        total = math.fsum(p[e] for e, _ in chosen)
        h, mag = [0.0] * len(p), [0.0] * len(p)
        if renormalize:
            mean = math.fsum(g * p[e] for e, g in chosen) / total if total else 0.0
            spread = math.fsum(abs(g) * p[e] for e, g in chosen) / total if total else 0.0
            for e, g in chosen:
                if total:
                    h[e] += scale * (g - mean) / total
                    mag[e] += abs(scale) * (abs(g) + spread) / total
        else:
            for e, g in chosen:
                h[e] += scale * g
                mag[e] += abs(scale * g)
        if score == "sigmoid":
            row = [v * s * (1 - s) for v, s in zip(h, p)]
            size.append([m * s for m, s in zip(mag, p)])
        else:
            dot = 0.0 if renormalize else math.fsum(v * s for v, s in zip(h, p))
            spread = 0.0 if renormalize else math.fsum(m * s for m, s in zip(mag, p))
            row = [s * (v - dot) for v, s in zip(h, p)]
            size.append([s * (m + spread) for m, s in zip(mag, p)])
        out.append(row)
    shape = (len(out), logits.shape[1])
    return torch.tensor(out, dtype=torch.float64).view(shape), torch.tensor(size, dtype=torch.float64).view(shape)
