"""Plain 64-bit forms of the FP8 group quantizer, the FP8 products and the expert
routing, on the CPU, for the tests.

A group's scale is 2^S, S = max(ceil(log2(amax / 448)), -127).  Products are
summed in 64 bits; `bounds` says how far a kernel may be from that: half a step
of the output's type, and for each of the R additions in fp32 one step of the sum
of magnitudes (2^-23: an addition may truncate).
"""
from __future__ import annotations

import numpy as np
import torch

GROUP = 128


def ceil_div(n, d=GROUP):
    return -(-n // d)


def scale_of(codes) -> torch.Tensor:
    """2^(code - 127) in 64 bits, NaN for 255."""
    c = codes.cpu().to(torch.float64)
    return torch.where(c == 255, torch.nan, torch.exp2(c - 127))


def payload_values(q) -> torch.Tensor:
    return q.cpu().view(torch.float8_e4m3fn).to(torch.float64)


def quantize_group(v: torch.Tensor):
    """(payload bytes, code) of one group of 64-bit values."""
    if not torch.isfinite(v).all():
        return torch.full(v.shape, 0x7F, dtype=torch.uint8), 255
    amax = float(v.abs().max()) if v.numel() else 0.0
    if amax == 0:
        code = 0
    else:
        m, e = np.frexp(amax)            # amax = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
        code = max(int(e) - 9 + (1 if m > 0.875 else 0), -127) + 127
    q = (v * 2.0 ** (127 - code)).to(torch.float32).to(torch.float8_e4m3fn)
    return q.view(torch.uint8), code


def quantize_rows(x: torch.Tensor):
    x = x.detach().cpu().to(torch.float64)
    rows, K = x.shape
    q = torch.zeros((rows, K), dtype=torch.uint8)
    codes = torch.zeros((rows, ceil_div(K)), dtype=torch.uint8)
    for r in range(rows):
        for b in range(ceil_div(K)):
            cols = slice(b * GROUP, min((b + 1) * GROUP, K))
            q[r, cols], codes[r, b] = quantize_group(x[r, cols])
    return q, codes


def segments(offsets, rows):
    """[(lo, hi)] of each expert, offsets clamped to [0, rows] and to a rising order."""
    if offsets is None:
        return [(0, rows)]
    out, top = [], 0
    v = [min(max(int(o), 0), rows) for o in offsets]
    for a, b in zip(v, v[1:]):
        lo = max(a, top)
        top = max(top, a, b)
        out.append((lo, max(lo, top)))
    return out


def quantize_cols(x: torch.Tensor, offsets=None):
    x = x.detach().cpu().to(torch.float64)
    rows, K = x.shape
    segs = segments(offsets, rows)
    groups = ceil_div(rows) if offsets is None else rows // GROUP + len(segs)
    q = torch.zeros((rows, K), dtype=torch.uint8)
    codes = torch.zeros((groups, K), dtype=torch.uint8)
    g = 0
    for lo, hi in segs:
        for r in range(lo, hi, GROUP):
            part = slice(r, min(r + GROUP, hi))
            for c in range(K):
                q[part, c], codes[g, c] = quantize_group(x[part, c])
            g += 1
    return q, codes


def gather(x: torch.Tensor, slots, top_k: int):
    x = x.detach().cpu()
    out = torch.zeros((len(slots), x.shape[1]), dtype=x.dtype)
    for r, s in enumerate(slots):
        if 0 <= s and s // top_k < x.shape[0]:
            out[r] = x[s // top_k]
    return out


def rows_values(q, codes):
    s = scale_of(codes).repeat_interleave(GROUP, 1)[:, :q.shape[1]]
    return payload_values(q) * s


def tiles_values(q, codes):
    s = scale_of(codes).repeat_interleave(GROUP, 0).repeat_interleave(GROUP, 1)
    return payload_values(q) * s[:q.shape[0], :q.shape[1]]


def cols_values(q, codes, lo, hi, first):
    """Rows [lo, hi) of a payload with column groups whose first group is `first`."""
    s = scale_of(codes)[first:first + max(1, ceil_div(hi - lo))].repeat_interleave(GROUP, 0)[:hi - lo]
    return payload_values(q)[lo:hi] * s


def product(v, u):
    """(v u^T, the sums of magnitudes) in 64 bits."""
    return v @ u.t(), v.abs() @ u.abs().t()


def matmul(q, codes, w, tiles, offsets=None, transpose=False):
    """y = x w^T, or with `transpose` dx = dy w -> (values, sums of magnitudes)."""
    v = rows_values(q, codes)
    ws = [w] if offsets is None else list(w)
    ts = [tiles] if offsets is None else list(tiles)
    cols = ws[0].shape[1] if transpose else ws[0].shape[0]
    y = torch.zeros((q.shape[0], cols), dtype=torch.float64)
    mag = torch.zeros_like(y)
    for (lo, hi), wi, ti in zip(segments(offsets, q.shape[0]), ws, ts):
        u = tiles_values(wi, ti)
        y[lo:hi], mag[lo:hi] = product(v[lo:hi], u.t() if transpose else u)
    return y, mag


def wgrad(dq, dcodes, xq, xcodes, offsets=None):
    out, first = [], 0
    for lo, hi in segments(offsets, dq.shape[0]):
        d, x = cols_values(dq, dcodes, lo, hi, first), cols_values(xq, xcodes, lo, hi, first)
        out.append(product(d.t(), x.t()))
        first += ceil_div(hi - lo)
    if offsets is None:
        return out[0]
    return torch.stack([y for y, _ in out]), torch.stack([m for _, m in out])


def bounds(want, mag, R, dtype):
    return torch.finfo(dtype).eps / 2 * want.abs() + 2.0 ** -23 * (R + 1) * mag + 2.0 ** -149


def check(got, want, mag, R, what=""):
    """got (on any device, bf16 / fp32) within its bounds of want; NaN exactly where want is NaN."""
    g = got.detach().cpu().to(torch.float64)
    assert g.shape == want.shape, f"{what}: {list(g.shape)} for {list(want.shape)}"
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(g), nan), f"{what}: NaN in other places"
    off = torch.where(nan, 0.0, (g - want).abs())
    allowed = torch.where(nan, 0.0, bounds(want, mag, R, got.dtype))
    worst = int((off - allowed).argmax()) if off.numel() else 0
    assert bool((off <= allowed).all()), (f"{what}: off by {off.reshape(-1)[worst]:.3g} where {allowed.reshape(-1)[worst]:.3g} "
                                          f"is allowed, at {np.unravel_index(worst, tuple(want.shape))}")


def sort_experts(ids, n_experts):
    flat = [int(i) for i in ids.reshape(-1)]
    key = [i if 0 <= i < n_experts else n_experts for i in flat]
    order = sorted(range(len(flat)), key=lambda s: key[s])
    offsets = [sum(k < e for k in key) for e in range(n_experts + 1)]
    slots, position = [], [0] * len(flat)
    for place, s in enumerate(order):
        dropped = key[s] == n_experts
        slots.append(~s if dropped else s)
        position[s] = ~place if dropped else place
    return offsets, slots, position
