"""A feed-forward layer of experts in FP8, forward and backward, on the package's calls.

    python examples/expert_layer.py [--tokens 2048 --experts 48 --top-k 6 --hidden 2048 --inner 1024]

Each expert is two matrices, up [inner, hidden] and down [hidden, inner], with
squared ReLU between them.  A training step converts the bf16 master weights to
128x128 blockwise FP8 (mxq_mxfp4_to_fp8_block128, so that the layer trains on
what an MXFP4 deployment will see), routes the tokens, runs the products by
expert and brings the rows back; the backward pass runs the same way in reverse
with straight-through gradients for the weights.  A decoding step routes a few
tokens through the same weights.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import microscaling_weight_quantization_amd as mxq  # noqa: E402


class ExpertLayer:
    def __init__(self, experts: int, hidden: int, inner: int, device="cuda", seed: int = 0):
        g = torch.Generator(device=device).manual_seed(seed)
        make = lambda n, k: (torch.randn(experts, n, k, generator=g, device=device) * k ** -0.5).to(torch.bfloat16)
        self.experts, self.up, self.down = experts, make(inner, hidden), make(hidden, inner)
        self.router = torch.randn(hidden, experts, generator=g, device=device) * hidden ** -0.5
        # FP8 payloads and tile codes of all experts, each expert's a slice, converted in one grouped call
        tiles = lambda n: (n + 127) // 128
        byte = lambda *s: torch.empty(s, dtype=torch.uint8, device=device)
        self.up8, self.up_codes = byte(experts, inner, hidden), byte(experts, tiles(inner), tiles(hidden))
        self.down8, self.down_codes = byte(experts, hidden, inner), byte(experts, tiles(hidden), tiles(inner))
        self._fold = [mxq.GroupedBlock128(list(w), list(q), list(c)) for w, q, c in (
            (self.up, self.up8, self.up_codes), (self.down, self.down8, self.down_codes))]
        self.refresh()

    def refresh(self):
        """Converts the master weights, after each step of an optimizer."""
        for fold in self._fold:
            fold()

    def route(self, x, top_k: int):
        """(experts int32 [tokens, top_k], their weights) of each token."""
        top = (x.float() @ self.router).topk(top_k, dim=1)
        return top.indices.int(), torch.softmax(top.values, dim=1)

    def forward(self, x, ids, weights, keep: bool = False):
        """y [tokens, hidden]; with `keep` also what backward needs."""
        top_k = ids.shape[1]
        offsets, slots, position = mxq.mxq_sort_experts(ids, self.experts)
        xq = mxq.mxq_quantize_fp8_group128_row_col(x, slots, top_k, offsets) if keep else \
            mxq.mxq_quantize_fp8_group128(x, slots, top_k)
        h = mxq.mxq_matmul_fp8_block128(xq[0], xq[1], self.up8, self.up_codes, offsets, fast_accum=True)
        a = torch.relu(h).square_()
        aq = mxq.mxq_quantize_fp8_group128_row_col(a, offsets=offsets) if keep else mxq.mxq_quantize_fp8_group128(a)
        rows = mxq.mxq_matmul_fp8_block128(aq[0], aq[1], self.down8, self.down_codes, offsets, fast_accum=True)
        y = mxq.mxq_combine_rows(rows, position, weights)
        return (y, (offsets, slots, position, xq, h, aq, rows, weights)) if keep else y

    def backward(self, dy, kept):
        """Gradients (dx, dweights, dup, ddown) for dy [tokens, hidden]."""
        offsets, slots, position, xq, h, aq, rows, weights = kept
        drows, dweights = mxq.mxq_combine_rows_backward(dy, rows, position, weights)
        gq = mxq.mxq_quantize_fp8_group128_row_col(drows, offsets=offsets)
        da = mxq.mxq_matmul_fp8_block128_dgrad(gq[0], gq[1], self.down8, self.down_codes, offsets, fast_accum=True)
        ddown = mxq.mxq_matmul_fp8_group128_wgrad(gq[2], gq[3], aq[2], aq[3], offsets)
        dh = da * (2 * torch.relu(h))
        hq = mxq.mxq_quantize_fp8_group128_row_col(dh, offsets=offsets)
        dxs = mxq.mxq_matmul_fp8_block128_dgrad(hq[0], hq[1], self.up8, self.up_codes, offsets, fast_accum=True)
        dup = mxq.mxq_matmul_fp8_group128_wgrad(hq[2], hq[3], xq[2], xq[3], offsets)
        return mxq.mxq_combine_rows(dxs, position), dweights, dup, ddown


def reference(layer: ExpertLayer, x, ids, weights):
    """The same layer in fp32 torch operations, on the weights that the layer's FP8 stands for."""
    tile = lambda q, c: torch.stack([mxq.mxq_dequantize(a, b, layout=mxq.MXQ_SCALE_TILE_128X128, out_dtype=torch.float32)
                                     for a, b in zip(q, c)])
    up, down = tile(layer.up8, layer.up_codes).requires_grad_(), tile(layer.down8, layer.down_codes).requires_grad_()
    x, weights = x.float().requires_grad_(), weights.clone().requires_grad_()
    y = torch.zeros_like(x)
    for e in range(layer.experts):
        token, choice = torch.nonzero(ids == e, as_tuple=True)
        out = torch.relu(x[token] @ up[e].t()).square() @ down[e].t()
        y = y.index_add(0, token, out * weights[token, choice][:, None])
    return y, (x, weights, up, down)


def relative(a, b):
    return float((a.float() - b.detach()).norm() / b.detach().norm())


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("tokens", 2048), ("experts", 48), ("top-k", 6), ("hidden", 2048), ("inner", 1024)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args(argv)
    layer = ExpertLayer(a.experts, a.hidden, a.inner)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(a.tokens, a.hidden, generator=g, device="cuda").to(torch.bfloat16)
    dy = torch.randn(a.tokens, a.hidden, generator=g, device="cuda").to(torch.bfloat16)
    ids, weights = layer.route(x, a.top_k)
    y, kept = layer.forward(x, ids, weights, keep=True)
    grads = layer.backward(dy, kept)
    want, leaves = reference(layer, x, ids, weights)
    want.backward(dy.float())
    off = {"y": relative(y, want)}
    off.update({n: relative(got, leaf.grad) for n, got, leaf in zip(("dx", "dweights", "dup", "ddown"), grads, leaves)})
    for n, v in off.items():
        print(f"{n:9s} {v:.4f} from fp32")
    token = layer.forward(x[:1], ids[:1], weights[:1])
    off["token"] = relative(token, want[:1].detach())
    print(f"one token {off['token']:.4f} from fp32", flush=True)
    return off


if __name__ == "__main__":
    main()
