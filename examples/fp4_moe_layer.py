"""A served mixture-of-experts layer on 4-bit weights: the scored router, the
routed SwiGLU experts and a shared expert's projection.

    python examples/fp4_moe_layer.py [--tokens 32] [--experts 64] [--top-k 6]
                                     [--hidden 1024] [--inner 512] [--format nv|mx]

Weights are random and quantised once, as a checkpoint would be when it loads;
the layer then runs on them and is compared with the same layer computed from
the dequantised weights in fp32 by torch.
"""
import argparse
import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import trellis_quantized_moe_sort_gb300 as tq


class Fp4Weights:
    """Matrices [E, N, K] as 4-bit codes, tiled block scales and one 32-bit scale each (NV)."""

    def __init__(self, w, fmt):
        E, N, K = w.shape
        self.fmt = fmt
        # the largest weight becomes 6 (E2M1's largest) times 448 (E4M3's)
        self.scale = (w.abs().amax((1, 2)) / (6.0 * 448.0)).float() if fmt == tq.FP4_NV else None
        self.packed = torch.empty((E, N, K // 2), dtype=torch.uint8, device=w.device)
        self.scales = torch.empty((E, N, K // (16 if fmt == tq.FP4_NV else 32)), dtype=torch.uint8, device=w.device)
        for e in range(E):
            tq.tq_fp4_quantize(w[e], fmt, self.global_scale(e), packed=self.packed[e], scales=self.scales[e])
        self.tiled = tq.tq_fp4_tile_scales(self.scales, fmt)

    def global_scale(self, e):
        return None if self.scale is None else self.scale[e:e + 1]

    def values(self, e):
        return tq.tq_fp4_dequantize(self.packed[e], self.scales[e], self.fmt, self.global_scale(e))


class Layer:
    """y = sum of the token's routed experts + the shared expert's projection."""

    def __init__(self, hidden, inner, experts, top_k, groups, top_groups, fmt, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *shape: torch.randn(shape, device="cuda", generator=g)
        self.top_k, self.groups, self.top_groups = top_k, groups, top_groups
        self.router = normal(hidden, experts) / math.sqrt(hidden)
        self.bias = 0.02 * normal(experts)
        self.gate_up = Fp4Weights(normal(experts, 2 * inner, hidden) / math.sqrt(hidden), fmt)
        self.down = Fp4Weights(normal(experts, hidden, inner) / math.sqrt(inner), fmt)
        self.shared = Fp4Weights(normal(1, hidden, hidden) / math.sqrt(hidden), fmt)
        self.fmt = fmt
        # activations' global scales, as calibration on sample data sets them
        scale = lambda largest: torch.full((1,), largest / (6.0 * 448.0), device="cuda") if fmt == tq.FP4_NV else None
        self.x_scale, self.h_scale = scale(6.0), scale(12.0)

    def route(self, x):
        return tq.tq_router_scored(x.float() @ self.router, self.top_k, score=tq.SCORE_SIGMOID, bias=self.bias,
                                   groups=self.groups, top_groups=self.top_groups, renormalize=True)

    def __call__(self, x):
        ids, w = self.route(x)
        y = tq.tq_fp4_moe_mlp_forward(x, self.gate_up.packed, self.gate_up.tiled, self.down.packed, self.down.tiled, ids, w,
                                      fmt=self.fmt, gu_scale=self.gate_up.scale, down_scale=self.down.scale,
                                      x_scale=self.x_scale, h_scale=self.h_scale)
        return y + tq.tq_fp4_linear(x, self.shared.packed[0], self.shared.tiled, fmt=self.fmt,
                                    w_scale=self.shared.scale, x_scale=self.x_scale)

    def reference(self, x):
        """The same from dequantised weights and activations, in fp32."""
        rounded = lambda t, s: tq.tq_fp4_dequantize(*tq.tq_fp4_quantize(t, self.fmt, s), self.fmt, s)
        ids, w = self.route(x)
        xq = rounded(x, self.x_scale)
        y = xq @ self.shared.values(0).t()
        for e in ids.unique().tolist():
            t, j = torch.nonzero(ids == e, as_tuple=True)
            gate, up = (xq[t] @ self.gate_up.values(e).t()).chunk(2, 1)
            h = rounded((torch.nn.functional.silu(gate) * up).contiguous(), self.h_scale)
            y.index_add_(0, t, (h @ self.down.values(e).t()) * w[t, j, None])
        return y


def run(tokens=32, experts=64, top_k=6, hidden=1024, inner=512, fmt=tq.FP4_NV, groups=8, top_groups=4, seed=0):
    """Builds the layer, runs it on random tokens and returns the 2-norm of its
    difference from the reference over the reference's."""
    tq.tq_init(0)
    layer = Layer(hidden, inner, experts, top_k, groups, top_groups, fmt, seed)
    x = torch.randn((tokens, hidden), device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed + 1)).bfloat16()
    y, want = layer(x).float(), layer.reference(x)
    code, where = tq.tq_device_error()
    if code:
        raise RuntimeError(f"device error {code} at {where}")
    return float((y - want).norm() / want.norm())


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=32)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--top-k", type=int, default=6)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--inner", type=int, default=512)
    ap.add_argument("--format", choices=("nv", "mx"), default="nv")
    a = ap.parse_args()
    off = run(a.tokens, a.experts, a.top_k, a.hidden, a.inner, tq.FP4_NV if a.format == "nv" else tq.FP4_MX)
    print(f"{a.tokens} tokens, top-{a.top_k} of {a.experts} experts, {a.hidden} -> {a.inner} -> {a.hidden}, {a.format}: "
          f"off by {off:.2e} of the reference's 2-norm")


if __name__ == "__main__":
    main()
