"""The 4-bit experts and SwiGLU experts with global scales on both sides, every
output against the fp64 definition.

Experts: both sides' values are those of the definition (global scales are
powers of two), what differs is the fp32 sum: below 2^-16 of sum |w| |x|, and the
one rounding to the output's type.

SwiGLU experts: h is quantised from fp32 sums of the first product, so a value of
h on an edge may fall to either side.  With delta the sum's bound for gate and up,
h is within 1.1 |up| delta_gate + |silu(gate)| delta_up + 2^-20 |h| of its fp64
value (silu's slope is below 1.1).  Where the two ends of that range have other
codes an output may differ by the weight times their distance; where they have
another block scale, by the weight times two of the larger scale's largest half
steps (a code is at most 1 from its quotient) for each value of the block."""
import numpy as np
import pytest
import torch

import oracle.moe_operators as M
import trellis_quantized_moe_sort_gb300 as tq
from gpu_util import check_no_device_error

pytestmark = pytest.mark.gpu
FMT = {"nv": tq.FP4_NV, "mx": tq.FP4_MX}
ROUND = {torch.float32: 2.0 ** -23, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -10}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from trellis_quantized_moe_sort_gb300 import build
    build.build()
    tq.tq_init(0)


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _scale(g):
    return None if g is None else torch.tensor([g], dtype=torch.float32, device="cuda")


class Experts:
    """E seeded matrices N(0, 1/K) with global scales of their own, quantised by the definition."""

    def __init__(self, rng, E, N, K, fmt):
        w = rng.standard_normal((E, N, K)) / np.sqrt(K)
        g = 2.0 ** -(8.0 + np.arange(E) % 3) if fmt == "nv" else np.ones(E)
        parts = [M.quantize(w[e], fmt, g[e]) for e in range(E)]
        self.packed = torch.from_numpy(np.stack([M.pack(p[0]) for p in parts])).cuda()
        self.tiled = tq.tq_fp4_tile_scales(torch.from_numpy(np.stack([p[1] for p in parts])).cuda(), FMT[fmt])
        self.scale = torch.from_numpy(g.astype(np.float32)).cuda() if fmt == "nv" else None
        self.values = np.stack([p[2] for p in parts])


def _routing(rng, n, E, k):
    ids = np.stack([rng.permutation(E)[:k] for _ in range(n)]).astype(np.int32)
    return ids, rng.standard_normal((n, k)).astype(np.float32)


def _activations(rng, n, K, dtype):
    x = rng.standard_normal((n, K)) * np.exp(0.5 * rng.standard_normal(K))
    return torch.from_numpy(x.astype(np.float32)).to(dtype)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("dtype", sorted(ROUND, key=str))
@pytest.mark.parametrize("n,E,k,K,N", [(1, 8, 2, 512, 130), (3, 64, 6, 288, 64), (70, 8, 2, 1056, 129), (500, 4, 3, 256, 257)])
def test_experts_with_global_scales(fmt, dtype, n, E, k, K, N):
    rng = np.random.default_rng([n, E, K])
    w = Experts(rng, E, N, K, fmt)
    x, (ids, tw) = _activations(rng, n, K, dtype), _routing(rng, n, E, k)
    g = 2.0 ** -8 if fmt == "nv" else None
    y = tq.tq_fp4_moe_forward(x.cuda(), w.packed, w.tiled, torch.from_numpy(ids).cuda(), torch.from_numpy(tw).cuda(),
                              fmt=FMT[fmt], w_scale=w.scale, x_scale=_scale(g))
    check_no_device_error()
    want, size = M.moe(M.quantize(_f64(x), fmt, 1.0 if g is None else g)[2], ids, tw, w.values)
    assert y.dtype == dtype
    assert (np.abs(_f64(y) - want) <= 2.0 ** -16 * size + ROUND[dtype] * np.abs(want) + 6e-8).all()


def _quantised_range(h, off, fmt, g):
    """(values of h, how far those of anything within `off` of it may be from them)."""
    _, byte, values = M.quantize(h, fmt, g)
    sign = np.where(np.signbit(h), -1.0, 1.0)
    (_, low_byte, low), (_, high_byte, high) = (M.quantize(sign * np.maximum(np.abs(h) + d, 0.0), fmt, g)
                                                for d in (-off, off))
    apart = np.maximum(np.abs(low - values), np.abs(high - values))
    largest = M.dequantize(M.pack(np.full(h.shape, 2, np.uint8)), high_byte, fmt, g)       # code 2 is 1: the scale
    unclear = np.repeat((low_byte != byte) | (high_byte != byte), M.BLOCK[fmt], -1)
    return values, np.where(unclear, np.maximum(apart, 2.0 * largest), apart)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,E,k,H,I", [(1, 8, 2, 256, 1056), (5, 16, 6, 512, 288), (40, 2, 1, 256, 2048), (60, 8, 2, 544, 512),
                                       (400, 4, 2, 288, 544)])
def test_swiglu_experts_output_by_output(fmt, dtype, n, E, k, H, I):
    rng = np.random.default_rng([n, H, I])
    gu, down = Experts(rng, E, 2 * I, H, fmt), Experts(rng, E, H, I, fmt)
    x, (ids, tw) = _activations(rng, n, H, dtype), _routing(rng, n, E, k)
    xs, hs = (2.0 ** -8, 2.0 ** -7) if fmt == "nv" else (None, None)
    y = tq.tq_fp4_moe_mlp_forward(x.cuda(), gu.packed, gu.tiled, down.packed, down.tiled, torch.from_numpy(ids).cuda(),
                                  torch.from_numpy(tw).cuda(), fmt=FMT[fmt], gu_scale=gu.scale, down_scale=down.scale,
                                  x_scale=_scale(xs), h_scale=_scale(hs))
    check_no_device_error()
    xq = M.quantize(_f64(x), fmt, 1.0 if xs is None else xs)[2]
    want, limit = np.zeros((n, H)), np.zeros((n, H))
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if not t.size:
            continue
        z, size = xq[t] @ gu.values[e].T, np.abs(xq[t]) @ np.abs(gu.values[e]).T
        gate, up, delta = z[:, :I], z[:, I:], 2.0 ** -16 * size
        silu = gate / (1.0 + np.exp(-gate))
        h = silu * up
        off = 1.1 * np.abs(up) * delta[:, :I] + np.abs(silu) * delta[:, I:] + 2.0 ** -20 * np.abs(h)
        hq, apart = _quantised_range(h, off, fmt, 1.0 if hs is None else hs)
        c, W = tw[t, j, None].astype(np.float64), np.abs(down.values[e]).T
        np.add.at(want, t, c * (hq @ down.values[e].T))
        np.add.at(limit, t, np.abs(c) * (2.0 ** -16 * (np.abs(hq) @ W) + apart @ W))
    assert y.dtype == dtype
    assert (np.abs(_f64(y) - want) <= limit + ROUND[dtype] * np.abs(want) + 6e-8).all()
