"""The scored router's gradient and the 4-bit operators at the ends of the fp32
range, and with scales that are zero or no number."""
import numpy as np
import pytest
import torch

import oracle.moe_operators as M
import trellis_quantized_moe_sort_gb300 as tq
from gpu_util import check_no_device_error

pytestmark = pytest.mark.gpu
FMT = {"nv": tq.FP4_NV, "mx": tq.FP4_MX}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from trellis_quantized_moe_sort_gb300 import build
    build.build()
    tq.tq_init(0)


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _scale(*g):
    return torch.tensor(g, dtype=torch.float32, device="cuda")


class Matrices:
    """E seeded matrices N(0, factor^2 / K), quantised by the definition."""

    def __init__(self, rng, E, N, K, fmt, factor=1.0):
        self.g = 2.0 ** -9 if fmt == "nv" else 1.0
        code, byte, values = M.quantize(factor * rng.standard_normal((E * N, K)) / np.sqrt(K), fmt, self.g)
        self.packed = torch.from_numpy(M.pack(code).reshape(E, N, K // 2)).cuda()
        self.byte = byte.reshape(E, N, -1)
        self.tiled = tq.tq_fp4_tile_scales(torch.from_numpy(self.byte).cuda(), FMT[fmt])
        self.scale = torch.full((E,), self.g, device="cuda") if fmt == "nv" else None
        self.values = values.reshape(E, N, K)


def _arms(call):
    """call()'s result and whether it took the one launch for few rows."""
    before = tq.tq_launch_counts_all()
    y = call()
    after = tq.tq_launch_counts_all()
    few, many = (after[c] - before[c] for c in ("fp4_gemv", "fp4_gemm"))
    assert few + many == 1
    return y, few == 1


# Both sides' values are those of the definition, so what differs is the fp32
# sum: at most K / 64 + 64 roundings of partial sums no larger than sum |w| |x|.
@pytest.mark.parametrize("n", [1, 300])
@pytest.mark.parametrize("dtype,special,factor", [
    (torch.bfloat16, float("inf"), 1.0), (torch.float16, float("-inf"), 1.0), (torch.float32, float("inf"), 1.0),
    (torch.float32, 2.0 ** 124, 1.0), (torch.bfloat16, -2.0 ** 126, 2.0 ** -100), (torch.float32, 2.0 ** 123, 2.0 ** -20),
    (torch.float32, 3e38, 1.0)])
@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_largest_activations(fmt, dtype, special, factor, n):
    """An infinity counts as the largest finite number, in every product; a block of such values
    against weights that cancel it out is 0."""
    rng = np.random.default_rng([n, 5])
    E, N, K = 3, 129, 512
    w = Matrices(rng, E, N, K, fmt, factor if fmt == "mx" else 1.0)
    x = torch.from_numpy(rng.standard_normal((n, K)).astype(np.float32)).to(dtype)
    x[:, 7] = special
    x[n // 2, 40] = -special
    g = 2.0 ** 110 if fmt == "nv" and dtype != torch.float16 else None
    xs = None if g is None else _scale(g)
    xq = M.quantize(_f64(x), fmt, 1.0 if g is None else g)[2]
    x = x.cuda()
    y, few = _arms(lambda: tq.tq_fp4_linear(x, w.packed[0], w.tiled[: w.tiled.numel() // E], fmt=FMT[fmt],
                                            w_scale=None if w.scale is None else w.scale[:1], x_scale=xs,
                                            y=torch.empty(n, N, device="cuda")))
    assert few == (n == 1)
    want, size = xq @ w.values[0].T, np.abs(xq) @ np.abs(w.values[0]).T
    assert (np.abs(_f64(y) - want) <= 2.0 ** -16 * size + 2.0 ** -23 * np.abs(want)).all()
    ids = np.stack([rng.permutation(E)[:2] for _ in range(n)]).astype(np.int32)
    tw = (0.5 * rng.random((n, 2))).astype(np.float32)
    y, few = _arms(lambda: tq.tq_fp4_moe_forward(x, w.packed, w.tiled, torch.from_numpy(ids).cuda(),
                                                 torch.from_numpy(tw).cuda(), fmt=FMT[fmt], w_scale=w.scale, x_scale=xs,
                                                 y=torch.empty(n, N, device="cuda")))
    assert few == (n == 1)
    check_no_device_error()
    want, size = M.moe(xq, ids, tw, w.values)
    assert (np.abs(_f64(y) - want) <= 2.0 ** -16 * size + 2.0 ** -23 * np.abs(want)).all()


@pytest.mark.parametrize("n", [1, 300])
@pytest.mark.parametrize("x_factor,w_factor", [(2.0 ** -110, 2.0 ** 115), (2.0 ** 122, 2.0 ** -120), (2.0 ** -60, 2.0 ** -40)])
def test_scales_far_apart(x_factor, w_factor, n):
    """Power-of-two scales whose product is an ordinary number, or near fp32's smallest ones."""
    rng = np.random.default_rng([n, 6])
    N, K = 130, 512
    w = Matrices(rng, 1, N, K, "mx", w_factor)
    x = torch.from_numpy((x_factor * rng.standard_normal((n, K))).astype(np.float32))
    xq = M.quantize(_f64(x), "mx")[2]
    y, few = _arms(lambda: tq.tq_fp4_linear(x.cuda(), w.packed[0], w.tiled, fmt=tq.FP4_MX))
    assert few == (n == 1)
    want, size = xq @ w.values[0].T, np.abs(xq) @ np.abs(w.values[0]).T
    assert (np.abs(_f64(y) - want) <= 2.0 ** -16 * size + 2.0 ** -23 * np.abs(want)).all()


@pytest.mark.parametrize("n", [1, 300])
def test_mx_scale_that_is_no_number(n):
    """E8M0's byte 255 is NaN: all values of its block, and the outputs of its weight row alone."""
    rng = np.random.default_rng(n)
    N, K = 130, 512
    w = Matrices(rng, 1, N, K, "mx")
    byte = w.byte.copy()
    byte[0, 77, 3] = 255
    scales = torch.from_numpy(byte).cuda()
    want = torch.zeros(N, K, dtype=torch.bool)
    want[77, 96:128] = True
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        got = tq.tq_fp4_dequantize(w.packed[0], scales[0], tq.FP4_MX, dtype=dtype)
        assert torch.equal(torch.isnan(got).cpu(), want) and torch.isfinite(got[~want.cuda()]).all()
    y, few = _arms(lambda: tq.tq_fp4_linear(torch.randn(n, K, device="cuda"), w.packed[0],
                                            tq.tq_fp4_tile_scales(scales, tq.FP4_MX), fmt=tq.FP4_MX))
    assert few == (n == 1)
    assert torch.isnan(y[:, 77]).all() and torch.isfinite(y[:, :77]).all() and torch.isfinite(y[:, 78:]).all()


@pytest.mark.parametrize("n", [1, 300])
def test_zeros_with_a_global_scale_of_zero(n):
    """amax / (6 * 448) of an all-zero tensor is 0: its values are 0, and so are its products."""
    N, K = 129, 512
    zero = _scale(0.0)
    packed, scales = tq.tq_fp4_quantize(torch.zeros(N, K, device="cuda"), tq.FP4_NV, zero)
    assert not packed.any() and not scales.any()
    assert not tq.tq_fp4_dequantize(packed, scales, tq.FP4_NV, zero).any()
    w = Matrices(np.random.default_rng(n), 1, N, K, "nv")
    for x, x_scale, codes, byte, w_scale in (
            (torch.randn(n, K, device="cuda"), _scale(2.0 ** -9), packed, scales, zero),
            (torch.zeros(n, K, device="cuda"), zero, w.packed[0], torch.from_numpy(w.byte[0]).cuda(), w.scale),
            (torch.randn(n, K, device="cuda"), zero, w.packed[0], torch.from_numpy(w.byte[0]).cuda(), w.scale)):
        tiled = tq.tq_fp4_tile_scales(byte)
        y, few = _arms(lambda: tq.tq_fp4_linear(x, codes, tiled, w_scale=w_scale, x_scale=x_scale))
        assert few == (n == 1) and bool((y == 0).all())
        ids, tw = torch.zeros(n, 1, dtype=torch.int32, device="cuda"), torch.ones(n, 1, device="cuda")
        y = tq.tq_fp4_moe_forward(x, codes[None], tiled, ids, tw, w_scale=w_scale, x_scale=x_scale)
        assert bool((y == 0).all())
    check_no_device_error()


# Scores of the chosen near fp32's smallest normal number (1.2e-38): their
# relative error is at most expf's 2 ulp, an addition's and a reciprocal's
# rounding, and half of a subnormal's last place (2^-22 of 2.9e-39 or more), below 2^-20;
# a quotient of two of them 2^-19, the row's dot product and the rest a few 2^-24
# more: within 2^-18 of the sum of the gradients' magnitudes.
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,k", [(8, 2), (64, 6), (200, 9)])
def test_gradient_of_tiny_scores(score, E, k):
    rng = np.random.default_rng([E, k])
    n = 40
    if score == "sigmoid":
        x, bias = -88.5 + 0.7 * rng.random((n, E)), None
    else:                                    # the bias picks experts far below the row's largest
        x, bias = -87.0 + 0.5 * rng.random((n, E)), np.zeros(E, np.float32)
        x[:, 0], bias[1:] = 0.0, 2.0
    x = x.astype(np.float32)
    g = (1000.0 * rng.standard_normal((n, k))).astype(np.float32)
    code = tq.SCORE_SIGMOID if score == "sigmoid" else tq.SCORE_SOFTMAX
    logits = torch.from_numpy(x).cuda()
    ids, w = tq.tq_router_scored(logits, k, score=code, bias=None if bias is None else torch.from_numpy(bias).cuda(),
                                 renormalize=True, scale=2.5)
    assert torch.allclose(w.sum(1), torch.full((n,), 2.5, device="cuda"), rtol=1e-5)
    got = _f64(tq.tq_router_scored_backward(logits, ids, w, torch.from_numpy(g).cuda(), score=code, renormalize=True,
                                            scale=2.5))
    check_no_device_error()
    ids = ids.cpu().numpy()
    want = M.router_backward(x, ids, np.ones((n, k)), g, score, True, 2.5)
    size = 2.5 * np.abs(g).astype(np.float64).sum(1, keepdims=True)
    assert (np.abs(got - want) <= 2.0 ** -18 * size).all()


# p (1 - p) of a score near 1: each factor has expf's 2 ulp, an addition's and a
# reciprocal's rounding (2^-21 together), the products three more.
@pytest.mark.parametrize("dtype,rounding", [(torch.float32, 0.0), (torch.bfloat16, 2.0 ** -8)])
def test_gradient_of_saturated_sigmoid_scores(dtype, rounding):
    rng = np.random.default_rng(1)
    n, E, k = 60, 32, 4
    logits = torch.from_numpy((3.0 + 77.0 * rng.random((n, E))).astype(np.float32)).to(dtype)
    x = _f64(logits)
    ids = torch.stack([torch.randperm(E)[:k] for _ in range(n)]).int()
    g = rng.standard_normal((n, k)).astype(np.float32)
    got = _f64(tq.tq_router_scored_backward(logits.cuda(), ids.cuda(), torch.ones(n, k, device="cuda"),
                                            torch.from_numpy(g).cuda(), score=tq.SCORE_SIGMOID, renormalize=False))
    check_no_device_error()
    i = ids.numpy().astype(np.int64)
    slope = np.exp(-x) / (1.0 + np.exp(-x)) ** 2
    want = np.zeros((n, E))
    np.put_along_axis(want, i, g * np.take_along_axis(slope, i, 1), 1)
    assert (np.abs(got - want) <= (2.0 ** -19 + rounding) * np.abs(want)).all()
    assert (got[want != 0] != 0).all()
    p = np.take_along_axis(1.0 / (1.0 + np.exp(-x)), i, 1)
    got = _f64(tq.tq_router_scored_backward(logits.cuda(), ids.cuda(), torch.ones(n, k, device="cuda"),
                                            torch.from_numpy(g).cuda(), score=tq.SCORE_SIGMOID, renormalize=True))
    q = p / p.sum(1, keepdims=True)
    per = q * (1.0 / (1.0 + np.exp(np.take_along_axis(x, i, 1))))
    want = np.zeros((n, E))
    np.put_along_axis(want, i, per * (g - (g * q).sum(1, keepdims=True)), 1)
    size = np.zeros((n, E))
    np.put_along_axis(size, i, per * (np.abs(g) + np.abs(g * q).sum(1, keepdims=True)), 1)
    assert (np.abs(got - want) <= 2.0 ** -19 * size + rounding * np.abs(want)).all()
