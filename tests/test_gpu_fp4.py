"""4-bit microscaled quantisation and products against the fp64 definition.

Quantisation is compared bit for bit: a 16-bit value x against a midpoint m s of
the grid (m and s of 3 and 4 bits, g a power of two) is equal or at least 2^-18
apart in relation, so that one fp32 division cannot cross it.  With any other
global scale a quotient may round onto a midpoint; there a code may be one step
off in one value of 10^5.

Products: both sides' values are those of the definition (the quantisation is
exact for these inputs), so what is left is the fp32 sum.  At most K / 64 + 64
roundings of partial sums no larger than sum |w| |x|, each 2^-24: below 2^-16 of
it for K <= 8192, and the one rounding to the output's type."""
import numpy as np
import pytest
import torch

import oracle.moe_operators as M
import trellis_quantized_moe_sort_gb300 as tq
from gpu_util import check_no_device_error

pytestmark = pytest.mark.gpu
FMT = {"nv": tq.FP4_NV, "mx": tq.FP4_MX}
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
ROUND = {"fp32": 2.0 ** -23, "bf16": 2.0 ** -8, "fp16": 2.0 ** -10}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from trellis_quantized_moe_sort_gb300 import build
    build.build()
    tq.tq_init(0)


def _x(rng, n, K, dtype, spread=3.0):
    """Rows of 16-bit values with blocks of different sizes."""
    x = rng.standard_normal((n, K)) * np.exp(spread * rng.standard_normal((n, K // 16)).repeat(16, 1) / 3)
    t = torch.from_numpy(x.astype(np.float32))
    return t.to(DTYPES[dtype]) if dtype != "fp32" else t.to(torch.bfloat16).float()


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _dev_scale(g):
    return None if g is None else torch.tensor([g], dtype=torch.float32, device="cuda")


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("n,K", [(1, 32), (3, 64), (5, 96), (2, 4096), (37, 288), (129, 1056), (700, 544)])
def test_quantize_bit_exact(fmt, dtype, n, K):
    rng = np.random.default_rng([n, K])
    x = _x(rng, n, K, dtype)
    x[0, :32] = 0
    for g in ((None, 2.0 ** -5) if fmt == "nv" else (None,)):
        packed, scales = tq.tq_fp4_quantize(x.cuda(), FMT[fmt], _dev_scale(g))
        code, byte, values = M.quantize(_f64(x), fmt, 1.0 if g is None else g)
        assert np.array_equal(scales.cpu().numpy(), byte)
        assert np.array_equal(packed.cpu().numpy(), M.pack(code))
        for out in sorted(DTYPES):
            got = tq.tq_fp4_dequantize(packed, scales, FMT[fmt], _dev_scale(g), dtype=DTYPES[out])
            assert got.shape == (n, K)
            want = torch.from_numpy(values).to(DTYPES[out]).float()
            assert torch.equal(got.float().cpu(), want)
    check_no_device_error()


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_quantize_ties_and_special_values(fmt):
    x = torch.zeros(8, 64)
    x[0, :17] = torch.tensor([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, -6, 0.])
    x[1, 0], x[1, 40] = float("nan"), 3.0
    x[2, 0], x[2, 1], x[2, 63] = float("inf"), 1.0, float("-inf")
    x[3] = torch.finfo(torch.float32).max
    x[4] = torch.finfo(torch.float32).tiny
    x[5] = 2.0 ** -149
    x[6] = -0.0
    x[7, ::2], x[7, 1::2] = 448.0 * 6, 1.0
    packed, scales = tq.tq_fp4_quantize(x.cuda(), FMT[fmt])
    code, byte, values = M.quantize(_f64(x), fmt)
    assert np.array_equal(scales.cpu().numpy(), byte) and np.array_equal(packed.cpu().numpy(), M.pack(code))
    got = tq.tq_fp4_dequantize(packed, scales, FMT[fmt])
    assert torch.isfinite(got).all()
    assert np.array_equal(_f64(got), values.astype(np.float32))


def test_quantize_any_global_scale():
    rng = np.random.default_rng(4)
    x = _x(rng, 400, 1024, "fp32") * 1.0001
    g = 0.0371
    packed, scales = tq.tq_fp4_quantize(x.cuda(), tq.FP4_NV, _dev_scale(g))
    g32 = float(np.float32(g))
    code, byte, values = M.quantize(_f64(x), "nv", g32)
    assert (scales.cpu().numpy() != byte).mean() <= 1e-5
    got = _f64(tq.tq_fp4_dequantize(packed, scales, tq.FP4_NV, _dev_scale(g)))
    off = np.abs(got - values) > 1e-6 * np.abs(values)
    assert off.mean() <= 1e-5
    step = np.repeat(M.dequantize(M.pack(np.full_like(code, 4)), byte, "nv", g32)[:, ::16], 16, 1)
    assert (np.abs(got - values) <= step * 1.001 + 1e-6 * np.abs(values)).all()


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_strided_rows_outputs_and_no_rows(fmt):
    rng = np.random.default_rng(8)
    wide = _x(rng, 40, 512, "bf16").cuda()
    view = wide[::2, 128:384]
    a = tq.tq_fp4_quantize(view, FMT[fmt])
    packed = torch.zeros(20, 128, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(20, 256 // M.BLOCK[fmt], dtype=torch.uint8, device="cuda")
    b = tq.tq_fp4_quantize(view.contiguous(), FMT[fmt], packed=packed, scales=scales)
    assert b[0] is packed and b[1] is scales
    assert torch.equal(a[0], packed) and torch.equal(a[1], scales)
    empty = tq.tq_fp4_quantize(wide[:0], FMT[fmt])
    assert empty[0].shape == (0, 256) and tq.tq_fp4_dequantize(*empty, FMT[fmt]).shape == (0, 512)
    with pytest.raises(tq.TQError):                      # rows off a 16-byte boundary
        tq.tq_fp4_quantize(wide[:, 1:257], FMT[fmt])
    with pytest.raises(tq.TQError):                      # K no multiple of 32
        tq.tq_fp4_quantize(torch.zeros(4, 48, device="cuda"), FMT[fmt])
    with pytest.raises(ValueError):
        tq.tq_fp4_quantize(wide.t(), FMT[fmt])
    with pytest.raises(TypeError):
        tq.tq_fp4_quantize(wide.double(), FMT[fmt])
    with pytest.raises(ValueError):
        tq.tq_fp4_quantize(wide, 5)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("E,N,K", [(1, 1, 32), (2, 128, 256), (3, 129, 288), (1, 300, 1056), (2, 31, 4096)])
def test_tile_scales(fmt, E, N, K):
    rng = np.random.default_rng([E, N, K])
    byte = rng.integers(0, 256, (E, N, K // M.BLOCK[fmt])).astype(np.uint8)
    want = M.tile_scales(byte, fmt)
    got = tq.tq_fp4_tile_scales(torch.from_numpy(byte).cuda(), FMT[fmt])
    assert got.numel() == tq.tq_fp4_tiled_scales_size(E, N, K, FMT[fmt]) == want.size
    assert np.array_equal(got.cpu().numpy(), want)
    if E == 1:
        assert torch.equal(tq.tq_fp4_tile_scales(torch.from_numpy(byte[0]).cuda(), FMT[fmt]), got)


class Weights:
    """E seeded matrices N(0, 1/K), quantised by the definition."""

    def __init__(self, rng, E, N, K, fmt):
        w = rng.standard_normal((E * N, K)) / np.sqrt(K)
        w *= np.exp(0.5 * rng.standard_normal((E * N, 1)))
        self.g = np.full(E, 2.0 ** -9) * (1 + np.arange(E) % 3) if fmt == "nv" else np.ones(E)
        parts = [M.quantize(w[e * N:(e + 1) * N], fmt, self.g[e]) for e in range(E)]
        self.fmt = FMT[fmt]
        self.packed = torch.from_numpy(np.stack([M.pack(p[0]) for p in parts])).cuda()
        byte = np.stack([p[1] for p in parts])
        self.tiled = tq.tq_fp4_tile_scales(torch.from_numpy(byte).cuda(), self.fmt)
        self.scale = torch.from_numpy(self.g.astype(np.float32)).cuda() if fmt == "nv" else None
        self.values = np.stack([p[2] for p in parts])


def _close(y, want, size, dtype):
    got = _f64(y)
    assert np.isfinite(got).all()
    limit = 2.0 ** -16 * size + ROUND[dtype] * np.abs(want) + 6e-8
    assert (np.abs(got - want) <= limit).all(), float((np.abs(got - want) / limit).max())


LINEAR = [(1, 32, 1), (1, 4096, 2048), (2, 288, 129), (3, 96, 5), (5, 1056, 515), (8, 256, 128), (16, 4096, 130),
          (17, 512, 127), (33, 64, 1), (64, 2048, 256), (100, 288, 384), (129, 800, 4), (200, 256, 300), (224, 544, 129),
          (225, 96, 131), (450, 1024, 257), (701, 352, 250)]


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("n,K,N", LINEAR)
def test_linear(fmt, dtype, n, K, N):
    rng = np.random.default_rng([n, K, N])
    w = Weights(rng, 1, N, K, fmt)
    x = _x(rng, n, K, dtype, spread=1.0)
    g = 2.0 ** -7 if fmt == "nv" else None
    y = tq.tq_fp4_linear(x.cuda(), w.packed[0], w.tiled, fmt=w.fmt, w_scale=w.scale, x_scale=_dev_scale(g))
    check_no_device_error()
    assert y.dtype == DTYPES[dtype] and y.shape == (n, N)
    xq = M.quantize(_f64(x), fmt, 1.0 if g is None else g)[2]
    _close(y, xq @ w.values[0].T, np.abs(xq) @ np.abs(w.values[0]).T, dtype)


@pytest.mark.parametrize("n", [2, 300])
@pytest.mark.parametrize("N,offset", [(256, 1), (256, 2), (255, 1), (130, 8)])
def test_linear_into_a_given_buffer(n, N, offset):
    """y of another type than x, at any alignment of its elements; strided x."""
    rng = np.random.default_rng([n, N])
    w = Weights(rng, 1, N, 512, "nv")
    wide = _x(rng, n, 1024, "bf16", spread=1.0).cuda()
    x = wide[:, 256:768]
    xq = M.quantize(_f64(x), "nv")[2]
    want, size = xq @ w.values[0].T, np.abs(xq) @ np.abs(w.values[0]).T
    for dtype in sorted(DTYPES):
        buffer = torch.full((n * N + 64,), 7.0, dtype=DTYPES[dtype], device="cuda")
        y = buffer[offset:offset + n * N].view(n, N)
        got = tq.tq_fp4_linear(x, w.packed[0], w.tiled, w_scale=w.scale, y=y)
        assert got is y
        _close(y, want, size, dtype)
        assert (buffer[:offset] == 7).all() and (buffer[offset + n * N:] == 7).all()


@pytest.mark.parametrize("fmt,dtype", [("nv", "bf16"), ("mx", "fp16")])
@pytest.mark.parametrize("n,N", [(70, 1), (70, 7), (71, 9), (77, 24), (130, 127), (250, 128), (259, 131), (300, 264),
                                 (500, 385), (1000, 520)])
def test_linear_rows_at_every_alignment(n, N, fmt, dtype):
    """One step of K, so no splits: 16-bit rows that start anywhere in their 16 bytes."""
    rng = np.random.default_rng([n, N])
    w = Weights(rng, 1, N, 64, fmt)
    x = _x(rng, n, 64, dtype, spread=1.0)
    xq = M.quantize(_f64(x), fmt)[2]
    want, size = xq @ w.values[0].T, np.abs(xq) @ np.abs(w.values[0]).T
    x = x.cuda()
    for offset in range(8):
        buffer = torch.full((n * N + 64,), 7.0, dtype=DTYPES[dtype], device="cuda")
        y = buffer[offset:offset + n * N].view(n, N)
        tq.tq_fp4_linear(x, w.packed[0], w.tiled, fmt=w.fmt, w_scale=w.scale, y=y)
        check_no_device_error()
        _close(y, want, size, dtype)
        assert (buffer[:offset] == 7).all() and (buffer[offset + n * N:] == 7).all()


# tokens, experts, top_k, K, N: few tokens (one launch), every m-tile size, experts
# without tokens, one with all of them
EXPERTS = [(1, 8, 2, 512, 256), (1, 256, 6, 256, 64), (2, 4, 4, 96, 5), (5, 1, 1, 288, 129), (40, 8, 2, 512, 257),
           (64, 64, 6, 544, 130), (100, 2, 2, 64, 3), (150, 8, 3, 256, 128), (300, 4, 1, 1056, 131), (333, 4, 3, 96, 200),
           (700, 3, 2, 288, 65), (900, 64, 8, 64, 129)]


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("n,E,k,K,N", EXPERTS)
@pytest.mark.parametrize("dtype", sorted(DTYPES))
def test_experts(fmt, n, E, k, K, N, dtype):
    rng = np.random.default_rng([n, E, k, K])
    w = Weights(rng, E, N, K, fmt)
    x = _x(rng, n, K, dtype, spread=1.0)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(n)]).astype(np.int32)
    if n > 100:
        ids[: n // 3] = ids[0]                       # a few experts take a third of the tokens
    weights = rng.standard_normal((n, k)).astype(np.float32)
    weights[0, 0] = 0.0
    y = tq.tq_fp4_moe_forward(x.cuda(), w.packed, w.tiled, torch.from_numpy(ids).cuda(), torch.from_numpy(weights).cuda(),
                              fmt=w.fmt, w_scale=w.scale)
    check_no_device_error()
    want, size = M.moe(M.quantize(_f64(x), fmt)[2], ids, weights, w.values)
    assert y.dtype == DTYPES[dtype]
    _close(y, want, size, dtype)


@pytest.mark.parametrize("n", [1, 50, 400])
def test_experts_out_of_range_add_nothing_and_are_reported(n):
    rng = np.random.default_rng(n)
    w = Weights(rng, 8, 130, 256, "mx")
    x = _x(rng, n, 256, "bf16", spread=1.0)
    ids = np.stack([rng.permutation(8)[:3] for _ in range(n)]).astype(np.int32)
    ids[0, 1], ids[n // 2, 2] = 8, -5
    weights = rng.random((n, 3)).astype(np.float32)
    work = torch.full((tq.tq_fp4_moe_workspace_size(n, 3, 8, 256, 130, tq.FP4_MX),), 255, dtype=torch.uint8, device="cuda")
    y = tq.tq_fp4_moe_forward(x.cuda(), w.packed, w.tiled, torch.from_numpy(ids).cuda(), torch.from_numpy(weights).cuda(),
                              fmt=tq.FP4_MX, workspace=work)
    torch.cuda.synchronize()
    assert tq.tq_device_error()[0] == -1
    want, size = M.moe(M.quantize(_f64(x), "mx")[2], ids, weights, w.values)
    _close(y, want, size, "bf16")


def test_every_pair_out_of_range():
    rng = np.random.default_rng(1)
    w = Weights(rng, 8, 64, 64, "nv")
    ids = torch.full((60, 2), -1, dtype=torch.int32, device="cuda")
    y = tq.tq_fp4_moe_forward(torch.ones(60, 64, device="cuda"), w.packed, w.tiled, ids, torch.ones(60, 2, device="cuda"),
                              w_scale=w.scale)
    torch.cuda.synchronize()
    assert tq.tq_device_error()[0] == -1 and not y.any()


@pytest.mark.parametrize("n", [0, 1, 30, 500])
def test_results_repeat_on_streams_and_in_graphs(n):
    rng = np.random.default_rng(n)
    w = Weights(rng, 16, 200, 512, "nv")
    x = _x(rng, n, 512, "bf16").cuda()
    ids = torch.from_numpy(rng.integers(0, 16, (n, 4)).astype(np.int32)).cuda()
    weights = torch.rand(n, 4, device="cuda")

    def call(stream=None):
        return (tq.tq_fp4_moe_forward(x, w.packed, w.tiled, ids, weights, w_scale=w.scale, stream=stream),
                tq.tq_fp4_linear(x, w.packed[3], w.tiled[: w.tiled.numel() // 16], w_scale=w.scale[3:4], stream=stream))

    want = call()
    assert want[0].shape == (n, 200)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b = call()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    check_no_device_error()
    for got in (a, b, call()):
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_a_given_stream_owns_the_memory(monkeypatch):
    """Everything that a call allocates comes from the stream that it runs on, so
    that no other stream's work can be given it before the call has run."""
    rng = np.random.default_rng(4)
    w = Weights(rng, 4, 128, 256, "nv")
    x = _x(rng, 40, 256, "bf16").cuda()
    ids = torch.from_numpy(rng.integers(0, 4, (40, 2)).astype(np.int32)).cuda()
    weights = torch.rand(40, 2, device="cuda")
    logits = torch.randn(40, 64, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    seen, empty = [], torch.empty

    def record(*args, **kwargs):
        seen.append(torch.cuda.current_stream())
        return empty(*args, **kwargs)

    def all_calls(stream):
        moe = tq.tq_fp4_moe_forward(x, w.packed, w.tiled, ids, weights, w_scale=w.scale, stream=stream)
        picks = tq.tq_router_scored(logits, 2, stream=stream)
        grad = tq.tq_router_scored_backward(logits, *picks, weights, stream=stream)
        packed, scales = tq.tq_fp4_quantize(x, stream=stream)
        tiled = tq.tq_fp4_tile_scales(scales, stream=stream)
        linear = tq.tq_fp4_linear(x, packed, tiled, stream=stream)
        return moe, *picks, grad, packed, scales, tiled, linear, tq.tq_fp4_dequantize(packed, scales, stream=stream)

    want = all_calls(None)
    torch.cuda.synchronize()
    monkeypatch.setattr(torch, "empty", record)
    got = all_calls(side)
    monkeypatch.undo()
    side.synchronize()
    check_no_device_error()
    assert len(seen) >= len(got) and all(s == side for s in seen)
    assert torch.cuda.current_stream() != side
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_both_arms_of_a_linear_agree():
    """A row alone (one launch) and among others (tensor cores): the same values to fp32 rounding."""
    rng = np.random.default_rng(77)
    w = Weights(rng, 1, 257, 2048, "nv")
    x = _x(rng, 300, 2048, "fp32", spread=1.0).cuda()
    before = tq.tq_launch_counts_all()
    many = tq.tq_fp4_linear(x, w.packed[0], w.tiled, w_scale=w.scale)
    one = tq.tq_fp4_linear(x[7:8], w.packed[0], w.tiled, w_scale=w.scale)
    after = tq.tq_launch_counts_all()
    assert after["fp4_gemm"] == before["fp4_gemm"] + 1 and after["fp4_gemv"] == before["fp4_gemv"] + 1
    xq = M.quantize(_f64(x[7:8]), "nv")[2]
    size = np.abs(xq) @ np.abs(w.values[0]).T
    assert (np.abs(_f64(one) - _f64(many[7:8])) <= 2.0 ** -15 * size).all()


# A value of h on the edge of two codes may fall to either side (its fp32 sums
# differ from fp64 by 2^-16 of their terms at most, so one in about 10^4 does):
# that moves an output by a code's step, a few per cent of one of I terms.  The
# 2-norm over all outputs stays within 2^-8 beside the output's own rounding.
@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("n,E,k,H,I", [(1, 8, 2, 256, 128), (3, 16, 6, 512, 96), (60, 8, 2, 288, 256), (400, 8, 3, 256, 160)])
def test_mlp(fmt, n, E, k, H, I):
    rng = np.random.default_rng([n, H, I])
    gu, down = Weights(rng, E, 2 * I, H, fmt), Weights(rng, E, H, I, fmt)
    x = _x(rng, n, H, "bf16", spread=1.0)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(n)]).astype(np.int32)
    weights = rng.random((n, k)).astype(np.float32)
    hs = 2.0 ** -6 if fmt == "nv" else None
    y = tq.tq_fp4_moe_mlp_forward(x.cuda(), gu.packed, gu.tiled, down.packed, down.tiled, torch.from_numpy(ids).cuda(),
                                  torch.from_numpy(weights).cuda(), fmt=gu.fmt, gu_scale=gu.scale, down_scale=down.scale,
                                  h_scale=_dev_scale(hs))
    check_no_device_error()
    xq = M.quantize(_f64(x), fmt)[2]
    want = np.zeros((n, H))
    for j in range(k):
        z = np.stack([gu.values[ids[t, j]] @ xq[t] for t in range(n)])
        gate, up = z[:, :I], z[:, I:]
        h = M.quantize((gate / (1 + np.exp(-gate)) * up).astype(np.float32), fmt, 1.0 if hs is None else hs)[2]
        want += weights[:, j:j + 1] * np.stack([down.values[ids[t, j]] @ h[t] for t in range(n)])
    off = np.linalg.norm(_f64(y) - want) / np.linalg.norm(want)
    assert off <= 2.0 ** -8 + 2.0 ** -8


def test_router_to_experts():
    """The layer as it is served: routed by the scored router, masked tokens contribute nothing."""
    rng = np.random.default_rng(2)
    E, k, H, I, n = 32, 4, 256, 128, 90
    gu, down = Weights(rng, E, 2 * I, H, "nv"), Weights(rng, E, H, I, "nv")
    x = _x(rng, n, H, "bf16", spread=1.0).cuda()
    logits = torch.from_numpy(rng.standard_normal((n, E)).astype(np.float32)).cuda()
    logits[5] = float("-inf")
    ids, w = tq.tq_router_scored(logits, k, groups=8, top_groups=4)
    y = tq.tq_fp4_moe_mlp_forward(x, gu.packed, gu.tiled, down.packed, down.tiled, ids, w, gu_scale=gu.scale,
                                  down_scale=down.scale)
    check_no_device_error()
    assert torch.isfinite(y).all() and not y[5].any() and y[4].any()


def test_argument_errors():
    w = Weights(np.random.default_rng(0), 4, 64, 64, "nv")
    x, ids, tw = torch.ones(3, 64, device="cuda"), torch.zeros(3, 2, dtype=torch.int32, device="cuda"), torch.ones(3, 2, device="cuda")
    ok = tq.tq_fp4_moe_forward(x, w.packed, w.tiled, ids, tw)
    assert ok.shape == (3, 64)
    for bad in (dict(x=x.cpu()), dict(x=x[0]), dict(x=torch.ones(3, 32, device="cuda")), dict(ids=ids[:2]), dict(tw=tw[:, :1]),
                dict(tiled=w.tiled[:-1]), dict(w_scale=torch.ones(3, device="cuda")), dict(x_scale=torch.ones(2, device="cuda")),
                dict(y=torch.ones(3, 63, device="cuda"))):
        a = dict(x=x, ids=ids, tw=tw, tiled=w.tiled, w_scale=None, x_scale=None, y=None) | bad
        with pytest.raises(ValueError):
            tq.tq_fp4_moe_forward(a["x"], w.packed, a["tiled"], a["ids"], a["tw"], w_scale=a["w_scale"], x_scale=a["x_scale"],
                                  y=a["y"])
    for bad in (dict(ids=ids.long()), dict(tw=tw.double()), dict(packed=w.packed.int()), dict(y=torch.ones(3, 64, device="cuda").double())):
        a = dict(ids=ids, tw=tw, packed=w.packed, y=None) | bad
        with pytest.raises(TypeError):
            tq.tq_fp4_moe_forward(x, a["packed"], w.tiled, a["ids"], a["tw"], y=a["y"])
    with pytest.raises(tq.TQError):                                  # MX has no global scales
        tq.tq_fp4_linear(x, w.packed[0], w.tiled[: w.tiled.numel() // 8], fmt=tq.FP4_MX, w_scale=torch.ones(1, device="cuda"))


# Many pairs to an expert, rows of very different sizes, an id out of range.
@pytest.mark.parametrize("N", [1024, 1027, 1006])
@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_experts_many_pairs(fmt, N):
    rng = np.random.default_rng(N)
    n, E, k, K = 1500, 8, 3, 96
    w = Weights(rng, E, N, K, fmt)
    x = _x(rng, n, K, "bf16", spread=1.0)
    x[3] = 0
    x[4] *= 2.0 ** 60
    x[5] *= 2.0 ** -60
    ids = np.stack([rng.permutation(E)[:k] for _ in range(n)]).astype(np.int32)
    ids[7, 1] = 99
    weights = rng.standard_normal((n, k)).astype(np.float32)
    args = (x.cuda(), w.packed, w.tiled, torch.from_numpy(ids).cuda(), torch.from_numpy(weights).cuda())
    y = tq.tq_fp4_moe_forward(*args, fmt=w.fmt, w_scale=w.scale)
    torch.cuda.synchronize()
    assert tq.tq_device_error()[0] == -1                      # of the one id
    xq = M.quantize(_f64(x), fmt)[2]
    want, size = np.zeros((n, N)), np.zeros((n, N))
    for e in range(E):
        t, j = np.nonzero(ids == e)
        p = xq[t] @ w.values[e].T
        c = weights[t, j, None].astype(np.float64)
        np.add.at(want, t, c * p)
        np.add.at(size, t, np.abs(c) * (np.abs(xq[t]) @ np.abs(w.values[e]).T))
    got = _f64(y)
    limit = 2.0 ** -16 * size + 2.0 ** -8 * np.abs(want) + 1e-37
    assert (np.abs(got - want) <= limit).all()
    # values themselves, not only the largest: the 2-norm is that of bf16 rounding
    rows = np.setdiff1d(np.arange(n), [4])
    assert np.linalg.norm(got[rows] - want[rows]) <= 2.0 ** -9 * np.linalg.norm(want[rows])
    y32 = tq.tq_fp4_moe_forward(*args, fmt=w.fmt, w_scale=w.scale, y=torch.empty(n, N, device="cuda"))
    tq.tq_device_error()
    assert (np.abs(_f64(y32) - want) <= 2.0 ** -16 * size + 2.0 ** -22 * np.abs(want) + 1e-37).all()


def test_not_finite_weights_stay_in_their_outputs():
    """A NaN scale in one weight row: that output is NaN for the tokens of its expert, its neighbours are not."""
    rng = np.random.default_rng(6)
    n, E, k, K, N = 1500, 8, 3, 64, 1024
    w = Weights(rng, E, N, K, "nv")
    byte = np.zeros((E, N, K // 16), np.uint8) + 0x38
    byte[2, 100, 1] = 0x7f
    tiled = tq.tq_fp4_tile_scales(torch.from_numpy(byte).cuda(), tq.FP4_NV)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(n)]).astype(np.int32)
    y = tq.tq_fp4_moe_forward(_x(rng, n, K, "bf16").cuda(), w.packed, tiled, torch.from_numpy(ids).cuda(),
                              torch.ones(n, k, device="cuda"))
    bad = torch.isnan(y).cpu().numpy()
    want = np.zeros((n, N), bool)
    want[(ids == 2).any(1), 100] = True
    assert np.array_equal(bad, want) and torch.isfinite(y[~torch.isnan(y)]).all()


def test_weights_past_four_gigabytes():
    """Experts whose codes start past 2^32 bytes, on both arms."""
    E, N, K = 600, 4096, 4096
    g = torch.Generator(device="cuda").manual_seed(3)
    packed = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.randint(0x28, 0x40, (E, N, K // 16), dtype=torch.uint8, device="cuda", generator=g)
    tiled = tq.tq_fp4_tile_scales(scales)
    x = torch.randn(70, K, device="cuda", generator=g).bfloat16()
    xq = tq.tq_fp4_dequantize(*tq.tq_fp4_quantize(x)).double()
    used = [0, 300, 599]
    values = {e: tq.tq_fp4_dequantize(packed[e], scales[e]).double() for e in used}
    before = tq.tq_launch_counts_all()
    for n in (2, 70):
        ids = torch.tensor(used, dtype=torch.int32, device="cuda").repeat(n, 1)
        w = torch.rand(n, 3, device="cuda", generator=g)
        y = tq.tq_fp4_moe_forward(x[:n], packed, tiled, ids, w, y=torch.empty(n, N, device="cuda"))
        check_no_device_error()
        want = sum(w[:, j, None].double() * (xq[:n] @ values[e].t()) for j, e in enumerate(used))
        size = sum(w[:, j, None].double() * (xq[:n].abs() @ values[e].abs().t()) for j, e in enumerate(used))
        assert bool(((y.double() - want).abs() <= 2.0 ** -16 * size).all())
    after = tq.tq_launch_counts_all()
    assert after["fp4_gemv"] == before["fp4_gemv"] + 1 and after["fp4_gemm"] == before["fp4_gemm"] + 1


def test_outputs_past_two_to_the_32():
    """More than 2^32 results, and more than 2^32 partial sums of pairs."""
    K, N = 32, 8192
    rng = np.random.default_rng(1)
    w = Weights(rng, 4, N, K, "mx")
    values = torch.from_numpy(w.values).cuda()
    n = 530_000
    x = torch.randn(n, K, device="cuda").bfloat16()
    xq = tq.tq_fp4_dequantize(*tq.tq_fp4_quantize(x, tq.FP4_MX), tq.FP4_MX).double()
    rows = torch.tensor([0, 1, 262_143, 262_144, 400_001, n - 1], device="cuda")
    y = tq.tq_fp4_linear(x, w.packed[1], w.tiled[w.tiled.numel() // 4: w.tiled.numel() // 2], fmt=tq.FP4_MX)
    check_no_device_error()
    want, size = xq[rows] @ values[1].t(), xq[rows].abs() @ values[1].abs().t()
    assert bool(((y[rows].double() - want).abs() <= 2.0 ** -16 * size + 2.0 ** -8 * want.abs()).all())
    del y
    n, k = 180_000, 3
    ids = torch.stack([torch.randperm(4, device="cuda")[:k] for _ in range(64)]).int().repeat(n // 64 + 1, 1)[:n].contiguous()
    tw = torch.rand(n, k, device="cuda")
    y = tq.tq_fp4_moe_forward(x[:n], w.packed, w.tiled, ids, tw, fmt=tq.FP4_MX)
    check_no_device_error()
    for t in (0, 100_003, 174_762, 174_763, n - 1):
        e = ids[t].long()
        want = (tw[t, :, None].double() * (values[e] @ xq[t])).sum(0)
        size = (tw[t, :, None].double() * (values[e].abs() @ xq[t].abs())).sum(0)
        assert bool(((y[t].double() - want).abs() <= 2.0 ** -16 * size + 2.0 ** -8 * want.abs()).all())
