"""8-bit block-scaled quantisation and products against the fp64 definition.

Quantisation: scale and quotient are rounded to fp32 by definition, so codes and
scales are compared bit for bit.

Products: both sides' values are those of the codes, so what is left is the sum.  A
block of 128 products is accumulated by the tensor cores, at most 128 roundings (or
truncations, twice as large) of partial sums no larger than sum |w| |x| of the block;
the scaled blocks add up in fp32 with a rounding of both scales' product, of each
addition and of the splits' and pairs' sums: fewer than K / 128 + 16 + 3 top_k more.
With 2^-23 each, (160 + K / 128 + 3 top_k) 2^-23 of sum |w| |x|; then the one rounding
to the output's type."""
import numpy as np
import pytest
import torch

import oracle.block_operators as B
import trellis_quantized_moe_sort_gb300 as tq
from gpu_util import check_no_device_error

pytestmark = pytest.mark.gpu
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
HALF = {k: torch.finfo(v).eps / 2 for k, v in DTYPES.items()}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from trellis_quantized_moe_sort_gb300 import build
    build.build()
    tq.tq_init(0)


def _f64(t):
    return t.detach().double().cpu().numpy()


def _x(rng, n, K, dtype="bf16"):
    x = rng.standard_normal((n, K)) * np.exp(rng.standard_normal(K))
    return torch.from_numpy(x.astype(np.float32)).to(DTYPES[dtype]).cuda()


def _roundings(K, top_k=0):
    return (160 + K / 128 + 3 * top_k) * 2.0 ** -23


class Weights:
    """E seeded matrices with random codes of all magnitudes and random scales."""

    def __init__(self, seed, E, N, K):
        g = torch.Generator(device="cuda").manual_seed(seed)
        v = torch.randn((E, N, K), device="cuda", generator=g) * 100.0
        self.codes = v.clamp(-448, 448).to(torch.float8_e4m3fn)
        kb, nb = -(-K // 128), -(-N // 128)
        self.scales = torch.exp(torch.randn((E, nb, kb), device="cuda", generator=g)) / (100.0 * K ** 0.5)
        rows = torch.arange(N, device="cuda") // 128
        cols = torch.arange(K, device="cuda") // 128
        self.values = self.codes.double() * self.scales.double()[:, rows][:, :, cols]


def _rows64(codes, scales):
    K = codes.shape[1]
    return codes.double() * scales.double()[:, torch.arange(K, device="cuda") // 128]


def _check(y, want, size, K, dtype, top_k=0):
    """want and size (the sum of magnitudes) in fp64 on the device."""
    bound = HALF[dtype] * want.abs() + _roundings(K, top_k) * size + 1e-30
    worst = ((y.double() - want).abs() / bound).max().item() if y.numel() else 0.0
    assert worst <= 1.0, worst


# ------------------------------------------------------------------ quantise

@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("n,K", [(1, 16), (3, 128), (5, 144), (2, 4096), (37, 272), (129, 1056), (300, 2064)])
def test_quantize_bit_exact(dtype, n, K):
    rng = np.random.default_rng([n, K])
    x = _x(rng, n, K, dtype)
    x[0, :16] = 0
    for rows in (1, 128):
        codes, scales = tq.tq_fp8_quantize(x, rows)
        q, s = B.quantize(_f64(x), rows)
        assert scales.shape == s.shape and codes.dtype == torch.float8_e4m3fn
        assert np.array_equal(_f64(scales), s)
        assert np.array_equal(_f64(codes), q)
        for out in sorted(DTYPES):
            got = tq.tq_fp8_dequantize(codes, scales, rows, dtype=DTYPES[out])
            want = torch.from_numpy(B.values(q, s, rows)).float().to(DTYPES[out])
            assert torch.equal(got.cpu(), want)
    check_no_device_error()


def test_quantize_matrices_strides_and_ties():
    rng = np.random.default_rng(4)
    x = _x(rng, 3 * 200, 160).view(3, 200, 160)
    codes, scales = tq.tq_fp8_quantize(x, 128)
    assert scales.shape == (3, 2, 2)
    for e in range(3):
        c, s = tq.tq_fp8_quantize(x[e], 128)
        assert torch.equal(codes[e].view(torch.uint8), c.view(torch.uint8)) and torch.equal(scales[e], s)
    assert torch.equal(tq.tq_fp8_dequantize(codes, scales, 128)[1], tq.tq_fp8_dequantize(codes[1], scales[1], 128))
    big = _x(rng, 70, 512)
    part = big[:, 64:64 + 272]
    a, b = tq.tq_fp8_quantize(part), tq.tq_fp8_quantize(part.contiguous())
    assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8)) and torch.equal(a[1], b[1])
    # every midpoint of the grid, at a scale of 1
    grid = np.sort(np.unique(B.code_value(np.arange(127))))
    mid = (grid[1:] + grid[:-1]) / 2
    t = torch.zeros(1, 128)
    t[0, :126] = torch.from_numpy(mid[:126]).float()
    t[0, 127] = 448.0
    codes, scales = tq.tq_fp8_quantize(t.cuda())
    assert scales.item() == 1.0
    assert np.array_equal(_f64(codes)[0, :126], B.e4m3(mid[:126]))


def test_quantize_special_values():
    x = torch.zeros(8, 256)
    x[1, 0], x[1, 200] = float("nan"), 3.0
    x[2, 0], x[2, 1], x[2, 255] = float("inf"), 1.0, float("-inf")
    x[3] = torch.finfo(torch.float32).max
    x[4] = torch.finfo(torch.float32).tiny
    x[5] = 2.0 ** -149
    x[6] = -0.0
    x[7, ::2], x[7, 1::2] = 1e-40, -2e-39
    codes, scales = tq.tq_fp8_quantize(x.cuda())
    q, s = B.quantize(x.double().numpy())
    assert np.array_equal(_f64(scales), s)
    assert np.array_equal(_f64(codes), q, equal_nan=True)
    assert np.isnan(_f64(codes)[1, 0]) and _f64(codes)[2, 0] == 448.0 and _f64(codes)[2, 255] == -448.0
    values = tq.tq_fp8_dequantize(codes, scales)
    assert torch.isfinite(values[2:]).all() and values[1, 200] == 3.0
    empty = tq.tq_fp8_quantize(torch.empty(0, 64, device="cuda"))
    assert empty[0].shape == (0, 64) and empty[1].shape == (0, 1)
    check_no_device_error()


# ------------------------------------------------------------------ products

LINEAR = [(1, 16, 1), (1, 128, 16), (2, 144, 17), (3, 4096, 2048), (8, 256, 130), (9, 400, 33), (16, 1040, 300),
          (17, 512, 64), (40, 128, 128), (100, 2064, 257), (129, 384, 1000), (257, 1024, 511), (300, 4096, 515),
          (1000, 256, 256), (2049, 640, 769), (5000, 16, 3)]


@pytest.mark.parametrize("n,K,N", LINEAR)
def test_linear(n, K, N):
    rng = np.random.default_rng([n, K, N])
    dtype = sorted(DTYPES)[(n + N) % 3]
    codes, scales = tq.tq_fp8_quantize(_x(rng, n, K))
    w = Weights(n + K + N, 1, N, K)
    x64 = _rows64(codes, scales)
    want, size = x64 @ w.values[0].t(), x64.abs() @ w.values[0].abs().t()
    y = tq.tq_fp8_linear(codes, scales, w.codes[0], w.scales[0], dtype=DTYPES[dtype])
    assert y.dtype == DTYPES[dtype] and y.shape == (n, N)
    _check(y, want, size, K, dtype)
    again = tq.tq_fp8_linear(codes.view(torch.uint8), scales, w.codes[0].view(torch.uint8), w.scales[0],
                             dtype=DTYPES[dtype])
    assert torch.equal(again, y)
    check_no_device_error()


def test_linear_nan_and_infinite_rows_stay_apart():
    """A NaN row of x gives a NaN row of y and touches no other."""
    rng = np.random.default_rng(9)
    for n in (5, 200):
        x = _x(rng, n, 256, "fp32")
        x[1, 3] = float("nan")
        codes, scales = tq.tq_fp8_quantize(x)
        w = Weights(n, 1, 200, 256)
        y = tq.tq_fp8_linear(codes, scales, w.codes[0], w.scales[0], dtype=torch.float32)
        assert torch.isnan(y[1]).all()
        rest = torch.arange(n) != 1
        assert torch.isfinite(y[rest.cuda()]).all()


def _routing(rng, n, E, k, skew=0.0):
    logits = rng.standard_normal((n, E)) + skew * rng.standard_normal(E)
    ids = np.argsort(-logits, axis=1)[:, :k].astype(np.int32)
    w = rng.random((n, k)).astype(np.float32) + 0.1
    return torch.from_numpy(np.ascontiguousarray(ids)).cuda(), torch.from_numpy(w).cuda()


def _moe64(rows, values, ids, topk_w):
    """(sum over pairs in fp64, the same of magnitudes); an id out of range adds nothing."""
    n, k = ids.shape
    y = torch.zeros((n, values.shape[1]), dtype=torch.float64, device="cuda")
    size = torch.zeros_like(y)
    for e in range(values.shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel():
            r = rows(t, j)
            c = topk_w[t, j].double()[:, None]
            y.index_add_(0, t, (r @ values[e].t()) * c)
            size.index_add_(0, t, (r.abs() @ values[e].abs().t()) * c.abs())
    return y, size


MOE = [(900, 4, 2, 512, 700), (3, 256, 6, 1040, 272), (1, 8, 2, 256, 128), (2, 16, 4, 128, 72), (7, 64, 6, 144, 130), (32, 64, 6, 512, 256), (64, 8, 2, 384, 257),
       (50, 4, 1, 400, 100), (300, 8, 2, 256, 512), (1000, 4, 2, 272, 300), (700, 16, 3, 1024, 384), (129, 1, 1, 256, 256),
       (3000, 16, 2, 144, 130), (2500, 4, 1, 400, 100), (1100, 300, 3, 272, 257), (700, 64, 6, 1040, 640), (4000, 8, 1, 16, 33),
       (64, 8, 2, 4096, 1025), (20, 4, 2, 4112, 2050), (300, 16, 2, 512, 1000)]


@pytest.mark.parametrize("skew", [0.0, 3.0])
@pytest.mark.parametrize("n,E,k,K,N", MOE)
def test_experts(n, E, k, K, N, skew):
    rng = np.random.default_rng([n, E, k, K])
    dtype = sorted(DTYPES)[(n + K // 16) % 3]
    codes, scales = tq.tq_fp8_quantize(_x(rng, n, K))
    w = Weights(n + E, E, N, K)
    ids, topk_w = _routing(rng, n, E, k, skew)
    x64 = _rows64(codes, scales)
    want, size = _moe64(lambda t, j: x64[t], w.values, ids, topk_w)
    y = tq.tq_fp8_moe_forward(codes, scales, w.codes, w.scales, ids, topk_w, dtype=DTYPES[dtype])
    _check(y, want, size, K, dtype, k)
    assert torch.equal(y, tq.tq_fp8_moe_forward(codes, scales, w.codes, w.scales, ids, topk_w, dtype=DTYPES[dtype]))
    check_no_device_error()


@pytest.mark.parametrize("n", [1, 40, 600])
def test_experts_bad_ids_add_nothing(n):
    rng = np.random.default_rng(n)
    E, k, K, N = 8, 3, 256, 192
    codes, scales = tq.tq_fp8_quantize(_x(rng, n, K))
    w = Weights(n, E, N, K)
    ids, topk_w = _routing(rng, n, E, k)
    ids[0, 1], ids[n // 2, 0] = -1, E
    x64 = _rows64(codes, scales)
    want, size = _moe64(lambda t, j: x64[t], w.values, ids, topk_w)
    y = tq.tq_fp8_moe_forward(codes, scales, w.codes, w.scales, ids, topk_w, dtype=torch.float32)
    _check(y, want, size, K, "fp32", k)
    torch.cuda.synchronize()
    assert tq.tq_device_error()[0] == -1


def test_experts_same_expert_twice_and_all_to_one():
    """A token that names an expert twice counts it twice; every pair of a batch to one expert."""
    rng = np.random.default_rng(11)
    E, k, K, N = 16, 2, 256, 128
    for n in (1, 9, 500):
        codes, scales = tq.tq_fp8_quantize(_x(rng, n, K))
        w = Weights(n, E, N, K)
        ids = torch.full((n, k), 5, dtype=torch.int32, device="cuda")
        topk_w = torch.rand((n, k), device="cuda")
        x64 = _rows64(codes, scales)
        want, size = _moe64(lambda t, j: x64[t], w.values, ids, topk_w)
        _check(tq.tq_fp8_moe_forward(codes, scales, w.codes, w.scales, ids, topk_w), want, size, K, "bf16", k)
    check_no_device_error()


def _mlp64(x64, gu, down, ids, topk_w):
    """y and, for its bound, the sums of magnitudes and of what the codes of h may differ by.

    gate and up are off by at most r = (160 + H / 128) 2^-23 of their sums of magnitudes G
    and U, h so by dh = 1.1 |up| r G + |silu| r U (silu's slope is below 1.1) and a few
    2^-24 of itself.  A code of h next to a border falls to its other side: where h / s is
    within dh / s (and the change of s) of a midpoint, one step of E4M3, at most 2^-3 of
    the value and 2^-9 s; s itself moves by 2^-22 and the largest dh / 448."""
    n, k = ids.shape
    H, I = gu.shape[2], down.shape[2]
    y = torch.zeros((n, down.shape[1]), dtype=torch.float64, device="cuda")
    slack = torch.zeros_like(y)
    r = (160 + H / 128) * 2.0 ** -23
    for e in range(gu.shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if not t.numel():
            continue
        s = x64[t] @ gu[e].t()
        m = x64[t].abs() @ gu[e].abs().t()
        gate, up = s[:, :I], s[:, I:]
        act = gate * torch.sigmoid(gate)
        h = act * up
        dh = 1.1 * up.abs() * r * m[:, :I] + act.abs() * r * m[:, I:] + 8 * 2.0 ** -24 * h.abs()
        hb, db = h.view(-1, I // 128, 128), dh.view(-1, I // 128, 128)
        scale = (hb.abs().amax(-1, keepdim=True) / 448.0).float().double()
        dscale = 2.0 ** -22 * scale + db.amax(-1, keepdim=True) / 448.0
        q = hb / torch.clamp(scale, min=1e-300)
        dq = db / torch.clamp(scale, min=1e-300) + q.abs() * dscale / torch.clamp(scale, min=1e-300)
        lo, hi = (q - dq).to(torch.float8_e4m3fn), (q + dq).to(torch.float8_e4m3fn)
        code = q.float().to(torch.float8_e4m3fn).double()
        moved = torch.maximum((hi.double() - code).abs(), (code - lo.double()).abs())
        value = (code * scale).view(-1, I)
        error = (moved * scale + (code.abs() + moved) * dscale).view(-1, I)
        c = topk_w[t, j].double()[:, None]
        y.index_add_(0, t, (value @ down[e].t()) * c)
        slack.index_add_(0, t, (error @ down[e].abs().t() + _roundings(I, k) * (value.abs() @ down[e].abs().t())) * c)
    return y, slack


MLP = [(1200, 4, 2, 256, 384), (2, 64, 6, 1040, 384), (1, 8, 2, 256, 128), (3, 16, 4, 144, 256), (40, 16, 3, 512, 384), (200, 4, 2, 272, 128), (600, 4, 2, 384, 640),
       (1500, 2, 1, 256, 256), (64, 1, 1, 1024, 512), (2000, 16, 4, 144, 256), (2500, 4, 2, 272, 128), (40, 16, 3, 2064, 640),
       (7, 8, 2, 1040, 384), (20, 4, 1, 144, 128)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n,E,k,H,I", MLP)
def test_expert_mlp(n, E, k, H, I, dtype):
    rng = np.random.default_rng([n, E, k, H, I])
    codes, scales = tq.tq_fp8_quantize(_x(rng, n, H))
    gu, down = Weights(n, E, 2 * I, H), Weights(n + 1, E, H, I)
    ids, topk_w = _routing(rng, n, E, k)
    want, slack = _mlp64(_rows64(codes, scales), gu.values, down.values, ids, topk_w)
    y = tq.tq_fp8_moe_mlp_forward(codes, scales, gu.codes, gu.scales, down.codes, down.scales, ids, topk_w,
                                  dtype=DTYPES[dtype])
    worst = ((y.double() - want).abs() / (HALF[dtype] * want.abs() + slack * 1.01 + 1e-30)).max().item()
    assert worst <= 1.0, worst
    assert torch.equal(y, tq.tq_fp8_moe_mlp_forward(codes, scales, gu.codes, gu.scales, down.codes, down.scales, ids,
                                                    topk_w, dtype=DTYPES[dtype]))
    check_no_device_error()


def test_a_layer_in_a_graph_and_on_another_stream():
    """Norm, router, SwiGLU experts and a shared linear, as a layer runs them: the same bits eagerly, on
    another stream, and from two graphs that share a workspace and are replayed in turn."""
    rng = np.random.default_rng(21)
    E, k, H, I = 16, 3, 512, 256
    gu, down, shared = Weights(1, E, 2 * I, H), Weights(2, E, H, I), Weights(3, 1, 200, H)
    weight = torch.rand(H, device="cuda") + 0.5
    gate = torch.randn(E, H, device="cuda") / H ** 0.5

    def layer(x, res, work=None, stream=None):
        y = torch.empty_like(x)
        codes, scales, r = tq.tq_rms_norm_fp8(x, weight, residual=res, y=y, stream=stream)
        logits = (y.float()[:, None, :] * gate).sum(-1)
        ids, w = tq.tq_router_scored(logits, k, stream=stream)
        out = tq.tq_fp8_moe_mlp_forward(codes, scales, gu.codes, gu.scales, down.codes, down.scales, ids, w,
                                        workspace=work, stream=stream)
        return out, r, tq.tq_fp8_linear(codes, scales, shared.codes[0], shared.scales[0], stream=stream)

    for n in (1, 24, 500):
        xs = [(_x(rng, n, H), _x(rng, n, H)) for _ in range(2)]
        want = [layer(*x) for x in xs]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = layer(*xs[0], stream=side)
        side.synchronize()
        for a, b in zip(want[0], other):
            assert torch.equal(a, b)
        work = torch.empty(tq.tq_fp8_moe_mlp_workspace_size(n, k, E, H, I), dtype=torch.uint8, device="cuda")
        graphs, got = [], []
        for x in xs:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                got.append(layer(*x, work=work))
            graphs.append(graph)
        for _ in range(2):
            for graph in graphs:
                graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            for s, t in zip(a, b):
                assert torch.equal(s, t)
    check_no_device_error()


def test_no_pair_in_range():
    """Every id out of range: zeros, and an error that names the fault."""
    rng = np.random.default_rng(13)
    for n in (1, 300):
        codes, scales = tq.tq_fp8_quantize(_x(rng, n, 256))
        w, down = Weights(n, 4, 256, 256), Weights(n, 4, 256, 128)
        ids = torch.full((n, 2), -1, dtype=torch.int32, device="cuda")
        topk_w = torch.ones((n, 2), device="cuda")
        assert (tq.tq_fp8_moe_forward(codes, scales, w.codes, w.scales, ids, topk_w) == 0).all()
        torch.cuda.synchronize()
        assert tq.tq_device_error()[0] == -1
        assert (tq.tq_fp8_moe_mlp_forward(codes, scales, w.codes, w.scales, down.codes, down.scales, ids, topk_w) == 0).all()
        torch.cuda.synchronize()
        assert tq.tq_device_error()[0] == -1


def test_arms():
    """Few rows take the few-rows kernel, many the tiles; both sides of the change agree."""
    rng = np.random.default_rng(17)
    w = Weights(17, 1, 2048, 2048)
    codes, scales = tq.tq_fp8_quantize(_x(rng, 300, 2048))
    taken = {}
    rows = {}
    for n in (1, 8, 9, 32, 300):
        before = tq.tq_launch_counts_all()
        rows[n] = tq.tq_fp8_linear(codes[:n], scales[:n], w.codes[0], w.scales[0], dtype=torch.float32)
        after = tq.tq_launch_counts_all()
        taken[n] = tuple(after[c] - before[c] for c in ("few_rows", "fp8_gemm"))
        assert sum(taken[n]) == 1
    assert taken[1] == (1, 0) and taken[300] == (0, 1)
    size = _rows64(codes, scales).abs() @ w.values[0].abs().t()
    for n in (1, 8, 9, 32):
        assert ((rows[n] - rows[300][:n]).abs() <= 2 * _roundings(2048) * size[:n] + 2.0 ** -23 * rows[n].abs()).all()
    check_no_device_error()


def test_arms_of_experts():
    """Tokens go by themselves or in tiles of sorted pairs, by what either would read; the results agree."""
    rng = np.random.default_rng(18)
    E, k, K, N = 8, 2, 512, 768
    w = Weights(18, E, N, K)
    codes, scales = tq.tq_fp8_quantize(_x(rng, 600, K))
    ids, topk_w = _routing(rng, 600, E, k)
    rows = {}
    for n, arm in ((4, "few_rows"), (600, "fp8_gemm")):
        before = tq.tq_launch_counts_all()
        rows[n] = tq.tq_fp8_moe_forward(codes[:n], scales[:n], w.codes, w.scales, ids[:n], topk_w[:n], dtype=torch.float32)
        after = tq.tq_launch_counts_all()
        assert {c: after[c] - before[c] for c in ("few_rows", "fp8_gemm")} == {"few_rows": 0, "fp8_gemm": 0, arm: 1}
    _, size = _moe64(lambda t, j: _rows64(codes, scales)[t], w.values, ids, topk_w)
    bound = 2 * _roundings(K, k) * size[:4] + 2.0 ** -23 * rows[4].abs()
    assert ((rows[4] - rows[600][:4]).abs() <= bound).all()
    check_no_device_error()


def test_two_streams_at_once():
    """Calls that overlap, each with its own workspace and output, keep their results."""
    rng = np.random.default_rng(19)
    E, k, H, I, n = 8, 2, 512, 256, 400
    gu, down = Weights(1, E, 2 * I, H), Weights(2, E, H, I)
    inputs = []
    for _ in range(2):
        codes, scales = tq.tq_fp8_quantize(_x(rng, n, H))
        inputs.append((codes, scales, gu.codes, gu.scales, down.codes, down.scales, *_routing(rng, n, E, k)))
    want = [tq.tq_fp8_moe_mlp_forward(*a) for a in inputs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    torch.cuda.synchronize()
    for _ in range(8):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(tq.tq_fp8_moe_mlp_forward(*inputs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for y in got[i]:
            assert torch.equal(y, want[i])
    check_no_device_error()


def test_weights_past_four_gigabytes():
    """The last experts of 4.9 GB of weights, by either arm, and codes past 2^32 bytes."""
    E, N, K = 300, 4096, 4096
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of free device memory")
    codes = torch.zeros((E, N, K), dtype=torch.uint8, device="cuda")
    codes[E - 1] = torch.randint(0, 120, (N, K), dtype=torch.uint8, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    scales = torch.full((E, N // 128, K // 128), 1.0 / 8192, device="cuda")
    rng = np.random.default_rng(23)
    for n in (1, 200):
        x, xs = tq.tq_fp8_quantize(_x(rng, n, K))
        ids = torch.stack((torch.full((n,), E - 1), torch.arange(n) % (E - 1)), 1).int().cuda()
        topk_w = torch.ones((n, 2), device="cuda")
        x64 = _rows64(x, xs)
        values = codes[E - 1].view(torch.float8_e4m3fn).double() / 8192
        want, size = x64 @ values.t(), x64.abs() @ values.abs().t()
        _check(tq.tq_fp8_moe_forward(x, xs, codes, scales, ids, topk_w, dtype=torch.float32), want, size, K, "fp32", 2)
    back = tq.tq_fp8_dequantize(codes, scales, 128, dtype=torch.bfloat16)
    assert torch.equal(back[E - 1].double(), (codes[E - 1].view(torch.float8_e4m3fn).double() / 8192))
    again, s = tq.tq_fp8_quantize(back, 128)
    alone, s1 = tq.tq_fp8_quantize(back[E - 1].clone(), 128)
    assert torch.equal(again[E - 1].view(torch.uint8), alone.view(torch.uint8)) and torch.equal(s[E - 1], s1)
    assert (again[E - 2].view(torch.uint8) == 0).all()
    check_no_device_error()


def test_outputs_past_four_gigabytes():
    """Results, pairs' partial sums and rows whose offsets pass 2^32 bytes, and 2^31 values: the last rows' are right."""
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of free device memory")
    g = torch.Generator("cuda").manual_seed(5)
    n, K, N = 600_000, 128, 4096
    x = torch.randn((n, K), device="cuda", generator=g).bfloat16()
    codes, scales = tq.tq_fp8_quantize(x)
    w = Weights(5, 2, N, K)
    some = torch.tensor([0, 1, 255, n // 2 + 3, n - 130, n - 2, n - 1], device="cuda")
    rows = _rows64(codes[some], scales[some])
    want, size = rows @ w.values[0].t(), rows.abs() @ w.values[0].abs().t()
    y = tq.tq_fp8_linear(codes, scales, w.codes[0], w.scales[0])
    _check(y[some], want, size, K, "bf16")
    del y
    n = 150_000   # 2.5 GB of results, 4.9 GB of partial sums
    ids = (torch.arange(2 * n, device="cuda") % 2).int().view(n, 2)
    topk_w = torch.rand((n, 2), device="cuda", generator=g)
    some = torch.tensor([0, 130, n // 2, n - 1], device="cuda")
    want, size = _moe64(lambda t, j: _rows64(codes[some], scales[some])[t], w.values, ids[some], topk_w[some])
    y = tq.tq_fp8_moe_forward(codes[:n], scales[:n], w.codes, w.scales, ids, topk_w, dtype=torch.float32)
    _check(y[some], want, size, K, "fp32", 2)
    del y, x
    x = torch.randn((n, 16384), device="cuda", generator=g).bfloat16()
    y, _, rstd = tq.tq_rms_norm(x)
    gx, gw = tq.tq_rms_norm_backward(y, x, torch.ones(16384, device="cuda"), rstd)
    back, _, again = tq.tq_rms_norm(x[some])
    assert torch.equal(y[some], back) and torch.equal(rstd[some], again)
    assert torch.equal(gx[some], tq.tq_rms_norm_backward(back, x[some], torch.ones(16384, device="cuda"), again)[0])
    c8, s8, _ = tq.tq_rms_norm_fp8(x)
    want, wants, _ = tq.tq_rms_norm_fp8(x[some])
    assert torch.equal(c8[some].view(torch.uint8), want.view(torch.uint8)) and torch.equal(s8[some], wants)
    check_no_device_error()


@pytest.mark.parametrize("dtype", sorted(DTYPES))
def test_results_from_any_element_on(dtype):
    """y from an address that is a multiple of its elements' size alone: the same results, by every way that writes them."""
    rng = np.random.default_rng(37)

    def same(call, n, N):
        room = torch.full((n * N + 9,), 7.0, dtype=DTYPES[dtype], device="cuda")
        want = call(None)
        for lead in (1, 2, 4):
            room.fill_(7.0)
            y = room[lead:lead + n * N].view(n, N)
            assert call(y) is y and torch.equal(y, want)
            assert (room[:lead] == 7.0).all() and (room[lead + n * N:] == 7.0).all()

    for n, K, N in ((5, 256, 136), (97, 4096, 256), (97, 4096, 131), (600, 256, 512)):   # few rows, K split twice, tiles
        codes, scales = tq.tq_fp8_quantize(_x(rng, n, K))
        w = Weights(n, 1, N, K)
        same(lambda y: tq.tq_fp8_linear(codes, scales, w.codes[0], w.scales[0], y=y, dtype=DTYPES[dtype]), n, N)
    for n, N in ((3, 136), (1000, 136), (1000, 137)):   # tokens by themselves, sorted pairs
        codes, scales = tq.tq_fp8_quantize(_x(rng, n, 256))
        w = Weights(n, 4, N, 256)
        ids, topk_w = _routing(rng, n, 4, 2)
        same(lambda y: tq.tq_fp8_moe_forward(codes, scales, w.codes, w.scales, ids, topk_w, y=y, dtype=DTYPES[dtype]), n, N)
    check_no_device_error()


def test_no_rows():
    """Empty batches give empty results, without a launch."""
    w, down = Weights(1, 4, 256, 128), Weights(2, 4, 128, 128)
    x = torch.empty((0, 128), dtype=torch.bfloat16, device="cuda")
    before = tq.tq_launch_counts_all()
    codes, scales = tq.tq_fp8_quantize(x)
    assert codes.shape == (0, 128) and scales.shape == (0, 1)
    assert tq.tq_fp8_dequantize(codes, scales).shape == (0, 128)
    assert [t.shape[0] for t in tq.tq_fp8_quantize(x, 128)] == [0, 0]
    ids, topk_w = torch.empty((0, 2), dtype=torch.int32, device="cuda"), torch.empty((0, 2), device="cuda")
    assert tq.tq_fp8_linear(codes, scales, w.codes[0], w.scales[0]).shape == (0, 256)
    assert tq.tq_fp8_moe_forward(codes, scales, w.codes, w.scales, ids, topk_w).shape == (0, 256)
    assert tq.tq_fp8_moe_mlp_forward(codes, scales, w.codes, w.scales, down.codes, down.scales, ids, topk_w).shape == (0, 128)
    assert [t.shape[0] for t in tq.tq_rms_norm_fp8(x)] == [0, 0, 0]
    assert tq.tq_launch_counts_all() == before
    check_no_device_error()


def test_rows_behind_the_output_stay():
    """Nothing is written past the results of each operator."""
    rng = np.random.default_rng(31)
    for n, K, N in ((3, 256, 100), (140, 256, 131), (300, 512, 256)):
        codes, scales = tq.tq_fp8_quantize(_x(rng, n, K))
        w = Weights(n, 1, N, K)
        room = torch.full((n * N + 4096,), 7.0, dtype=torch.bfloat16, device="cuda")
        y = room[:n * N].view(n, N)
        tq.tq_fp8_linear(codes, scales, w.codes[0], w.scales[0], y=y)
        assert (room[n * N:] == 7.0).all() and not (y == 7.0).all()
        ids, topk_w = _routing(rng, n, 1, 1)
        room.fill_(7.0)
        tq.tq_fp8_moe_forward(codes, scales, w.codes, w.scales, ids, topk_w, y=y)
        assert (room[n * N:] == 7.0).all() and not (y == 7.0).all()
    check_no_device_error()


def test_refusals():
    x = torch.zeros(4, 64, device="cuda")
    codes, scales = tq.tq_fp8_quantize(x)
    w, ws = tq.tq_fp8_quantize(torch.zeros(32, 64, device="cuda"), 128)
    ids, topk_w = torch.zeros(4, 1, dtype=torch.int32, device="cuda"), torch.ones(4, 1, device="cuda")
    assert tq.tq_fp8_linear(codes, scales, w, ws).shape == (4, 32)
    for bad in (lambda: tq.tq_fp8_quantize(x, 2), lambda: tq.tq_fp8_quantize(x[0]), lambda: tq.tq_fp8_quantize(x.cpu()),
                lambda: tq.tq_fp8_linear(codes, scales[:3], w, ws), lambda: tq.tq_fp8_linear(codes, scales, w[:, :32], ws),
                lambda: tq.tq_fp8_linear(codes, scales, w, ws.repeat(2, 1)), lambda: tq.tq_fp8_linear(codes.cpu(), scales, w, ws),
                lambda: tq.tq_fp8_moe_forward(codes, scales, w[None], ws[None], ids[:3], topk_w),
                lambda: tq.tq_fp8_linear(codes, scales, w, ws, y=torch.zeros(4, 33, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: tq.tq_fp8_linear(x, scales, w, ws), lambda: tq.tq_fp8_linear(codes, scales.half(), w, ws),
                lambda: tq.tq_fp8_linear(codes, scales, w, ws, dtype=torch.float64),
                lambda: tq.tq_fp8_moe_forward(codes, scales, w[None], ws[None], ids.long(), topk_w)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(tq.TQError):
        tq.tq_fp8_quantize(torch.zeros(4, 40, device="cuda"))
    with pytest.raises(tq.TQError):
        tq.tq_fp8_moe_mlp_forward(codes, scales, torch.zeros(1, 128, 64, dtype=torch.uint8, device="cuda"),
                                  torch.zeros(1, 1, 1, device="cuda"), torch.zeros(1, 64, 64, dtype=torch.uint8, device="cuda"),
                                  torch.zeros(1, 1, 1, device="cuda"), ids, topk_w)
