"""RMS norm, its 8-bit output and its gradient against the fp64 definition.

Tolerances.  Half a step of a type is 2^-24 (fp32), 2^-8 (bf16) or 2^-11 (fp16) of
the value.  r: one rounding of an exact sum of two numbers, which fp32 may round once
before (bf16 and fp16 sums are exact in fp32 but for exponents far apart, where the
first rounding is far below the second): equal to torch's fp32 sum.  rstd: the sum
carries its errors, one rounding of the result, 2^-24, and a margin of 2^-40.  y: the
roundings of rstd and of two products in fp32, 3 x 2^-24, and the one to the type.
Codes and scales: equal to those of fp32 arithmetic from the returned rstd.

Gradient: rstd 2^-24, and per value a, x rstd, their difference, the products: below
8 x 2^-24 of each of the terms added; the mean's sum of K values in a tree of at most
16 + 10 additions: 26 x 2^-24 of the mean of magnitudes; then the type's rounding.
grad_weight: rows in a chain of at most n / blocks + blocks / 32 + 5 additions of n
values, at most n of them, each 2^-24 of the sum of magnitudes."""
import numpy as np
import pytest
import torch

import oracle.block_operators as B
import trellis_quantized_moe_sort_gb300 as tq
from gpu_util import check_no_device_error

pytestmark = pytest.mark.gpu
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
HALF = {k: torch.finfo(v).eps / 2 for k, v in DTYPES.items()}
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from trellis_quantized_moe_sort_gb300 import build
    build.build()
    tq.tq_init(0)


def _f64(t):
    return t.detach().double().cpu().numpy()


def _rows(rng, n, K, dtype, spread=1.0):
    x = rng.standard_normal((n, K)) * np.exp(spread * rng.standard_normal(K))
    return torch.from_numpy(x.astype(np.float32)).to(DTYPES[dtype]).cuda()


def _weight(rng, K, dtype):
    return torch.from_numpy((1.0 + 0.3 * rng.standard_normal(K)).astype(np.float32)).to(DTYPES[dtype]).cuda()


def _tiny(dtype):
    return float(torch.finfo(DTYPES[dtype]).tiny) * HALF[dtype] * 2


SIZES = [(1, 1), (1, 7), (2, 16), (3, 31), (5, 128), (4, 513), (7, 1000), (33, 2048), (3, 4096), (2, 4097), (3, 8192),
         (2, 8193), (2, 12000), (1, 16384), (2, 16383)]


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("n,K", SIZES)
def test_norm_and_gradient(dtype, n, K):
    rng = np.random.default_rng([n, K])
    x, res = _rows(rng, n, K, dtype), _rows(rng, n, K, dtype, 2.0)
    w_type = ("fp32", dtype)[K % 2]
    w = _weight(rng, K, w_type)
    y, r, rstd = tq.tq_rms_norm(x, w, eps=1e-5, residual=res)
    assert y.dtype == r.dtype == x.dtype and rstd.shape == (n,)
    assert torch.equal(r, (x.float() + res.float()).to(x.dtype))
    eps = float(np.float32(1e-5))
    want, want_rstd = B.rms_norm(_f64(r), _f64(w), eps)
    assert np.all(np.abs(_f64(rstd)[:, None] - want_rstd) <= (U + 2.0 ** -40) * want_rstd)
    assert np.all(np.abs(_f64(y) - want) <= (HALF[dtype] + 4 * U) * np.abs(want) + _tiny(dtype))

    dy, dr = _rows(rng, n, K, dtype), _rows(rng, n, K, dtype)
    gx, gw = tq.tq_rms_norm_backward(dy, r, w, rstd, grad_residual=dr)
    want_x, want_w = B.rms_norm_grad(_f64(dy), _f64(r), _f64(w), eps, _f64(dr))
    a, v = np.abs(_f64(dy) * _f64(w)), np.abs(_f64(r))
    terms = want_rstd * (a + v * want_rstd ** 2 * (a * v).mean(-1, keepdims=True)) + np.abs(_f64(dr))
    assert gx.dtype == x.dtype and gw.dtype == w.dtype
    assert np.all(np.abs(_f64(gx) - want_x) <= HALF[dtype] * np.abs(want_x) + 36 * U * terms + _tiny(dtype))
    magnitudes = (np.abs(_f64(dy)) * v * want_rstd).sum(0)
    assert np.all(np.abs(_f64(gw) - want_w) <= HALF[w_type] * np.abs(want_w) + (n + 4) * U * magnitudes + _tiny(w_type))
    # without a residual's gradient, and without a weight
    gx0, gw0 = tq.tq_rms_norm_backward(dy, r, None, rstd)
    assert gw0 is None
    want_x, _ = B.rms_norm_grad(_f64(dy), _f64(r), None, eps)
    d = np.abs(_f64(dy))
    terms = want_rstd * (d + v * want_rstd ** 2 * (d * v).mean(-1, keepdims=True))
    assert np.all(np.abs(_f64(gx0) - want_x) <= HALF[dtype] * np.abs(want_x) + 36 * U * terms + _tiny(dtype))
    check_no_device_error()


def _codes_of(r, rstd, w):
    """Codes and scales of fp32 arithmetic."""
    y = r.float().cpu().numpy() * rstd.cpu().numpy()[:, None]
    if w is not None:
        y = y * w.float().cpu().numpy()
    assert y.dtype == np.float32
    return B.quantize(y), y


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("n,K", [(1, 16), (3, 128), (5, 144), (2, 512), (17, 1040), (9, 4096), (4, 8192), (2, 8208),
                                 (1, 16384)])
def test_norm_fp8(dtype, n, K):
    rng = np.random.default_rng([n, K, 8])
    x, res, w = _rows(rng, n, K, dtype), _rows(rng, n, K, dtype, 2.0), _weight(rng, K, "fp32")
    y, r, rstd = tq.tq_rms_norm(x, w, residual=res)
    both = torch.empty_like(x)
    codes, scales, r8 = tq.tq_rms_norm_fp8(x, w, residual=res, y=both)
    assert codes.dtype == torch.float8_e4m3fn and scales.shape == (n, -(-K // 128))
    assert torch.equal(r8, r) and torch.equal(both, y)
    (q, s), y32 = _codes_of(r, rstd, w)
    assert np.array_equal(_f64(scales), s)
    assert np.array_equal(_f64(codes), q)
    # the quantiser gives the same of the same numbers
    c2, s2 = tq.tq_fp8_quantize(torch.from_numpy(y32).cuda())
    assert torch.equal(c2.view(torch.uint8), codes.view(torch.uint8)) and torch.equal(s2, scales)
    check_no_device_error()


def test_strides_alignment_and_in_place():
    rng = np.random.default_rng(3)
    for dtype in sorted(DTYPES):
        for K, lead in ((256, 0), (256, 1), (250, 3)):
            big = _rows(rng, 6, 2 * K + 8, dtype)
            x, res = big[:, lead:lead + K], _rows(rng, 6, K + 9, dtype)[:, lead:lead + K]
            w = _weight(rng, K + 1, "bf16")[1:]
            y, r, rstd = tq.tq_rms_norm(x, w, residual=res)
            y2, r2, rstd2 = tq.tq_rms_norm(x.contiguous(), w.clone(), residual=res.contiguous())
            # neighbours of a thread differ between the two ways to read a row; rstd is rounded once either way
            assert torch.equal(r, r2) and torch.equal(rstd, rstd2) and torch.equal(y, y2)
        x, res, w = _rows(rng, 5, 512, dtype), _rows(rng, 5, 512, dtype), _weight(rng, 512, "fp32")
        y, r, _ = tq.tq_rms_norm(x, w, residual=res)
        place = res.clone()
        y2, r2, _ = tq.tq_rms_norm(x, w, residual=place, residual_out=place)
        assert r2 is place and torch.equal(r2, r) and torch.equal(y2, y)
        again = x.clone()
        y3, same, rstd = tq.tq_rms_norm(again, w, y=again)
        assert same is again and torch.equal(y3, tq.tq_rms_norm(x, w)[0])
        dy = _rows(rng, 5, 512, dtype)
        gx, gw = tq.tq_rms_norm_backward(dy, x, w, rstd)
        gx2, gw2 = tq.tq_rms_norm_backward(dy, x, w, rstd, grad_x=dy)
        assert gx2 is dy and torch.equal(gx, gx2) and torch.equal(gw, gw2)


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("n,K", [(400, 8208), (330, 16384), (160, 12304)])
def test_gradient_of_many_wide_rows(n, K, dtype):
    """Blocks take several rows of more than 8192 values each, with and without a residual's gradient, also in place."""
    rng = np.random.default_rng([n, K, 1])
    x, dy, dr = (_rows(rng, n, K, dtype) for _ in range(3))
    w = _weight(rng, K, "fp32")
    _, _, rstd = tq.tq_rms_norm(x, w)
    eps = float(np.float32(1e-6))
    for g in (None, dr):
        gx, gw = tq.tq_rms_norm_backward(dy, x, w, rstd, grad_residual=g)
        want_x, want_w = B.rms_norm_grad(_f64(dy), _f64(x), _f64(w), eps, None if g is None else _f64(g))
        a, v, r = np.abs(_f64(dy) * _f64(w)), np.abs(_f64(x)), _f64(rstd)[:, None]
        terms = r * (a + v * r ** 2 * (a * v).mean(-1, keepdims=True)) + (0 if g is None else np.abs(_f64(g)))
        assert np.all(np.abs(_f64(gx) - want_x) <= HALF[dtype] * np.abs(want_x) + 36 * U * terms + _tiny(dtype))
        magnitudes = (np.abs(_f64(dy)) * v * r).sum(0)
        assert np.all(np.abs(_f64(gw) - want_w) <= (n + 4) * U * magnitudes + U * np.abs(want_w))
        again = dy.clone()
        gx2, gw2 = tq.tq_rms_norm_backward(again, x, w, rstd, grad_residual=g, grad_x=again)
        assert torch.equal(gx2, gx) and torch.equal(gw2, gw)
    check_no_device_error()


def test_outputs_over_inputs():
    """Dense rows may be written in their place by each output; rows that they would only partly cover are refused."""
    rng = np.random.default_rng(11)
    for n, K in ((700, 512), (300, 250)):
        x, res, w = _rows(rng, n, K, "bf16"), _rows(rng, n, K, "bf16"), _weight(rng, K, "fp32")
        dy, dr = _rows(rng, n, K, "bf16"), _rows(rng, n, K, "bf16")
        y, r, rstd = tq.tq_rms_norm(x, w, residual=res)
        for first, second in ((x, res), (res, x)):
            a, b = first.clone(), second.clone()
            y2, r2, rstd2 = tq.tq_rms_norm(a if first is x else b, w, residual=b if first is x else a, residual_out=a, y=b)
            assert torch.equal(y2, y) and torch.equal(r2, r) and torch.equal(rstd2, rstd)
        gx, gw = tq.tq_rms_norm_backward(dy, r, w, rstd, grad_residual=dr)
        for place in range(3):
            args = [dy.clone(), r.clone(), dr.clone()]
            gx2, gw2 = tq.tq_rms_norm_backward(args[0], args[1], w, rstd, grad_residual=args[2], grad_x=args[place])
            assert gx2 is args[place] and torch.equal(gx2, gx) and torch.equal(gw2, gw)
        pad = torch.cat((x, x), 1)
        with pytest.raises(tq.TQError):
            tq.tq_rms_norm(pad[:, :K], w, y=pad.view(2 * n, K)[:n])
        with pytest.raises(tq.TQError):
            tq.tq_rms_norm(x[1:], w, y=x[:-1])
    check_no_device_error()


def test_rows_out_of_the_ordinary():
    K = 384
    for dtype in ("fp32", "bf16"):
        x = torch.zeros(8, K, dtype=DTYPES[dtype])
        x[1] = 1e-30
        x[2] = 1e25
        x[3], x[3, 5] = 1.0, float("nan")
        x[4], x[4, 5] = 1.0, float("inf")
        x[5] = float(torch.finfo(DTYPES[dtype]).max)
        x[6, 7] = -3.0
        x[7] = -1e-38
        x = x.cuda()
        codes, scales, r = tq.tq_rms_norm_fp8(x, None, eps=1e-6)
        y, _, rstd = tq.tq_rms_norm(x, None, eps=1e-6)
        eps = float(np.float32(1e-6))
        with np.errstate(all="ignore"):
            want, want_rstd = B.rms_norm(_f64(x), None, eps)
        for i in (0, 1, 2, 5, 6, 7):
            assert np.abs(_f64(rstd)[i] - want_rstd[i, 0]) <= (U + 2.0 ** -40) * want_rstd[i, 0] + 2.0 ** -150
            assert np.all(np.abs(_f64(y)[i] - want[i]) <= (HALF[dtype] + 2.0 ** -20) * np.abs(want[i]) + 2.0 ** -140)
        assert torch.isnan(y[3]).all() and torch.isnan(y[4, 5]) and (y[4, :5] == 0).all()
        assert np.all(_f64(codes)[0] == 0) and np.all(_f64(scales)[0] == 0)
        assert np.isnan(_f64(codes)[3]).all()
        assert _f64(codes)[6, 7] == -448.0
        # without eps tiny rows count, down to those whose squares are no fp32 numbers
        tiny = torch.full((1, K), 3e-33, dtype=DTYPES[dtype], device="cuda")
        y1, _, _ = tq.tq_rms_norm(tiny, None, eps=0.0)
        assert torch.allclose(y1.float(), torch.ones(1, device="cuda"), rtol=4 * U, atol=0.0)
        # eps 0 and a row of zeros: 0 times infinity
        y0, _, rstd0 = tq.tq_rms_norm(x[:1], None, eps=0.0)
        assert torch.isinf(rstd0).all() and torch.isnan(y0).all()
    empty = torch.empty(0, 64, device="cuda")
    y, r, rstd = tq.tq_rms_norm(empty, None)
    assert y.shape == (0, 64) and rstd.shape == (0,)
    gx, gw = tq.tq_rms_norm_backward(empty, empty, torch.ones(64, device="cuda"), rstd)
    assert gx.shape == (0, 64) and (gw == 0).all()
    check_no_device_error()


def test_many_rows_repeat():
    """More rows than blocks of the gradient: the same bits every time, on another stream and from a graph."""
    rng = np.random.default_rng(5)
    n, K = 5000, 1024
    x, dy, w = _rows(rng, n, K, "bf16"), _rows(rng, n, K, "bf16"), _weight(rng, K, "fp32")
    _, _, rstd = tq.tq_rms_norm(x, w)
    gx, gw = tq.tq_rms_norm_backward(dy, x, w, rstd)
    _, want = B.rms_norm_grad(_f64(dy), _f64(x), _f64(w), float(np.float32(1e-6)))
    magnitudes = np.abs(_f64(dy) * _f64(x) * _f64(rstd)[:, None]).sum(0)
    assert np.all(np.abs(_f64(gw) - want) <= 128 * U * magnitudes)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    gx2, gw2 = tq.tq_rms_norm_backward(dy, x, w, rstd, stream=side)
    side.synchronize()
    assert torch.equal(gx, gx2) and torch.equal(gw, gw2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gx3, gw3 = tq.tq_rms_norm_backward(dy, x, w, rstd)
    for t in (gx3, gw3):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(gx, gx3) and torch.equal(gw, gw3)
    check_no_device_error()


def test_refusals():
    x, w = torch.zeros(4, 64, device="cuda"), torch.ones(64, device="cuda")
    with pytest.raises(ValueError):
        tq.tq_rms_norm(x, torch.ones(63, device="cuda"))
    with pytest.raises(TypeError):
        tq.tq_rms_norm(x, w, residual=x.half())
    with pytest.raises(ValueError):
        tq.tq_rms_norm(x, w, residual=x[:3])
    with pytest.raises(ValueError):
        tq.tq_rms_norm(x, w, residual_out=x)
    with pytest.raises(ValueError):
        tq.tq_rms_norm(x.t(), w)
    with pytest.raises(TypeError):
        tq.tq_rms_norm(x.double(), w)
    with pytest.raises(tq.TQError):
        tq.tq_rms_norm(x, w, eps=-1.0)
    with pytest.raises(tq.TQError):
        tq.tq_rms_norm(torch.zeros(1, 16400, device="cuda"))
    with pytest.raises(tq.TQError):
        tq.tq_rms_norm_fp8(torch.zeros(4, 72, device="cuda"))
    with pytest.raises(tq.TQError):
        tq.tq_rms_norm_fp8(torch.zeros(4, 65, device="cuda")[:, 1:])
    with pytest.raises(ValueError):
        tq.tq_rms_norm(x.cpu(), w)
    with pytest.raises(tq.TQError):
        tq.tq_rms_norm_backward(x, x, w, x[:, 0].contiguous(), workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
