"""Gated projection and its gradients against the fp64 definition.

Tolerances.  gate and up: 16-bit products are exact in fp32; a sum of H of them is
accumulated with at most H roundings or truncations, in practice one per 16, of partial
sums below the sum of magnitudes: r = (H / 16 + 32) 2^-23 of it.  h = silu(gate) up: 1.1
|up| r G + |silu| r U, 8 x 2^-24 of itself for the activation, and the one rounding to
the type.  d = [dgate dup]: their fp32 errors by the slopes (silu' is below 1.1, its own
slope below 0.5) and half a step of the type; the two products add half a step of each
d they sum, (terms / 16 + 32) 2^-23 of the sums of magnitudes, 16 splits, and the
rounding of the result."""
import numpy as np
import pytest
import torch

import oracle.block_operators as B
import trellis_quantized_moe_sort_gb300 as tq
from gpu_util import check_no_device_error

pytestmark = pytest.mark.gpu
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
HALF = {k: torch.finfo(v).eps / 2 for k, v in DTYPES.items()}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from trellis_quantized_moe_sort_gb300 import build
    build.build()
    tq.tq_init(0)


def _problem(seed, n, H, I, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((n, H), device="cuda", generator=g).to(DTYPES[dtype])
    w = (torch.randn((2 * I, H), device="cuda", generator=g) / H ** 0.5).to(DTYPES[dtype])
    dh = torch.randn((n, I), device="cuda", generator=g).to(DTYPES[dtype])
    return x, w, dh


def _tiny(dtype):
    return float(torch.finfo(DTYPES[dtype]).tiny) * HALF[dtype] * 2


def _r(terms):
    return (terms / 16 + 32) * 2.0 ** -23


def _reference(x, w, dh, dtype):
    x, w, dh = x.double(), w.double(), dh.double()
    n, H = x.shape
    I = w.shape[0] // 2
    s, m = x @ w.t(), x.abs() @ w.abs().t()
    gate, up, G, U = s[:, :I], s[:, I:], m[:, :I], m[:, I:]
    sig = torch.sigmoid(gate)
    act, slope = gate * sig, sig * (1 + gate * (1 - sig))
    r = _r(H)
    h = act * up
    h_bound = 1.1 * up.abs() * r * G + act.abs() * r * U + (8 * 2.0 ** -24 + HALF[dtype]) * h.abs() + _tiny(dtype)
    d = torch.cat((dh * up * slope, dh * act), -1)
    e = torch.cat((dh.abs() * (r * U * 1.1 + up.abs() * 0.5 * r * G), dh.abs() * 1.1 * r * G), -1)
    # the fp32 arithmetic of d, by its terms, and its rounding to 16 bits
    e = e + 16 * 2.0 ** -24 * torch.cat((dh.abs() * up.abs() * (1 + gate.abs()), dh.abs() * gate.abs()), -1)
    e = e + HALF[dtype] * (d.abs() + e) + _tiny(dtype)
    gx, gw = d @ w, d.t() @ x
    gx_bound = e @ w.abs() + _r(2 * I) * ((d.abs() + e) @ w.abs()) + HALF[dtype] * gx.abs()
    gw_bound = e.t() @ x.abs() + _r(n) * ((d.abs() + e).t() @ x.abs()) + HALF[dtype] * gw.abs()
    return (h, h_bound), (gx, gx_bound * 1.01 + _tiny(dtype)), (gw, gw_bound * 1.01 + _tiny(dtype)), s, m


def _check(got, want):
    worst = ((got.double() - want[0]).abs() / want[1]).max().item()
    assert worst <= 1.0, worst


SIZES = [(1, 8, 8), (1, 64, 16), (2, 72, 24), (8, 256, 128), (9, 136, 40), (16, 1024, 264), (17, 64, 64), (33, 520, 72),
         (100, 256, 128), (128, 1032, 136), (130, 64, 520), (300, 512, 256), (513, 2048, 120), (1000, 136, 1000),
         (2050, 264, 72), (4000, 8, 8)]


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("n,H,I", SIZES)
def test_forward_and_gradients(n, H, I, dtype):
    x, w, dh = _problem(n + H + I, n, H, I, dtype)
    want_h, want_gx, want_gw, s, m = _reference(x, w, dh, dtype)
    h = tq.tq_swiglu_linear(x, w)
    assert h.dtype == x.dtype and h.shape == (n, I)
    _check(h, want_h)
    gate_up = torch.full((n, 2 * I), float("nan"), device="cuda")
    assert torch.equal(tq.tq_swiglu_linear(x, w, gate_up=gate_up), h)
    _check(gate_up, (s, _r(H) * m + 1e-30))
    gx, gw = tq.tq_swiglu_linear_backward(x, w, dh, gate_up=gate_up)
    assert gx.dtype == gw.dtype == x.dtype
    _check(gx, want_gx)
    _check(gw, want_gw)
    again = tq.tq_swiglu_linear_backward(x, w, dh)
    assert torch.equal(again[0], gx) and torch.equal(again[1], gw)
    check_no_device_error()


def test_gradient_is_the_oracles_and_a_difference():
    """Along a direction: the gradients' products with it are the loss's difference in fp64."""
    x, w, dh = _problem(5, 40, 64, 48, "fp16")
    gx, gw = tq.tq_swiglu_linear_backward(x, w, dh)
    f64 = lambda t: t.double().cpu().numpy()
    ox, ow, _ = B.gated_grad(f64(x), f64(w), f64(dh))
    rng = np.random.default_rng(5)
    ax, aw = rng.standard_normal(ox.shape), rng.standard_normal(ow.shape)
    step = 1e-5
    loss = lambda a, b: (B.gated(a, b)[0] * f64(dh)).sum()
    diff = (loss(f64(x) + step * ax, f64(w) + step * aw) - loss(f64(x) - step * ax, f64(w) - step * aw)) / (2 * step)
    assert abs(diff - (ox * ax).sum() - (ow * aw).sum()) <= 1e-5 * abs(diff) + 1e-4
    got = (f64(gx) * ax).sum() + (f64(gw) * aw).sum()
    # two roundings of 2^-11 of each element, added up over the direction
    room = 2.5 * 2.0 ** -11 * ((np.abs(ox) * np.abs(ax)).sum() + (np.abs(ow) * np.abs(aw)).sum())
    assert abs(got - diff) <= room


def test_strided_rows_and_one_gradient():
    big, w, dh = _problem(7, 200, 256, 64, "bf16")
    x = big[:, 64:192]
    w = w[:, :128].contiguous()
    h = tq.tq_swiglu_linear(x, w)
    assert torch.equal(h, tq.tq_swiglu_linear(x.contiguous(), w))
    a, b = tq.tq_swiglu_linear_backward(x, w, dh), tq.tq_swiglu_linear_backward(x.contiguous(), w, dh)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    few = big[:9, 64:192]
    assert torch.equal(tq.tq_swiglu_linear(few, w), tq.tq_swiglu_linear(few.contiguous(), w))
    check_no_device_error()


def test_large_values_and_no_rows():
    """Gates far from 0: silu is 0 or the gate itself, its slope 0 or 1, and nothing overflows on the way."""
    x = torch.full((20, 8), 30.0, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((16, 8), dtype=torch.bfloat16, device="cuda")
    w[0], w[1], w[8:] = 10.0, -10.0, 1.0
    dh = torch.ones((20, 8), dtype=torch.bfloat16, device="cuda")
    h = tq.tq_swiglu_linear(x, w)
    assert (h[:, 0] == 2400.0 * 240.0).all() and (h[:, 1:] == 0).all()
    gx, gw = tq.tq_swiglu_linear_backward(x, w, dh)
    assert torch.isfinite(gx).all() and torch.isfinite(gw).all()
    # dgate = up = 240 and dup = gate = 2400 of the first, dgate = up / 2 of the six zero gates (whose weights are 0)
    assert (gx == 2400.0 + 2400.0).all()
    h0 = tq.tq_swiglu_linear(x[:0], w)
    gx0, gw0 = tq.tq_swiglu_linear_backward(x[:0], w, dh[:0])
    assert h0.shape == (0, 8) and gx0.shape == (0, 8) and (gw0 == 0).all()
    check_no_device_error()


def test_rows_past_four_gigabytes():
    """gate_up of 4.9 GB: the last rows of every result are those of the rows alone."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of free device memory")
    n, H, I = 300_000, 64, 2048
    x, w, dh = _problem(13, n, H, I, "bf16")
    gate_up = torch.empty((n, 2 * I), device="cuda")
    h = tq.tq_swiglu_linear(x, w, gate_up=gate_up)
    gx, gw = tq.tq_swiglu_linear_backward(x, w, dh, gate_up=gate_up)
    for rows in (slice(0, 256), slice(n - 288, n)):
        want_h, want_gx, _, s, m = _reference(x[rows], w, dh[rows], "bf16")
        _check(h[rows], want_h)
        _check(gate_up[rows], (s, _r(H) * m + 1e-30))
        _check(gx[rows], want_gx)
    # the weights' gradient over all rows: added up in fp64 from slices
    want, bound = 0, 0
    for i in range(0, n, 30_000):
        _, _, part, _, _ = _reference(x[i:i + 30_000], w, dh[i:i + 30_000], "bf16")
        want, bound = want + part[0], bound + part[1]
    bound = bound + HALF["bf16"] * want.abs()
    # longer sums in fp32: n / 16 additions in place of 30000 / 16, of magnitudes below those that the slices' bounds hold
    assert ((gw.double() - want).abs() <= bound * (_r(n) / _r(30_000))).all()
    check_no_device_error()


def test_training_step_in_a_graph():
    """Forward and backward captured together replay to the same bits, also beside an eager call."""
    x, w, dh = _problem(9, 300, 256, 128, "bf16")

    def step():
        gate_up = torch.empty((300, 256), device="cuda")
        h = tq.tq_swiglu_linear(x, w, gate_up=gate_up)
        return (h, *tq.tq_swiglu_linear_backward(x, w, dh, gate_up=gate_up))

    want = step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    eager = step()
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, got, eager):
        assert torch.equal(a, b) and torch.equal(a, c)
    check_no_device_error()


def test_refusals():
    x, w, dh = _problem(1, 20, 64, 16, "bf16")
    for bad in (lambda: tq.tq_swiglu_linear(x.float(), w.float()), lambda: tq.tq_swiglu_linear(x, w.half()),
                lambda: tq.tq_swiglu_linear_backward(x, w, dh.half())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: tq.tq_swiglu_linear(x, w[:, :32]), lambda: tq.tq_swiglu_linear(x.t(), w),
                lambda: tq.tq_swiglu_linear(x, w[:31]), lambda: tq.tq_swiglu_linear_backward(x, w, dh[:3]),
                lambda: tq.tq_swiglu_linear(x, w, gate_up=torch.zeros(20, 16, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(tq.TQError):
        tq.tq_swiglu_linear(x[:, :60].contiguous(), w[:, :60].contiguous())
    with pytest.raises(tq.TQError):
        tq.tq_swiglu_linear(torch.zeros(4, 68, dtype=torch.bfloat16, device="cuda")[:, :64], w)
    with pytest.raises(tq.TQError):
        tq.tq_swiglu_linear_backward(x, w, dh, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
