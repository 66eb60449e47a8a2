"""Edges of the 8-bit and gated operators' number ranges: signs of zero, gates whose
exponential leaves fp32's range, scales and router weights far from 1, and gradients
asked for one at a time."""
import pytest
import torch

import trellis_quantized_moe_sort_gb300 as tq
from gpu_util import check_no_device_error

pytestmark = pytest.mark.gpu
BF16 = torch.finfo(torch.bfloat16).eps / 2


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from trellis_quantized_moe_sort_gb300 import build
    build.build()
    tq.tq_init(0)


def _ran(call, *kernels):
    """call's result, after checking that it launched these kernels."""
    before = tq.tq_launch_counts_all()
    result = call()
    after = tq.tq_launch_counts_all()
    for kernel in kernels:
        assert after[kernel] > before[kernel], kernel
    return result


# ------------------------------------------------------------------ codes

@pytest.mark.parametrize("dtype", (torch.float32, torch.bfloat16, torch.float16))
@pytest.mark.parametrize("rows", (1, 128))
def test_code_bytes_keep_the_sign_of_zero(dtype, rows):
    """The codes, as bytes, are torch's conversions of the quotients: -0 and negative values
    that round to 0 are 0x80, in blocks of ordinary and of extreme scales."""
    g = torch.Generator().manual_seed(3)
    most = 3e38 if dtype != torch.float16 else 6e4
    sizes = torch.tensor([1.0, 1e-3, 448.0, most, 1e-30 if dtype != torch.float16 else 1e-7, 3e-38, 1e-6, 1.0])
    # (a block of 128 x 128 has one size)
    x = torch.randn((256 * 8, 256), generator=g).clamp(-3, 3) / 3 * sizes.repeat_interleave(256)[:, None]
    x[:, ::5] = 0.0
    x[:, 1::5] = -0.0
    x[:, 2::7] *= 1e-4
    x = x.to(dtype).cuda()
    codes, scales = tq.tq_fp8_quantize(x, rows)
    wide = scales.repeat_interleave(rows, 0).repeat_interleave(128, 1)
    assert (wide == 0).sum().item() < wide.numel() // 2
    want = (x.float() / wide).to(torch.float8_e4m3fn).view(torch.uint8)
    want = torch.where(wide > 0, want, torch.zeros_like(want))   # no scale: all is 0
    got = codes.view(torch.uint8)
    assert torch.equal(got, want), (got != want).sum().item()
    assert (got == 0x80).any()
    check_no_device_error()


def test_norm_codes_keep_the_sign_of_zero():
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((9, 512), device="cuda", generator=g)
    x[:, ::3] = 0.0
    x[:, 1::3] *= torch.tensor(-0.0, device="cuda")   # zeros of both signs
    weight = torch.randn(512, device="cuda", generator=g)
    y = torch.empty_like(x)
    codes, scales, _ = tq.tq_rms_norm_fp8(x, weight, y=y)
    plain = tq.tq_fp8_quantize(y)
    assert torch.equal(scales, plain[1])
    want = (y / scales.repeat_interleave(128, 1)).to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(codes.view(torch.uint8), want) and torch.equal(plain[0].view(torch.uint8), want)
    assert (want == 0x80).any() and (want == 0).any()
    check_no_device_error()


# ------------------------------------------------------------------ gates

# Tolerance of h = g e u / (1 + e), e = exp(-|g|) for these gates: e is off by two of its own
# steps (2^-149 where it is subnormal), the other operations by 6 x 2^-24 together, and h is
# rounded once.
def _gated(gates, up):
    g = gates.double()
    e = torch.exp(g)
    h = g * e / (1 + e) * up
    return h, (2 * 2.0 ** -149 * g.abs() * up + 12 * 2.0 ** -24 * h.abs()), e


@pytest.mark.parametrize("n,H,I,kernels", [(4, 64, 64, ("few_rows",)), (128, 4096, 2048, ("gemm_f16", "swiglu_sum")),
                                           (1500, 64, 64, ("gemm_f16",))])
def test_gates_of_large_magnitude(n, H, I, kernels):
    """silu of gates around -88, whose exponential passes 2^126, is still a number: -5e-37, and
    with a large up projection an ordinary one."""
    up = 2.0 ** 40
    values = torch.arange(-94.0, -80.0, 0.5)   # each has 8 bits
    gates = values.repeat(I // len(values) + 1)[:I].cuda()
    x = torch.zeros((n, H), dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1.0
    w = torch.zeros((2 * I, H), dtype=torch.bfloat16, device="cuda")
    w[:I, 0], w[I:, 0] = gates.to(torch.bfloat16), up
    want, bound, e = _gated(gates, up)
    gate_up = torch.empty((n, 2 * I), device="cuda")
    h = _ran(lambda: tq.tq_swiglu_linear(x, w, gate_up=gate_up), *kernels)
    assert torch.equal(gate_up[:, :I], gates.expand(n, I)) and (gate_up[:, I:] == up).all()
    assert ((h.double() - want).abs() <= bound + BF16 * want.abs()).all()
    # d = [dgate dup] by grad_w of a single row (the others' dh is 0): x is 1 in its first column
    dh = torch.zeros((n, I), dtype=torch.bfloat16, device="cuda")
    dh[0] = 1.0
    _, grad_w = _ran(lambda: tq.tq_swiglu_linear_backward(x, w, dh, gate_up=gate_up), "swiglu_grad")
    g, s = gates.double(), e / (1 + e)
    d = torch.cat((up * s * (1 + g * (1 - s)), g * s))
    wide = torch.cat((2 * 2.0 ** -149 * up * (1 + g.abs()), 2 * 2.0 ** -149 * g.abs())) + 16 * 2.0 ** -24 * d.abs()
    # the product reads d rounded to the type, and is rounded itself (to bf16's smallest step at least)
    assert ((grad_w[:, 0].double() - d).abs() <= wide + 2.01 * BF16 * d.abs() + 2.0 ** -133).all()
    assert (grad_w[:, 1:] == 0).all()
    check_no_device_error()


@pytest.mark.parametrize("n,kernel", [(1, "few_rows"), (2048, "fp8_gemm")])
def test_expert_gates_of_large_magnitude(n, kernel):
    """The same in 8 bits: gates of -88 and around it, one to each block of 128."""
    H, I, up = 256, 512, 448.0 * 2.0 ** 30
    x = torch.zeros((n, H), dtype=torch.float8_e4m3fn, device="cuda").view(torch.uint8)
    x[:, 0] = 0x38   # 1
    x_scales = torch.ones((n, 2), device="cuda")
    w_gu = torch.zeros((1, 2 * I, H), dtype=torch.uint8, device="cuda")
    w_gu[0, :I, 0] = torch.tensor(-88.0).to(torch.float8_e4m3fn).view(torch.uint8).item()
    w_gu[0, I:, 0] = 0x7e   # 448
    gu_scales = torch.ones((1, 8, 2), device="cuda")
    gu_scales[0, :4, 0] = torch.tensor([0.995, 1.0, 1.003, 1.006], device="cuda")
    gu_scales[0, 4:] = 2.0 ** 30
    # y[j] = h of column 128 j, for j < 4
    w_down = torch.zeros((1, H, I), dtype=torch.uint8, device="cuda")
    for j in range(4):
        w_down[0, j, 128 * j] = 0x38
    down_scales = torch.ones((1, 2, 4), device="cuda")
    ids = torch.zeros((n, 1), dtype=torch.int32, device="cuda")
    y = _ran(lambda: tq.tq_fp8_moe_mlp_forward(x, x_scales, w_gu, gu_scales, w_down, down_scales, ids,
                                               torch.ones((n, 1), device="cuda"), dtype=torch.float32), kernel)
    # h is the largest of its block: code 448, scale h / 448 rounded, and their product rounded
    gates = (-88.0 * gu_scales[0, :4, 0].double()).float()
    want, bound, _ = _gated(gates, up)
    # (the gate is rounded to 2^-24 of itself, by which h moves 88 times as much)
    assert ((y[:, :4].double() - want).abs() <= bound + (4 + 90) * 2.0 ** -24 * want.abs()).all()
    assert (y[:, 4:] == 0).all()
    check_no_device_error()


# ------------------------------------------------------------------ router weights

@pytest.mark.parametrize("x_exp,w_exp,weight_exp", [(-50, -60, -30), (40, 60, -110), (-100, 120, 10), (100, -120, -10),
                                                    (0, 0, 0)])
@pytest.mark.parametrize("n,E,kernel", [(2, 64, "few_rows"), (2048, 4, "fp8_gemm")])
def test_scales_and_router_weights_far_from_one(n, E, kernel, x_exp, w_exp, weight_exp):
    """The scales' product is in fp32's range, and so are W x of each expert and the result: a
    router weight that takes one of the scales out of that range changes nothing."""
    K, N, top_k = 400, 48, 2
    g = torch.Generator(device="cuda").manual_seed(8)
    codes = lambda *s: (100.0 * torch.randn(s, device="cuda", generator=g)).clamp(-448, 448).to(torch.float8_e4m3fn)
    x, w = codes(n, K), codes(E, N, K)
    x_scales = torch.full((n, 4), 2.0 ** x_exp, device="cuda")
    w_scales = torch.full((E, 1, 4), 2.0 ** w_exp, device="cuda")
    ids = (torch.arange(n * top_k, device="cuda", dtype=torch.int32) % E).view(n, top_k)
    topk_w = (1 + torch.rand((n, top_k), device="cuda", generator=g)) * 2.0 ** weight_exp
    y = _ran(lambda: tq.tq_fp8_moe_forward(x, x_scales, w, w_scales, ids, topk_w, dtype=torch.float32), kernel)
    scale = 2.0 ** (x_exp + w_exp)
    picked = w.double()[ids.long()]   # [n, top_k, N, K]
    want = torch.einsum("nk,nj,njrk->nr", x.double(), topk_w.double(), picked) * scale
    size = torch.einsum("nk,nj,njrk->nr", x.double().abs(), topk_w.double(), picked.abs()) * scale
    # a block of 128 in any order, four blocks, two pairs and their weights; results near the smallest normal number
    bound = (160 + 4 + 6) * 2.0 ** -23 * size + 8 * 2.0 ** -149
    assert want.abs().max() > 2.0 ** -126
    assert ((y.double() - want).abs() <= bound).all()
    check_no_device_error()


# ------------------------------------------------------------------ workspaces

def test_results_in_a_used_workspace_are_refused():
    """Where K is split the partial sums are read while results are written."""
    g = torch.Generator(device="cuda").manual_seed(2)
    n, K, N = 300, 4096, 256
    x, x_scales = tq.tq_fp8_quantize(torch.randn((n, K), device="cuda", generator=g))
    w, w_scales = tq.tq_fp8_quantize(torch.randn((N, K), device="cuda", generator=g), 128)
    size = tq.tq_fp8_linear_workspace_size(n, K, N)
    assert size > 256
    work = torch.empty(size, dtype=torch.uint8, device="cuda")
    y = tq.tq_fp8_linear(x, x_scales, w, w_scales, workspace=work)
    inside = work[:2 * n * N].view(torch.bfloat16).view(n, N)
    with pytest.raises(tq.TQError):
        tq.tq_fp8_linear(x, x_scales, w, w_scales, workspace=work, y=inside)
    assert torch.equal(y, tq.tq_fp8_linear(x, x_scales, w, w_scales))
    n, H, I = 128, 4096, 2048
    x = torch.randn((n, H), device="cuda", generator=g).bfloat16()
    w = (torch.randn((2 * I, H), device="cuda", generator=g) / H ** 0.5).bfloat16()
    size = tq.tq_swiglu_linear_workspace_size(n, H, I)
    assert size > 256
    work = torch.empty(size, dtype=torch.uint8, device="cuda")
    with pytest.raises(tq.TQError):
        tq.tq_swiglu_linear(x, w, h=work[:2 * n * I].view(torch.bfloat16).view(n, I), workspace=work)
    assert torch.equal(tq.tq_swiglu_linear(x, w, workspace=work), tq.tq_swiglu_linear(x, w))
    check_no_device_error()


def test_one_workspace_for_batches_of_many_sizes():
    """Sizes asked for each batch: a smaller batch can need more (K split), and the largest
    serves them all."""
    g = torch.Generator(device="cuda").manual_seed(6)
    K, N, batches = 4096, 256, (1, 40, 300, 1000, 8000)
    w, w_scales = tq.tq_fp8_quantize(torch.randn((N, K), device="cuda", generator=g), 128)
    sizes = [tq.tq_fp8_linear_workspace_size(n, K, N) for n in batches]
    assert max(sizes) > sizes[-1]
    work = torch.empty(max(sizes), dtype=torch.uint8, device="cuda")
    for n, size in zip(batches, sizes):
        x, x_scales = tq.tq_fp8_quantize(torch.randn((n, K), device="cuda", generator=g))
        want = tq.tq_fp8_linear(x, x_scales, w, w_scales)
        assert torch.equal(tq.tq_fp8_linear(x, x_scales, w, w_scales, workspace=work), want)
        if size > 256:
            with pytest.raises(tq.TQError):
                tq.tq_fp8_linear(x, x_scales, w, w_scales, workspace=work[:size - 256])
    H, I, batches = 4096, 2048, (1, 128, 2000)
    w = (torch.randn((2 * I, H), device="cuda", generator=g) / H ** 0.5).bfloat16()
    sizes = [tq.tq_swiglu_linear_workspace_size(n, H, I) for n in batches]
    assert max(sizes) > sizes[-1]
    work = torch.empty(max(sizes), dtype=torch.uint8, device="cuda")
    for n in batches:
        x = torch.randn((n, H), device="cuda", generator=g).bfloat16()
        assert torch.equal(tq.tq_swiglu_linear(x, w, workspace=work), tq.tq_swiglu_linear(x, w))
    check_no_device_error()


# ------------------------------------------------------------------ one gradient alone

def _ptr(t):
    return None if t is None else t.data_ptr()


@pytest.mark.parametrize("n,H,I", [(20, 64, 16), (300, 512, 256), (1000, 136, 1000)])
@pytest.mark.parametrize("keep", (True, False))
def test_one_gradient_of_the_gated_projection(n, H, I, keep):
    """A C caller leaves out either gradient: the other has the same bits."""
    g = torch.Generator(device="cuda").manual_seed(n)
    x = torch.randn((n, H), device="cuda", generator=g).bfloat16()
    w = (torch.randn((2 * I, H), device="cuda", generator=g) / H ** 0.5).bfloat16()
    dh = torch.randn((n, I), device="cuda", generator=g).bfloat16()
    gate_up = None
    if keep:
        gate_up = torch.empty((n, 2 * I), device="cuda")
        tq.tq_swiglu_linear(x, w, gate_up=gate_up)
    want = tq.tq_swiglu_linear_backward(x, w, dh, gate_up=gate_up)
    size = tq.tq_swiglu_linear_backward_workspace_size(n, H, I, keep)
    for which in (0, 1):
        out = torch.full_like(want[which], float("nan"))
        work = torch.empty(size, dtype=torch.uint8, device="cuda")
        grads = (out, None) if which == 0 else (None, out)
        rc = tq.lib().tq_swiglu_linear_backward(_ptr(x), 1, H, _ptr(w), _ptr(gate_up), _ptr(dh), n, H, I, _ptr(work), size,
                                                _ptr(grads[0]), _ptr(grads[1]), torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        assert torch.equal(out, want[which])
    check_no_device_error()


@pytest.mark.parametrize("n,K", [(5, 144), (300, 2048), (200, 1023), (160, 12304)])
def test_norm_gradient_without_the_weights(n, K):
    """Without grad_weight, and without a workspace, grad_x has the same bits."""
    g = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randn((n, K), device="cuda", generator=g).bfloat16()
    dy = torch.randn((n, K), device="cuda", generator=g).bfloat16()
    weight = torch.randn(K, device="cuda", generator=g)
    _, _, rstd = tq.tq_rms_norm(x, weight)
    want, _ = tq.tq_rms_norm_backward(dy, x, weight, rstd)
    out = torch.full_like(want, float("nan"))
    rc = tq.lib().tq_rms_norm_backward(_ptr(dy), K, _ptr(x), 1, K, _ptr(weight), 0, _ptr(rstd), None, 0, n, K, None, 0,
                                       _ptr(out), None, torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    assert torch.equal(out, want)
    check_no_device_error()
