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
