"""What the scored router and the 4-bit operators refuse, before any device
work: with no GPU present a bad size, type, option or alignment is reported as
such (the addresses below are never dereferenced)."""
import pytest

INVALID, WORKSPACE = -1, -8
A = 0x10000            # 256-byte aligned stand-in address


@pytest.fixture(scope="module")
def tq():
    from trellis_quantized_moe_sort_gb300 import build
    build.build()
    import trellis_quantized_moe_sort_gb300 as tq
    return tq


def test_router_refusals(tq):
    def call(logits=A, dtype=0, stride=64, n=4, E=64, k=6, score=1, groups=8, top_groups=4, ids=A, w=A):
        return tq.lib().tq_router_scored(logits, dtype, stride, None, n, E, k, score, groups, top_groups, 1, 1.0, ids, w,
                                         None)

    for bad in (dict(dtype=3), dict(dtype=-1), dict(stride=63), dict(n=-1), dict(E=0), dict(E=1025, stride=1025),
                dict(k=0), dict(k=33), dict(score=2), dict(groups=0), dict(groups=7), dict(groups=64, top_groups=8),
                dict(top_groups=0), dict(top_groups=9), dict(k=9, top_groups=1), dict(logits=None), dict(ids=None),
                dict(w=None), dict(n=1 << 31)):
        assert call(**bad) == INVALID, bad

    def back(dtype=0, stride=64, n=4, E=64, k=6, score=1, grad=A, out=A):
        return tq.lib().tq_router_scored_backward(A, dtype, stride, A, A, grad, n, E, k, score, 1, 1.0, out, None)

    for bad in (dict(dtype=3), dict(stride=63), dict(n=-1), dict(E=2000, stride=2000), dict(k=65), dict(score=-1),
                dict(grad=None), dict(out=None)):
        assert back(**bad) == INVALID, bad


def test_quantize_refusals(tq):
    def call(x=A, dtype=1, stride=64, n=4, K=64, fmt=0, g=None, packed=A, scales=A):
        return tq.lib().tq_fp4_quantize(x, dtype, stride, n, K, fmt, g, packed, scales, None)

    for bad in (dict(dtype=9), dict(stride=32), dict(stride=65), dict(n=-1), dict(K=0), dict(K=48), dict(K=16), dict(fmt=2),
                dict(fmt=1, g=A), dict(x=None), dict(x=A + 8), dict(packed=None), dict(packed=A + 4), dict(scales=None)):
        assert call(**bad) == INVALID, bad

    def back(packed=A, scales=A, n=4, K=64, fmt=0, g=None, out=A, dtype=0):
        return tq.lib().tq_fp4_dequantize(packed, scales, n, K, fmt, g, out, dtype, None)

    for bad in (dict(packed=None), dict(packed=A + 2), dict(scales=None), dict(n=-1), dict(K=40), dict(fmt=-1),
                dict(fmt=1, g=A), dict(out=None), dict(out=A + 8), dict(dtype=3)):
        assert back(**bad) == INVALID, bad
    assert tq.tq_fp4_tiled_scales_size(0, 1, 32) == 0 and tq.tq_fp4_tiled_scales_size(1, 1, 33) == 0
    assert tq.tq_fp4_tiled_scales_size(1, 1, 32, tq.FP4_NV) == 2048 and tq.tq_fp4_tiled_scales_size(1, 1, 32, tq.FP4_MX) == 1024
    assert tq.tq_fp4_tiled_scales_size(3, 129, 257 * 32, tq.FP4_NV) == 3 * 256 * (33 * 256 // 16)
    assert tq.lib().tq_fp4_tile_scales(None, 1, 1, 32, 0, A, None) == INVALID
    assert tq.lib().tq_fp4_tile_scales(A, 1, 1, 32, 0, A + 8, None) == INVALID


def test_product_refusals(tq):
    def linear(x=A, dtype=1, stride=64, packed=A, tiled=A, fmt=0, ws=None, n=40, K=64, N=128, work=A, size=1 << 30, y=A,
               y_type=1):
        return tq.lib().tq_fp4_linear(x, dtype, stride, packed, tiled, fmt, ws, None, n, K, N, work, size, y, y_type, None)

    for bad in (dict(x=None), dict(x=A + 8), dict(dtype=7), dict(stride=60), dict(packed=None), dict(packed=A + 8),
                dict(tiled=None), dict(tiled=A + 8), dict(fmt=3), dict(fmt=1, ws=A), dict(n=-1), dict(K=100), dict(N=0),
                dict(y=None), dict(y=A + 1), dict(y_type=5), dict(n=1 << 31)):
        assert linear(**bad) == INVALID, bad
    big = dict(n=200, K=4096, N=4096, stride=4096)
    need = tq.tq_fp4_linear_workspace_size(200, 4096, 4096)
    assert linear(**big, size=need - 1) == WORKSPACE
    assert linear(**big, work=None) == WORKSPACE and linear(**big, work=A + 128) == WORKSPACE

    def moe(n=40, k=6, E=64, K=64, N=128, fmt=0, ids=A, w=A, work=A, size=1 << 30, y=A):
        return tq.lib().tq_fp4_moe_forward(A, 1, K, A, A, fmt, None, None, ids, w, n, k, E, K, N, work, size, y, 1, None)

    for bad in (dict(n=-1), dict(k=0), dict(k=65), dict(k=33), dict(E=0), dict(E=1025), dict(K=36), dict(N=0), dict(fmt=2),
                dict(ids=None), dict(w=None), dict(y=None)):
        assert moe(**bad) == INVALID, bad
    big = dict(n=500, K=4096, N=2048)
    need = tq.tq_fp4_moe_workspace_size(500, 6, 64, 4096, 2048)
    assert moe(**big, size=need - 1) == WORKSPACE and moe(**big, work=None) == WORKSPACE

    def mlp(n=40, k=6, E=64, H=128, I=64, fmt=0, down=A, work=A, size=1 << 34, y=A):
        return tq.lib().tq_fp4_moe_mlp_forward(A, 1, H, A, A, None, down, A, None, fmt, None, None, A, A, n, k, E, H, I,
                                               work, size, y, 1, None)

    for bad in (dict(n=-1), dict(k=33), dict(E=1025), dict(H=100), dict(I=48), dict(I=0), dict(fmt=2), dict(down=None),
                dict(down=A + 4), dict(y=None)):
        assert mlp(**bad) == INVALID, bad
    assert mlp(size=tq.tq_fp4_moe_mlp_workspace_size(40, 6, 64, 128, 64) - 1) == WORKSPACE
    assert mlp(work=None) == WORKSPACE
    for size in (tq.tq_fp4_linear_workspace_size(-1, 64, 1), tq.tq_fp4_linear_workspace_size(1, 65, 1),
                 tq.tq_fp4_moe_workspace_size(4, 9, 8, 64, 64), tq.tq_fp4_moe_mlp_workspace_size(4, 2, 8, 64, 30),
                 tq.tq_fp4_moe_workspace_size(4, 2, 8, 64, 64, 7)):
        assert size == 0


def test_binding_refuses_without_a_gpu(tq):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a CUDA device is present")
    with pytest.raises(RuntimeError, match="needs a CUDA device"):
        tq.tq_router_scored(torch.zeros(4, 8), 2)
    with pytest.raises(RuntimeError, match="needs a CUDA device"):
        tq.tq_fp4_quantize(torch.zeros(4, 32))


def test_short_calls_take_the_headers_arguments(tq):
    """The C wrappers of the binding: each takes the arguments the header
    declares, in kind and number (a float where it declares one, no text, no
    integer past an int), and refuses others before the library is called."""
    import os
    import re
    tq.lib()
    header = open(os.path.join(os.path.dirname(tq.__file__), "..", "include", "tqmoe.h")).read()
    header = re.sub(r"/\*.*?\*/", "", header, flags=re.S)
    for name in tq._CALLS:
        call = tq._call(name)
        args = re.search(name + r"\s*\(([^;]*)\);", header, re.S).group(1).split(",")
        # as many zeros as arguments: refused by the library, not by the wrapper
        zeros = [None if "*" in a or "tq_stream_t" in a else 0.0 if "float" in a else 0 for a in args]
        assert call(*zeros) == INVALID, name
        if type(call).__name__ != "builtin_function_or_method":
            continue
        with pytest.raises(TypeError):
            call(*zeros[:-1])
        for k, a in enumerate(args):
            wrong = list(zeros)
            wrong[k] = "text"
            with pytest.raises(TypeError):
                call(*wrong)
            if "*" not in a and "tq_stream_t" not in a and "float" not in a:
                wrong[k] = 1 << 40
                if "int64" in a or "size_t" in a:
                    assert call(*wrong) == INVALID
                else:
                    with pytest.raises(OverflowError):
                        call(*wrong)


def test_sizes_past_a_size_t_are_refused(tq):
    """Rows x N values whose fp32 partial sums need 2^63 bytes or more."""
    big = 1 << 30
    assert tq.lib().tq_fp4_linear_workspace_size(big, 32, big, 0) == 0
    assert tq.lib().tq_fp4_linear(A, 1, 32, A, A, 0, None, None, big, 32, big, A, 1 << 20, A, 1, None) == INVALID
    assert tq.lib().tq_fp4_moe_workspace_size(big, 1, 1, 32, big, 0) == 0
    assert tq.lib().tq_fp4_moe_forward(A, 1, 32, A, A, 0, None, None, A, A, big, 1, 1, 32, big, A, 1 << 20, A, 1,
                                       None) == INVALID
    assert tq.lib().tq_fp4_moe_mlp_workspace_size(big, 1, 1, 32, 1 << 28, 0) == 0
    assert tq.lib().tq_fp4_linear_workspace_size(big, 32, 1 << 20, 0) > 1 << 35   # within it
