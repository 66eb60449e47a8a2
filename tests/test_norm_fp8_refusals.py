"""What the norm, the 8-bit operators and the gated projection refuse, before any
device work: with no GPU present a bad size, type, option or alignment is reported as
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


def test_norm_refusals(tq):
    def call(x=A, dtype=1, stride=64, res=A, res_stride=64, w=A, w_type=0, eps=1e-6, n=4, K=64, r=A + 4096, y=A + 8192,
             rstd=A, codes=None, scales=None):
        return tq.lib().tq_rms_norm(x, dtype, stride, res, res_stride, w, w_type, eps, n, K, r, y, rstd, codes, scales,
                                    None)

    for bad in (dict(x=None), dict(dtype=3), dict(dtype=-1), dict(stride=63), dict(res_stride=63), dict(w_type=5),
                dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")), dict(n=-1), dict(n=1 << 31), dict(K=0),
                dict(K=16385, stride=16385, res_stride=16385), dict(r=None), dict(res=None), dict(y=None),
                dict(y=A + 4096), dict(codes=A), dict(scales=A), dict(x=A + 1), dict(w=A + 2), dict(rstd=A + 2),
                dict(codes=A + 8, scales=A), dict(codes=A, scales=A, K=72, stride=72, res_stride=72),
                dict(codes=A, scales=A, x=A + 2), dict(codes=A, scales=A, stride=65), dict(codes=A, scales=A, y=A + 2),
                dict(stride=1 << 60), dict(res_stride=1 << 60)):
        assert call(**bad) == INVALID, bad

    def back(dy=A, dy_stride=64, x=A, dtype=1, stride=64, w=A, w_type=0, rstd=A, g=A, g_stride=64, n=4, K=64, work=A,
             size=1 << 30, gx=A, gw=A):
        return tq.lib().tq_rms_norm_backward(dy, dy_stride, x, dtype, stride, w, w_type, rstd, g, g_stride, n, K, work,
                                             size, gx, gw, None)

    for bad in (dict(dy=None), dict(dy_stride=1), dict(x=None), dict(dtype=9), dict(stride=0), dict(w=None), dict(w_type=-1),
                dict(rstd=None), dict(g_stride=63), dict(n=-1), dict(K=20000, dy_stride=20000, stride=20000, g_stride=20000),
                dict(gx=None), dict(dy=A + 1), dict(gw=A + 2), dict(rstd=A + 1)):
        assert back(**bad) == INVALID, bad
    for bad in (dict(work=None), dict(work=A + 16), dict(size=16)):
        assert back(**bad) == WORKSPACE, bad
    assert tq.tq_rms_norm_backward_workspace_size(-1, 64) == 0 and tq.tq_rms_norm_backward_workspace_size(4, 0) == 0
    assert tq.tq_rms_norm_backward_workspace_size(4, 16385) == 0 and tq.tq_rms_norm_backward_workspace_size(0, 64) == 256


def test_quantize_refusals(tq):
    def call(x=A, dtype=1, stride=64, E=2, n=4, K=64, rows=1, codes=A, scales=A):
        return tq.lib().tq_fp8_quantize(x, dtype, stride, E, n, K, rows, codes, scales, None)

    for bad in (dict(x=None), dict(x=A + 8), dict(dtype=7), dict(stride=48), dict(stride=65), dict(E=-1), dict(n=-1),
                dict(n=1 << 31), dict(E=1 << 20, n=1 << 20), dict(K=0), dict(K=8), dict(K=72, stride=72), dict(rows=0),
                dict(rows=2), dict(rows=64), dict(codes=None), dict(codes=A + 8), dict(scales=None), dict(scales=A + 2),
                dict(rows=128, E=65536), dict(rows=128, E=1, n=65536 * 128), dict(stride=1 << 60)):
        assert call(**bad) == INVALID, bad

    def back(codes=A, scales=A, E=2, n=4, K=64, rows=128, out=A, dtype=0):
        return tq.lib().tq_fp8_dequantize(codes, scales, E, n, K, rows, out, dtype, None)

    for bad in (dict(codes=None), dict(codes=A + 8), dict(scales=None), dict(n=-1), dict(K=40), dict(rows=7), dict(out=None),
                dict(out=A + 8), dict(dtype=3), dict(E=1 << 30, n=1 << 30)):
        assert back(**bad) == INVALID, bad


def test_product_refusals(tq):
    def linear(x=A, xs=A, w=A, ws=A, n=40, K=64, N=128, work=A, size=1 << 40, y=A, y_type=1):
        return tq.lib().tq_fp8_linear(x, xs, w, ws, n, K, N, work, size, y, y_type, None)

    for bad in (dict(x=None), dict(xs=None), dict(w=None), dict(ws=None), dict(y=None), dict(n=-1), dict(n=(1 << 31) - 1024),
                dict(K=0), dict(K=24), dict(N=0), dict(N=(1 << 31) - 1024), dict(y_type=3), dict(x=A + 8), dict(w=A + 8),
                dict(xs=A + 2), dict(ws=A + 2), dict(y=A + 1)):
        assert linear(**bad) == INVALID, bad
    assert tq.tq_fp8_linear_workspace_size(-1, 64, 64) == 0 and tq.tq_fp8_linear_workspace_size(4, 63, 64) == 0
    assert tq.tq_fp8_linear_workspace_size(4, 64, 0) == 0

    def moe(x=A, xs=A, w=A, ws=A, ids=A, tw=A, n=40, k=2, E=8, K=64, N=128, work=A, size=1 << 40, y=A, y_type=1):
        return tq.lib().tq_fp8_moe_forward(x, xs, w, ws, ids, tw, n, k, E, K, N, work, size, y, y_type, None)

    for bad in (dict(x=None), dict(ids=None), dict(tw=None), dict(n=-1), dict(k=0), dict(k=9), dict(E=0), dict(E=1025, k=33),
                dict(K=8), dict(N=0), dict(E=1024, N=1 << 21), dict(n=1 << 30), dict(y_type=-1), dict(w=A + 4),
                dict(y=A + 1), dict(ws=A + 1)):
        assert moe(**bad) == INVALID, bad
    for bad in (dict(work=None), dict(work=A + 64), dict(size=1000)):
        assert moe(**bad) == WORKSPACE, bad
    assert tq.tq_fp8_moe_workspace_size(4, 9, 8, 64, 64) == 0 and tq.tq_fp8_moe_workspace_size(1 << 30, 4, 8, 64, 64) == 0

    def mlp(x=A, gu=A, gus=A, down=A, downs=A, ids=A, tw=A, n=40, k=2, E=8, H=64, I=128, work=A, size=1 << 40, y=A, y_type=1):
        return tq.lib().tq_fp8_moe_mlp_forward(x, A, gu, gus, down, downs, ids, tw, n, k, E, H, I, work, size, y, y_type, None)

    for bad in (dict(I=64), dict(I=0), dict(I=130), dict(H=8), dict(H=72), dict(gu=None), dict(gus=None), dict(down=A + 8),
                dict(downs=None), dict(E=1024, I=1 << 21), dict(I=1 << 30), dict(y_type=4), dict(k=33, E=64)):
        assert mlp(**bad) == INVALID, bad
    assert mlp(work=None) == WORKSPACE and mlp(size=4096) == WORKSPACE
    assert tq.tq_fp8_moe_mlp_workspace_size(4, 2, 8, 64, 64) == 0


def test_gated_refusals(tq):
    def call(x=A, dtype=1, stride=64, w=A, n=40, H=64, I=32, work=A, size=1 << 40, h=A, gu=None):
        return tq.lib().tq_swiglu_linear(x, dtype, stride, w, n, H, I, work, size, h, gu, None)

    for bad in (dict(x=None), dict(x=A + 8), dict(dtype=0), dict(dtype=3), dict(stride=60), dict(stride=66), dict(stride=1 << 39),
                dict(w=None), dict(w=A + 2), dict(n=-1), dict(n=(1 << 31) - 1), dict(H=4), dict(H=68, stride=72), dict(I=0),
                dict(I=12), dict(I=1 << 30), dict(h=None), dict(h=A + 8), dict(gu=A + 4)):
        assert call(**bad) == INVALID, bad

    def back(x=A, dtype=1, stride=64, w=A, gu=A, gh=A, n=40, H=64, I=32, work=A, size=1 << 40, gx=A, gw=A):
        return tq.lib().tq_swiglu_linear_backward(x, dtype, stride, w, gu, gh, n, H, I, work, size, gx, gw, None)

    for bad in (dict(x=None), dict(dtype=0), dict(stride=56), dict(w=None), dict(gu=A + 8), dict(gh=None), dict(gh=A + 2),
                dict(n=-1), dict(H=12), dict(I=4), dict(gx=None, gw=None), dict(gx=A + 8), dict(gw=A + 8)):
        assert back(**bad) == INVALID, bad
    for bad in (dict(work=None), dict(work=A + 128), dict(size=100)):
        assert back(**bad) == WORKSPACE, bad
    assert tq.tq_swiglu_linear_workspace_size(4, 12, 8) == 0
    assert tq.tq_swiglu_linear_backward_workspace_size(4, 12, 8) == 0
