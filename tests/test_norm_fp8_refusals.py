"""What the norm, the 8-bit operators and the gated projection refuse, before any
device work: with no GPU present a bad size, type, option or alignment is reported as
such (the addresses below are never dereferenced)."""
import pytest

INVALID, WORKSPACE = -1, -8
A = 0x10000            # 256-byte aligned stand-in addresses, far apart
B, C, D = A + (1 << 42), A + (1 << 44), A + (1 << 46)


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
                dict(y=A + 4096), dict(codes=B), dict(scales=A), dict(x=A + 1), dict(w=A + 2), dict(rstd=A + 2),
                dict(codes=B + 8, scales=A), dict(codes=B, scales=A, K=72, stride=72, res_stride=72),
                dict(codes=B, scales=A, x=A + 2), dict(codes=B, scales=A, stride=65), dict(codes=B, scales=A, y=A + 2),
                dict(stride=1 << 60), dict(res_stride=1 << 60),
                # over rows: not from their start, not as dense as they are; over another output
                dict(y=A + 16), dict(y=A, stride=72), dict(r=A, stride=128), dict(r=A + 128), dict(res=B, y=B + 256),
                dict(res=B, res_stride=80, r=B), dict(y=C, r=C + 511), dict(y=C + 511, r=C), dict(codes=A, scales=D),
                dict(codes=A + 8192 + 16, scales=D), dict(codes=A + 4096 + 256, scales=D),
                dict(res=B, codes=B + 256, scales=D)):
        assert call(**bad) == INVALID, bad

    def back(dy=A, dy_stride=64, x=A, dtype=1, stride=64, w=A, w_type=0, rstd=A, g=A, g_stride=64, n=4, K=64, work=A,
             size=1 << 30, gx=A, gw=A):
        return tq.lib().tq_rms_norm_backward(dy, dy_stride, x, dtype, stride, w, w_type, rstd, g, g_stride, n, K, work,
                                             size, gx, gw, None)

    for bad in (dict(dy=None), dict(dy_stride=1), dict(x=None), dict(dtype=9), dict(stride=0), dict(w=None), dict(w_type=-1),
                dict(rstd=None), dict(g_stride=63), dict(n=-1), dict(K=20000, dy_stride=20000, stride=20000, g_stride=20000),
                dict(gx=None), dict(dy=A + 1), dict(gw=A + 2), dict(rstd=A + 1), dict(x=B, gx=B + 128), dict(dy=B, gx=B + 256),
                dict(g=B, gx=B - 256), dict(g=B, g_stride=66, gx=B), dict(dy=C, dy_stride=128, gx=C)):
        assert back(**bad) == INVALID, bad
    for bad in (dict(work=None), dict(work=A + 16), dict(size=16)):
        assert back(**bad) == WORKSPACE, bad
    assert tq.tq_rms_norm_backward_workspace_size(-1, 64) == 0 and tq.tq_rms_norm_backward_workspace_size(4, 0) == 0
    assert tq.tq_rms_norm_backward_workspace_size(4, 16385) == 0 and tq.tq_rms_norm_backward_workspace_size(0, 64) == 256


def test_quantize_refusals(tq):
    def call(x=A, dtype=1, stride=64, E=2, n=4, K=64, rows=1, codes=B, scales=A):
        return tq.lib().tq_fp8_quantize(x, dtype, stride, E, n, K, rows, codes, scales, None)

    for bad in (dict(x=None), dict(x=A + 8), dict(dtype=7), dict(stride=48), dict(stride=65), dict(E=-1), dict(n=-1),
                dict(n=1 << 31), dict(E=1 << 20, n=1 << 20), dict(K=0), dict(K=8), dict(K=72, stride=72), dict(rows=0),
                dict(rows=2), dict(rows=64), dict(codes=None), dict(codes=B + 8), dict(scales=None), dict(scales=A + 2),
                dict(codes=A), dict(codes=A + 1008), dict(rows=128, E=65536), dict(rows=128, E=1, n=65536 * 128), dict(stride=1 << 60)):
        assert call(**bad) == INVALID, bad

    def back(codes=A, scales=A, E=2, n=4, K=64, rows=128, out=B, dtype=0):
        return tq.lib().tq_fp8_dequantize(codes, scales, E, n, K, rows, out, dtype, None)

    for bad in (dict(codes=None), dict(codes=A + 8), dict(scales=None), dict(n=-1), dict(K=40), dict(rows=7), dict(out=None),
                dict(out=B + 8), dict(out=A), dict(out=A + 496), dict(codes=B + 2032), dict(dtype=3), dict(E=1 << 30, n=1 << 30)):
        assert back(**bad) == INVALID, bad


def test_product_refusals(tq):
    def linear(x=A, xs=A, w=B, ws=A, n=40, K=64, N=128, work=A, size=1 << 40, y=C, y_type=1):
        return tq.lib().tq_fp8_linear(x, xs, w, ws, n, K, N, work, size, y, y_type, None)

    for bad in (dict(x=None), dict(xs=None), dict(w=None), dict(ws=None), dict(y=None), dict(n=-1), dict(n=(1 << 31) - 1024),
                dict(K=0), dict(K=24), dict(N=0), dict(N=(1 << 31) - 1024), dict(y_type=3), dict(x=A + 8), dict(w=B + 8),
                dict(xs=A + 2), dict(ws=A + 2), dict(y=C + 1), dict(y=A), dict(y=A + 2558), dict(y=B + 8190), dict(y=B - 2)):
        assert linear(**bad) == INVALID, bad
    assert tq.tq_fp8_linear_workspace_size(-1, 64, 64) == 0 and tq.tq_fp8_linear_workspace_size(4, 63, 64) == 0
    assert tq.tq_fp8_linear_workspace_size(4, 64, 0) == 0

    def moe(x=A, xs=A, w=B, ws=A, ids=A, tw=A, n=40, k=2, E=8, K=64, N=128, work=A, size=1 << 40, y=C, y_type=1):
        return tq.lib().tq_fp8_moe_forward(x, xs, w, ws, ids, tw, n, k, E, K, N, work, size, y, y_type, None)

    for bad in (dict(x=None), dict(ids=None), dict(tw=None), dict(n=-1), dict(k=0), dict(k=9), dict(E=0), dict(E=1025, k=33),
                dict(K=8), dict(N=0), dict(E=1024, N=1 << 21), dict(n=1 << 30), dict(y_type=-1), dict(w=B + 4),
                dict(y=C + 1), dict(ws=A + 1), dict(y=A), dict(y=B + 65534), dict(x=C + 10224)):
        assert moe(**bad) == INVALID, bad
    for bad in (dict(work=None), dict(work=A + 64), dict(size=1000)):   # of many tokens: sorted pairs and partial sums
        assert moe(n=4000, **bad) == WORKSPACE, bad
    assert tq.tq_fp8_moe_workspace_size(4, 9, 8, 64, 64) == 0 and tq.tq_fp8_moe_workspace_size(1 << 30, 4, 8, 64, 64) == 0

    def mlp(x=A, gu=B, gus=A, down=C, downs=A, ids=A, tw=A, n=40, k=2, E=8, H=64, I=128, work=A, size=1 << 40, y=D, y_type=1):
        return tq.lib().tq_fp8_moe_mlp_forward(x, A, gu, gus, down, downs, ids, tw, n, k, E, H, I, work, size, y, y_type, None)

    for bad in (dict(I=64), dict(I=0), dict(I=130), dict(H=8), dict(H=72), dict(gu=None), dict(gus=None), dict(down=C + 8),
                dict(y=A), dict(y=C + 65534), dict(downs=None), dict(E=1024, I=1 << 21), dict(I=1 << 30), dict(y_type=4), dict(k=33, E=64)):
        assert mlp(**bad) == INVALID, bad
    assert mlp(work=None) == WORKSPACE and mlp(size=4096) == WORKSPACE
    assert tq.tq_fp8_moe_mlp_workspace_size(4, 2, 8, 64, 64) == 0


def test_gated_refusals(tq):
    def call(x=A, dtype=1, stride=64, w=B, n=40, H=64, I=32, work=A, size=1 << 40, h=C, gu=None):
        return tq.lib().tq_swiglu_linear(x, dtype, stride, w, n, H, I, work, size, h, gu, None)

    for bad in (dict(x=None), dict(x=A + 8), dict(dtype=0), dict(dtype=3), dict(stride=60), dict(stride=66), dict(stride=1 << 39),
                dict(w=None), dict(w=B + 2), dict(n=-1), dict(n=(1 << 31) - 1), dict(H=4), dict(H=68, stride=72), dict(I=0),
                dict(I=12), dict(I=1 << 30), dict(h=None), dict(h=C + 8), dict(gu=D + 4), dict(h=A), dict(h=A + 39 * 128 + 112),
                dict(h=B + 4096), dict(gu=A), dict(gu=B - 16), dict(gu=C + 2544), dict(x=C + 2544)):
        assert call(**bad) == INVALID, bad

    def back(x=A, dtype=1, stride=64, w=B, gu=A, gh=A, n=40, H=64, I=32, work=A, size=1 << 40, gx=C, gw=D):
        return tq.lib().tq_swiglu_linear_backward(x, dtype, stride, w, gu, gh, n, H, I, work, size, gx, gw, None)

    for bad in (dict(x=None), dict(dtype=0), dict(stride=56), dict(w=None), dict(gu=A + 8), dict(gh=None), dict(gh=A + 2),
                dict(n=-1), dict(H=12), dict(I=4), dict(gx=None, gw=None), dict(gx=C + 8), dict(gw=D + 8), dict(gx=A),
                dict(gx=B), dict(gw=A + 16), dict(gw=B - 16), dict(gx=D + 8176), dict(gw=C + 5104)):
        assert back(**bad) == INVALID, bad
    for bad in (dict(work=None), dict(work=A + 128), dict(size=100)):
        assert back(**bad) == WORKSPACE, bad
    assert tq.tq_swiglu_linear_workspace_size(4, 12, 8) == 0
    assert tq.tq_swiglu_linear_backward_workspace_size(4, 12, 8) == 0


def test_tensors_of_another_device_are_refused(tq, monkeypatch):
    """Device 0 is current: a call with any one of its tensors on device 1 is refused before the library is called."""
    import torch

    from test_operator_limits import _OnDevice
    bf16, f32, i32, f8, u8 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn, torch.uint8
    for name, value in (("_torch_mod", torch), ("_common", None), ("_type_codes", None), ("_code_types", None),
                        ("_raw_stream_fn", lambda device: 0)):
        monkeypatch.setattr(tq, name, value)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    called = []
    monkeypatch.setattr(tq, "_calls", {name: (lambda *a, name=name: called.append(name) or 0) for name in tq._CALLS})
    monkeypatch.setattr(tq, "_workspace_bytes", lambda *a: 4096)
    n, E, k, K, N, I = 40, 8, 2, 256, 128, 128
    ids, tw, work = (i32, n, k), (f32, n, k), (u8, 1 << 20)
    calls = {
        "norm": (lambda a: tq.tq_rms_norm(a["x"], a["w"], 1e-6, a["res"], a["y"], a["r"], a["rstd"]),
                 dict(x=(bf16, n, K), w=(f32, K), res=(bf16, n, K), y=(bf16, n, K), r=(bf16, n, K), rstd=(f32, n))),
        "norm to 8 bits": (lambda a: tq.tq_rms_norm_fp8(a["x"], a["w"], 1e-6, a["res"], a["c"], a["s"], a["y"], a["r"]),
                           dict(x=(bf16, n, K), w=(f32, K), res=(bf16, n, K), c=(f8, n, K), s=(f32, n, 2), y=(bf16, n, K),
                                r=(bf16, n, K))),
        "norm backward": (lambda a: tq.tq_rms_norm_backward(a["dy"], a["x"], a["w"], a["rstd"], a["g"], a["gx"], a["gw"],
                                                            a["work"]),
                          dict(dy=(bf16, n, K), x=(bf16, n, K), w=(f32, K), rstd=(f32, n), g=(bf16, n, K), gx=(bf16, n, K),
                               gw=(f32, K), work=work)),
        "quantize": (lambda a: tq.tq_fp8_quantize(a["x"], 1, a["c"], a["s"]),
                     dict(x=(bf16, n, K), c=(f8, n, K), s=(f32, n, 2))),
        "dequantize": (lambda a: tq.tq_fp8_dequantize(a["c"], a["s"], 1, out=a["out"]),
                       dict(c=(f8, n, K), s=(f32, n, 2), out=(bf16, n, K))),
        "linear": (lambda a: tq.tq_fp8_linear(a["x"], a["xs"], a["w"], a["ws"], None, a["work"], a["y"]),
                   dict(x=(f8, n, K), xs=(f32, n, 2), w=(f8, N, K), ws=(f32, 1, 2), work=work, y=(bf16, n, N))),
        "experts": (lambda a: tq.tq_fp8_moe_forward(a["x"], a["xs"], a["w"], a["ws"], a["ids"], a["tw"], None, a["work"], a["y"]),
                    dict(x=(f8, n, K), xs=(f32, n, 2), w=(f8, E, N, K), ws=(f32, E, 1, 2), ids=ids, tw=tw, work=work,
                         y=(bf16, n, N))),
        "expert MLP": (lambda a: tq.tq_fp8_moe_mlp_forward(a["x"], a["xs"], a["gu"], a["gus"], a["d"], a["ds"], a["ids"],
                                                           a["tw"], None, a["work"], a["y"]),
                       dict(x=(f8, n, K), xs=(f32, n, 2), gu=(f8, E, 2 * I, K), gus=(f32, E, 2, 2), d=(f8, E, K, I),
                            ds=(f32, E, 2, 1), ids=ids, tw=tw, work=work, y=(bf16, n, K))),
        "gated": (lambda a: tq.tq_swiglu_linear(a["x"], a["w"], a["h"], a["gu"], a["work"]),
                  dict(x=(bf16, n, K), w=(bf16, 2 * I, K), h=(bf16, n, I), gu=(f32, n, 2 * I), work=work)),
        "gated backward": (lambda a: tq.tq_swiglu_linear_backward(a["x"], a["w"], a["gh"], a["gu"], a["gx"], a["gw"], a["work"]),
                           dict(x=(bf16, n, K), w=(bf16, 2 * I, K), gh=(bf16, n, I), gu=(f32, n, 2 * I), gx=(bf16, n, K),
                                gw=(bf16, 2 * I, K), work=work)),
    }
    for what, (call, args) in calls.items():
        make = lambda other: {name: _OnDevice(*spec, device=int(name == other)) for name, spec in args.items()}
        call(make(None))
        assert len(called) == 1, what
        called.clear()
        for name in args:
            with pytest.raises(ValueError, match="cuda:1"):
                call(make(name))
            assert not called, (what, name)
