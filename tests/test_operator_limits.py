"""What the scored router and the 4-bit operators do at the ends of their
arguments' ranges, and their binding apart from any device: no GPU is needed."""
import os
import subprocess
import sys

import pytest

INVALID = -1
A = 0x10000            # 256-byte aligned stand-in address, never dereferenced


@pytest.fixture(scope="module")
def tq():
    from trellis_quantized_moe_sort_gb300 import build
    build.build()
    import trellis_quantized_moe_sort_gb300 as tq
    return tq


# n * top_k is 2^64 or a multiple of it for each of these, 0 in 64 bits
@pytest.mark.parametrize("n,k", [(1 << 62, 4), (1 << 60, 16), (1 << 59, 32), (3 << 61, 8)])
def test_pairs_that_wrap_are_refused(tq, n, k):
    lib = tq.lib()
    assert n * k % (1 << 64) == 0 and n < 1 << 63
    assert lib.tq_router_scored(A, 0, 64, None, n, 64, k, 1, 1, 1, 1, 1.0, A, A, None) == INVALID
    assert lib.tq_router_scored_backward(A, 0, 64, A, A, A, n, 64, k, 1, 1, 1.0, A, None) == INVALID
    assert lib.tq_fp4_moe_workspace_size(n, k, 64, 64, 64, 0) == 0
    assert lib.tq_fp4_moe_mlp_workspace_size(n, k, 64, 64, 64, 0) == 0
    assert lib.tq_fp4_moe_forward(A, 1, 64, A, A, 0, None, None, A, A, n, k, 64, 64, 64, A, 1 << 30, A, 1, None) == INVALID
    assert lib.tq_fp4_moe_mlp_forward(A, 1, 64, A, A, None, A, A, None, 0, None, None, A, A, n, k, 64, 64, 64, A, 1 << 30,
                                      A, 1, None) == INVALID


def test_values_that_wrap_are_refused(tq):
    lib = tq.lib()
    n = 1 << 59                # times 32 values of 4 bytes, 0 in 64 bits
    assert lib.tq_fp4_quantize(A, 0, 32, n, 32, 0, None, A, A, None) == INVALID
    assert lib.tq_fp4_dequantize(A, A, n, 32, 0, None, A, 0, None) == INVALID
    # rows 2^62 elements apart: the second one's address wraps
    assert lib.tq_fp4_quantize(A, 0, 1 << 62, 2, 32, 0, None, A, A, None) == INVALID
    assert lib.tq_fp4_linear(A, 0, 1 << 62, A, A, 0, None, None, 2, 32, 32, None, 0, A, 0, None) == INVALID


def test_longest_rows(tq):
    """K up to the largest multiple of 32 that an int holds: sizes grow with it and do not wrap."""
    longest = (1 << 31) - 32
    for fmt, per in ((tq.FP4_NV, 2048), (tq.FP4_MX, 1024)):
        assert tq.tq_fp4_tiled_scales_size(1, 1, longest, fmt) == (1 << 23) * per
        assert tq.tq_fp4_tiled_scales_size(2, 129, longest, fmt) == 4 * (1 << 23) * per
        for K in ((1 << 31) - 256, longest):
            size = tq.lib().tq_fp4_linear_workspace_size(100, K, 1, fmt)
            assert 100 * (K // 2) + -(-K // 256) * per <= size < 1 << 42
            size = tq.lib().tq_fp4_moe_workspace_size(100, 1, 1, K, 1, fmt)
            assert 100 * (K // 2) + -(-K // 256) * per <= size < 1 << 42


def test_scale_tiling_keeps_to_the_products_sizes(tq):
    most = (1 << 31) - 1024
    assert tq.tq_fp4_tiled_scales_size(1, most - 1, 32) == (1 << 24) * 2048 - 8 * 2048
    for E, N in ((1, most), (1, (1 << 31) - 1), (1024, most // 1024 + 1), ((1 << 31) - 1, (1 << 31) - 1)):
        assert tq.tq_fp4_tiled_scales_size(E, N, 32) == 0
        assert tq.lib().tq_fp4_tile_scales(A, E, N, 32, 0, A, None) == INVALID
    assert tq.tq_fp4_tiled_scales_size((1 << 31) - 1025, 1, (1 << 31) - 32) == 0     # bytes past a size_t


def test_other_threads_run_during_a_short_call(tq):
    """A wrapper of the binding bound to a function that sleeps for as many microseconds as its first argument says:
    another thread gets on meanwhile."""
    tq.lib()
    if type(tq._call("tq_fp4_dequantize")).__name__ != "builtin_function_or_method":
        pytest.skip("the calls go through ctypes")
    program = """
import ctypes, threading, time
from trellis_quantized_moe_sort_gb300 import _tqcall
usleep = ctypes.CDLL(None).usleep
_tqcall.bind("tq_fp4_dequantize", ctypes.cast(usleep, ctypes.c_void_p).value)
seen, stop = [], threading.Event()
def tick():
    while not stop.is_set():
        seen.append(time.monotonic())
        time.sleep(0.005)
t = threading.Thread(target=tick)
t.start()
time.sleep(0.05)
start = time.monotonic()
_tqcall.tq_fp4_dequantize(500000, None, 0, 0, 0, None, None, 0, None)
end = time.monotonic()
stop.set()
t.join()
assert end - start >= 0.4, end - start
print(sum(start + 0.1 < s < end - 0.1 for s in seen))
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(tq.__file__)))
    r = subprocess.run([sys.executable, "-c", program], capture_output=True, text=True, cwd=root, timeout=120)
    assert r.returncode == 0, r.stderr
    assert int(r.stdout) > 0


def test_a_failing_compiler_leaves_the_calls_to_ctypes(tq, monkeypatch, tmp_path, capsys):
    """The short calls are an extra: where gcc cannot build them the rest is built all the same, and no
    earlier one stays in their place."""
    import importlib.machinery
    import types
    from trellis_quantized_moe_sort_gb300 import build
    if not build.python_include():
        pytest.skip("no Python.h or no gcc")
    assert os.path.basename(build.CALLS) == "_tqcall" + importlib.machinery.EXTENSION_SUFFIXES[0]
    calls = tmp_path / os.path.basename(build.CALLS)
    monkeypatch.setattr(build, "CALLS", str(calls))
    assert build.build_calls(True) and calls.exists()
    stamp = calls.stat().st_mtime_ns
    assert build.build_calls() and calls.stat().st_mtime_ns == stamp      # nothing to do
    ran = []

    def run(cmd, **kwargs):
        ran.append(cmd[0])
        return types.SimpleNamespace(returncode=1, stdout="", stderr="no such file")

    monkeypatch.setattr(build.subprocess, "run", run)
    assert not build.build_calls(True) and not calls.exists() and ran == ["gcc"]
    assert "ctypes" in capsys.readouterr().err
    assert build.build() == build.LIB                                     # the library is up to date without them
    assert "nvcc" not in " ".join(ran)


class _OnDevice:
    """What the binding asks of a tensor on CUDA device `device`."""
    is_cuda = True

    def __init__(self, dtype, *shape, device=0):
        import torch
        self.dtype, self.shape, self._device = dtype, torch.Size(shape), device

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return A

    def get_device(self):
        return self._device

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()


def test_tensors_of_another_device_are_refused(tq, monkeypatch):
    """Device 0 is current: a call with any one of its tensors on device 1 is refused before the library is called."""
    import torch
    f32, i32, u8 = torch.float32, torch.int32, torch.uint8
    for name, value in (("_torch_mod", torch), ("_common", None), ("_type_codes", None), ("_raw_stream_fn", lambda device: 0)):
        monkeypatch.setattr(tq, name, value)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    called = []
    monkeypatch.setattr(tq, "_calls", {name: (lambda *a, name=name: called.append(name) or 0) for name in tq._CALLS})
    monkeypatch.setattr(tq.lib(), "tq_fp4_tile_scales", lambda *a: called.append("tq_fp4_tile_scales") or 0)
    n, E, k, K, N = 4, 8, 2, 64, 96

    def rows(v):
        return -(-v // 128) * 128

    weights = lambda e, r, c: dict(packed=(u8, e, r, c // 2), tiled=(u8, e * rows(r) * (-(-c // 256) * 256 // 16)))
    t = lambda dtype, *shape: (dtype, *shape)
    calls = {
        "router": (lambda a: tq.tq_router_scored(a["x"], k, bias=a["bias"], topk_ids=a["ids"], topk_w=a["w"]),
                   dict(x=t(f32, n, E), bias=t(f32, E), ids=t(i32, n, k), w=t(f32, n, k))),
        "router backward": (lambda a: tq.tq_router_scored_backward(a["x"], a["ids"], a["w"], a["g"], grad_logits=a["out"]),
                            dict(x=t(f32, n, E), ids=t(i32, n, k), w=t(f32, n, k), g=t(f32, n, k), out=t(f32, n, E))),
        "quantize": (lambda a: tq.tq_fp4_quantize(a["x"], tq.FP4_NV, a["g"], a["packed"], a["scales"]),
                     dict(x=t(f32, n, K), g=t(f32, 1), packed=t(u8, n, K // 2), scales=t(u8, n, K // 16))),
        "dequantize": (lambda a: tq.tq_fp4_dequantize(a["packed"], a["scales"], tq.FP4_NV, a["g"], out=a["out"]),
                       dict(packed=t(u8, n, K // 2), scales=t(u8, n, K // 16), g=t(f32, 1), out=t(f32, n, K))),
        "tile scales": (lambda a: tq.tq_fp4_tile_scales(a["scales"], tq.FP4_NV, a["tiled"]),
                        dict(scales=t(u8, N, K // 16), tiled=t(u8, 128 * 16))),
        "linear": (lambda a: tq.tq_fp4_linear(a["x"], a["packed"], a["tiled"], tq.FP4_NV, a["ws"], a["xs"], a["work"], a["y"]),
                   dict(x=t(f32, n, K), **weights(1, N, K), ws=t(f32, 1), xs=t(f32, 1), work=t(u8, 1 << 20), y=t(f32, n, N))),
        "experts": (lambda a: tq.tq_fp4_moe_forward(a["x"], a["packed"], a["tiled"], a["ids"], a["w"], tq.FP4_NV, a["ws"],
                                                    a["xs"], a["work"], a["y"]),
                    dict(x=t(f32, n, K), **weights(E, N, K), ids=t(i32, n, k), w=t(f32, n, k), ws=t(f32, E), xs=t(f32, 1),
                         work=t(u8, 1 << 20), y=t(f32, n, N))),
        "mlp": (lambda a: tq.tq_fp4_moe_mlp_forward(a["x"], a["gu"], a["gut"], a["packed"], a["tiled"], a["ids"], a["w"],
                                                    tq.FP4_NV, a["gs"], a["ds"], a["xs"], a["hs"], a["work"], a["y"]),
                dict(x=t(f32, n, K), gu=t(u8, E, 2 * N, K // 2), gut=t(u8, E * rows(2 * N) * 16), **weights(E, K, N),
                     ids=t(i32, n, k), w=t(f32, n, k), gs=t(f32, E), ds=t(f32, E), xs=t(f32, 1), hs=t(f32, 1),
                     work=t(u8, 1 << 20), y=t(f32, n, K))),
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


def test_workspace_sizes_follow_the_device(tq, monkeypatch, request):
    """The library's answer depends on the current device: the sizes are asked anew, and a call keeps them by device."""
    import torch
    request.addfinalizer(tq._workspace_bytes.cache_clear)     # of the sizes made up here
    current = [0]
    sizes = {0: 4096, 1: 8192}
    monkeypatch.setattr(tq, "_torch_mod", torch)
    monkeypatch.setattr(tq, "_common", None)
    for name, args in (("tq_fp4_linear_workspace_size", (300, 96, 33)), ("tq_fp4_moe_workspace_size", (300, 2, 8, 96, 33)),
                       ("tq_fp4_moe_mlp_workspace_size", (300, 2, 8, 96, 32))):
        monkeypatch.setattr(tq.lib(), name, lambda *a: sizes[current[0]])
        made = []
        monkeypatch.setattr(tq, "_empty", lambda n, dtype, device, stream:
                            made.append((n, device)) or torch.empty(n, dtype=dtype))
        size = getattr(tq, name)
        for device in (0, 1, 0):
            current[0] = device
            assert size(*args) == sizes[device], name
            assert tq._workspace(None, size, device, None, *args, tq.FP4_NV)[1] == sizes[device], name
        assert made == [(4096, 0), (8192, 1), (4096, 0)]
