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
