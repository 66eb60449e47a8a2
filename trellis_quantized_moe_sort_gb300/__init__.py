"""Python binding of libtqmoe.so (C ABI: include/tqmoe.h).

Argument marshalling only: every step of the MoE path runs in the library's
CUDA kernels.  PyTorch provides device memory and the current stream.  There
is no CPU fallback: if the library is missing or no sm_103a device is present,
calls raise.

Tensor conventions: bf16 activations (torch.bfloat16 or 16-bit integer views),
packed bitstreams torch.uint8 [E, N, K/4], LUT fp16 (torch.float16 or 16-bit
integer view) [2^L], router ids torch.int32 [n, top_k], router weights
torch.float32 [n, top_k].
"""
from __future__ import annotations

import ctypes
import functools
import os

__all__ = [
    "TQError", "lib", "lib_path", "tq_init", "tq_arch_witness", "tq_pairs_per_woken_expert",
    "tq_tiles_amortize", "tq_grouped_min_tokens", "tq_tile_map_capacity", "tq_native_tile_m", "TILE_NATIVE", "tq_select_arm",
    "tq_route", "tq_router_topk", "tq_route_logits", "tq_build_tile_map", "tq_gather_rows", "tq_prepare", "tq_grouped_gemm", "tq_gemv", "tq_combine",
    "tq_moe_workspace_size", "tq_moe_forward", "tq_moe_forward_static", "tq_device_error", "tq_launch_counts",
    "tq_status_string", "tq_probe_lut_rate", "tq_probe_wait_timeout", "tq_grouped_gemm_pairs", "tq_swiglu",
    "tq_moe_mlp_workspace_size", "tq_moe_mlp_forward", "tq_dequantize", "tq_grouped_gemm_dense",
    "tq_moe_dequant_workspace_size", "tq_moe_forward_dequant", "ARM_AUTO", "ARM_GEMV", "ARM_GROUPED", "ARM_MEASURED", "EXPORTED_SYMBOLS",
    "X_TOKENS", "X_PAIR_SORTED", "GATHER_MAX_TILE_M",
    "tq_router_scored", "tq_router_scored_backward", "SCORE_SOFTMAX", "SCORE_SIGMOID",
    "tq_fp4_quantize", "tq_fp4_dequantize", "tq_fp4_tiled_scales_size", "tq_fp4_tile_scales",
    "tq_fp4_linear_workspace_size", "tq_fp4_linear", "tq_fp4_moe_workspace_size", "tq_fp4_moe_forward",
    "tq_fp4_moe_mlp_workspace_size", "tq_fp4_moe_mlp_forward", "FP4_NV", "FP4_MX", "tq_launch_counts_all",
    "tq_rms_norm", "tq_rms_norm_fp8", "tq_rms_norm_backward_workspace_size", "tq_rms_norm_backward",
    "tq_fp8_quantize", "tq_fp8_dequantize", "tq_fp8_linear_workspace_size", "tq_fp8_linear", "tq_fp8_moe_workspace_size",
    "tq_fp8_moe_forward", "tq_fp8_moe_mlp_workspace_size", "tq_fp8_moe_mlp_forward", "FP8_BLOCK",
    "tq_swiglu_linear_workspace_size", "tq_swiglu_linear", "tq_swiglu_linear_backward_workspace_size", "tq_swiglu_linear_backward",
]

ARM_AUTO, ARM_GEMV, ARM_GROUPED, ARM_MEASURED = 0, 1, 2, 3
TILE_NATIVE = 0          # tile_m of the whole-product calls: the kernel's native m-tile
X_TOKENS, X_PAIR_SORTED = 0, 1   # activation layouts of tq_grouped_gemm / tq_grouped_gemm_dense
GATHER_MAX_TILE_M = 16   # the whole-product calls gather rows in the kernel up to this m-tile
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1   # scores of tq_router_scored
FP4_NV, FP4_MX = 0, 1    # 4-bit formats: blocks of 16 with E4M3 scales, blocks of 32 with E8M0 scales
FP8_BLOCK = 128          # values of a row, or rows and columns of a matrix, that share an 8-bit scale
_HERE = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_HERE, "libtqmoe.so")

_c_i64, _c_int, _c_dbl, _c_p, _c_sz = ctypes.c_int64, ctypes.c_int, ctypes.c_double, ctypes.c_void_p, ctypes.c_size_t
_c_flt = ctypes.c_float

# name -> (restype, argtypes); the same set include/tqmoe.h declares
_SIGS = {
    "tq_status_string": (ctypes.c_char_p, [_c_int]),
    "tq_init": (_c_int, [_c_int]),
    "tq_arch_witness": (_c_int, [_c_int, ctypes.POINTER(_c_int)]),
    "tq_pairs_per_woken_expert": (_c_dbl, [_c_i64, _c_int, _c_int]),
    "tq_tiles_amortize": (_c_int, [_c_i64, _c_int, _c_int, _c_int]),
    "tq_grouped_min_tokens": (_c_i64, [_c_int, _c_int, _c_int]),
    "tq_tile_map_capacity": (_c_i64, [_c_i64, _c_int, _c_int, _c_int]),
    "tq_native_tile_m": (_c_int, [_c_i64, _c_int, _c_int]),
    "tq_select_arm": (_c_int, [_c_i64, _c_int, _c_int, _c_int, _c_int]),
    "tq_route": (_c_int, [_c_p, _c_i64, _c_int, _c_int, _c_p, _c_p, _c_p, _c_p]),
    "tq_build_tile_map": (_c_int, [_c_p, _c_int, _c_int, _c_p, _c_p, _c_i64, _c_p]),
    "tq_router_topk": (_c_int, [_c_p, _c_i64, _c_int, _c_int, _c_p, _c_p, _c_p]),
    "tq_route_logits": (_c_int, [_c_p, _c_i64, _c_int, _c_int, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p]),
    "tq_grouped_gemm": (_c_int, [_c_p, _c_int, _c_p, _c_p, _c_int, _c_p, _c_p, _c_p, _c_p, _c_i64, _c_i64,
                                 _c_int, _c_int, _c_int, _c_int, _c_int, _c_p, _c_p]),
    "tq_gemv": (_c_int, [_c_p, _c_p, _c_p, _c_int, _c_p, _c_p, _c_i64, _c_int, _c_int, _c_int,
                         _c_int, _c_p, _c_p]),
    "tq_combine": (_c_int, [_c_p, _c_p, _c_i64, _c_p]),
    "tq_gather_rows": (_c_int, [_c_p, _c_p, _c_i64, _c_int, _c_int, _c_p, _c_p]),
    "tq_prepare": (_c_int, [_c_p, _c_p, _c_i64, _c_int, _c_int, _c_int, _c_int, _c_p, _c_p, _c_p, _c_p, _c_p,
                            _c_i64, _c_p, _c_p, _c_i64, _c_p]),
    "tq_moe_workspace_size": (_c_sz, [_c_i64, _c_int, _c_int, _c_int, _c_int, _c_int]),
    "tq_moe_forward": (_c_int, [_c_p, _c_p, _c_p, _c_int, _c_p, _c_p, _c_i64, _c_int, _c_int,
                                _c_int, _c_int, _c_int, _c_int, _c_p, _c_sz, _c_p,
                                ctypes.POINTER(_c_int), _c_p]),
    "tq_moe_forward_static": (_c_int, [_c_p, _c_p, _c_p, _c_int, _c_p, _c_p, _c_i64, _c_int, _c_int,
                                       _c_int, _c_int, _c_int, _c_int, _c_p, ctypes.POINTER(_c_int), _c_p]),
    "tq_probe_lut_rate": (_c_int, [_c_p, _c_int, _c_int, _c_p, _c_p, _c_p]),
    "tq_probe_wait_timeout": (_c_int, [_c_i64, _c_p, _c_p]),
    "tq_grouped_gemm_pairs": (_c_int, [_c_p, _c_p, _c_p, _c_int, _c_p, _c_p, _c_p, _c_i64, _c_i64, _c_int, _c_int,
                                       _c_int, _c_int, _c_int, _c_p, _c_p]),
    "tq_swiglu": (_c_int, [_c_p, _c_i64, _c_int, _c_p, _c_p]),
    "tq_moe_mlp_workspace_size": (_c_sz, [_c_i64, _c_int, _c_int, _c_int, _c_int, _c_int]),
    "tq_moe_mlp_forward": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_int, _c_p, _c_p, _c_i64, _c_int, _c_int, _c_int,
                                    _c_int, _c_int, _c_int, _c_p, _c_sz, _c_p, ctypes.POINTER(_c_int), _c_p]),
    "tq_dequantize": (_c_int, [_c_p, _c_p, _c_int, _c_p, _c_int, _c_int, _c_int, _c_int, _c_p, _c_p]),
    "tq_grouped_gemm_dense": (_c_int, [_c_p, _c_int, _c_p, _c_p, _c_p, _c_p, _c_p, _c_i64, _c_i64, _c_int, _c_int,
                                       _c_int,
                                       _c_int, _c_int, _c_p, _c_p]),
    "tq_moe_dequant_workspace_size": (_c_sz, [_c_i64, _c_int, _c_int, _c_int, _c_int, _c_int]),
    "tq_moe_forward_dequant": (_c_int, [_c_p, _c_p, _c_p, _c_int, _c_p, _c_p, _c_i64, _c_int, _c_int, _c_int,
                                        _c_int, _c_int, _c_p, _c_sz, _c_p, _c_p]),
    "tq_device_error": (_c_int, [ctypes.POINTER(_c_int), ctypes.POINTER(_c_int)]),
    "tq_launch_counts": (None, [ctypes.POINTER(_c_i64)]),
    "tq_launch_counts_all": (_c_int, [ctypes.POINTER(_c_i64), _c_int]),
    "tq_router_scored": (_c_int, [_c_p, _c_int, _c_i64, _c_p, _c_i64, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int,
                                  _c_flt, _c_p, _c_p, _c_p]),
    "tq_router_scored_backward": (_c_int, [_c_p, _c_int, _c_i64, _c_p, _c_p, _c_p, _c_i64, _c_int, _c_int, _c_int,
                                           _c_int, _c_flt, _c_p, _c_p]),
    "tq_fp4_quantize": (_c_int, [_c_p, _c_int, _c_i64, _c_i64, _c_int, _c_int, _c_p, _c_p, _c_p, _c_p]),
    "tq_fp4_dequantize": (_c_int, [_c_p, _c_p, _c_i64, _c_int, _c_int, _c_p, _c_p, _c_int, _c_p]),
    "tq_fp4_tiled_scales_size": (_c_sz, [_c_int, _c_int, _c_int, _c_int]),
    "tq_fp4_tile_scales": (_c_int, [_c_p, _c_int, _c_int, _c_int, _c_int, _c_p, _c_p]),
    "tq_fp4_linear_workspace_size": (_c_sz, [_c_i64, _c_int, _c_int, _c_int]),
    "tq_fp4_linear": (_c_int, [_c_p, _c_int, _c_i64, _c_p, _c_p, _c_int, _c_p, _c_p, _c_i64, _c_int, _c_int, _c_p,
                               _c_sz, _c_p, _c_int, _c_p]),
    "tq_fp4_moe_workspace_size": (_c_sz, [_c_i64, _c_int, _c_int, _c_int, _c_int, _c_int]),
    "tq_fp4_moe_forward": (_c_int, [_c_p, _c_int, _c_i64, _c_p, _c_p, _c_int, _c_p, _c_p, _c_p, _c_p, _c_i64, _c_int,
                                    _c_int, _c_int, _c_int, _c_p, _c_sz, _c_p, _c_int, _c_p]),
    "tq_fp4_moe_mlp_workspace_size": (_c_sz, [_c_i64, _c_int, _c_int, _c_int, _c_int, _c_int]),
    "tq_fp4_moe_mlp_forward": (_c_int, [_c_p, _c_int, _c_i64, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_int, _c_p, _c_p,
                                        _c_p, _c_p, _c_i64, _c_int, _c_int, _c_int, _c_int, _c_p, _c_sz, _c_p, _c_int,
                                        _c_p]),
    "tq_rms_norm": (_c_int, [_c_p, _c_int, _c_i64, _c_p, _c_i64, _c_p, _c_int, _c_flt, _c_i64, _c_int, _c_p, _c_p, _c_p,
                             _c_p, _c_p, _c_p]),
    "tq_rms_norm_backward_workspace_size": (_c_sz, [_c_i64, _c_int]),
    "tq_rms_norm_backward": (_c_int, [_c_p, _c_i64, _c_p, _c_int, _c_i64, _c_p, _c_int, _c_p, _c_p, _c_i64, _c_i64, _c_int,
                                      _c_p, _c_sz, _c_p, _c_p, _c_p]),
    "tq_fp8_quantize": (_c_int, [_c_p, _c_int, _c_i64, _c_int, _c_i64, _c_int, _c_int, _c_p, _c_p, _c_p]),
    "tq_fp8_dequantize": (_c_int, [_c_p, _c_p, _c_int, _c_i64, _c_int, _c_int, _c_p, _c_int, _c_p]),
    "tq_fp8_linear_workspace_size": (_c_sz, [_c_i64, _c_int, _c_int]),
    "tq_fp8_linear": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_i64, _c_int, _c_int, _c_p, _c_sz, _c_p, _c_int, _c_p]),
    "tq_fp8_moe_workspace_size": (_c_sz, [_c_i64, _c_int, _c_int, _c_int, _c_int]),
    "tq_fp8_moe_forward": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_i64, _c_int, _c_int, _c_int, _c_int, _c_p,
                                    _c_sz, _c_p, _c_int, _c_p]),
    "tq_fp8_moe_mlp_workspace_size": (_c_sz, [_c_i64, _c_int, _c_int, _c_int, _c_int]),
    "tq_fp8_moe_mlp_forward": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_i64, _c_int, _c_int, _c_int,
                                        _c_int, _c_p, _c_sz, _c_p, _c_int, _c_p]),
    "tq_swiglu_linear_workspace_size": (_c_sz, [_c_i64, _c_int, _c_int]),
    "tq_swiglu_linear": (_c_int, [_c_p, _c_int, _c_i64, _c_p, _c_i64, _c_int, _c_int, _c_p, _c_sz, _c_p, _c_p, _c_p]),
    "tq_swiglu_linear_backward_workspace_size": (_c_sz, [_c_i64, _c_int, _c_int, _c_int]),
    "tq_swiglu_linear_backward": (_c_int, [_c_p, _c_int, _c_i64, _c_p, _c_p, _c_p, _c_i64, _c_int, _c_int, _c_p, _c_sz,
                                           _c_p, _c_p, _c_p]),
}
EXPORTED_SYMBOLS = tuple(_SIGS)

_lib = None


class TQError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {tq_status_string(status)} ({status})" if what else
                         f"{tq_status_string(status)} ({status})")


def lib() -> ctypes.CDLL:
    """Load libtqmoe.so (built by __graft_entry__.build()); raise if missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(lib_path):
            raise RuntimeError(f"{lib_path} is not built; run `python -c 'import __graft_entry__ as g; "
                               f"g.build()'` (nvcc, sm_103a)")
        h = ctypes.CDLL(lib_path)
        for name, (res, args) in _SIGS.items():
            fn = getattr(h, name)
            fn.restype = res
            fn.argtypes = args
        _lib = h
        _bind_calls(h)
    return _lib


# The calls of the scored router, the norm and the 4-, 8- and 16-bit operators, by name: the C wrappers of
# csrc/tq_python.c, or ctypes' functions where those are not built.
_CALLS = ("tq_router_scored", "tq_router_scored_backward", "tq_fp4_quantize", "tq_fp4_dequantize", "tq_fp4_linear",
          "tq_fp4_moe_forward", "tq_fp4_moe_mlp_forward", "tq_rms_norm", "tq_rms_norm_backward", "tq_fp8_quantize",
          "tq_fp8_dequantize", "tq_fp8_linear", "tq_fp8_moe_forward", "tq_fp8_moe_mlp_forward", "tq_swiglu_linear",
          "tq_swiglu_linear_backward")
_calls: dict = {}


def _bind_calls(h: ctypes.CDLL) -> None:
    try:
        from . import _tqcall
    except ImportError:
        _tqcall = None
    for name in _CALLS:
        if _tqcall is None:
            _calls[name] = getattr(h, name)
        else:
            _tqcall.bind(name, ctypes.cast(getattr(h, name), ctypes.c_void_p).value)
            _calls[name] = getattr(_tqcall, name)


def _call(name: str):
    if not _calls:
        lib()
    return _calls[name]


def tq_status_string(status: int) -> str:
    return lib().tq_status_string(int(status)).decode()


def _check(rc: int, what: str):
    if rc != 0:
        raise TQError(rc, what)


# ------------------------------------------------------------------ torch glue

_torch_mod = None


def _torch():
    """torch, once a CUDA device has been seen (checked on the first call only)."""
    global _torch_mod
    if _torch_mod is None:
        import torch
        if not torch.cuda.is_available():
            raise RuntimeError("trellis_quantized_moe_sort_gb300 needs a CUDA device (sm_103a); none found")
        _torch_mod = torch
    return _torch_mod


def _dev_ptr(t, dtypes, name):
    """Device address of a contiguous CUDA tensor of one of `dtypes`."""
    try:
        ok = t.is_cuda and (not dtypes or t.dtype in dtypes) and t.is_contiguous()
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None
    if not ok:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if dtypes and t.dtype not in dtypes:
            raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


_raw_stream_fn = None


def _stream(stream, device=None):
    """Raw handle of the given stream, or of torch's current one on the device
    (by default the current one)."""
    global _raw_stream_fn
    if stream is not None:
        return stream.cuda_stream
    torch = _torch()
    if _raw_stream_fn is None:
        # the C-level getter of torch's current stream (a plain integer), when
        # this torch build has it; else the public (slower) route
        _raw_stream_fn = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda device: torch.cuda.current_stream(device).cuda_stream)
    return _raw_stream_fn(torch.cuda.current_device() if device is None else device)


_bits16_types = None


def _bits16():
    global _bits16_types
    if _bits16_types is None:
        torch = _torch()
        _bits16_types = (torch.bfloat16, torch.float16, torch.int16, torch.uint16)
    return _bits16_types


# ------------------------------------------------------------------ API

def tq_init(device: int = 0) -> None:
    _check(lib().tq_init(device), "tq_init")


def tq_arch_witness(device: int = 0) -> int:
    arch = ctypes.c_int(0)
    _check(lib().tq_arch_witness(device, ctypes.byref(arch)), "tq_arch_witness")
    return arch.value


def tq_pairs_per_woken_expert(n: int, top_k: int, E: int) -> float:
    return lib().tq_pairs_per_woken_expert(n, top_k, E)


def tq_tiles_amortize(n: int, top_k: int, E: int, tile_m: int) -> bool:
    rc = lib().tq_tiles_amortize(n, top_k, E, tile_m)
    if rc < 0:
        raise TQError(rc, "tq_tiles_amortize")
    return bool(rc)


def tq_grouped_min_tokens(top_k: int, E: int, tile_m: int) -> int:
    rc = lib().tq_grouped_min_tokens(top_k, E, tile_m)
    if rc < 0:
        raise TQError(int(rc), "tq_grouped_min_tokens")
    return int(rc)


def tq_native_tile_m(n: int, top_k: int, E: int) -> int:
    v = lib().tq_native_tile_m(n, top_k, E)
    if v < 0:
        raise TQError(v, "tq_native_tile_m")
    return int(v)


def tq_tile_map_capacity(n: int, top_k: int, E: int, tile_m: int) -> int:
    rc = lib().tq_tile_map_capacity(n, top_k, E, tile_m)
    if rc < 0:
        raise TQError(int(rc), "tq_tile_map_capacity")
    return int(rc)


def tq_select_arm(n: int, top_k: int, E: int, tile_m: int, pin: int = ARM_AUTO) -> int:
    rc = lib().tq_select_arm(n, top_k, E, tile_m, pin)
    if rc < 0:
        raise TQError(rc, "tq_select_arm")
    return rc


def tq_route(topk_ids, E: int, counts=None, offsets=None, sorted_pairs=None, stream=None):
    """Stable sort of pairs by expert -> (counts[E], offsets[E+1], sorted_pairs[P])."""
    torch = _torch()
    n, k = topk_ids.shape
    dev = topk_ids.device
    counts = torch.empty(E, dtype=torch.int32, device=dev) if counts is None else counts
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev) if offsets is None else offsets
    if sorted_pairs is None:
        sorted_pairs = torch.empty(max(n * k, 1), dtype=torch.int32, device=dev)
    _check(lib().tq_route(_dev_ptr(topk_ids, (torch.int32,), "topk_ids"), n, k, E,
                          _dev_ptr(counts, (torch.int32,), "counts"),
                          _dev_ptr(offsets, (torch.int32,), "offsets"),
                          _dev_ptr(sorted_pairs, (torch.int32,), "sorted_pairs"), _stream(stream)),
           "tq_route")
    return counts, offsets, sorted_pairs[: n * k]


def tq_router_topk(logits, top_k: int, topk_ids=None, topk_w=None, stream=None):
    """Per-token top_k experts and softmax weights from fp32 logits [n, E]."""
    torch = _torch()
    n, E = logits.shape
    topk_ids = torch.empty((n, top_k), dtype=torch.int32, device=logits.device) if topk_ids is None else topk_ids
    topk_w = torch.empty((n, top_k), dtype=torch.float32, device=logits.device) if topk_w is None else topk_w
    _check(lib().tq_router_topk(_dev_ptr(logits, (torch.float32,), "logits"), n, E, top_k,
                                _dev_ptr(topk_ids, (torch.int32,), "topk_ids"),
                                _dev_ptr(topk_w, (torch.float32,), "topk_w"), _stream(stream)), "tq_router_topk")
    return topk_ids, topk_w


def tq_route_logits(logits, top_k: int, stream=None):
    """Router top-k then the routing sort -> (ids, w, counts, offsets, sorted_pairs)."""
    torch = _torch()
    n, E = logits.shape
    dev = logits.device
    ids = torch.empty((n, top_k), dtype=torch.int32, device=dev)
    w = torch.empty((n, top_k), dtype=torch.float32, device=dev)
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    sp = torch.empty(max(n * top_k, 1), dtype=torch.int32, device=dev)
    _check(lib().tq_route_logits(_dev_ptr(logits, (torch.float32,), "logits"), n, E, top_k,
                                 _dev_ptr(ids, (torch.int32,), "topk_ids"), _dev_ptr(w, (torch.float32,), "topk_w"),
                                 _dev_ptr(counts, (torch.int32,), "counts"), _dev_ptr(offsets, (torch.int32,), "offsets"),
                                 _dev_ptr(sp, (torch.int32,), "sorted_pairs"), _stream(stream)), "tq_route_logits")
    return ids, w, counts, offsets, sp[: n * top_k]


def tq_build_tile_map(offsets, tile_m: int, cap: int, tiles=None, num_tiles=None, stream=None):
    """m-tile map -> (tiles[cap, 3], num_tiles[1]) (device)."""
    torch = _torch()
    E = offsets.numel() - 1
    dev = offsets.device
    tiles = torch.empty((cap, 3), dtype=torch.int32, device=dev) if tiles is None else tiles
    num_tiles = torch.empty(1, dtype=torch.int32, device=dev) if num_tiles is None else num_tiles
    _check(lib().tq_build_tile_map(_dev_ptr(offsets, (torch.int32,), "offsets"), E, tile_m,
                                   _dev_ptr(tiles, (torch.int32,), "tiles"),
                                   _dev_ptr(num_tiles, (torch.int32,), "num_tiles"), cap, _stream(stream)),
           "tq_build_tile_map")
    return tiles, num_tiles


def _shapes(x, packed, lut):
    n, K = x.shape
    E, N, kb = packed.shape
    if kb * 4 != K:
        raise ValueError(f"packed has {kb} bytes per row, expected K/4 = {K // 4}")
    L = lut.numel().bit_length() - 1
    if lut.numel() != (1 << L):
        raise ValueError("lut must have 2^L entries")
    return n, K, E, N, L


def tq_gather_rows(x, sorted_pairs, top_k: int, x_sorted=None, stream=None):
    """Pair-sorted copy of the activations: x_sorted[s] = x[sorted_pairs[s] // top_k]."""
    torch = _torch()
    n, K = x.shape
    P = n * top_k
    x_sorted = torch.empty((max(P, 1), K), dtype=x.dtype, device=x.device) if x_sorted is None else x_sorted
    _check(lib().tq_gather_rows(_dev_ptr(x, _bits16(), "x"), _dev_ptr(sorted_pairs, (torch.int32,), "sorted_pairs"),
                                n, top_k, K, _dev_ptr(x_sorted, _bits16(), "x_sorted"), _stream(stream)),
           "tq_gather_rows")
    return x_sorted[:P]


def tq_prepare(topk_ids, x, E: int, tile_m: int, cap: int, counts, offsets, sorted_pairs, tiles, num_tiles,
               x_sorted=None, y32=None, stream=None) -> None:
    """Route + tile map in one launch, clearing y32 (fp32) in the same launch
    when it is given; with x_sorted, also the pair-sorted copy of x (what
    tq_grouped_gemm_pairs reads; tq_grouped_gemm gathers the rows itself)."""
    torch = _torch()
    n, top_k = topk_ids.shape
    K = x.shape[1]
    y32_ptr = None if y32 is None else _dev_ptr(y32, (torch.float32,), "y32")
    xs_ptr = None if x_sorted is None else _dev_ptr(x_sorted, _bits16(), "x_sorted")
    _check(lib().tq_prepare(_dev_ptr(topk_ids, (torch.int32,), "topk_ids"), _dev_ptr(x, _bits16(), "x"), n, top_k,
                            E, K, tile_m, _dev_ptr(counts, (torch.int32,), "counts"),
                            _dev_ptr(offsets, (torch.int32,), "offsets"),
                            _dev_ptr(sorted_pairs, (torch.int32,), "sorted_pairs"),
                            _dev_ptr(tiles, (torch.int32,), "tiles"), _dev_ptr(num_tiles, (torch.int32,), "num_tiles"),
                            cap, xs_ptr, y32_ptr, 0 if y32 is None else y32.numel(), _stream(stream)), "tq_prepare")


def _x_rows(x, x_layout: int, top_k: int) -> int:
    """Tokens n of an activation tensor in either layout."""
    if x_layout == X_TOKENS:
        return x.shape[0]
    if x_layout != X_PAIR_SORTED:
        raise ValueError(f"x_layout must be X_TOKENS or X_PAIR_SORTED, not {x_layout}")
    if x.shape[0] % top_k:
        raise ValueError("pair-sorted x must have n*top_k rows")
    return x.shape[0] // top_k


def tq_grouped_gemm(x, packed, lut, sorted_pairs, topk_w, tiles, num_tiles, top_k: int, tile_m: int,
                    y32, x_layout: int = X_TOKENS, stream=None) -> None:
    """y32 += grouped product (y32 fp32 [n, N], zero it for a plain product).
    x: the token activations [n, K] (X_TOKENS: the kernel gathers each m-tile's
    rows through sorted_pairs) or their pair-sorted copy [n*top_k, K] from
    tq_gather_rows (X_PAIR_SORTED)."""
    torch = _torch()
    n = _x_rows(x, x_layout, top_k)
    K = x.shape[1]
    E, N, kb = packed.shape
    if kb * 4 != K:
        raise ValueError(f"packed has {kb} bytes per row, expected K/4 = {K // 4}")
    L = lut.numel().bit_length() - 1
    cap = tiles.shape[0]
    _check(lib().tq_grouped_gemm(_dev_ptr(x, _bits16(), "x"), x_layout, _dev_ptr(packed, (torch.uint8,), "packed"),
                                 _dev_ptr(lut, _bits16(), "lut"), L,
                                 _dev_ptr(sorted_pairs, (torch.int32,), "sorted_pairs"),
                                 _dev_ptr(topk_w, (torch.float32,), "topk_w"),
                                 _dev_ptr(tiles, (torch.int32,), "tiles"),
                                 _dev_ptr(num_tiles, (torch.int32,), "num_tiles"), cap, n, top_k, E, K, N,
                                 tile_m, _dev_ptr(y32, (torch.float32,), "y32"), _stream(stream)),
           "tq_grouped_gemm")


def tq_gemv(x, packed, lut, topk_ids, topk_w, y32, stream=None) -> None:
    """y32 += per-pair GEMV product."""
    torch = _torch()
    n, K, E, N, L = _shapes(x, packed, lut)
    top_k = topk_ids.shape[1]
    _check(lib().tq_gemv(_dev_ptr(x, _bits16(), "x"), _dev_ptr(packed, (torch.uint8,), "packed"),
                         _dev_ptr(lut, _bits16(), "lut"), L, _dev_ptr(topk_ids, (torch.int32,), "topk_ids"),
                         _dev_ptr(topk_w, (torch.float32,), "topk_w"), n, top_k, E, K, N,
                         _dev_ptr(y32, (torch.float32,), "y32"), _stream(stream)), "tq_gemv")


def tq_combine(y32, y=None, stream=None):
    """bf16 (round to nearest even) copy of y32."""
    torch = _torch()
    y = torch.empty(y32.shape, dtype=torch.bfloat16, device=y32.device) if y is None else y
    _check(lib().tq_combine(_dev_ptr(y32, (torch.float32,), "y32"), _dev_ptr(y, _bits16(), "y"),
                            y32.numel(), _stream(stream)), "tq_combine")
    return y


def tq_moe_workspace_size(n: int, top_k: int, E: int, K: int, N: int, tile_m: int) -> int:
    return int(lib().tq_moe_workspace_size(n, top_k, E, K, N, tile_m))


def tq_moe_forward(x, packed, lut, topk_ids, topk_w, tile_m: int = 16, pin: int = ARM_AUTO,
                   workspace=None, y=None, stream=None):
    """Whole routed-expert product -> (y bf16 [n, N], arm used)."""
    torch = _torch()
    n, K, E, N, L = _shapes(x, packed, lut)
    top_k = topk_ids.shape[1]
    need = tq_moe_workspace_size(n, top_k, E, K, N, tile_m)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=x.device)
    y = torch.empty((n, N), dtype=torch.bfloat16, device=x.device) if y is None else y
    arm = ctypes.c_int(-1)
    _check(lib().tq_moe_forward(_dev_ptr(x, _bits16(), "x"), _dev_ptr(packed, (torch.uint8,), "packed"),
                                _dev_ptr(lut, _bits16(), "lut"), L,
                                _dev_ptr(topk_ids, (torch.int32,), "topk_ids"),
                                _dev_ptr(topk_w, (torch.float32,), "topk_w"), n, top_k, E, K, N, tile_m, pin,
                                _dev_ptr(workspace, (torch.uint8,), "workspace"), workspace.numel(),
                                _dev_ptr(y, _bits16(), "y"), ctypes.byref(arm), _stream(stream)),
           "tq_moe_forward")
    return y, arm.value


STATIC_SCRATCH_BYTES = 16 * 1024 * 1024   # TQ_STATIC_SCRATCH_BYTES in include/tqmoe.h


def tq_moe_forward_static(x, packed, lut, topk_ids, topk_w, tile_m: int = 16, pin: int = ARM_AUTO,
                          y=None, stream=None):
    """Whole routed-expert product with the library's fixed scratch array
    instead of a workspace (for callers that cannot allocate device memory;
    here only `y` is allocated, and only when not given) -> (y, arm used).
    Calls sharing a device must not overlap on the GPU."""
    torch = _torch()
    n, K, E, N, L = _shapes(x, packed, lut)
    top_k = topk_ids.shape[1]
    y = torch.empty((n, N), dtype=torch.bfloat16, device=x.device) if y is None else y
    arm = ctypes.c_int(-1)
    _check(lib().tq_moe_forward_static(_dev_ptr(x, _bits16(), "x"), _dev_ptr(packed, (torch.uint8,), "packed"),
                                       _dev_ptr(lut, _bits16(), "lut"), L,
                                       _dev_ptr(topk_ids, (torch.int32,), "topk_ids"),
                                       _dev_ptr(topk_w, (torch.float32,), "topk_w"), n, top_k, E, K, N, tile_m,
                                       pin, _dev_ptr(y, _bits16(), "y"), ctypes.byref(arm), _stream(stream)),
           "tq_moe_forward_static")
    return y, arm.value


def tq_probe_wait_timeout(timeout_ns: int, stream=None) -> tuple[bool, int]:
    """Run the bounded-wait probe: (whether the wait completed, microseconds
    waited).  The give-up is recorded in the device error word."""
    torch = _torch()
    out = torch.full((2,), -1, dtype=torch.int32, device="cuda")
    _check(lib().tq_probe_wait_timeout(int(timeout_ns), _dev_ptr(out, (torch.int32,), "out"), _stream(stream)),
           "tq_probe_wait_timeout")
    torch.cuda.synchronize()
    done, us = out.tolist()
    return bool(done), int(us)


def tq_probe_lut_rate(warps_per_sm: int = 8, iters: int = 512, stream=None) -> float:
    """Measured random 16-bit shared-memory lookups per clock per SM (the
    resource that bounds the trellis decode)."""
    torch = _torch()
    sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    table = torch.zeros(65536, dtype=torch.int16, device="cuda")
    sink = torch.empty(sms * warps_per_sm * 32, dtype=torch.int32, device="cuda")
    cycles = torch.zeros(sms, dtype=torch.int64, device="cuda")
    _check(lib().tq_probe_lut_rate(_dev_ptr(table, _bits16(), "table"), warps_per_sm, iters,
                                   _dev_ptr(sink, (torch.int32,), "sink"), _dev_ptr(cycles, (torch.int64,), "cycles"),
                                   _stream(stream)), "tq_probe_lut_rate")
    torch.cuda.synchronize()
    c = float(cycles.double().mean())
    return warps_per_sm * 32 * iters * 16 / c


def tq_moe_mlp_workspace_size(n: int, top_k: int, E: int, H: int, I: int, tile_m: int) -> int:
    return int(lib().tq_moe_mlp_workspace_size(n, top_k, E, H, I, tile_m))


def tq_moe_mlp_forward(x, packed_gu, lut_gu, packed_down, lut_down, topk_ids, topk_w, tile_m: int = 16,
                       pin: int = ARM_AUTO, workspace=None, y=None, stream=None):
    """Whole SwiGLU expert MLP -> (y bf16 [n, H], arm used)."""
    torch = _torch()
    n, H = x.shape
    E, I2, hb = packed_gu.shape
    I = I2 // 2
    if hb * 4 != H or tuple(packed_down.shape) != (E, H, I // 4):
        raise ValueError("packed_gu must be [E, 2I, H/4] and packed_down [E, H, I/4]")
    L = lut_gu.numel().bit_length() - 1
    if lut_down.numel() != lut_gu.numel():
        raise ValueError("both LUTs need 2^L entries")
    top_k = topk_ids.shape[1]
    need = tq_moe_mlp_workspace_size(n, top_k, E, H, I, tile_m)
    workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=x.device) if workspace is None else workspace
    y = torch.empty((n, H), dtype=torch.bfloat16, device=x.device) if y is None else y
    arm = ctypes.c_int(-1)
    _check(lib().tq_moe_mlp_forward(_dev_ptr(x, _bits16(), "x"), _dev_ptr(packed_gu, (torch.uint8,), "packed_gu"),
                                    _dev_ptr(lut_gu, _bits16(), "lut_gu"),
                                    _dev_ptr(packed_down, (torch.uint8,), "packed_down"),
                                    _dev_ptr(lut_down, _bits16(), "lut_down"), L,
                                    _dev_ptr(topk_ids, (torch.int32,), "topk_ids"),
                                    _dev_ptr(topk_w, (torch.float32,), "topk_w"), n, top_k, E, H, I, tile_m,
                                    pin, _dev_ptr(workspace, (torch.uint8,), "workspace"), workspace.numel(),
                                    _dev_ptr(y, _bits16(), "y"), ctypes.byref(arm), _stream(stream)),
           "tq_moe_mlp_forward")
    return y, arm.value


def tq_swiglu(gate_up, h=None, stream=None):
    """h = bf16(silu(gate) * up) for gate_up fp32 [P, 2I]."""
    torch = _torch()
    P, I2 = gate_up.shape
    h = torch.empty((P, I2 // 2), dtype=torch.bfloat16, device=gate_up.device) if h is None else h
    _check(lib().tq_swiglu(_dev_ptr(gate_up, (torch.float32,), "gate_up"), P, I2 // 2, _dev_ptr(h, _bits16(), "h"),
                           _stream(stream)), "tq_swiglu")
    return h


def tq_dequantize(packed, lut, expert_ids=None, w_out=None, stream=None):
    """Materialized bf16 weights [m, N, K] of the listed experts (all E when
    expert_ids is None) -- the dequantize-materialize comparator's first step."""
    torch = _torch()
    E, N, kb = packed.shape
    K = kb * 4
    L = lut.numel().bit_length() - 1
    if lut.numel() != (1 << L):
        raise ValueError("lut must have 2^L entries")
    m = E if expert_ids is None else expert_ids.numel()
    w_out = torch.empty((m, N, K), dtype=torch.bfloat16, device=packed.device) if w_out is None else w_out
    ids = None if expert_ids is None else _dev_ptr(expert_ids, (torch.int32,), "expert_ids")
    _check(lib().tq_dequantize(_dev_ptr(packed, (torch.uint8,), "packed"), _dev_ptr(lut, _bits16(), "lut"), L, ids,
                               m, E, N, K, _dev_ptr(w_out, _bits16(), "w_out"), _stream(stream)), "tq_dequantize")
    return w_out


def tq_grouped_gemm_dense(x, w_dense, sorted_pairs, topk_w, tiles, num_tiles, top_k: int, tile_m: int,
                          y32, x_layout: int = X_TOKENS, stream=None) -> None:
    """y32 += grouped product with dense bf16 weights w_dense [E, N, K];
    x and x_layout as in tq_grouped_gemm."""
    torch = _torch()
    n = _x_rows(x, x_layout, top_k)
    K = x.shape[1]
    E, N, K2 = w_dense.shape
    if K2 != K:
        raise ValueError(f"w_dense has K = {K2}, x has {K}")
    _check(lib().tq_grouped_gemm_dense(_dev_ptr(x, _bits16(), "x"), x_layout,
                                       _dev_ptr(w_dense, _bits16(), "w_dense"),
                                       _dev_ptr(sorted_pairs, (torch.int32,), "sorted_pairs"),
                                       _dev_ptr(topk_w, (torch.float32,), "topk_w"),
                                       _dev_ptr(tiles, (torch.int32,), "tiles"),
                                       _dev_ptr(num_tiles, (torch.int32,), "num_tiles"), tiles.shape[0], n,
                                       top_k, E, K, N, tile_m, _dev_ptr(y32, (torch.float32,), "y32"),
                                       _stream(stream)), "tq_grouped_gemm_dense")


def tq_moe_dequant_workspace_size(n: int, top_k: int, E: int, K: int, N: int, tile_m: int) -> int:
    return int(lib().tq_moe_dequant_workspace_size(n, top_k, E, K, N, tile_m))


def tq_moe_forward_dequant(x, packed, lut, topk_ids, topk_w, tile_m: int = 16, workspace=None, y=None,
                           stream=None):
    """Dequantize-materialize comparator: the routed-expert product through
    dense bf16 copies of the woken experts -> y bf16 [n, N]."""
    torch = _torch()
    n, K, E, N, L = _shapes(x, packed, lut)
    top_k = topk_ids.shape[1]
    need = tq_moe_dequant_workspace_size(n, top_k, E, K, N, tile_m)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=x.device)
    y = torch.empty((n, N), dtype=torch.bfloat16, device=x.device) if y is None else y
    _check(lib().tq_moe_forward_dequant(_dev_ptr(x, _bits16(), "x"), _dev_ptr(packed, (torch.uint8,), "packed"),
                                        _dev_ptr(lut, _bits16(), "lut"), L,
                                        _dev_ptr(topk_ids, (torch.int32,), "topk_ids"),
                                        _dev_ptr(topk_w, (torch.float32,), "topk_w"), n, top_k, E, K, N, tile_m,
                                        _dev_ptr(workspace, (torch.uint8,), "workspace"), workspace.numel(),
                                        _dev_ptr(y, _bits16(), "y"), _stream(stream)), "tq_moe_forward_dequant")
    return y


def tq_device_error() -> tuple[int, int]:
    """(code, where) of the first device-side error since the last call; clears it."""
    code, where = ctypes.c_int(0), ctypes.c_int(0)
    _check(lib().tq_device_error(ctypes.byref(code), ctypes.byref(where)), "tq_device_error")
    return code.value, where.value


LAUNCH_COUNTERS = ("route", "tile_map", "grouped", "gemv", "combine", "gather", "router", "dequant",
                   "route_tile_map", "clear", "swiglu")


def tq_launch_counts() -> dict:
    arr = (ctypes.c_int64 * len(LAUNCH_COUNTERS))()
    lib().tq_launch_counts(arr)
    return dict(zip(LAUNCH_COUNTERS, list(arr)))


def tq_launch_counts_all() -> dict:
    """tq_launch_counts and the counters of the scored router and the 4-bit operators."""
    arr = (ctypes.c_int64 * len(ALL_LAUNCH_COUNTERS))()
    lib().tq_launch_counts_all(arr, len(ALL_LAUNCH_COUNTERS))
    return dict(zip(ALL_LAUNCH_COUNTERS, list(arr)))


ALL_LAUNCH_COUNTERS = LAUNCH_COUNTERS + ("router_scored", "router_scored_backward", "fp4_quantize", "fp4_dequantize",
                                         "fp4_tile_scales", "fp4_stage", "fp4_gemm", "fp4_combine", "fp4_swiglu",
                                         "fp4_gemv", "rms_norm", "rms_norm_backward", "rms_norm_weight", "fp8_quantize",
                                         "fp8_dequantize", "fp8_gemm", "few_rows", "gemm_f16",
                                         "swiglu_sum", "swiglu_grad")


# ------------------------------------------------------------------ scored router, 4-bit operators

_type_codes = None


def _type_code(dtype, name):
    """TQ_FP32, TQ_BF16 or TQ_FP16 of a torch dtype."""
    global _type_codes
    if _type_codes is None:
        torch = _torch()
        _type_codes = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
    code = _type_codes.get(dtype)
    if code is None:
        raise TypeError(f"{name} has dtype {dtype}, expected one of {tuple(_type_codes)}")
    return code


def _current_device():
    return _torch().cuda.current_device()


def _elsewhere(t, device, name):
    """The kernels run on the current device: every tensor of a call has to be there."""
    return ValueError(f"{name} is on cuda:{t.get_device()}, the call runs on cuda:{device}" if t.is_cuda
                      else f"{name} must be a CUDA tensor")


def _rows(t, name):
    """(address, type code, elements between rows, rows, elements, device) of a 2-D
    tensor with contiguous rows on the current CUDA device."""
    try:
        code = _type_codes.get(t.dtype) if _type_codes is not None else None
        if code is None:
            code = _type_code(t.dtype, name)
        device = _current_device()
        if t.get_device() != device:
            raise _elsewhere(t, device, name)
        shape = t.shape
        if len(shape) != 2:
            raise ValueError(f"{name} must have two dimensions, not {len(shape)}")
        n, width = shape
        if t.is_contiguous():
            return t.data_ptr(), code, width, n, width, device
        step, inner = t.stride()
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None
    if inner != 1 and width > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return t.data_ptr(), code, step if n > 1 else width, n, width, device


def _there(t, dtypes, name, device):
    """Address of a contiguous tensor of one of `dtypes` on the device."""
    try:
        if t.get_device() == device and (not dtypes or t.dtype in dtypes) and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _dev_ptr(t, dtypes, name)     # raises, unless the device is all that is wrong
    raise _elsewhere(t, device, name)


def _given(t, shape, dtypes, name, device):
    """Address of an argument of a known shape: a contiguous tensor on the device."""
    ptr = _there(t, dtypes, name, device)
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return ptr


_common = None


def _types():
    """torch, its fp32, int32 and uint8 as tuples of one: what the calls below compare with."""
    global _common
    if _common is None:
        torch = _torch()
        _common = torch, (torch.float32,), (torch.int32,), (torch.uint8,)
    return _common


def _scale_ptr(t, count, name, device):
    """Address of `count` fp32 scales, or None."""
    if t is None:
        return None
    ptr = _there(t, _types()[1], name, device)
    if t.numel() != count:
        raise ValueError(f"{name} has {t.numel()} values, expected {count}")
    return ptr


def _empty(shape, dtype, device, stream):
    """A new tensor in the memory of the stream that the call runs on: memory of
    another stream's may still be in use there, or be given away there before
    the call has run."""
    torch = _types()[0]
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def tq_router_scored(logits, top_k: int, score: int = SCORE_SIGMOID, bias=None, groups: int = 1, top_groups: int = 1,
                     renormalize: bool = True, scale: float = 1.0, topk_ids=None, topk_w=None, stream=None):
    """Top-k experts by score + bias within the best groups -> (topk_ids int32 [n, top_k], topk_w fp32 [n, top_k]).

    logits [n, E] fp32, bf16 or fp16 (rows may be strided); score SCORE_SIGMOID
    or SCORE_SOFTMAX; bias fp32 [E] moves the choice, not the weights; of
    `groups` equal groups the `top_groups` with the largest two best values
    stay; the weights are the chosen scores, divided by their sum with
    `renormalize`, times `scale`.  A non-finite logit masks its expert; a row
    with none left has weights 0."""
    torch, fp32, int32, _ = _types()
    ptr, code, step, n, E, device = _rows(logits, "logits")
    if topk_ids is None:
        topk_ids = _empty((n, top_k), torch.int32, logits.device, stream)
        ids_ptr = topk_ids.data_ptr()
    else:
        ids_ptr = _given(topk_ids, (n, top_k), int32, "topk_ids", device)
    if topk_w is None:
        topk_w = _empty((n, top_k), torch.float32, logits.device, stream)
        w_ptr = topk_w.data_ptr()
    else:
        w_ptr = _given(topk_w, (n, top_k), fp32, "topk_w", device)
    rc = _call("tq_router_scored")(ptr, code, step, _scale_ptr(bias, E, "bias", device), n, E, top_k, score, groups,
                                   top_groups, 1 if renormalize else 0, scale, ids_ptr, w_ptr, _stream(stream, device))
    if rc:
        raise TQError(rc, "tq_router_scored")
    return topk_ids, topk_w


def tq_router_scored_backward(logits, topk_ids, topk_w, grad_w, score: int = SCORE_SIGMOID, renormalize: bool = True,
                              scale: float = 1.0, grad_logits=None, stream=None):
    """Gradient of the logits from the gradient of topk_w (fp32 [n, top_k]), in
    the logits' dtype; topk_ids, topk_w and the options are those of the
    forward call."""
    torch, fp32, int32, _ = _types()
    ptr, code, step, n, E, device = _rows(logits, "logits")
    shape = (n, topk_ids.shape[1])
    if grad_logits is None:
        grad_logits = _empty((n, E), logits.dtype, logits.device, stream)
        out = grad_logits.data_ptr()
    else:
        out = _given(grad_logits, (n, E), (logits.dtype,), "grad_logits", device)
    rc = _call("tq_router_scored_backward")(
        ptr, code, step, _given(topk_ids, shape, int32, "topk_ids", device),
        _given(topk_w, shape, fp32, "topk_w", device), _given(grad_w, shape, fp32, "grad_w", device), n, E, shape[1],
        score, 1 if renormalize else 0, scale, out, _stream(stream, device))
    if rc:
        raise TQError(rc, "tq_router_scored_backward")
    return grad_logits


def _fp4_block(fmt):
    if fmt != FP4_NV and fmt != FP4_MX:
        raise ValueError(f"fmt must be FP4_NV or FP4_MX, not {fmt}")
    return 16 if fmt == FP4_NV else 32


def tq_fp4_quantize(x, fmt: int = FP4_NV, global_scale=None, packed=None, scales=None, stream=None):
    """4-bit microscaled copy of x [n, K] (fp32, bf16 or fp16; 16-byte aligned
    rows; K % 32 == 0) -> (packed uint8 [n, K/2], scales uint8 [n, K/16] for
    FP4_NV or [n, K/32] for FP4_MX).  global_scale: fp32 [1] on the device
    (FP4_NV only)."""
    torch, _, _, uint8 = _types()
    ptr, code, step, n, K, device = _rows(x, "x")
    kb = K // _fp4_block(fmt)
    if packed is None:
        packed = _empty((n, K // 2), torch.uint8, x.device, stream)
        p_ptr = packed.data_ptr()
    else:
        p_ptr = _given(packed, (n, K // 2), uint8, "packed", device)
    if scales is None:
        scales = _empty((n, kb), torch.uint8, x.device, stream)
        s_ptr = scales.data_ptr()
    else:
        s_ptr = _given(scales, (n, kb), uint8, "scales", device)
    rc = _call("tq_fp4_quantize")(ptr, code, step, n, K, fmt, _scale_ptr(global_scale, 1, "global_scale", device),
                                  p_ptr, s_ptr, _stream(stream, device))
    if rc:
        raise TQError(rc, "tq_fp4_quantize")
    return packed, scales


def tq_fp4_dequantize(packed, scales, fmt: int = FP4_NV, global_scale=None, dtype=None, out=None, stream=None):
    """The values of tq_fp4_quantize's output, [..., K] of `dtype` (fp32 when
    neither it nor `out` is given)."""
    torch, _, _, uint8 = _types()
    device = torch.cuda.current_device()
    p_ptr, s_ptr = _there(packed, uint8, "packed", device), _there(scales, uint8, "scales", device)
    K = 2 * packed.shape[-1]
    n = packed.numel() // max(K // 2, 1)
    if scales.numel() != n * (K // _fp4_block(fmt)):
        raise ValueError("scales do not match packed")
    shape = (*packed.shape[:-1], K)
    if out is None:
        out = _empty(shape, torch.float32 if dtype is None else dtype, packed.device, stream)
        o_ptr = out.data_ptr()
    else:
        if dtype is not None and out.dtype != dtype:
            raise TypeError(f"out has dtype {out.dtype}, not {dtype}")
        o_ptr = _given(out, shape, (), "out", device)
    rc = _call("tq_fp4_dequantize")(p_ptr, s_ptr, n, K, fmt, _scale_ptr(global_scale, 1, "global_scale", device), o_ptr,
                                    _type_code(out.dtype, "out"), _stream(stream, device))
    if rc:
        raise TQError(rc, "tq_fp4_dequantize")
    return out


def tq_fp4_tiled_scales_size(E: int, N: int, K: int, fmt: int = FP4_NV) -> int:
    return int(lib().tq_fp4_tiled_scales_size(E, N, K, fmt))


def tq_fp4_tile_scales(scales, fmt: int = FP4_NV, tiled=None, stream=None):
    """Block scales [N, K/block] or [E, N, K/block] in the tiled layout the
    products read (1-D uint8); done once, when weights load."""
    torch = _torch()
    E, N, kb = scales.shape if scales.dim() == 3 else (1, *scales.shape)
    K = kb * _fp4_block(fmt)
    size = tq_fp4_tiled_scales_size(E, N, K, fmt)
    tiled = _empty(size, torch.uint8, scales.device, stream) if tiled is None else tiled
    if tiled.numel() != size:
        raise ValueError(f"tiled has {tiled.numel()} bytes, expected {size}")
    device = torch.cuda.current_device()
    _check(lib().tq_fp4_tile_scales(_there(scales, (torch.uint8,), "scales", device), E, N, K, fmt,
                                    _there(tiled, (torch.uint8,), "tiled", device), _stream(stream, device)),
           "tq_fp4_tile_scales")
    return tiled


def _fp4_matrix(packed, tiled_scales, E, N, K, fmt, name, device):
    """Addresses of a 4-bit weight matrix (or E of them), sizes checked."""
    uint8 = _types()[3]
    if packed.shape[-1] != K // 2 or packed.shape[-2] != N or packed.numel() != E * N * (K // 2):
        raise ValueError(f"{name} has shape {tuple(packed.shape)}, expected {(E, N, K // 2)}")
    if tiled_scales.numel() != E * (-(-N // 128) * 128) * (-(-K // 256) * 256 // _fp4_block(fmt)):
        raise ValueError(f"the scales of {name} are not the tiled layout of {E} x {N} x {K}")
    return _there(packed, uint8, name, device), _there(tiled_scales, uint8, "tiled scales", device)


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(size, device, *args):
    """size(*args), which depends on the device's SM count too; `device` is the current one."""
    return size(*args)


def _workspace(workspace, size, device, stream, *args, keep_small=False):
    """(address, bytes) of the caller's workspace, or of a new one of
    size(*args) bytes (none where the call needs none: 256 reported, unless
    keep_small), and the tensor, to be kept until the call is enqueued."""
    torch, _, _, uint8 = _types()
    if workspace is None:
        need = _workspace_bytes(size, device, *args)
        if need <= (0 if keep_small else 256):
            return None, 0, None
        workspace = _empty(need, torch.uint8, device, stream)
        return workspace.data_ptr(), need, workspace
    return _there(workspace, uint8, "workspace", device), workspace.numel(), workspace


def _output(y, shape, x, stream, device):
    """(y, address, type code): the caller's, or a new one in x's dtype."""
    if y is None:
        y = _empty(shape, x.dtype, x.device, stream)
        return y, y.data_ptr(), _type_code(y.dtype, "y")
    return y, _given(y, shape, (), "y", device), _type_code(y.dtype, "y")


def tq_fp4_linear_workspace_size(n: int, K: int, N: int, fmt: int = FP4_NV) -> int:
    return lib().tq_fp4_linear_workspace_size(n, K, N, fmt)


def tq_fp4_linear(x, packed, tiled_scales, fmt: int = FP4_NV, w_scale=None, x_scale=None, workspace=None, y=None,
                  stream=None):
    """x [n, K], quantised by the call, times a 4-bit matrix packed [N, K/2]
    with tiled_scales (tq_fp4_tile_scales) -> y [n, N] in x's dtype (or y's).
    w_scale, x_scale: fp32 [1] global scales (FP4_NV)."""
    ptr, code, step, n, K, device = _rows(x, "x")
    N = packed.shape[-2]
    w_ptr, s_ptr = _fp4_matrix(packed, tiled_scales, 1, N, K, fmt, "packed", device)
    ws_ptr, ws_bytes, workspace = _workspace(workspace, tq_fp4_linear_workspace_size, device, stream, n, K, N, fmt)
    y, y_ptr, y_code = _output(y, (n, N), x, stream, device)
    rc = _call("tq_fp4_linear")(ptr, code, step, w_ptr, s_ptr, fmt, _scale_ptr(w_scale, 1, "w_scale", device),
                                _scale_ptr(x_scale, 1, "x_scale", device), n, K, N, ws_ptr, ws_bytes, y_ptr, y_code,
                                _stream(stream, device))
    if rc:
        raise TQError(rc, "tq_fp4_linear")
    return y


def tq_fp4_moe_workspace_size(n: int, top_k: int, E: int, K: int, N: int, fmt: int = FP4_NV) -> int:
    return lib().tq_fp4_moe_workspace_size(n, top_k, E, K, N, fmt)


def tq_fp4_moe_forward(x, packed, tiled_scales, topk_ids, topk_w, fmt: int = FP4_NV, w_scale=None, x_scale=None,
                       workspace=None, y=None, stream=None):
    """Routed-expert product over 4-bit experts packed [E, N, K/2] with
    tiled_scales (tq_fp4_tile_scales) -> y [n, N] in x's dtype (or y's):
    y[t] = sum_j topk_w[t, j] * W_{topk_ids[t, j]} x[t].  w_scale fp32 [E],
    x_scale fp32 [1]: global scales (FP4_NV)."""
    _, fp32, int32, _ = _types()
    ptr, code, step, n, K, device = _rows(x, "x")
    E, N, _ = packed.shape
    top_k = topk_ids.shape[1]
    w_ptr, s_ptr = _fp4_matrix(packed, tiled_scales, E, N, K, fmt, "packed", device)
    ws_ptr, ws_bytes, workspace = _workspace(workspace, tq_fp4_moe_workspace_size, device, stream, n, top_k, E, K, N,
                                             fmt)
    y, y_ptr, y_code = _output(y, (n, N), x, stream, device)
    rc = _call("tq_fp4_moe_forward")(ptr, code, step, w_ptr, s_ptr, fmt, _scale_ptr(w_scale, E, "w_scale", device),
                                     _scale_ptr(x_scale, 1, "x_scale", device),
                                     _given(topk_ids, (n, top_k), int32, "topk_ids", device),
                                     _given(topk_w, (n, top_k), fp32, "topk_w", device), n, top_k, E, K, N, ws_ptr,
                                     ws_bytes, y_ptr, y_code, _stream(stream, device))
    if rc:
        raise TQError(rc, "tq_fp4_moe_forward")
    return y


def tq_fp4_moe_mlp_workspace_size(n: int, top_k: int, E: int, H: int, I: int, fmt: int = FP4_NV) -> int:
    return lib().tq_fp4_moe_mlp_workspace_size(n, top_k, E, H, I, fmt)


def tq_fp4_moe_mlp_forward(x, packed_gu, tiled_gu, packed_down, tiled_down, topk_ids, topk_w, fmt: int = FP4_NV,
                           gu_scale=None, down_scale=None, x_scale=None, h_scale=None, workspace=None, y=None,
                           stream=None):
    """SwiGLU expert MLP over 4-bit experts: packed_gu [E, 2I, H/2] (gate rows,
    then up rows), packed_down [E, H, I/2] -> y [n, H] in x's dtype (or y's).
    gu_scale, down_scale fp32 [E]; x_scale, h_scale fp32 [1], the global scales
    of x and of h = silu(gate) * up (FP4_NV)."""
    _, fp32, int32, _ = _types()
    ptr, code, step, n, H, device = _rows(x, "x")
    E, I = packed_gu.shape[0], packed_gu.shape[1] // 2
    top_k = topk_ids.shape[1]
    gu_ptr, gus_ptr = _fp4_matrix(packed_gu, tiled_gu, E, 2 * I, H, fmt, "packed_gu", device)
    d_ptr, ds_ptr = _fp4_matrix(packed_down, tiled_down, E, H, I, fmt, "packed_down", device)
    ws_ptr, ws_bytes, workspace = _workspace(workspace, tq_fp4_moe_mlp_workspace_size, device, stream, n, top_k, E, H,
                                             I, fmt)
    y, y_ptr, y_code = _output(y, (n, H), x, stream, device)
    rc = _call("tq_fp4_moe_mlp_forward")(
        ptr, code, step, gu_ptr, gus_ptr, _scale_ptr(gu_scale, E, "gu_scale", device), d_ptr, ds_ptr,
        _scale_ptr(down_scale, E, "down_scale", device), fmt, _scale_ptr(x_scale, 1, "x_scale", device),
        _scale_ptr(h_scale, 1, "h_scale", device), _given(topk_ids, (n, top_k), int32, "topk_ids", device),
        _given(topk_w, (n, top_k), fp32, "topk_w", device), n, top_k, E, H, I, ws_ptr, ws_bytes, y_ptr, y_code,
        _stream(stream, device))
    if rc:
        raise TQError(rc, "tq_fp4_moe_mlp_forward")
    return y


# ------------------------------------------------------------------ norm

def _same_rows(t, n, K, dtype, name):
    """(address, elements between rows) of rows that go with x [n, K]."""
    ptr, _, step, rows, width, _ = _rows(t, name)
    if rows != n or width != K:
        raise ValueError(f"{name} has shape {(rows, width)}, expected {(n, K)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    return ptr, step


def _norm_weight(weight, K, device):
    """(address, type code) of the weights, or of none."""
    if weight is None:
        return None, 0
    return _given(weight, (K,), (), "weight", device), _type_code(weight.dtype, "weight")


def _norm_rows(x, weight, residual, residual_out, stream):
    """What both forms of the norm take: x's, the residual's and the weight's addresses
    and strides, and residual_out."""
    ptr, code, step, n, K, device = _rows(x, "x")
    w_ptr, w_code = _norm_weight(weight, K, device)
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out is an output of the addition of a residual")
        return n, K, device, (ptr, code, step, None, 0, w_ptr, w_code), x, None
    dtype = x.dtype
    r_ptr, r_step = _same_rows(residual, n, K, dtype, "residual")
    if residual_out is None:
        residual_out = _empty((n, K), dtype, x.device, stream)
        o_ptr = residual_out.data_ptr()
    else:
        o_ptr = _given(residual_out, (n, K), (dtype,), "residual_out", device)
    return n, K, device, (ptr, code, step, r_ptr, r_step, w_ptr, w_code), residual_out, o_ptr


def tq_rms_norm(x, weight=None, eps: float = 1e-6, residual=None, y=None, residual_out=None, rstd=None, stream=None):
    """RMS norm of r = x + residual over rows x [n, K] (fp32, bf16 or fp16; rows may
    be strided) -> (y, r, rstd): y = r * rstd * weight in x's dtype; r as the next
    block's residual and the gradient take it (x itself without a residual; in place
    with residual_out=residual); rstd fp32 [n] = 1 / sqrt(mean(r^2) + eps).  weight:
    [K] of any of the three types, or None for ones."""
    torch, fp32, _, _ = _types()
    n, K, device, rows, r, o_ptr = _norm_rows(x, weight, residual, residual_out, stream)
    if y is None:
        y = _empty((n, K), x.dtype, x.device, stream)
        y_ptr = y.data_ptr()
    else:
        y_ptr = _given(y, (n, K), (x.dtype,), "y", device)
    if rstd is None:
        rstd = _empty((n,), torch.float32, x.device, stream)
        rstd_ptr = rstd.data_ptr()
    else:
        rstd_ptr = _given(rstd, (n,), fp32, "rstd", device)
    rc = _call("tq_rms_norm")(*rows, eps, n, K, o_ptr, y_ptr, rstd_ptr, None, None, _stream(stream, device))
    if rc:
        raise TQError(rc, "tq_rms_norm")
    return y, r, rstd


def tq_rms_norm_fp8(x, weight=None, eps: float = 1e-6, residual=None, codes=None, scales=None, y=None,
                    residual_out=None, stream=None):
    """tq_rms_norm with its output in 8 bits, as tq_fp8_linear and the experts read
    it -> (codes float8_e4m3fn [n, K], scales fp32 [n, ceil(K / 128)], r).  K a
    multiple of 16, rows 16-byte aligned.  With y (a tensor [n, K] in x's dtype) the
    unquantised output is written too."""
    torch, fp32, _, _ = _types()
    n, K, device, rows, r, o_ptr = _norm_rows(x, weight, residual, residual_out, stream)
    y_ptr = None if y is None else _given(y, (n, K), (x.dtype,), "y", device)
    blocks = (K + 127) // 128
    if codes is None:
        codes = _empty((n, K), torch.float8_e4m3fn, x.device, stream)
        c_ptr = codes.data_ptr()
    else:
        c_ptr = _given(codes, (n, K), _fp8(), "codes", device)
    if scales is None:
        scales = _empty((n, blocks), torch.float32, x.device, stream)
        s_ptr = scales.data_ptr()
    else:
        s_ptr = _given(scales, (n, blocks), fp32, "scales", device)
    rc = _call("tq_rms_norm")(*rows, eps, n, K, o_ptr, y_ptr, None, c_ptr, s_ptr, _stream(stream, device))
    if rc:
        raise TQError(rc, "tq_rms_norm_fp8")
    return codes, scales, r


def tq_rms_norm_backward_workspace_size(n: int, K: int) -> int:
    return lib().tq_rms_norm_backward_workspace_size(n, K)


def tq_rms_norm_backward(grad_y, x, weight, rstd, grad_residual=None, grad_x=None, grad_weight=None, workspace=None,
                         stream=None):
    """Gradients of tq_rms_norm -> (grad_x, grad_weight): x is the normed r and rstd
    what that call returned, grad_residual the gradient that arrives through r.
    grad_x, in x's dtype, is the gradient of the call's x and residual alike;
    grad_weight has the weight's dtype (None without a weight)."""
    torch, fp32, _, _ = _types()
    ptr, code, step, n, K, device = _rows(x, "x")
    dy_ptr, dy_step = _same_rows(grad_y, n, K, x.dtype, "grad_y")
    w_ptr, w_code = _norm_weight(weight, K, device)
    g_ptr, g_step = (None, 0) if grad_residual is None else _same_rows(grad_residual, n, K, x.dtype, "grad_residual")
    grad_x, gx_ptr = _dense(grad_x, n, K, x, "grad_x", device, stream)
    gw_ptr = ws_ptr = None
    ws_bytes = 0
    if weight is not None:
        if grad_weight is None:
            grad_weight = _empty((K,), weight.dtype, x.device, stream)
            gw_ptr = grad_weight.data_ptr()
        else:
            gw_ptr = _given(grad_weight, (K,), (weight.dtype,), "grad_weight", device)
        ws_ptr, ws_bytes, workspace = _workspace(workspace, tq_rms_norm_backward_workspace_size, device, stream, n, K,
                                                 keep_small=True)
    elif grad_weight is not None:
        raise ValueError("grad_weight needs a weight")
    rc = _call("tq_rms_norm_backward")(dy_ptr, dy_step, ptr, code, step, w_ptr, w_code,
                                       _given(rstd, (n,), fp32, "rstd", device), g_ptr, g_step, n, K, ws_ptr, ws_bytes,
                                       gx_ptr, gw_ptr, _stream(stream, device))
    if rc:
        raise TQError(rc, "tq_rms_norm_backward")
    return grad_x, grad_weight


def _dense(t, rows, width, x, name, device, stream):
    """(tensor, address) of a dense output [rows, width] in x's dtype: the caller's, or a new one."""
    if t is None:
        t = _empty((rows, width), x.dtype, x.device, stream)
        return t, t.data_ptr()
    return t, _given(t, (rows, width), (x.dtype,), name, device)


# ------------------------------------------------------------------ 8-bit operators

_code_types = None


def _fp8():
    """The dtypes that 8-bit codes may have."""
    global _code_types
    if _code_types is None:
        torch = _torch()
        _code_types = (torch.float8_e4m3fn, torch.uint8)
    return _code_types


def _fp8_rows(x, x_scales):
    """(address, scales' address, rows, K, device) of 8-bit activations [n, K]."""
    device = _current_device()
    ptr = _there(x, _fp8(), "x", device)
    shape = x.shape
    if len(shape) != 2:
        raise ValueError(f"x must have two dimensions, not {len(shape)}")
    n, K = shape
    return ptr, _given(x_scales, (n, (K + 127) // 128), _types()[1], "x_scales", device), n, K, device


def _fp8_matrix(w, scales, E, N, K, name, device):
    """Addresses of 8-bit weights [N, K] (E None) or [E, N, K] and of their scales."""
    blocks = ((N + 127) // 128, (K + 127) // 128)
    return (_given(w, (N, K) if E is None else (E, N, K), _fp8(), name, device),
            _given(scales, blocks if E is None else (E, *blocks), _types()[1], f"the scales of {name}", device))


def _fp8_blocking(shape, rows_per_block, name):
    """(matrices, rows of each, K, shape of the scales) of values [n, K] or [E, n, K]."""
    if rows_per_block != 1 and rows_per_block != FP8_BLOCK:
        raise ValueError(f"rows_per_block must be 1 or {FP8_BLOCK}, not {rows_per_block}")
    if len(shape) == 2:
        n, K = shape
        return 1, n, K, (-(-n // rows_per_block), (K + 127) // 128)
    if len(shape) != 3:
        raise ValueError(f"{name} must have two or three dimensions, not {len(shape)}")
    E, n, K = shape
    return E, n, K, (E, -(-n // rows_per_block), (K + 127) // 128)


def tq_fp8_quantize(x, rows_per_block: int = 1, codes=None, scales=None, stream=None):
    """8-bit block-scaled copy of x [n, K] or [E, n, K] (fp32, bf16 or fp16; 16-byte
    aligned rows; K % 16 == 0) -> (codes float8_e4m3fn of x's shape, scales fp32
    [.., ceil(n / rows_per_block), ceil(K / 128)]).  rows_per_block: 1 for
    activations (rows may be strided), 128 for weights."""
    torch, fp32, _, _ = _types()
    shape = x.shape
    E, n, K, blocks = _fp8_blocking(shape, rows_per_block, "x")
    if len(shape) == 3:
        if not x.is_contiguous():
            raise ValueError("x [E, n, K] must be contiguous")
        x = x.view(E * n, K)
    ptr, code, step, _, _, device = _rows(x, "x")
    if codes is None:
        codes = _empty(shape, torch.float8_e4m3fn, x.device, stream)
        c_ptr = codes.data_ptr()
    else:
        c_ptr = _given(codes, shape, _fp8(), "codes", device)
    if scales is None:
        scales = _empty(blocks, torch.float32, x.device, stream)
        s_ptr = scales.data_ptr()
    else:
        s_ptr = _given(scales, blocks, fp32, "scales", device)
    rc = _call("tq_fp8_quantize")(ptr, code, step, E, n, K, rows_per_block, c_ptr, s_ptr, _stream(stream, device))
    if rc:
        raise TQError(rc, "tq_fp8_quantize")
    return codes, scales


def tq_fp8_dequantize(codes, scales, rows_per_block: int = 1, dtype=None, out=None, stream=None):
    """The values of tq_fp8_quantize's output, in `dtype` (fp32 when neither it nor
    `out` is given)."""
    torch, fp32, _, _ = _types()
    device = _current_device()
    c_ptr = _there(codes, _fp8(), "codes", device)
    shape = codes.shape
    E, n, K, blocks = _fp8_blocking(shape, rows_per_block, "codes")
    s_ptr = _given(scales, blocks, fp32, "scales", device)
    if out is None:
        out = _empty(shape, torch.float32 if dtype is None else dtype, codes.device, stream)
        o_ptr = out.data_ptr()
    else:
        if dtype is not None and out.dtype != dtype:
            raise TypeError(f"out has dtype {out.dtype}, not {dtype}")
        o_ptr = _given(out, shape, (), "out", device)
    rc = _call("tq_fp8_dequantize")(c_ptr, s_ptr, E, n, K, rows_per_block, o_ptr, _type_code(out.dtype, "out"),
                                    _stream(stream, device))
    if rc:
        raise TQError(rc, "tq_fp8_dequantize")
    return out


def _result(y, shape, dtype, x, stream, device):
    """(y, address, type code) of a product: the caller's, or a new one of `dtype` (bf16 by default)."""
    if y is None:
        y = _empty(shape, _types()[0].bfloat16 if dtype is None else dtype, x.device, stream)
        return y, y.data_ptr(), _type_code(y.dtype, "y")
    if dtype is not None and y.dtype != dtype:
        raise TypeError(f"y has dtype {y.dtype}, not {dtype}")
    return y, _given(y, shape, (), "y", device), _type_code(y.dtype, "y")


def tq_fp8_linear_workspace_size(n: int, K: int, N: int) -> int:
    return lib().tq_fp8_linear_workspace_size(n, K, N)


def tq_fp8_linear(x, x_scales, w, w_scales, dtype=None, workspace=None, y=None, stream=None):
    """8-bit rows x [n, K] (tq_fp8_quantize or tq_rms_norm_fp8) times an 8-bit matrix
    w [N, K] with scales [ceil(N / 128), ceil(K / 128)] -> y [n, N] in `dtype`
    (bf16 by default)."""
    ptr, xs_ptr, n, K, device = _fp8_rows(x, x_scales)
    N = w.shape[0]
    w_ptr, ws_ptr = _fp8_matrix(w, w_scales, None, N, K, "w", device)
    work_ptr, work_bytes, workspace = _workspace(workspace, tq_fp8_linear_workspace_size, device, stream, n, K, N)
    y, y_ptr, y_code = _result(y, (n, N), dtype, x, stream, device)
    rc = _call("tq_fp8_linear")(ptr, xs_ptr, w_ptr, ws_ptr, n, K, N, work_ptr, work_bytes, y_ptr, y_code,
                                _stream(stream, device))
    if rc:
        raise TQError(rc, "tq_fp8_linear")
    return y


def tq_fp8_moe_workspace_size(n: int, top_k: int, E: int, K: int, N: int) -> int:
    return lib().tq_fp8_moe_workspace_size(n, top_k, E, K, N)


def tq_fp8_moe_forward(x, x_scales, w, w_scales, topk_ids, topk_w, dtype=None, workspace=None, y=None, stream=None):
    """Routed-expert product over 8-bit experts w [E, N, K] with scales [E,
    ceil(N / 128), ceil(K / 128)] -> y [n, N] in `dtype` (bf16 by default):
    y[t] = sum_j topk_w[t, j] * W_{topk_ids[t, j]} x[t]."""
    _, fp32, int32, _ = _types()
    ptr, xs_ptr, n, K, device = _fp8_rows(x, x_scales)
    E, N = w.shape[0], w.shape[1]
    top_k = topk_ids.shape[1]
    w_ptr, ws_ptr = _fp8_matrix(w, w_scales, E, N, K, "w", device)
    work_ptr, work_bytes, workspace = _workspace(workspace, tq_fp8_moe_workspace_size, device, stream, n, top_k, E, K, N,
                                                 keep_small=True)
    y, y_ptr, y_code = _result(y, (n, N), dtype, x, stream, device)
    rc = _call("tq_fp8_moe_forward")(ptr, xs_ptr, w_ptr, ws_ptr, _given(topk_ids, (n, top_k), int32, "topk_ids", device),
                                     _given(topk_w, (n, top_k), fp32, "topk_w", device), n, top_k, E, K, N, work_ptr,
                                     work_bytes, y_ptr, y_code, _stream(stream, device))
    if rc:
        raise TQError(rc, "tq_fp8_moe_forward")
    return y


def tq_fp8_moe_mlp_workspace_size(n: int, top_k: int, E: int, H: int, I: int) -> int:
    return lib().tq_fp8_moe_mlp_workspace_size(n, top_k, E, H, I)


def tq_fp8_moe_mlp_forward(x, x_scales, w_gu, gu_scales, w_down, down_scales, topk_ids, topk_w, dtype=None,
                           workspace=None, y=None, stream=None):
    """SwiGLU expert MLP over 8-bit experts: w_gu [E, 2I, H] (gate rows, then up
    rows), w_down [E, H, I], I a multiple of 128 -> y [n, H] in `dtype` (bf16 by
    default).  h = silu(gate) * up is kept in 8 bits between the products."""
    _, fp32, int32, _ = _types()
    ptr, xs_ptr, n, H, device = _fp8_rows(x, x_scales)
    E, I = w_gu.shape[0], w_gu.shape[1] // 2
    top_k = topk_ids.shape[1]
    gu_ptr, gus_ptr = _fp8_matrix(w_gu, gu_scales, E, 2 * I, H, "w_gu", device)
    d_ptr, ds_ptr = _fp8_matrix(w_down, down_scales, E, H, I, "w_down", device)
    work_ptr, work_bytes, workspace = _workspace(workspace, tq_fp8_moe_mlp_workspace_size, device, stream, n, top_k, E, H,
                                                 I, keep_small=True)
    y, y_ptr, y_code = _result(y, (n, H), dtype, x, stream, device)
    rc = _call("tq_fp8_moe_mlp_forward")(
        ptr, xs_ptr, gu_ptr, gus_ptr, d_ptr, ds_ptr, _given(topk_ids, (n, top_k), int32, "topk_ids", device),
        _given(topk_w, (n, top_k), fp32, "topk_w", device), n, top_k, E, H, I, work_ptr, work_bytes, y_ptr, y_code,
        _stream(stream, device))
    if rc:
        raise TQError(rc, "tq_fp8_moe_mlp_forward")
    return y


# ------------------------------------------------------------------ gated projection

def _rows16(x):
    """_rows of a 16-bit tensor."""
    rows = _rows(x, "x")
    if rows[1] == 0:
        raise TypeError(f"x has dtype {x.dtype}, expected bf16 or fp16")
    return rows


def tq_swiglu_linear_workspace_size(n: int, H: int, I: int) -> int:
    return lib().tq_swiglu_linear_workspace_size(n, H, I)


def tq_swiglu_linear(x, w_gu, h=None, gate_up=None, workspace=None, stream=None):
    """h [n, I] = silu(x Wg^T) * (x Wu^T) for x [n, H] in bf16 or fp16 (rows may be
    strided) and w_gu [2I, H] of the same dtype, gate rows first; H and I multiples
    of 8.  With gate_up (fp32 [n, 2I]) gate and up are kept there for the gradient."""
    _, fp32, _, _ = _types()
    ptr, code, step, n, H, device = _rows16(x)
    I = w_gu.shape[0] // 2
    w_ptr = _given(w_gu, (2 * I, H), (x.dtype,), "w_gu", device)
    h, h_ptr = _dense(h, n, I, x, "h", device, stream)
    gu_ptr = None if gate_up is None else _given(gate_up, (n, 2 * I), fp32, "gate_up", device)
    work_ptr, work_bytes, workspace = _workspace(workspace, tq_swiglu_linear_workspace_size, device, stream, n, H, I)
    rc = _call("tq_swiglu_linear")(ptr, code, step, w_ptr, n, H, I, work_ptr, work_bytes, h_ptr, gu_ptr,
                                   _stream(stream, device))
    if rc:
        raise TQError(rc, "tq_swiglu_linear")
    return h


def tq_swiglu_linear_backward_workspace_size(n: int, H: int, I: int, has_gate_up: bool = True) -> int:
    return lib().tq_swiglu_linear_backward_workspace_size(n, H, I, 1 if has_gate_up else 0)


def tq_swiglu_linear_backward(x, w_gu, grad_h, gate_up=None, grad_x=None, grad_w_gu=None, workspace=None, stream=None):
    """Gradients of tq_swiglu_linear from that of h -> (grad_x [n, H], grad_w_gu
    [2I, H]) in x's dtype.  gate_up: what the forward call kept, or None to compute
    it again."""
    _, fp32, _, _ = _types()
    ptr, code, step, n, H, device = _rows16(x)
    I = w_gu.shape[0] // 2
    w_ptr = _given(w_gu, (2 * I, H), (x.dtype,), "w_gu", device)
    gh_ptr = _given(grad_h, (n, I), (x.dtype,), "grad_h", device)
    gu_ptr = None if gate_up is None else _given(gate_up, (n, 2 * I), fp32, "gate_up", device)
    grad_x, gx_ptr = _dense(grad_x, n, H, x, "grad_x", device, stream)
    grad_w_gu, gw_ptr = _dense(grad_w_gu, 2 * I, H, x, "grad_w_gu", device, stream)
    work_ptr, work_bytes, workspace = _workspace(workspace, tq_swiglu_linear_backward_workspace_size, device, stream, n,
                                                 H, I, gate_up is not None, keep_small=True)
    rc = _call("tq_swiglu_linear_backward")(ptr, code, step, w_ptr, gu_ptr, gh_ptr, n, H, I, work_ptr, work_bytes, gx_ptr,
                                            gw_ptr, _stream(stream, device))
    if rc:
        raise TQError(rc, "tq_swiglu_linear_backward")
    return grad_x, grad_w_gu
