// Gated projection in 16 bits and its gradient: the entry points, and the gradient of
// the activation.
#include <cuda_runtime.h>

#include <algorithm>

#include "tq_device.cuh"
#include "tq_internal.h"
#include "tq_tiling.h"
#include "tq_types.cuh"

namespace tq {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxIndex = (static_cast<int64_t>(1) << 31) - 1024;
size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// d = [dgate dup] of 8 columns a thread; reads gate, up and grad_h once: bound by memory.
template <typename T>
__global__ void __launch_bounds__(kThreads)
swiglu_grad_kernel(const float* __restrict__ gate_up, const T* __restrict__ grad_h, long long rows, int I,
                   T* __restrict__ d) {
  pdl_wait();
  pdl_trigger();
  const int items = I / 8;
  const long long total = rows * items, step = static_cast<long long>(gridDim.x) * kThreads;
  for (long long i = blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x; i < total; i += step) {
    const long long row = i / items;
    const int col = 8 * static_cast<int>(i - row * items);
    const float4* const g = reinterpret_cast<const float4*>(gate_up + row * 2 * I + col);
    const float4* const u = g + I / 4;
    float4 gv[2] = {__ldcs(g), __ldcs(g + 1)}, uv[2] = {__ldcs(u), __ldcs(u + 1)};
    const uint4 raw = __ldg(reinterpret_cast<const uint4*>(grad_h) + i);
    const T* const h = reinterpret_cast<const T*>(&raw);
    const float* const gs = reinterpret_cast<const float*>(gv);
    const float* const us = reinterpret_cast<const float*>(uv);
    T dg[8], du[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float s = 1.f / (1.f + expf(-gs[j])), dh = widen(h[j]);
      dg[j] = narrow<T>(dh * us[j] * (s * (1.f + gs[j] * (1.f - s))));
      du[j] = narrow<T>(dh * (gs[j] * s));
    }
    T* const out = d + row * 2 * I + col;
    *reinterpret_cast<uint4*>(out) = *reinterpret_cast<const uint4*>(dg);
    *reinterpret_cast<uint4*>(out + I) = *reinterpret_cast<const uint4*>(du);
  }
}

bool bad_sizes(int64_t n, int H, int I) {
  return n < 0 || n >= kMaxIndex || H < 8 || H % 8 != 0 || H >= kMaxIndex || I < 8 || I % 8 != 0 || 2ll * I >= kMaxIndex ||
         static_cast<double>(n) * H >= 0x1p57 || 2.0 * n * I >= 0x1p57 || 2.0 * I * H >= 0x1p57;
}
bool bad_type16(int type) { return type != TQ_BF16 && type != TQ_FP16; }
bool bad_x(const void* x, int64_t stride, int64_t n, int H) {
  return stride < H || stride % 8 != 0 || (n > 1 && static_cast<double>(n) * static_cast<double>(stride) >= 0x1p57) ||
         stride >= (1ll << 38) || (n > 0 && (!x || !aligned(x, 16)));
}

constexpr int64_t kFewRowsMost = 16;

int forward(const void* x, int type, int64_t x_stride, const void* w, int64_t n, int H, int I, void* h, float* gate_up,
            int* err, cudaStream_t s) {
  if (n <= kFewRowsMost) {
    FewRows f{};
    f.w = static_cast<const uint8_t*>(w);
    f.x = static_cast<const uint8_t*>(x);
    f.row_bytes = 2ll * H;
    f.x_stride = 2 * x_stride;
    f.M = static_cast<int>(n);
    f.E = f.top_k = f.segments = 1;
    f.N = I;
    f.steps = (H + 63) / 64;
    f.y = h;
    f.y_type = type;
    f.gate_up = gate_up;
    f.err = err;
    return launch_few_rows(f, type, true, n <= 8 ? 8 : 16, 1, s);
  }
  const TileChoice t = choose_tile(static_cast<double>(n), 1.0, (H + 63) / 64, I, true, TileRows::kOne, false, false);
  GemmF16 g{type, x, x_stride, w, H, n, I, H, false, false, true, t.tile_m, t.cols, 1, h, type, gate_up, err};
  return launch_gemm_f16(g, s);
}

// The two products of the gradient.
TileChoice tile_x(int64_t n, int H, int I) {
  return choose_tile(static_cast<double>(n), 1.0, static_cast<int>((2ll * I + 63) / 64), H, false, TileRows::kOne, false, true);
}
TileChoice tile_w(int64_t n, int H, int I) {
  return choose_tile(2.0 * I, 1.0, static_cast<int>((n + 63) / 64), H, false, TileRows::kOne, false, true);
}
TileChoice at_least_64(TileChoice t) {   // operands across K come in boxes of 64 columns
  t.cols = std::max(t.cols, 64);
  return t;
}

struct GradPlan {
  TileChoice x, w;
  size_t gate_up, d, part, bytes;   // offsets
};
GradPlan plan(int64_t n, int H, int I, bool has_gate_up) {
  GradPlan p;
  p.x = at_least_64(tile_x(n, H, I));
  p.w = at_least_64(tile_w(n, H, I));
  size_t used = 0;
  auto take = [&](double values, size_t size) {
    const size_t at = used;
    used += align256(static_cast<size_t>(values) * size);
    return at;
  };
  p.gate_up = take(has_gate_up ? 0 : 2.0 * n * I, 4);
  p.d = take(2.0 * n * I, 2);
  const double sums_x = p.x.splits > 1 ? static_cast<double>(p.x.splits) * n * H : 0;
  const double sums_w = p.w.splits > 1 ? static_cast<double>(p.w.splits) * 2 * I * H : 0;
  p.part = take(std::max(sums_x, sums_w), 4);   // in turn: the second product starts after the first's sums are read
  p.bytes = std::max<size_t>(used, 256);
  return p;
}

int product(GemmF16 g, TileChoice t, void* part, void* y, int type, cudaStream_t s) {
  g.tile_m = t.tile_m;
  g.cols = t.cols;
  g.splits = t.splits;
  g.y = t.splits > 1 ? part : y;
  g.y_type = t.splits > 1 ? TQ_FP32 : type;
  const int rc = launch_gemm_f16(g, s);
  if (rc != TQ_OK || t.splits == 1) return rc;
  return launch_fp4_combine(static_cast<const float*>(part), g.M * g.N, t.splits, nullptr, nullptr, nullptr, nullptr,
                            g.M, 1, 1, static_cast<int>(g.N), y, type, s);
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" {

int tq_swiglu_linear(const void* x, int type, int64_t x_stride, const void* w_gu, int64_t n, int H, int I, void* h,
                     float* gate_up, tq_stream_t stream) {
  if (bad_sizes(n, H, I) || bad_type16(type) || bad_x(x, x_stride, n, H)) return TQ_ERR_INVALID_ARG;
  if (n > 0 && (!w_gu || (!h && !gate_up) || !aligned(w_gu, 16) || !aligned(h, 16) || !aligned(gate_up, 16)))
    return TQ_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int rc = require_sm103(s);
  if (rc != TQ_OK || n == 0) return rc;
  int* err = error_word(&rc);
  if (!err) return rc;
  return forward(x, type, x_stride, w_gu, n, H, I, h, gate_up, err, s);
}

size_t tq_swiglu_linear_backward_workspace_size(int64_t n, int H, int I, int has_gate_up) {
  return bad_sizes(n, H, I) ? 0 : plan(n, H, I, has_gate_up != 0).bytes;
}

int tq_swiglu_linear_backward(const void* x, int type, int64_t x_stride, const void* w_gu, const float* gate_up,
                              const void* grad_h, int64_t n, int H, int I, void* workspace, size_t workspace_bytes,
                              void* grad_x, void* grad_w_gu, tq_stream_t stream) {
  if (bad_sizes(n, H, I) || bad_type16(type) || bad_x(x, x_stride, n, H) || (!grad_x && !grad_w_gu))
    return TQ_ERR_INVALID_ARG;
  if (n > 0 && (!w_gu || !grad_h || !aligned(w_gu, 16) || !aligned(grad_h, 16) || !aligned(gate_up, 16) ||
                !aligned(grad_x, 16) || !aligned(grad_w_gu, 16)))
    return TQ_ERR_INVALID_ARG;
  const GradPlan p = plan(n, H, I, gate_up != nullptr);
  if (n > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < p.bytes)) return TQ_ERR_WORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int rc = require_sm103(s);
  if (rc != TQ_OK) return rc;
  if (n == 0) {   // a sum over no rows
    if (grad_w_gu && cudaMemsetAsync(grad_w_gu, 0, 4ull * I * H, s) != cudaSuccess) return launch_status();
    return TQ_OK;
  }
  int* err = error_word(&rc);
  if (!err) return rc;
  uint8_t* const base = static_cast<uint8_t*>(workspace);
  if (!gate_up) {
    float* const again = reinterpret_cast<float*>(base + p.gate_up);
    rc = forward(x, type, x_stride, w_gu, n, H, I, nullptr, again, err, s);
    if (rc != TQ_OK) return rc;
    gate_up = again;
  }
  void* const d = base + p.d;
  const int blocks = static_cast<int>(std::min<int64_t>((n * (I / 8) + kThreads - 1) / kThreads, sm_count() * 16ll));
  rc = type == TQ_BF16
           ? launch_pdl(swiglu_grad_kernel<__nv_bfloat16>, dim3(blocks), dim3(kThreads), 0, s, gate_up,
                        static_cast<const __nv_bfloat16*>(grad_h), static_cast<long long>(n), I,
                        static_cast<__nv_bfloat16*>(d))
           : launch_pdl(swiglu_grad_kernel<__half>, dim3(blocks), dim3(kThreads), 0, s, gate_up,
                        static_cast<const __half*>(grad_h), static_cast<long long>(n), I, static_cast<__half*>(d));
  if (rc != TQ_OK) return rc;
  count_launch(kCntSwigluGrad);
  if (grad_x) {
    GemmF16 g{type, d, 2ll * I, w_gu, H, n, H, 2ll * I, false, true, false, 0, 0, 0, nullptr, 0, nullptr, err};
    rc = product(g, p.x, base + p.part, grad_x, type, s);
    if (rc != TQ_OK) return rc;
  }
  if (!grad_w_gu) return TQ_OK;
  GemmF16 g{type, d, 2ll * I, x, x_stride, 2ll * I, H, n, true, true, false, 0, 0, 0, nullptr, 0, nullptr, err};
  return product(g, p.w, base + p.part, grad_w_gu, type, s);
}

}  // extern "C"
