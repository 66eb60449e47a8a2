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

// d = [dgate dup] of 8 columns a thread; reads gate, up and grad_h once: bound by memory
// (8192 rows of 2048: 30 us for 235 MB, most of its writes left in L2).
//
// d is rounded to the type: it is an operand of both products, and the tensor cores take
// operands of 16 bits.  The gradients are off by 2.3e-3 of themselves for it (rms, bf16, 8192
// rows 4096 -> 2 x 2048), where their own rounding is 1.7e-3; with d in two parts, each
// product run twice, they would take 300 us more of 545.
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
      const float s = sigmoid(gs[j]), dh = widen(h[j]);
      dg[j] = narrow<T>(dh * us[j] * (s * (1.f + gs[j] * (1.f - s))));
      du[j] = narrow<T>(dh * (gs[j] * s));
    }
    T* const out = d + row * 2 * I + col;
    *reinterpret_cast<uint4*>(out) = *reinterpret_cast<const uint4*>(dg);
    *reinterpret_cast<uint4*>(out + I) = *reinterpret_cast<const uint4*>(du);
  }
}

// h (and gate and up) from the gate and up projections' partial sums, added in order: 4
// columns a thread.
template <typename T>
__global__ void __launch_bounds__(kThreads)
swiglu_sum_kernel(const float* __restrict__ part, long long split_stride, int splits, long long rows, int I,
                  T* __restrict__ h, float* __restrict__ gate_up) {
  pdl_wait();
  pdl_trigger();
  const int items = I / 4;
  const long long total = rows * items, step = static_cast<long long>(gridDim.x) * kThreads;
  for (long long i = blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x; i < total; i += step) {
    const long long row = i / items, at = row * 2 * I + 4 * (i - row * items);
    float4 g = make_float4(0.f, 0.f, 0.f, 0.f), u = g;
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
      const float4 a = __ldcs(reinterpret_cast<const float4*>(part + s * split_stride + at));
      const float4 b = __ldcs(reinterpret_cast<const float4*>(part + s * split_stride + at + I));
      g = make_float4(g.x + a.x, g.y + a.y, g.z + a.z, g.w + a.w);
      u = make_float4(u.x + b.x, u.y + b.y, u.z + b.z, u.w + b.w);
    }
    if (gate_up) {
      *reinterpret_cast<float4*>(gate_up + at) = g;
      *reinterpret_cast<float4*>(gate_up + at + I) = u;
    }
    if (!h) continue;
    const float gs[4] = {g.x, g.y, g.z, g.w}, us[4] = {u.x, u.y, u.z, u.w};
    T out[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) out[j] = narrow<T>(silu(gs[j]) * us[j]);
    *reinterpret_cast<uint2*>(h + 4 * i) = *reinterpret_cast<const uint2*>(out);
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

// How gate, up and h are computed: by the few-rows kernel; in one launch of tiles; or,
// where few rows make few tiles, in tiles with K split and a launch that adds up (128
// rows 4096 -> 2 x 2048 took 25.7 us in one launch of 32 tiles).
struct ForwardPlan {
  bool few, split;
  TileChoice tile;
  size_t part;   // bytes of partial sums
};
ForwardPlan plan_forward(int64_t n, int H, int I) {
  ForwardPlan f{};
  const int steps = (H + 63) / 64;
  f.tile = choose_tile(false, static_cast<double>(std::max<int64_t>(n, 1)), 1.0, steps, I, true, TileRows::kOne, false, false);
  const TileChoice plain = choose_tile(false, static_cast<double>(std::max<int64_t>(n, 1)), 1.0, steps, 2ll * I, false,
                                       TileRows::kOne, true, true, 64);
  f.few = few_rows_cost(n, 4.0 * I * H, false) < std::min(plain.cost, f.tile.cost);
  f.split = !f.few && plain.cost < f.tile.cost;
  if (f.split) {
    f.tile = plain;
    f.part = align256(static_cast<size_t>(plain.splits) * n * 2 * I * sizeof(float));
  }
  return f;
}

// Blocks of the kernels that walk rows * columns items.
int walk_blocks(int64_t items) {
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((items + kThreads - 1) / kThreads, sm_count() * 16ll)));
}

int forward(const ForwardPlan& f, const void* x, int type, int64_t x_stride, const void* w, int64_t n, int H, int I,
            void* part, void* h, float* gate_up, int* err, cudaStream_t s) {
  if (f.few) {
    FewRows r{};
    r.w = static_cast<const uint8_t*>(w);
    r.x = static_cast<const uint8_t*>(x);
    r.row_bytes = 2ll * H;
    r.x_stride = 2 * x_stride;
    r.M = static_cast<int>(n);
    r.E = r.top_k = r.segments = 1;
    r.N = I;
    r.steps = (H + 63) / 64;
    r.y = h;
    r.y_type = type;
    r.gate_up = gate_up;
    r.err = err;
    return launch_few_rows(r, type, s);
  }
  GemmF16 g{type, x, x_stride, w, H, n, I, H, false, false, true, f.tile.tile_m, f.tile.cols, 1, h, type, gate_up, err};
  if (!f.split) return launch_gemm_f16(g, s);
  g.N = 2ll * I;
  g.gated = false;
  g.splits = f.tile.splits;
  g.y = part;
  g.y_type = TQ_FP32;
  g.gate_up = nullptr;
  int rc = launch_gemm_f16(g, s);
  if (rc != TQ_OK) return rc;
  const dim3 blocks(walk_blocks(n * (I / 4)));
  const long long stride = 2ll * I * n;
  rc = type == TQ_BF16 ? launch_pdl(swiglu_sum_kernel<__nv_bfloat16>, blocks, dim3(kThreads), 0, s,
                                    static_cast<const float*>(part), stride, g.splits, static_cast<long long>(n), I,
                                    static_cast<__nv_bfloat16*>(h), gate_up)
                       : launch_pdl(swiglu_sum_kernel<__half>, blocks, dim3(kThreads), 0, s,
                                    static_cast<const float*>(part), stride, g.splits, static_cast<long long>(n), I,
                                    static_cast<__half*>(h), gate_up);
  if (rc == TQ_OK) count_launch(kCntSwigluSum);
  return rc;
}

// The two products of the gradient.
TileChoice tile_x(int64_t n, int H, int I) {
  return choose_tile(false, static_cast<double>(std::max<int64_t>(n, 1)), 1.0, static_cast<int>((2ll * I + 63) / 64), H,
                     false, TileRows::kOne, false, true);
}
TileChoice tile_w(int64_t n, int H, int I) {
  return choose_tile(false, 2.0 * I, 1.0, static_cast<int>((n + 63) / 64), H, false, TileRows::kOne, false, true);
}

struct GradPlan {
  TileChoice x, w;
  ForwardPlan forward;   // of gate and up again
  size_t gate_up, d, part, bytes;   // offsets
};
GradPlan plan(int64_t n, int H, int I, bool has_gate_up) {
  GradPlan p{};
  if (!has_gate_up) p.forward = plan_forward(n, H, I);
  p.x = tile_x(n, H, I);
  p.w = tile_w(n, H, I);
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
  // in turn: each product starts after the sums before it are read
  p.part = take(std::max({sums_x, sums_w, static_cast<double>(p.forward.part / 4)}), 4);
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
  return launch_fp4_combine(static_cast<const float*>(part), g.N, g.M * g.N, t.splits, nullptr, nullptr, nullptr, nullptr,
                            g.M, 1, 1, static_cast<int>(g.N), y, type, s);
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" {

size_t tq_swiglu_linear_workspace_size(int64_t n, int H, int I) {
  return bad_sizes(n, H, I) ? 0 : std::max<size_t>(256, plan_forward(n, H, I).part);
}

int tq_swiglu_linear(const void* x, int type, int64_t x_stride, const void* w_gu, int64_t n, int H, int I, void* workspace,
                     size_t workspace_bytes, void* h, float* gate_up, tq_stream_t stream) {
  if (bad_sizes(n, H, I) || bad_type16(type) || bad_x(x, x_stride, n, H)) return TQ_ERR_INVALID_ARG;
  if (n > 0 && (!w_gu || (!h && !gate_up) || !aligned(w_gu, 16) || !aligned(h, 16) || !aligned(gate_up, 16)))
    return TQ_ERR_INVALID_ARG;
  const ForwardPlan f = plan_forward(n, H, I);
  if (n > 0 && f.split && (!workspace || !aligned(workspace, 256) || workspace_bytes < f.part)) return TQ_ERR_WORKSPACE;
  const int64_t x_bytes = row_bytes(n, x_stride, H, 2), w_bytes = 4ll * I * H, h_bytes = 2 * n * I, gu_bytes = 8 * n * I;
  if (n > 0 && outputs_overlap({{h, h_bytes}, {gate_up, gu_bytes}, {f.split ? workspace : nullptr, static_cast<int64_t>(f.part)}},
                               {{x, x_bytes}, {w_gu, w_bytes}}))
    return TQ_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int rc = require_sm103(s);
  if (rc != TQ_OK || n == 0) return rc;
  int* err = error_word(&rc);
  if (!err) return rc;
  return forward(f, x, type, x_stride, w_gu, n, H, I, workspace, h, gate_up, err, s);
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
  // (grad_h and gate_up are read before either gradient is written)
  const int64_t x_bytes = row_bytes(n, x_stride, H, 2), gx_bytes = 2 * n * H, w_bytes = n > 0 ? 4ll * I * H : 0;
  const Span work{workspace, static_cast<int64_t>(p.bytes)};
  if (n > 0 && (outputs_overlap({{grad_x, gx_bytes}, {grad_w_gu, w_bytes}, work}, {{x, x_bytes}, {w_gu, w_bytes}}) ||
                outputs_overlap({work}, {{grad_h, 2 * n * I}, {gate_up, 8 * n * I}})))
    return TQ_ERR_INVALID_ARG;
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
    rc = forward(p.forward, x, type, x_stride, w_gu, n, H, I, base + p.part, nullptr, again, err, s);
    if (rc != TQ_OK) return rc;
    gate_up = again;
  }
  void* const d = base + p.d;
  const int blocks = walk_blocks(n * (I / 8));
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
