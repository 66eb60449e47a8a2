// Root-mean-square norm with the residual's addition, its output in the input's type
// or in 8 bits with block scales, and its gradient.
//
//   r = x + residual, rounded to the type and kept;  rstd = 1 / sqrt(mean(r^2) + eps);
//   y = (r rstd) w.
//   With a = grad_y w:  grad_x = rstd (a - r rstd^2 mean(a r)) + grad_residual,
//   grad_w = sum over rows of grad_y (r rstd).
//
// A block takes a row, 16 values a thread in registers, so that every byte moves once
// (the gradient: rows in turn, its share of grad_w in registers too).  Rows of any
// width and alignment take the same path with loads of single values, neighbouring
// threads neighbouring values.
//
// The sum of squares carries its rounding errors along (Knuth's two-sum: the sum of
// two numbers and its exact error), and rstd is the fp32 number nearest to the true
// one but in rare cases: 8-bit codes fall to one or the other side of a border by the
// last bit of y, and so do not depend on the order of a sum.
#include <cuda_runtime.h>

#include <algorithm>

#include "tq_fp8.cuh"
#include "tq_internal.h"

namespace tq {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kPer = 16;   // values per thread

// hi + lo = a sum and its rounding errors.
struct Sum2 {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float v) {
    const float s = __fadd_rn(hi, v), b = __fsub_rn(s, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(v, b)));
    hi = s;
  }
  __device__ __forceinline__ void add_square(float v) {
    const float p = __fmul_rn(v, v);
    add(p);
    lo = __fadd_rn(lo, __fmaf_rn(v, v, -p));   // 0 for 16-bit values
  }
};
__device__ __forceinline__ Sum2 warp_sum(Sum2 s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float hi = __shfl_xor_sync(kAll, s.hi, o), lo = __shfl_xor_sync(kAll, s.lo, o);
    s.add(hi);
    s.lo = __fadd_rn(s.lo, lo);
  }
  return s;
}
__device__ __forceinline__ float warp_sum(float s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
  return s;
}

// 1 / sqrt(m) rounded to fp32: one Newton step in 64 bits from the approximation.
__device__ __forceinline__ float rsqrt_rounded(double m) {
  double back = 1.0;
  if (m > 0x1p100) {
    m *= 0x1p-200;   // up to 2^256
    back = 0x1p-100;
  } else if (m < 0x1p-100) {
    m *= 0x1p200;
    back = 0x1p100;
  }
  const double r = rsqrtf(static_cast<float>(m));
  if (!(r < 3e38) || r == 0.0) return static_cast<float>(r);   // of 0, infinity or NaN
  return static_cast<float>(back * (r + 0.5 * r * (1.0 - m * r * r)));
}

// A thread's columns: 16 consecutive ones, or every blockDim.x-th.
template <bool kVec>
__device__ __forceinline__ int column(int i) {
  return kVec ? kPer * static_cast<int>(threadIdx.x) + i : static_cast<int>(threadIdx.x) + i * static_cast<int>(blockDim.x);
}

template <bool kVec, typename T>
__device__ __forceinline__ void load16(const T* __restrict__ p, int K, float (&v)[kPer]) {
  if constexpr (kVec) {
    T t[kPer];
    if (column<true>(0) < K) {
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(T)); ++i)
        reinterpret_cast<uint4*>(t)[i] = reinterpret_cast<const uint4*>(p + column<true>(0))[i];
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[i] = widen(t[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[i] = 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int c = column<false>(i);
      v[i] = c < K ? widen(p[c]) : 0.f;
    }
  }
}
template <bool kVec, typename T>
__device__ __forceinline__ void store16(T* __restrict__ p, int K, const float (&v)[kPer]) {
  if constexpr (kVec) {
    if (column<true>(0) >= K) return;
    T t[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) t[i] = narrow<T>(v[i]);
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)); ++i)
      reinterpret_cast<uint4*>(p + column<true>(0))[i] = reinterpret_cast<const uint4*>(t)[i];
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int c = column<false>(i);
      if (c < K) p[c] = narrow<T>(v[i]);
    }
  }
}
template <bool kVec>
__device__ __forceinline__ void load_weight(const void* w, int type, int K, float (&v)[kPer]) {
  if (type == TQ_FP32)
    load16<kVec>(static_cast<const float*>(w), K, v);
  else if (type == TQ_BF16)
    load16<kVec>(static_cast<const __nv_bfloat16*>(w), K, v);
  else
    load16<kVec>(static_cast<const __half*>(w), K, v);
}

template <typename T, bool kVec, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads) rms_norm_kernel(const NormArgs a) {
  __shared__ Sum2 parts[32];
  __shared__ float shared_rstd;
  pdl_wait();
  pdl_trigger();
  const int K = a.K, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x / 32;
  const long long row = blockIdx.x;
  float v[kPer];
  load16<kVec>(static_cast<const T*>(a.x) + row * a.x_stride, K, v);
  if (a.residual) {
    float r[kPer];
    load16<kVec>(static_cast<const T*>(a.residual) + row * a.residual_stride, K, r);
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = widen(narrow<T>(v[i] + r[i]));
    store16<kVec>(static_cast<T*>(a.residual_out) + row * K, K, v);
  }
  float w[kPer];
  if (a.weight) load_weight<kVec>(a.weight, a.w_type, K, w);   // under way while the row is summed

  // Squares of values beyond 2^63 overflow: such a row is summed again, 2^-96 of it.
  for (float scale = 1.f;; scale = 0x1p-96f) {
    Sum2 s;
#pragma unroll
    for (int i = 0; i < kPer; ++i) s.add_square(v[i] * scale);
    s = warp_sum(s);
    if (lane == 0) parts[warp] = s;
    __syncthreads();
    if (warp == 0) {
      s = lane < warps ? parts[lane] : Sum2();
      s = warp_sum(s);
      if (lane == 0) {
        if (scale == 1.f && s.hi > FLT_MAX) {
          shared_rstd = -1.f;
        } else {
          // (a sum that overflowed makes its error term NaN)
          double m = static_cast<double>(s.hi) + (s.hi <= FLT_MAX ? static_cast<double>(s.lo) : 0.0);
          if (scale != 1.f) m *= 0x1p192;
          shared_rstd = rsqrt_rounded(m / K + static_cast<double>(a.eps));
        }
      }
    }
    __syncthreads();
    if (shared_rstd >= 0.f || scale != 1.f || shared_rstd != shared_rstd) break;
  }
  const float rstd = shared_rstd;
  if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    v[i] = __fmul_rn(v[i], rstd);
    if (a.weight) v[i] = __fmul_rn(v[i], w[i]);
  }
  if (a.y) store16<kVec>(static_cast<T*>(a.y) + row * K, K, v);
  if constexpr (kVec) {
    if (a.codes) {   // a block of 128 is eight neighbouring threads
      float top = fp8_top<kPer>(v);
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
      if (column<true>(0) < K) {
        const Fp8Scale s(top);
        *reinterpret_cast<uint4*>(a.codes + row * K + column<true>(0)) = fp8_codes16(v, s);
        if ((lane & 7) == 0) a.scales[row * ((K + kFp8Block - 1) / kFp8Block) + threadIdx.x / 8] = s.s;
      }
    }
  }
}

template <typename T, bool kVec, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads) rms_norm_backward_kernel(const NormGradArgs a) {
  __shared__ float parts[2][32];
  pdl_wait();
  const int K = a.K, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x / 32;
  float w[kPer], gw[kPer] = {};
  if (a.weight) {
    load_weight<kVec>(a.weight, a.w_type, K, w);
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) w[i] = 1.f;
  }
  int buffer = 0;
  for (long long row = blockIdx.x; row < a.n; row += gridDim.x, buffer ^= 1) {
    float v[kPer], d[kPer], dot = 0.f;
    load16<kVec>(static_cast<const T*>(a.x) + row * a.x_stride, K, v);
    load16<kVec>(static_cast<const T*>(a.grad_y) + row * a.grad_y_stride, K, d);
    const float rstd = __ldg(a.rstd + row);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      gw[i] = fmaf(d[i], v[i] * rstd, gw[i]);
      d[i] *= w[i];
      v[i] *= rstd;
      dot = fmaf(d[i], v[i], dot);
    }
    dot = warp_sum(dot);
    if (lane == 0) parts[buffer][warp] = dot;   // read until the next row's barrier at the latest
    __syncthreads();
    dot = lane < warps ? parts[buffer][lane] : 0.f;
    dot = warp_sum(dot) / static_cast<float>(K);
#pragma unroll
    for (int i = 0; i < kPer; ++i) d[i] = rstd * (d[i] - v[i] * dot);
    if (a.grad_residual) {
      float g[kPer];
      load16<kVec>(static_cast<const T*>(a.grad_residual) + row * a.grad_residual_stride, K, g);
#pragma unroll
      for (int i = 0; i < kPer; ++i) d[i] += g[i];
    }
    store16<kVec>(static_cast<T*>(a.grad_x) + row * K, K, d);
  }
  pdl_trigger();
  if (a.part) store16<kVec>(a.part + static_cast<long long>(blockIdx.x) * K, K, gw);
}

// grad_w[k] = the sum of the blocks' shares, in order: 32 columns a block, each of its
// eight warps every eighth share.
__global__ void __launch_bounds__(256) rms_norm_weight_kernel(const float* __restrict__ part, int shares, int K,
                                                              void* grad_w, int type) {
  __shared__ float sums[8][32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < K) {
#pragma unroll 4
    for (int b = warp; b < shares; b += 8) s += __ldcs(part + static_cast<long long>(b) * K + c);
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < K) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += sums[i][lane];
    if (type == TQ_FP32)
      static_cast<float*>(grad_w)[c] = s;
    else if (type == TQ_BF16)
      static_cast<__nv_bfloat16*>(grad_w)[c] = narrow<__nv_bfloat16>(s);
    else
      static_cast<__half*>(grad_w)[c] = narrow<__half>(s);
  }
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool rows_in_vectors(const void* p, int64_t stride, int type) {
  return aligned(p, 16) && stride * static_cast<int64_t>(type_size(type)) % 16 == 0;
}
int block_threads(int K) { return ((K + kPer - 1) / kPer + 31) / 32 * 32; }
bool bad_rows(const void* p, int64_t stride, int64_t n, int K) {
  return stride < K || (n > 1 && static_cast<double>(n) * static_cast<double>(stride) >= 0x1p58) || (n > 0 && !p);
}
bool bad_width(int K) { return K < 1 || K > TQ_NORM_MAX_WIDTH; }

template <typename T>
int run_norm(const NormArgs& a, bool vec, cudaStream_t s) {
  const int threads = block_threads(a.K);
  auto kernel = vec ? (threads <= 512 ? rms_norm_kernel<T, true, 512> : rms_norm_kernel<T, true, 1024>)
                    : (threads <= 512 ? rms_norm_kernel<T, false, 512> : rms_norm_kernel<T, false, 1024>);
  return launch_pdl(kernel, dim3(static_cast<unsigned>(a.n)), dim3(threads), 0, s, a);
}

template <typename T>
int run_backward(const NormGradArgs& a, bool vec, int blocks, cudaStream_t s) {
  const int threads = block_threads(a.K);
  auto kernel = vec ? (threads <= 512 ? rms_norm_backward_kernel<T, true, 512> : rms_norm_backward_kernel<T, true, 1024>)
                    : (threads <= 512 ? rms_norm_backward_kernel<T, false, 512>
                                      : rms_norm_backward_kernel<T, false, 1024>);
  return launch_pdl(kernel, dim3(blocks), dim3(threads), 0, s, a);
}

// Blocks of the gradient: what the SMs hold at once at 64 registers a thread.
int backward_blocks(int64_t n, int K) {
  const int per_sm = std::max(1, std::min(16, 1024 / block_threads(K)));
  return static_cast<int>(std::min<int64_t>(n, static_cast<int64_t>(sm_count()) * per_sm));
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" {

int tq_rms_norm(const void* x, int x_type, int64_t x_stride, const void* residual, int64_t residual_stride,
                const void* weight, int w_type, float eps, int64_t n, int K, void* residual_out, void* y, float* rstd,
                uint8_t* codes, float* scales, tq_stream_t stream) {
  if (n < 0 || n > 0x7fffffff || bad_width(K) || bad_type(x_type) || bad_type(w_type) || !(eps >= 0.f) ||
      !(eps <= FLT_MAX) || bad_rows(x, x_stride, n, K))
    return TQ_ERR_INVALID_ARG;
  if (residual && (bad_rows(residual, residual_stride, n, K) || (n > 0 && !residual_out))) return TQ_ERR_INVALID_ARG;
  if (!residual && residual_out) return TQ_ERR_INVALID_ARG;
  if (n > 0 && !y && !codes) return TQ_ERR_INVALID_ARG;
  if ((codes == nullptr) != (scales == nullptr)) return TQ_ERR_INVALID_ARG;
  const size_t size = type_size(x_type);
  if (!aligned(x, size) || !aligned(residual, size) || !aligned(residual_out, size) || !aligned(y, size) ||
      !aligned(weight, type_size(w_type)) || !aligned(rstd, 4) || !aligned(scales, 4))
    return TQ_ERR_INVALID_ARG;
  const bool vec = K % kPer == 0 && rows_in_vectors(x, x_stride, x_type) &&
                   (!residual || rows_in_vectors(residual, residual_stride, x_type)) && aligned(residual_out, 16) &&
                   aligned(y, 16) && aligned(weight, 16);
  if (codes && (!vec || !aligned(codes, 16))) return TQ_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int rc = require_sm103(s);
  if (rc != TQ_OK || n == 0) return rc;
  const NormArgs a{x, residual, weight, residual_out, y, rstd, codes, scales, x_stride, residual_stride, n, K, w_type, eps};
  const int st = x_type == TQ_FP32   ? run_norm<float>(a, vec, s)
                 : x_type == TQ_BF16 ? run_norm<__nv_bfloat16>(a, vec, s)
                                     : run_norm<__half>(a, vec, s);
  if (st == TQ_OK) count_launch(kCntNorm);
  return st;
}

size_t tq_rms_norm_backward_workspace_size(int64_t n, int K) {
  if (n < 0 || n > 0x7fffffff || bad_width(K)) return 0;
  return std::max<size_t>(256, static_cast<size_t>(n ? backward_blocks(n, K) : 0) * K * sizeof(float));
}

int tq_rms_norm_backward(const void* grad_y, int64_t grad_y_stride, const void* x, int x_type, int64_t x_stride,
                         const void* weight, int w_type, const float* rstd, const void* grad_residual,
                         int64_t grad_residual_stride, int64_t n, int K, void* workspace, size_t workspace_bytes,
                         void* grad_x, void* grad_weight, tq_stream_t stream) {
  if (n < 0 || n > 0x7fffffff || bad_width(K) || bad_type(x_type) || bad_type(w_type) ||
      bad_rows(grad_y, grad_y_stride, n, K) || bad_rows(x, x_stride, n, K) ||
      (grad_residual && bad_rows(grad_residual, grad_residual_stride, n, K)) || (n > 0 && (!rstd || !grad_x)) ||
      (grad_weight && !weight))
    return TQ_ERR_INVALID_ARG;
  const size_t size = type_size(x_type);
  if (!aligned(grad_y, size) || !aligned(x, size) || !aligned(grad_residual, size) || !aligned(grad_x, size) ||
      !aligned(weight, type_size(w_type)) || !aligned(grad_weight, type_size(w_type)) || !aligned(rstd, 4))
    return TQ_ERR_INVALID_ARG;
  if (grad_weight && n > 0 &&
      (!workspace || !aligned(workspace, 256) || workspace_bytes < tq_rms_norm_backward_workspace_size(n, K)))
    return TQ_ERR_WORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int rc = require_sm103(s);
  if (rc != TQ_OK) return rc;
  if (n == 0) {   // a sum over no rows
    if (grad_weight && cudaMemsetAsync(grad_weight, 0, K * type_size(w_type), s) != cudaSuccess) return launch_status();
    return TQ_OK;
  }
  const bool vec = K % kPer == 0 && rows_in_vectors(x, x_stride, x_type) && rows_in_vectors(grad_y, grad_y_stride, x_type) &&
                   (!grad_residual || rows_in_vectors(grad_residual, grad_residual_stride, x_type)) &&
                   aligned(grad_x, 16) && aligned(weight, 16);
  const int blocks = backward_blocks(n, K);
  const NormGradArgs a{grad_y, x, weight, grad_residual, rstd, grad_x, grad_weight ? static_cast<float*>(workspace) : nullptr,
                       grad_y_stride, x_stride, grad_residual_stride, n, K, w_type};
  rc = x_type == TQ_FP32   ? run_backward<float>(a, vec, blocks, s)
       : x_type == TQ_BF16 ? run_backward<__nv_bfloat16>(a, vec, blocks, s)
                           : run_backward<__half>(a, vec, blocks, s);
  if (rc != TQ_OK) return rc;
  count_launch(kCntNormBackward);
  if (!grad_weight) return TQ_OK;
  rc = launch_pdl(rms_norm_weight_kernel, dim3((K + 31) / 32), dim3(256), 0, s, static_cast<const float*>(workspace),
                  blocks, K, grad_weight, w_type);
  if (rc == TQ_OK) count_launch(kCntNormWeight);
  return rc;
}

}  // extern "C"
