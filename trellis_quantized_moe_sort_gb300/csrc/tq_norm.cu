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
// threads neighbouring values, no row ahead and the weights read again, which leaves
// registers for more of them (gradient of 2048 rows of 16383 in bf16: 289 us with, 181 so).
//
// The sum of squares carries its rounding errors along (Knuth's two-sum: the sum of
// two numbers and its exact error), and rstd is the fp32 number nearest to the true
// one but in rare cases: 8-bit codes fall to one or the other side of a border by the
// last bit of y, and so do not depend on the order of a sum.
//
// Bound by the memory's rate, and for 8 bits by instructions too (63% of the issue slots:
// the codes and the exact sum).  Measured in bf16, rows of 4096 with residual: 8192 rows to
// 8 bits 44 us (235 MB, 80% of the measured copy rate); 4095 rows to 16 bits 24 us (134 MB,
// 82%), their gradient 24 us (134 MB, 84%) and the sum of grad_w's shares 7.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "tq_device.cuh"
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
};
// The sum of a thread's squares: two sums side by side, two operations an instruction.
// kExact: a square has no rounding error (values of 16 bits).
template <bool kExact>
__device__ __forceinline__ Sum2 sum_of_squares(const float (&v)[kPer], float scale) {
  float2 hi = make_float2(0.f, 0.f), lo = hi;
#pragma unroll
  for (int i = 0; i < kPer; i += 2) {
    float2 a = make_float2(v[i], v[i + 1]);
    if (!kExact) a = mul2(a, make_float2(scale, scale));
    const float2 p = mul2(a, a), s = add2(hi, p), b = sub2(s, hi);
    lo = add2(lo, add2(sub2(hi, sub2(s, b)), sub2(p, b)));
    if (!kExact) lo = add2(lo, fma2(a, a, make_float2(-p.x, -p.y)));
    hi = s;
  }
  Sum2 s;
  s.hi = hi.x;
  s.lo = lo.x;
  s.add(hi.y);
  s.lo = __fadd_rn(s.lo, lo.y);
  return s;
}
// Over the lanes, or the first `lanes` of them (a power of two).
__device__ __forceinline__ Sum2 warp_sum(Sum2 s, int lanes = 32) {
  for (int o = lanes / 2; o > 0; o >>= 1) {
    const float hi = __shfl_xor_sync(kAll, s.hi, o), lo = __shfl_xor_sync(kAll, s.lo, o);
    s.add(hi);
    s.lo = __fadd_rn(s.lo, lo);
  }
  return s;
}
__device__ __forceinline__ float warp_sum(float s, int lanes = 32) {
  for (int o = lanes / 2; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
  return s;
}

// 1 / sqrt(hi + lo), rounded to fp32: a Newton step from the approximation r, its
// residual 1 - m r^2 by exact products.  (In 64 bits the step would take longer than
// the row: an SM does two such operations a clock.)
__device__ __forceinline__ float rsqrt_rounded(float hi, float lo) {
  float back = 1.f;
  if (hi > 0x1p100f) {
    hi *= 0x1p-100f;
    lo *= 0x1p-100f;
    back = 0x1p-50f;
  } else if (hi < 0x1p-80f) {
    hi *= 0x1p60f;
    lo *= 0x1p60f;
    back = 0x1p30f;
  }
  const float r = rsqrtf(hi);
  if (!(r < 3e38f) || r == 0.f) return r;   // of 0, infinity or NaN
  const float t = __fmul_rn(r, r), t_lo = __fmaf_rn(r, r, -t);
  const float e = __fmaf_rn(-hi, t, 1.f) - hi * t_lo - lo * t;
  return __fmul_rn(__fmaf_rn(0.5f * r, e, r), back);
}
// 1 / sqrt(s / K + eps).
__device__ __forceinline__ float rstd_of(const Sum2& s, float K, float eps) {
  if (!(s.hi <= FLT_MAX)) return rsqrtf(s.hi);
  const float q = __fdiv_rn(s.hi, K), q_lo = __fdiv_rn(__fmaf_rn(-q, K, s.hi) + s.lo, K);
  Sum2 m;
  m.hi = q;
  m.add(eps);
  return rsqrt_rounded(m.hi, m.lo + q_lo);
}

// A thread's columns: 16 consecutive ones, or every blockDim.x-th.
template <bool kVec>
__device__ __forceinline__ int column(int i) {
  return kVec ? kPer * static_cast<int>(threadIdx.x) + i : static_cast<int>(threadIdx.x) + i * static_cast<int>(blockDim.x);
}

// A thread's values of a row as they are in memory; zeros past its end.
template <bool kVec, typename T>
struct Raw {
  alignas(16) T t[kPer];
  __device__ __forceinline__ void load(const T* p, int K) {
    if constexpr (kVec) {
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(T)); ++i)
        reinterpret_cast<uint4*>(t)[i] = column<true>(0) < K ? reinterpret_cast<const uint4*>(p + column<true>(0))[i]
                                                             : make_uint4(0u, 0u, 0u, 0u);
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) t[i] = column<false>(i) < K ? p[column<false>(i)] : narrow<T>(0.f);
    }
  }
  __device__ __forceinline__ void open(float (&v)[kPer]) const {
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = widen(t[i]);
  }
};
template <bool kVec, typename T>
__device__ __forceinline__ void load16(const T* p, int K, float (&v)[kPer]) {
  Raw<kVec, T> raw;
  raw.load(p, K);
  raw.open(v);
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

// Lanes that a sum over the block's warps takes.
__device__ __forceinline__ int power_above(int warps) { return warps > 1 ? 1 << (32 - __clz(warps - 1)) : 1; }

// rstd of a row from its threads' sums of squares times scale^2, or, for a first sum
// (scale 1) that did not keep its range, kTooLarge or kTooSmall.  One warp adds up and
// takes the root: with every warp doing so a block's eight of them spent a third of
// their instructions on it.
constexpr float kTooLarge = -1.f, kTooSmall = -2.f;
__device__ __forceinline__ float block_rstd(Sum2 s, float scale, const NormArgs& a, int lane, int warp, int warps,
                                            int lanes, int& buffer, Sum2 (&parts)[2][32], float (&result)[2]) {
  s = warp_sum(s);
  if (warps > 1) {
    if (lane == 0) parts[buffer][warp] = s;
    __syncthreads();
    if (warp == 0) {
      s = lane < warps ? parts[buffer][lane] : Sum2();
      s = warp_sum(s, lanes);
    }
  }
  if (warp == 0 && lane == 0) {
    float r = rstd_of(s, static_cast<float>(a.K), a.eps * scale * scale) * scale;
    if (scale == 1.f && s.hi > FLT_MAX) r = kTooLarge;
    if (scale == 1.f && s.hi < 0x1p-100f && a.eps < 0x1p-100f) r = kTooSmall;
    result[buffer] = r;
  }
  __syncthreads();
  // (written again after the next sum's first barrier; of one warp, after its second)
  const float r = result[buffer];
  buffer ^= 1;
  return r;
}

// Blocks walk the rows, the next row's loads under way while the present one is summed
// and written.
template <typename T, bool kVec, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads, kMaxThreads == 256 ? 4 : 1) rms_norm_kernel(const NormArgs a) {
  __shared__ Sum2 parts[2][32];
  __shared__ float result[2];
  pdl_wait();
  pdl_trigger();
  const int K = a.K, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x / 32;
  const int lanes = power_above(warps);
  const T* const x = static_cast<const T*>(a.x);
  const T* const residual = static_cast<const T*>(a.residual);
  Raw<kVec, T> next_x, next_r = {};
  auto fetch = [&](long long row) {
    next_x.load(x + row * a.x_stride, K);
    if (residual) next_r.load(residual + row * a.residual_stride, K);
  };
  if (kVec) fetch(blockIdx.x);
  float w[kPer];
  if (kVec && a.weight) load_weight<kVec>(a.weight, a.w_type, K, w);
  int buffer = 0;
  for (long long row = blockIdx.x; row < a.n; row += gridDim.x) {
    if (!kVec) fetch(row);
    Raw<kVec, T> r = next_x;
    float v[kPer];
    if (residual) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) r.t[i] = narrow<T>(widen(r.t[i]) + widen(next_r.t[i]));
    }
    if (kVec && row + gridDim.x < a.n) fetch(row + gridDim.x);
    r.open(v);
    if (residual) store16<kVec>(static_cast<T*>(a.residual_out) + row * K, K, v);

    // Squares of values beyond 2^63 overflow, and where eps does not count those of tiny
    // values underflow: such a row is summed again, 2^-96 or 2^90 of it.
    float rstd = block_rstd(sum_of_squares<sizeof(T) == 2>(v, 1.f), 1.f, a, lane, warp, warps, lanes, buffer, parts, result);
    if (rstd < 0.f) {
      const float scale = rstd == kTooLarge ? 0x1p-96f : 0x1p90f;
      rstd = block_rstd(sum_of_squares<false>(v, scale), scale, a, lane, warp, warps, lanes, buffer, parts, result);
    }
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
    if (!kVec && a.weight) load_weight<kVec>(a.weight, a.w_type, K, w);
#pragma unroll
    for (int i = 0; i < kPer; i += 2) {
      float2 t = mul2(make_float2(v[i], v[i + 1]), make_float2(rstd, rstd));
      if (a.weight) t = mul2(t, make_float2(w[i], w[i + 1]));
      v[i] = t.x;
      v[i + 1] = t.y;
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
}

template <typename T, bool kVec, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads) rms_norm_backward_kernel(const NormGradArgs a) {
  __shared__ float parts[2][32];
  pdl_wait();
  const int K = a.K, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x / 32;
  const int lanes = power_above(warps);
  const T* const x = static_cast<const T*>(a.x);
  const T* const grad_y = static_cast<const T*>(a.grad_y);
  const T* const grad_r = static_cast<const T*>(a.grad_residual);
  Raw<kVec, T> next_x, next_y, next_r = {};
  float next_rstd = 0.f;
  auto fetch = [&](long long row) {
    next_x.load(x + row * a.x_stride, K);
    next_y.load(grad_y + row * a.grad_y_stride, K);
    if (grad_r) next_r.load(grad_r + row * a.grad_residual_stride, K);
    next_rstd = a.rstd[row];
  };
  if (kVec) fetch(blockIdx.x);
  float w[kPer], gw[kPer] = {};
  auto weights = [&] {
    if (a.weight) {
      load_weight<kVec>(a.weight, a.w_type, K, w);
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) w[i] = 1.f;
    }
  };
  if (kVec) weights();
  int buffer = 0;
  for (long long row = blockIdx.x; row < a.n; row += gridDim.x, buffer ^= 1) {
    if (!kVec) {
      fetch(row);
      weights();
    }
    const Raw<kVec, T> g = next_r;
    const float rstd = next_rstd;
    float v[kPer], d[kPer], dot = 0.f;
    next_x.open(v);
    next_y.open(d);
    if (kVec && row + gridDim.x < a.n) fetch(row + gridDim.x);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      v[i] *= rstd;
      gw[i] = fmaf(d[i], v[i], gw[i]);
      d[i] *= w[i];
      dot = fmaf(d[i], v[i], dot);
    }
    dot = warp_sum(dot);
    if (lane == 0) parts[buffer][warp] = dot;   // read until the next row's barrier at the latest
    __syncthreads();
    dot = lane < warps ? parts[buffer][lane] : 0.f;
    dot = __shfl_sync(kAll, warp_sum(dot, lanes), 0) / static_cast<float>(K);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      d[i] = rstd * (d[i] - v[i] * dot);
      if (grad_r) d[i] += widen(g.t[i]);
    }
    store16<kVec>(static_cast<T*>(a.grad_x) + row * K, K, d);
  }
  pdl_trigger();
  if (a.part) store16<kVec>(a.part + static_cast<long long>(blockIdx.x) * K, K, gw);
}

// The same for rows of more than 8192 values, whose blocks of up to 1024 threads have 64
// registers a thread: the rows come through shared memory, each thread's values by its own
// asynchronous copies, the next row's under way where two of them fit (`buffers`), and are
// read twice from there.  (In registers, with spills, 2048 rows of 16384 in bf16 took 142
// us and in fp32 262, 93 and 160 so.)
template <typename T>
__global__ void __launch_bounds__(1024) rms_norm_backward_wide_kernel(const NormGradArgs a, const int buffers) {
  extern __shared__ uint4 rows[];   // [buffers][3][pieces][threads]
  __shared__ float parts[2][32];
  constexpr int kPieces = static_cast<int>(sizeof(T)), kEach = kPer / kPieces;   // 16-byte pieces of a thread, values of one
  pdl_wait();
  const int K = a.K, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x / 32;
  const int lanes = power_above(warps), at = column<true>(0);
  const bool in = at < K;
  const int arrays = a.grad_residual ? 3 : 2;
  auto fetch = [&](long long row, int buffer) {
    if (in && row < a.n) {
      const T* const from[3] = {static_cast<const T*>(a.x) + row * a.x_stride,
                                static_cast<const T*>(a.grad_y) + row * a.grad_y_stride,
                                static_cast<const T*>(a.grad_residual) + row * a.grad_residual_stride};
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        if (i == arrays) break;
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
          const uint32_t to = smem_u32(rows + ((buffer * arrays + i) * kPieces + j) * blockDim.x + threadIdx.x);
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from[i] + at + kEach * j) : "memory");
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  fetch(blockIdx.x, 0);
  float w[kPer], gw[kPer] = {};
  if (a.weight) {
    load_weight<true>(a.weight, a.w_type, K, w);
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) w[i] = 1.f;
  }
  float next_rstd = a.rstd[blockIdx.x];
  int parity = 0, buffer = 0;
  for (long long row = blockIdx.x; row < a.n; row += gridDim.x, parity ^= 1) {
    const float rstd = next_rstd;
    if (row + gridDim.x < a.n) next_rstd = a.rstd[row + gridDim.x];
    if (buffers == 2) {
      fetch(row + gridDim.x, buffer ^ 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    const uint4* const mine = rows + buffer * arrays * kPieces * blockDim.x + threadIdx.x;
    auto piece = [&](int array, int j, float (&v)[kEach]) {
      const uint4 raw = mine[(array * kPieces + j) * blockDim.x];
      T t[kEach];
      memcpy(t, &raw, 16);
#pragma unroll
      for (int i = 0; i < kEach; ++i) v[i] = widen(t[i]);
    };
    float dot = 0.f;
    if (in) {
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        float v[kEach], d[kEach];
        piece(0, j, v);
        piece(1, j, d);
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          const float u = v[i] * rstd;
          gw[kEach * j + i] = fmaf(d[i], u, gw[kEach * j + i]);
          dot = fmaf(d[i] * w[kEach * j + i], u, dot);
        }
      }
    }
    dot = warp_sum(dot);
    if (lane == 0) parts[parity][warp] = dot;   // read until the next row's barrier at the latest
    __syncthreads();
    dot = lane < warps ? parts[parity][lane] : 0.f;
    dot = __shfl_sync(kAll, warp_sum(dot, lanes), 0) / static_cast<float>(K);
    if (in) {
      T* const out = static_cast<T*>(a.grad_x) + row * K + at;
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        float v[kEach], d[kEach], g[kEach];
        T t[kEach];
        piece(0, j, v);
        piece(1, j, d);
        if (arrays == 3) piece(2, j, g);
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          float r = rstd * (d[i] * w[kEach * j + i] - v[i] * rstd * dot);
          if (arrays == 3) r += g[i];
          t[i] = narrow<T>(r);
        }
        uint4 raw;
        memcpy(&raw, t, 16);
        *reinterpret_cast<uint4*>(out + kEach * j) = raw;
      }
    }
    if (buffers == 2)
      buffer ^= 1;
    else
      fetch(row + gridDim.x, 0);   // (over values that this thread alone has read)
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  pdl_trigger();
  if (a.part) store16<true>(a.part + static_cast<long long>(blockIdx.x) * K, K, gw);
}

// grad_w[k] = the sum of the blocks' shares, in order: 32 columns a block, each of its
// warps every 32nd share.
__global__ void __launch_bounds__(1024) rms_norm_weight_kernel(const float* __restrict__ part, int shares, int K,
                                                              void* grad_w, int type) {
  __shared__ float sums[32][33];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < K) {
    for (int b = warp; b < shares; b += 32 * 12) {   // a dozen reads under way
      float v[12];
#pragma unroll
      for (int i = 0; i < 12; ++i) v[i] = b + 32 * i < shares ? __ldcs(part + static_cast<long long>(b + 32 * i) * K + c) : 0.f;
#pragma unroll
      for (int i = 0; i < 12; ++i) s += v[i];
    }
  }
  sums[warp][lane] = s;
  __syncthreads();
  // warp w adds up column w
  s = warp_sum(sums[lane][warp]);
  c = blockIdx.x * 32 + warp;
  if (lane == 0 && c < K) {
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
// An output may take the place of input rows, dense and from the same address: a row is
// read before it is written.  It may not share memory with rows in any other way.
bool bad_place(const void* out, const void* rows, int64_t stride, int64_t n, int K, int type) {
  const int64_t size = static_cast<int64_t>(type_size(type));
  return overlap(out, n * K * size, rows, row_bytes(n, stride, K, size)) && !(out == rows && (stride == K || n == 1));
}
bool bad_width(int K) { return K < 1 || K > TQ_NORM_MAX_WIDTH; }

// Blocks of a kernel that the device holds at once (asked once per kernel, block and device).
template <typename Kernel>
long long resident(Kernel kernel, int threads) {
  struct Entry {
    const void* kernel;
    int threads, sms, blocks;
  };
  static thread_local Entry kept[64];
  const int sms = sm_count();
  const void* const id = reinterpret_cast<const void*>(kernel);
  Entry& e = kept[(reinterpret_cast<uintptr_t>(id) / 16 + threads / 32) % 64];
  if (e.kernel != id || e.threads != threads || e.sms != sms) {
    int per_sm = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, 0) != cudaSuccess) cudaGetLastError();
    e = {id, threads, sms, sms * std::max(1, per_sm)};
  }
  return e.blocks;
}

template <typename T>
int run_norm(const NormArgs& a, bool vec, cudaStream_t s) {
  const int threads = block_threads(a.K);
  auto kernel = vec ? (threads <= 256   ? rms_norm_kernel<T, true, 256>
                       : threads <= 512 ? rms_norm_kernel<T, true, 512>
                                        : rms_norm_kernel<T, true, 1024>)
                    : (threads <= 512 ? rms_norm_kernel<T, false, 512> : rms_norm_kernel<T, false, 1024>);
  return launch_pdl(kernel, dim3(static_cast<unsigned>(std::min<long long>(a.n, resident(kernel, threads)))), dim3(threads),
                    0, s, a);
}

template <typename T>
int run_backward(const NormGradArgs& a, bool vec, int blocks, cudaStream_t s) {
  const int threads = block_threads(a.K);
  if (vec && threads > 512) {
    constexpr int kMost = 224 * 1024;
    auto wide = rms_norm_backward_wide_kernel<T>;
    static std::atomic<uint64_t> allowed{0};   // bit d: device d
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) {
      cudaGetLastError();
      return TQ_ERR_CUDA;
    }
    const uint64_t bit = 1ull << (device & 63);
    if (!(allowed.load() & bit)) {
      if (cudaFuncSetAttribute(wide, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost) != cudaSuccess) {
        cudaGetLastError();
        return TQ_ERR_CUDA;
      }
      allowed.fetch_or(bit);
    }
    const int bytes = (a.grad_residual ? 3 : 2) * kPer * static_cast<int>(sizeof(T)) * threads;   // of a row: at most 192 KB
    const int buffers = 2 * bytes <= kMost ? 2 : 1;
    return launch_pdl(wide, dim3(blocks), dim3(threads), buffers * bytes, s, a, buffers);
  }
  auto kernel = vec ? rms_norm_backward_kernel<T, true, 512>
                    : (threads <= 512 ? rms_norm_backward_kernel<T, false, 512>
                                      : rms_norm_backward_kernel<T, false, 1024>);
  return launch_pdl(kernel, dim3(blocks), dim3(threads), 0, s, a);
}

// Blocks of the gradient: what the SMs hold at once at 128 registers a thread.
int backward_blocks(int64_t n, int K) {
  const int per_sm = std::max(1, std::min(16, 512 / block_threads(K)));
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
  const int64_t each = static_cast<int64_t>(size), w_size = static_cast<int64_t>(type_size(w_type));
  const Span y_rows{y, n * K * each}, r_rows{residual_out, n * K * each}, rstds{rstd, 4 * n}, code_rows{codes, n * K},
      scale_rows{scales, 4 * n * ((K + kFp8Block - 1) / kFp8Block)}, weights{weight, K * w_size};
  for (const void* out : {static_cast<const void*>(y), static_cast<const void*>(residual_out)}) {
    if (bad_place(out, x, x_stride, n, K, x_type) || bad_place(out, residual, residual_stride, n, K, x_type))
      return TQ_ERR_INVALID_ARG;
  }
  if (n > 0 && (outputs_overlap({y_rows, r_rows, rstds, code_rows, scale_rows}, {weights}) ||
                outputs_overlap({rstds, code_rows, scale_rows}, {{x, row_bytes(n, x_stride, K, each)},
                                                                 {residual, row_bytes(n, residual_stride, K, each)}})))
    return TQ_ERR_INVALID_ARG;
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
  if (bad_place(grad_x, x, x_stride, n, K, x_type) || bad_place(grad_x, grad_y, grad_y_stride, n, K, x_type) ||
      bad_place(grad_x, grad_residual, grad_residual_stride, n, K, x_type))
    return TQ_ERR_INVALID_ARG;
  const int64_t each = static_cast<int64_t>(size), w_bytes = K * static_cast<int64_t>(type_size(w_type));
  const Span gw{grad_weight, w_bytes}, weights{weight, w_bytes}, rstds{rstd, 4 * n};
  const Span work{grad_weight ? workspace : nullptr, static_cast<int64_t>(tq_rms_norm_backward_workspace_size(n, K))};
  if (n > 0 && (outputs_overlap({{grad_x, n * K * each}, gw, work}, {weights, rstds}) ||
                outputs_overlap({gw, work}, {{x, row_bytes(n, x_stride, K, each)},
                                             {grad_y, row_bytes(n, grad_y_stride, K, each)},
                                             {grad_residual, row_bytes(n, grad_residual_stride, K, each)}})))
    return TQ_ERR_INVALID_ARG;
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
  rc = launch_pdl(rms_norm_weight_kernel, dim3((K + 31) / 32), dim3(1024), 0, s, static_cast<const float*>(workspace),
                  blocks, K, grad_weight, w_type);
  if (rc == TQ_OK) count_launch(kCntNormWeight);
  return rc;
}

}  // extern "C"
