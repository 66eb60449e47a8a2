// 4-bit microscaled values: quantise, dequantise, the tiled scale layout, the
// product's activation staging and the combine of its partial sums.
//
// All of these move bytes: a thread takes 16 consecutive values (two or four
// 16-byte loads), so a warp reads 1 or 2 KiB of a row at once and writes 256
// bytes of codes.  A block of 32 values is two neighbouring threads, which
// share their maximum by one shuffle.
//
// Measured for 8192 x 4096 bf16 values, NV: quantise 17.9 us for 86 MB (the
// issue of its instructions is 71% busy), dequantise 13.8 us for 86 MB (6.2
// TB/s); the two in turn 31.2 us.  Staging 2048 tokens for top-6 products: 15.5 us
// for 17 MB read and 28 MB written: a pair's scales are single words 16 bytes
// apart in the tiled layout, a 32-byte sector of L2 each, so that the scales
// take twice the sectors of the codes.  The combine of those 12288 x 2048
// partial sums: 23.6 us for 109 MB, of 8192 tokens 69 us for 436 MB (6.3 TB/s).
#include <cuda_runtime.h>

#include <algorithm>

#include "tq_fp4.cuh"
#include "tq_internal.h"

namespace tq {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kQuantThreads = 256;

// Quantises 16 values, the largest magnitude `top`, of a block (the whole of
// it, or one of its two halves in neighbouring lanes; every lane of the warp
// takes part): codes and scale byte.
template <int kFmt>
__device__ __forceinline__ uint2 quantize16(const float (&v)[16], float top, const GlobalScale& g, uint32_t* byte) {
  if (kFmt == TQ_FP4_MX) top = fmaxf(top, __shfl_xor_sync(kAll, top, 1));
  float d, r;
  *byte = fp4_block_scale<kFmt>(top, g, &d, &r);
  return fp4_codes16<kFmt>(v, d, r, top);
}

// A warp takes a chunk of 512 values at a time; the next chunk's loads are in
// flight while the present one is quantised.  Row and chunk advance by the
// launch's constant step (step_rows, step_chunks), without divisions.
template <typename T, int kFmt>
__global__ void __launch_bounds__(kQuantThreads)
fp4_quantize_kernel(const T* __restrict__ x, long long stride, long long n, int K, const float* __restrict__ scale,
                    int step_rows, int step_chunks, uint8_t* __restrict__ packed, uint8_t* __restrict__ scales) {
  pdl_wait();
  pdl_trigger();
  const GlobalScale g(scale);
  const int lane = threadIdx.x & 31;
  const int items = K / 16, chunks = (items + 31) / 32;
  const long long warp = blockIdx.x * (kQuantThreads / 32ll) + (threadIdx.x >> 5);
  long long row = warp / chunks;
  int chunk = static_cast<int>(warp - row * chunks);
  Piece<T> next = {};
  if (row < n && chunk * 32 + lane < items) next = load_piece(x + row * stride + 16 * (chunk * 32 + lane));
  while (row < n) {
    const Piece<T> piece = next;
    const int item = chunk * 32 + lane;
    const long long at = row;
    row += step_rows;
    chunk += step_chunks;
    if (chunk >= chunks) {
      chunk -= chunks;
      ++row;
    }
    if (row < n && chunk * 32 + lane < items) next = load_piece(x + row * stride + 16 * (chunk * 32 + lane));
    float v[16];
    const float top = open_piece(piece, v);   // lanes past the row hold an old piece and write nothing
    uint32_t byte;
    const uint2 q = quantize16<kFmt>(v, top, g, &byte);
    if (item < items) {
      *reinterpret_cast<uint2*>(packed + at * (K / 2) + 8 * item) = q;
      if (kFmt == TQ_FP4_NV)
        scales[at * items + item] = static_cast<uint8_t>(byte);
      else if ((lane & 1) == 0)
        scales[at * (items / 2) + item / 2] = static_cast<uint8_t>(byte);
    }
  }
}

// Two E2M1 codes (low half first) as fp32.
__device__ __forceinline__ float2 from_e2m1x2(uint32_t byte) {
  uint32_t h;
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}"
      : "=r"(h) : "r"(byte));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// A thread writes 16 bytes of consecutive values (8 of 16 bits, 4 of 32), so
// that a warp's stores are whole lines; kAhead of them at once.
template <typename T, int kFmt>
__global__ void __launch_bounds__(kQuantThreads)
fp4_dequantize_kernel(const uint8_t* __restrict__ packed, const uint8_t* __restrict__ scales, long long items,
                      const float* __restrict__ scale, T* __restrict__ out) {
  constexpr int kVals = 16 / static_cast<int>(sizeof(T)), kAhead = 4;
  using Codes = std::conditional_t<kVals == 8, uint32_t, uint16_t>;
  pdl_wait();
  pdl_trigger();
  const float g = scale ? *scale : 1.f;
  const long long step = static_cast<long long>(gridDim.x) * kQuantThreads;
  for (long long i0 = blockIdx.x * static_cast<long long>(kQuantThreads) + threadIdx.x; i0 < items;
       i0 += kAhead * step) {
    Codes q[kAhead];
    uint32_t b[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const long long i = i0 + a * step;
      if (i < items) {
        q[a] = __ldg(reinterpret_cast<const Codes*>(packed) + i);
        b[a] = __ldg(scales + i / (fp4_block(kFmt) / kVals));
      }
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const long long i = i0 + a * step;
      if (i >= items) break;
      const float s = fp4_scale_value<kFmt>(b[a]);
      T v[kVals];
#pragma unroll
      for (int j = 0; j < kVals / 2; ++j) {
        const float2 f = from_e2m1x2(static_cast<uint32_t>(q[a]) >> (8 * j));
        v[2 * j] = narrow<T>(__fmul_rn(__fmul_rn(f.x, s), g));
        v[2 * j + 1] = narrow<T>(__fmul_rn(__fmul_rn(f.y, s), g));
      }
      uint4 o;
      memcpy(&o, v, 16);
      reinterpret_cast<uint4*>(out)[i] = o;
    }
  }
}

// Row-major scales to the tiled layout: one thread per four blocks of a row,
// padding rows and blocks zero.
__global__ void __launch_bounds__(kQuantThreads)
fp4_tile_scales_kernel(const uint8_t* __restrict__ scales, int E, int N, int kb, int kb4, uint32_t* __restrict__ tiled) {
  pdl_wait();
  pdl_trigger();
  const int rows = (N + 127) / 128 * 128;
  const long long total = static_cast<long long>(E) * rows * kb4;
  const long long step = static_cast<long long>(gridDim.x) * kQuantThreads;
  for (long long i = blockIdx.x * static_cast<long long>(kQuantThreads) + threadIdx.x; i < total; i += step) {
    // i = ((e * row groups + group) * kb4 + b4) * 128 + (row % 32) * 4 + (row % 128) / 32
    const int in = static_cast<int>(i & 127);
    const long long tile = i >> 7;
    const int b4 = static_cast<int>(tile % kb4);
    const long long group = tile / kb4;
    const long long e = group / (rows / 128);
    const int r = static_cast<int>(group - e * (rows / 128)) * 128 + (in & 3) * 32 + (in >> 2);
    uint32_t word = 0;
    if (r < N) {
      const uint8_t* const src = scales + (e * N + r) * kb + 4 * b4;
#pragma unroll
      for (int j = 0; j < 4; ++j) word |= 4 * b4 + j < kb ? static_cast<uint32_t>(src[j]) << (8 * j) : 0u;
    }
    tiled[i] = word;
  }
}

// Where a pair's staged row goes: byte offsets of its codes and of its first
// scale in the tiled layout of its m-tile; codes -1 for a pair without a place
// (an expert out of range).
struct Place {
  long long codes, scales;
};

template <int kFmt>
__device__ __forceinline__ Place place_of(const Fp4Slots& s, long long pair, int tile_m, int K) {
  long long slot = pair, tile, row;
  if (s.slot_of) {
    const int e = __ldg(s.ids + pair);
    slot = __ldg(s.slot_of + pair);
    if (slot < 0) return {-1, 0};
    const int rank = static_cast<int>(slot) - __ldg(s.offsets + e);
    tile = __ldg(s.tile_first + e) + rank / tile_m;
    row = rank % tile_m;
  } else {
    tile = pair / tile_m;
    row = pair % tile_m;
  }
  const int steps = fp4_steps(K);
  const long long tile_bytes = static_cast<long long>((tile_m + 127) / 128) * steps * fp4_scale_step_bytes(kFmt);
  return {slot * (K / 2), tile * tile_bytes + static_cast<long long>(fp4_tiled_offset(kFmt, steps, row, 0))};
}

// One block's share of a staged row: 16 values per thread and their largest
// magnitude from load(item, v), their codes and scales to each of the row's places
// (blocks past K zero, so that the MMA's last step multiplies zeros by a finite
// scale).
template <int kFmt, typename Load>
__device__ __forceinline__ void stage_row(int K, const GlobalScale& g, const Place* places, int count,
                                          uint8_t* __restrict__ xq, uint8_t* __restrict__ xs, Load&& load) {
  const int steps = fp4_steps(K);
  const int items = K / 16, all = steps * (kFp4Step / 16);
  const int lane = threadIdx.x & 31;
  // whole warps stay in the loop together: all is a multiple of 16, a warp may end half empty
  for (int item0 = threadIdx.x - lane; item0 < all; item0 += blockDim.x) {
    const int item = item0 + lane;
    float v[16] = {}, top = 0.f;
    if (item < items) top = load(item, v);
    uint32_t byte;
    const uint2 q = quantize16<kFmt>(v, top, g, &byte);
    if (item >= items) byte = 0;
    // four blocks' scales in one word
    uint32_t word;
    int word_lane;   // lane of the word's first block
    if (kFmt == TQ_FP4_NV) {
      word_lane = lane & ~3;
      word = __shfl_sync(kAll, byte, word_lane) | __shfl_sync(kAll, byte, word_lane + 1) << 8 |
             __shfl_sync(kAll, byte, word_lane + 2) << 16 | __shfl_sync(kAll, byte, word_lane + 3) << 24;
    } else {
      word_lane = lane & ~7;
      word = __shfl_sync(kAll, byte, word_lane) | __shfl_sync(kAll, byte, word_lane + 2) << 8 |
             __shfl_sync(kAll, byte, word_lane + 4) << 16 | __shfl_sync(kAll, byte, word_lane + 6) << 24;
    }
    const int block = kFmt == TQ_FP4_NV ? item : item / 2;
    uint8_t* const codes = xq + 8 * item;
    uint8_t* const scales = xs + fp4_tiled_offset(kFmt, steps, 0, block);
    const bool writes_scales = item < all && lane == word_lane;
    for (int j = 0; j < count; ++j) {
      const Place p = places[j];
      if (p.codes < 0) continue;
      if (item < items) *reinterpret_cast<uint2*>(codes + p.codes) = q;
      if (writes_scales) *reinterpret_cast<uint32_t*>(scales + p.scales) = word;
    }
  }
}

// Quantises each token's row once and writes it where the product reads it,
// once per pair of the token.  Without slot_of a row's slot is its index and
// its tile index / tile_m.  One block per row.
template <typename T, int kFmt>
__global__ void __launch_bounds__(kQuantThreads)
fp4_stage_kernel(const T* __restrict__ x, long long stride, int K, const float* __restrict__ scale, int top_k,
                 const Fp4Slots slots, int tile_m, uint8_t* __restrict__ xq, uint8_t* __restrict__ xs) {
  __shared__ Place places[32];
  pdl_wait();
  pdl_trigger();
  const long long row = blockIdx.x;
  // the row's first values are under way while its places are looked up
  Piece<T> first = {};
  if (static_cast<int>(threadIdx.x) < K / 16) first = load_piece(x + row * stride + 16 * threadIdx.x);
  const GlobalScale g(scale);
  if (static_cast<int>(threadIdx.x) < top_k)
    places[threadIdx.x] = place_of<kFmt>(slots, row * top_k + threadIdx.x, tile_m, K);
  __syncthreads();
  stage_row<kFmt>(K, g, places, top_k, xq, xs, [&](int item, float (&v)[16]) {
    return open_piece(item == static_cast<int>(threadIdx.x) ? first : load_piece(x + row * stride + 16 * item), v);
  });
}

// h = silu(gate) * up of one pair per block, quantised from fp32.  gate and up
// are sums of the product's splits times x_scale * w_scale[expert].
template <int kFmt>
__global__ void __launch_bounds__(kQuantThreads)
fp4_stage_swiglu_kernel(const float* __restrict__ part, long long split_stride, int splits,
                        const float* __restrict__ x_scale, const float* __restrict__ w_scale, int E, int I,
                        const float* __restrict__ h_scale, const Fp4Slots slots, int tile_m,
                        uint8_t* __restrict__ hq, uint8_t* __restrict__ hs) {
  __shared__ Place place;
  pdl_wait();
  pdl_trigger();
  const long long pair = blockIdx.x;
  if (threadIdx.x == 0) place = place_of<kFmt>(slots, pair, tile_m, I);
  __syncthreads();
  const int e = __ldg(slots.ids + pair);
  if (place.codes < 0 || e < 0 || e >= E) return;   // a pair without a slot has no gate and up either
  const float alpha = (x_scale ? *x_scale : 1.f) * (w_scale ? __ldg(w_scale + e) : 1.f);
  const float* const row = part + pair * 2 * I;
  stage_row<kFmt>(I, GlobalScale(h_scale), &place, 1, hq, hs, [&](int item, float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
      for (int s = 0; s < splits; ++s) {
        const float* const src = row + s * split_stride + 16 * item + i;
        const float4 c = __ldcs(reinterpret_cast<const float4*>(src));
        const float4 d = __ldcs(reinterpret_cast<const float4*>(src + I));
        a = make_float4(a.x + c.x, a.y + c.y, a.z + c.z, a.w + c.w);
        b = make_float4(b.x + d.x, b.y + d.y, b.z + d.z, b.w + d.w);
      }
      const float gate[4] = {a.x * alpha, a.y * alpha, a.z * alpha, a.w * alpha};
      const float up[4] = {b.x * alpha, b.y * alpha, b.z * alpha, b.w * alpha};
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i + j] = gate[j] / (1.f + expf(-gate[j])) * up[j];
    }
    return fp4_max16(v);
  });
}

// y[t][r] = sum_j c_tj sum_s part[s][t * top_k + j][r] in that order, in fp32,
// rounded once; c_tj = topk_w[t][j] * x_scale * w_scale[expert].  A pair whose
// expert is out of range adds nothing (its partial sums were never written and
// are not read).  kVec columns per thread, two pairs' loads in flight: occupancy
// hides the latency better than more of them (8192 tokens of top-6, 2048
// columns: 69 us at two and 32 registers, 84 at four, 103 at eight).
template <typename T, int kVec>
__global__ void __launch_bounds__(kQuantThreads, 8)
fp4_combine_kernel(const float* __restrict__ part, long long part_ld, long long split_stride, int splits, const int32_t* __restrict__ ids,
                   const float* __restrict__ topk_w, const float* __restrict__ x_scale,
                   const float* __restrict__ w_scale, int top_k, int E, int N, int blocks_per_row, bool wide,
                   T* __restrict__ y) {
  constexpr int kAhead = 2;
  __shared__ float coef[32];
  __shared__ bool skip[32];
  pdl_wait();
  pdl_trigger();
  const long long t = blockIdx.x / blocks_per_row;
  const int c = (blockIdx.x - static_cast<int>(t * blocks_per_row)) * kQuantThreads + threadIdx.x;
  if (static_cast<int>(threadIdx.x) < top_k) {
    const long long pair = t * top_k + threadIdx.x;
    const int e = ids ? __ldg(ids + pair) : 0;
    const bool in = e >= 0 && e < E;
    skip[threadIdx.x] = !in;
    coef[threadIdx.x] = in ? (topk_w ? __ldg(topk_w + pair) : 1.f) *
                                 ((x_scale ? *x_scale : 1.f) * (w_scale ? __ldg(w_scale + e) : 1.f))
                           : 0.f;
  }
  __syncthreads();
  if (c * kVec >= N) return;
  float sum[kVec] = {};
  const float* const src = part + t * top_k * part_ld + static_cast<long long>(c) * kVec;
  for (int j0 = 0; j0 < top_k; j0 += kAhead) {
    float v[kAhead][kVec] = {};
    for (int s = 0; s < splits; ++s) {
      float f[kAhead][kVec] = {};
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int j = j0 + i;
        if (j >= top_k || skip[j]) continue;
        const float* const p = src + s * split_stride + static_cast<long long>(j) * part_ld;
        if constexpr (kVec == 4) {
          const float4 q = __ldcs(reinterpret_cast<const float4*>(p));
          f[i][0] = q.x;
          f[i][1] = q.y;
          f[i][2] = q.z;
          f[i][3] = q.w;
        } else {
          f[i][0] = __ldcs(p);
        }
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
#pragma unroll
        for (int q = 0; q < kVec; ++q) v[i][q] += f[i][q];
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (j0 + i >= top_k || skip[j0 + i]) continue;
#pragma unroll
      for (int q = 0; q < kVec; ++q) sum[q] = fmaf(coef[j0 + i], v[i][q], sum[q]);
    }
  }
  T out[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) out[i] = narrow<T>(sum[i]);
  T* const dst = y + t * N + static_cast<long long>(c) * kVec;
  if (kVec == 4 && !wide) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      if (c * kVec + i < N) dst[i] = out[i];
    }
  } else if constexpr (kVec == 4 && sizeof(T) == 4) {
    float4 o;
    memcpy(&o, out, 16);
    *reinterpret_cast<float4*>(dst) = o;
  } else if constexpr (kVec == 4) {
    uint2 o;
    memcpy(&o, out, 8);
    *reinterpret_cast<uint2*>(dst) = o;
  } else {
    dst[0] = out[0];
  }
}

// Threads of a block that stages one row: one per 16 values, 32 to 256.
int row_threads(int K) {
  return std::min(kQuantThreads, (fp4_steps(K) * (kFp4Step / 16) + 31) / 32 * 32);
}

int quant_blocks(long long warps_of_work) {
  const long long per = kQuantThreads / 32;
  return static_cast<int>(std::max<long long>(1, std::min<long long>((warps_of_work + per - 1) / per,
                                                                     static_cast<long long>(sm_count()) * 8)));
}

// f(T *, integral_constant fmt) for the element type and format.
template <typename F>
int by_type(int type, int fmt, F&& f) {
  using NV = std::integral_constant<int, TQ_FP4_NV>;
  using MX = std::integral_constant<int, TQ_FP4_MX>;
  switch (type) {
    case TQ_FP32: return fmt == TQ_FP4_NV ? f(static_cast<float*>(nullptr), NV()) : f(static_cast<float*>(nullptr), MX());
    case TQ_BF16:
      return fmt == TQ_FP4_NV ? f(static_cast<__nv_bfloat16*>(nullptr), NV())
                              : f(static_cast<__nv_bfloat16*>(nullptr), MX());
    default: return fmt == TQ_FP4_NV ? f(static_cast<__half*>(nullptr), NV()) : f(static_cast<__half*>(nullptr), MX());
  }
}

}  // namespace

int launch_fp4_quantize(const void* x, int type, int64_t stride, int64_t n, int K, int fmt, const float* scale,
                        uint8_t* packed, uint8_t* scales, cudaStream_t s) {
  const int chunks = (K / 16 + 31) / 32;
  const int blocks = quant_blocks(n * chunks), warps = blocks * (kQuantThreads / 32);
  const int st = by_type(type, fmt, [&](auto* t, auto f) {
    using T = std::remove_pointer_t<decltype(t)>;
    return launch_pdl(fp4_quantize_kernel<T, decltype(f)::value>, dim3(blocks), dim3(kQuantThreads), 0, s,
                      static_cast<const T*>(x), static_cast<long long>(stride), static_cast<long long>(n), K, scale,
                      warps / chunks, warps % chunks, packed, scales);
  });
  if (st == TQ_OK) count_launch(kCntFp4Quantize);
  return st;
}

int launch_fp4_dequantize(const uint8_t* packed, const uint8_t* scales, int64_t n, int K, int fmt, const float* scale,
                          void* out, int type, cudaStream_t s) {
  const long long items = n * K * static_cast<long long>(type_size(type)) / 16;
  const int st = by_type(type, fmt, [&](auto* t, auto f) {
    using T = std::remove_pointer_t<decltype(t)>;
    return launch_pdl(fp4_dequantize_kernel<T, decltype(f)::value>, dim3(quant_blocks((items + 31) / 32)),
                      dim3(kQuantThreads), 0, s, packed, scales, items, scale, static_cast<T*>(out));
  });
  if (st == TQ_OK) count_launch(kCntFp4Dequantize);
  return st;
}

int launch_fp4_tile_scales(const uint8_t* scales, int E, int N, int K, int fmt, uint8_t* tiled, cudaStream_t s) {
  const int kb = K / fp4_block(fmt), kb4 = fp4_steps(K) * (kFp4Step / fp4_block(fmt)) / 4;
  const long long words = static_cast<long long>(E) * ((N + 127) / 128 * 128) * kb4;
  const int st = launch_pdl(fp4_tile_scales_kernel, dim3(quant_blocks((words + 31) / 32)), dim3(kQuantThreads), 0, s, scales,
                    E, N, kb, kb4, reinterpret_cast<uint32_t*>(tiled));
  if (st == TQ_OK) count_launch(kCntFp4TileScales);
  return st;
}

int launch_fp4_stage(const void* x, int type, int64_t stride, int64_t n, int K, int fmt, const float* scale, int top_k,
                     const Fp4Slots& slots, int tile_m, uint8_t* xq, uint8_t* xs, cudaStream_t s) {
  const int st = by_type(type, fmt, [&](auto* t, auto f) {
    using T = std::remove_pointer_t<decltype(t)>;
    return launch_pdl(fp4_stage_kernel<T, decltype(f)::value>, dim3(static_cast<unsigned>(n)), dim3(row_threads(K)), 0,
                      s, static_cast<const T*>(x), static_cast<long long>(stride), K, scale, top_k, slots, tile_m, xq,
                      xs);
  });
  if (st == TQ_OK) count_launch(kCntFp4Stage);
  return st;
}

int launch_fp4_stage_swiglu(const float* part, int64_t split_stride, int splits, const float* x_scale,
                            const float* w_scale, int64_t P, int E, int I, int fmt, const float* h_scale,
                            const Fp4Slots& slots, int tile_m, uint8_t* hq, uint8_t* hs, cudaStream_t s) {
  auto kernel = fmt == TQ_FP4_NV ? fp4_stage_swiglu_kernel<TQ_FP4_NV> : fp4_stage_swiglu_kernel<TQ_FP4_MX>;
  const int st = launch_pdl(kernel, dim3(static_cast<unsigned>(P)), dim3(row_threads(I)), 0, s, part,
                            static_cast<long long>(split_stride), splits, x_scale, w_scale, E, I, h_scale, slots,
                            tile_m, hq, hs);
  if (st == TQ_OK) count_launch(kCntFp4Swiglu);
  return st;
}

int launch_fp4_combine(const float* part, int64_t part_ld, int64_t split_stride, int splits, const int32_t* ids, const float* topk_w,
                       const float* x_scale, const float* w_scale, int64_t n, int top_k, int E, int N, void* y,
                       int type, cudaStream_t s) {
  // partial sums in whole vectors, past N too, and results in them where their rows allow it
  const bool vec = part_ld % 4 == 0;
  const bool wide = N % 4 == 0 && (reinterpret_cast<uintptr_t>(y) & 15u) == 0;
  const int cols = vec ? (N - 1) / 4 + 1 : N;
  const int per_row = (cols + kQuantThreads - 1) / kQuantThreads;
  const long long blocks = n * per_row;
  if (blocks >= (1ll << 31)) return TQ_ERR_INVALID_ARG;
  const int st = by_type(type, TQ_FP4_NV, [&](auto* t, auto) {
    using T = std::remove_pointer_t<decltype(t)>;
    auto kernel = vec ? fp4_combine_kernel<T, 4> : fp4_combine_kernel<T, 1>;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(kQuantThreads), 0, s, part,
                      static_cast<long long>(part_ld), static_cast<long long>(split_stride), splits, ids, topk_w, x_scale,
                      w_scale, top_k, E, N, per_row, wide, static_cast<T*>(y));
  });
  if (st == TQ_OK) count_launch(kCntFp4Combine);
  return st;
}

}  // namespace tq
