// Product of 4-bit microscaled weights with few activation rows, in one
// launch: y[t] = sum_j c_tj W_{e(t,j)} x[t], c the router weight and the
// global scales.
//
// A block takes eight weight rows and one activation row, which it quantises
// itself (the same values as tq_fp4_quantize) into shared memory as fp16.  A
// warp takes two of the rows over half of every 4096 values, a lane 32
// consecutive codes at a time: a 16-byte load, their fp16 pairs and sixteen
// fp16 FMAs.  Eight products of E2M1 pairs sum to a multiple of 1/4 of at most
// 288, 1152 units: exact in fp16's 11 bits, so the only roundings are those of
// the fp32 accumulation over blocks.  The token's top_k experts add up in the
// same registers; there is no scratch, no second launch and one order of
// summation.
//
// The block's rows are 2a, 2a + 1 of each 32-row quarter of a 128-row group:
// their scales share the 32-byte sectors of the tiled layout, which the block
// copies to shared memory together (read row by row, their 512-byte strides
// cost more of the load path than the codes: 1.2 us per 8.4M codes against
// 0.8).  Two rows a warp halve the reads of x from shared memory.
//
// Bound: weight bytes (one token of top-6, 4096 -> 2048: 28 MB, 4.2 us at the
// copy's rate, 10.1 us measured; one row of a linear 3.4 us).  What is left above
// the bytes is the launch, each block's quantising of its row, and the first
// loads' latency: a block has six batches of codes to hide it behind.  The codes
// and scales of the next 4096 values are in flight while the present ones are
// multiplied.
#include <cuda_runtime.h>

#include <algorithm>

#include "tq_fp4.cuh"
#include "tq_internal.h"

namespace tq {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kChunk = 32;        // codes per lane and load
constexpr int kBatchCodes = 4096; // values of a row per batch, half for each of two warps
constexpr int kBatchChunks = kBatchCodes / kChunk;
constexpr int kLoads = kBatchChunks / 2 / 32;   // loads per lane, row and batch

struct GemvParams {
  const uint8_t* w;
  const uint8_t* w_scales;
  const float* w_scale;
  const float* x_scale;
  const int32_t* ids;     // nullptr: one matrix
  const float* topk_w;
  int* err;
  long long stride;
  int top_k, E, K, N;
};

__device__ __forceinline__ uint4 load_stream(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// Two ways from codes to fp16 pairs, for the two words of a 16-code piece: they
// run on different pipes, and together take less time than either alone.
//
// By the hardware's conversion: codes 2 i and 2 i + 1 of a word.
struct Pairs {
  __half2 h[4];
};
__device__ __forceinline__ Pairs pairs_by_conversion(uint32_t w) {
  uint32_t r[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(w));
  Pairs p;
  memcpy(&p, r, 16);
  return p;
}
// By shifts: codes i and i + 4 of a word, times 2^-14.  An E2M1 code's exponent
// and mantissa bits in the low end of fp16's exponent and the high end of its
// mantissa are its value with the exponent bias 15 in place of 1, subnormals
// included.
__device__ __forceinline__ Pairs pairs_by_shifts(uint32_t w) {
  const uint32_t r[4] = {((w << 12) & 0x80008000u) | ((w << 9) & 0x0e000e00u),
                         ((w << 8) & 0x80008000u) | ((w << 5) & 0x0e000e00u),
                         ((w << 4) & 0x80008000u) | ((w << 1) & 0x0e000e00u),
                         (w & 0x80008000u) | ((w >> 3) & 0x0e000e00u)};
  Pairs p;
  memcpy(&p, r, 16);
  return p;
}

constexpr float kPieceScale = 1.f / 128.f;   // of dot16's result

// kPieceScale times the dot product of 16 codes with the 16 values that
// piece_x laid out in a and b.
__device__ __forceinline__ float dot16(uint32_t w0, uint32_t w1, uint4 a, uint4 b) {
  const __half2* const xa = reinterpret_cast<const __half2*>(&a);
  const __half2* const xb = reinterpret_cast<const __half2*>(&b);
  const Pairs p0 = pairs_by_conversion(w0), p1 = pairs_by_shifts(w1);
  __half2 sum = __hmul2(p0.h[0], xa[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) sum = __hfma2(p0.h[i], xa[i], sum);
#pragma unroll
  for (int i = 0; i < 4; ++i) sum = __hfma2(p1.h[i], xb[i], sum);
  const float2 f = __half22float2(sum);
  return f.x + f.y;
}

// The 16 values of two words of codes in the order and scaling of the two ways
// above: 2^-7 x beside codes, 2^7 x beside codes times 2^-14.
__device__ __forceinline__ void piece_x(uint2 q, uint4* a, uint4* b) {
  Pairs p0 = pairs_by_conversion(q.x), p1 = pairs_by_shifts(q.y);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    p0.h[i] = __hmul2(p0.h[i], __float2half2_rn(kPieceScale));
    p1.h[i] = __hmul2(__hmul2(p1.h[i], __float2half2_rn(16384.f)), __float2half2_rn(1.f / kPieceScale));
  }
  memcpy(a, &p0, 16);
  memcpy(b, &p1, 16);
}

// The E8M0 scale 2^e of a block of x as two factors: a block's dot product takes
// the first (`second` 0; 2^7 above its part, for kPieceScale), the weights' scale
// and then the other.  One scale can be 2^125 where the other is small: their
// product, or that of one of them and kPieceScale's inverse, would be infinite,
// and NaN beside a sum of 0.  With 2^e in halves for e > 0 no step is infinite
// unless the result is; for e <= 0 the whole of it comes first and is exact (a
// sum is a multiple of 1/4).
static_assert(kPieceScale == 0x1p-7f, "mx_factor");
__device__ __forceinline__ float mx_factor(uint32_t byte, int second) {
  const int late = max(static_cast<int>(byte) - 127, 0) >> 1;
  return __uint_as_float(static_cast<uint32_t>(second ? late + 127 : static_cast<int>(byte) - late + 7) << 23);
}

template <typename TX, typename TY, int kFmt>
__global__ void __launch_bounds__(kThreads, 4)
fp4_gemv_kernel(const TX* __restrict__ x, const GemvParams p, TY* __restrict__ y) {
  extern __shared__ uint4 smem[];
  constexpr int kTiles = kBatchCodes / fp4_block(kFmt) / 4;   // scale tiles per batch
  __shared__ uint4 scale_tiles[2][kTiles][2];                 // [buffer][tile][row parity]: four quarters x four blocks
  __shared__ float halves[8];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int K = p.K, N = p.N, top_k = p.top_k, E = p.E, chunks = K / kChunk, items = K / 16;
  // x in four planes of 8 values: chunk c's values 8 i .. 8 i + 7 at plane[i * chunks + c],
  // so that neighbouring lanes read neighbouring 16 bytes; then the scales of its 16-value pieces
  // (MX: the two factors of its blocks')
  uint4* const plane = smem;
  float* const xs = reinterpret_cast<float*>(smem + 4 * chunks);
  const long long t = blockIdx.y;
  const int group = blockIdx.x / 16, a2 = 2 * (blockIdx.x % 16);   // rows a2, a2 + 1 of each quarter
  const int quarter = warp & 3, half = warp >> 2;
  const int row0 = group * 128 + 32 * quarter + a2;
  const int steps = fp4_steps(K);
  const size_t group_bytes = static_cast<size_t>(steps) * fp4_scale_step_bytes(kFmt);
  const size_t w_expert = static_cast<size_t>(N) * (K / 2), ws_expert = (N + 127) / 128 * group_bytes;
  const uint8_t* const w = p.w + static_cast<size_t>(row0) * (K / 2);
  const uint8_t* const ws = p.w_scales + group * group_bytes + a2 * 16;
  const int rows = max(0, min(2, N - row0));
  const int tiles = steps * (fp4_scale_step_bytes(kFmt) / 512);

  const int per = (K + kBatchCodes - 1) / kBatchCodes;   // batches per expert
  const int32_t* const ids = p.ids ? p.ids + t * top_k : nullptr;
  // expert of pair j; -1 when out of range
  auto expert = [&](int j) {
    if (!ids) return 0;
    const int e = __ldg(ids + j);
    return e >= 0 && e < E ? e : -1;
  };
  int j = 0, i = 0;       // pair and batch of `next`
  int e = expert(0);
  uint4 next[2][kLoads];
  auto fetch = [&](int buffer) {
    const uint8_t* const src = w + max(e, 0) * w_expert;
    const int c0 = i * kBatchChunks + half * (kBatchChunks / 2) + lane;
    // an expert or a row out of range: nothing is read, its terms are zero
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        const int c = c0 + 32 * k;
        next[r][k] = make_uint4(0u, 0u, 0u, 0u);
        if (e >= 0 && r < rows && c < chunks) next[r][k] = load_stream(src + r * (K / 2) + 16ll * c);
      }
    }
    if (threadIdx.x < 2 * kTiles) {
      const int tile = i * kTiles + threadIdx.x / 2;
      if (e >= 0 && tile < tiles)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(
                         smem_u32(&scale_tiles[buffer][threadIdx.x / 2][threadIdx.x & 1])),
                     "l"(ws + e * ws_expert + tile * 512ll + (threadIdx.x & 1) * 16)
                     : "memory");
    }
  };
  fetch(0);   // under way while x is quantised

  const TX* const row_x = x + t * p.stride;
  const GlobalScale g(p.x_scale);
  for (int item0 = threadIdx.x - lane; item0 < items; item0 += kThreads) {
    const int item = item0 + lane;
    float v[16] = {}, top = 0.f;
    if (item < items) top = open_piece(load_piece(row_x + 16 * item), v);
    if (kFmt == TQ_FP4_MX) top = fmaxf(top, __shfl_xor_sync(kAll, top, 1));
    float d, r;
    const uint32_t byte = fp4_block_scale<kFmt>(top, g, &d, &r);
    const uint2 q = fp4_codes16<kFmt>(v, d, r, top);
    if (item < items) {
      piece_x(q, &plane[(2 * (item & 1)) * chunks + item / 2], &plane[(2 * (item & 1) + 1) * chunks + item / 2]);
      xs[item] = kFmt == TQ_FP4_NV ? from_e4m3(byte) * (1.f / kPieceScale) : mx_factor(byte, item & 1);
    }
  }

  float total[2] = {0.f, 0.f}, part[2] = {0.f, 0.f};
  for (int n = 0; j < top_k; ++n) {
    uint4 q[2][kLoads];
    memcpy(q, next, sizeof(q));
    const int cj = j, ci = i, ce = e;
    // the scales of this batch (and, the first time, x) are in; the other
    // buffer has been read by every warp
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    if (++i == per) {
      i = 0;
      if (++j < top_k) e = expert(j);
    }
    if (j < top_k) fetch((n + 1) & 1);
    const uint8_t* const sw = reinterpret_cast<const uint8_t*>(scale_tiles[n & 1]) + 4 * quarter;
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      const int in = half * (kBatchChunks / 2) + 32 * k + lane;   // chunk inside the batch
      const int c = ci * kBatchChunks + in;
      if (ce < 0 || c >= chunks) break;
      const uint4 x0 = plane[c], x1 = plane[chunks + c], x2 = plane[2 * chunks + c], x3 = plane[3 * chunks + c];
      const float2 s = reinterpret_cast<const float2*>(xs)[c];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float d0 = dot16(q[r][k].x, q[r][k].y, x0, x1);
        const float d1 = dot16(q[r][k].z, q[r][k].w, x2, x3);
        if (kFmt == TQ_FP4_NV) {
          uint32_t h;
          asm("cvt.rn.f16x2.e4m3x2 %0, %1;"
              : "=r"(h) : "h"(*reinterpret_cast<const uint16_t*>(sw + (in / 2) * 32 + r * 16 + (in & 1) * 2)));
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
          part[r] = fmaf(d0, s.x * f.x, part[r]);
          part[r] = fmaf(d1, s.y * f.y, part[r]);
        } else {
          part[r] = fmaf((d0 + d1) * s.x * from_e8m0(sw[(in / 4) * 32 + r * 16 + (in & 3)]), s.y, part[r]);
        }
      }
    }
    if (ci == per - 1) {
      if (ce < 0) {
        if (threadIdx.x == 0) record_error(p.err, TQ_ERR_INVALID_ARG, kWhereFp4Gemv);
      } else {
        const float c =
            (p.topk_w ? __ldg(p.topk_w + t * top_k + cj) : 1.f) * (g.g * (p.w_scale ? __ldg(p.w_scale + ce) : 1.f));
        total[0] = fmaf(c, part[0], total[0]);
        total[1] = fmaf(c, part[1], total[1]);
      }
      part[0] = part[1] = 0.f;
    }
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total[r] += __shfl_xor_sync(kAll, total[r], o);
    if (half == 1 && lane == 0) halves[2 * quarter + r] = total[r];
  }
  __syncthreads();
  if (half == 0 && lane < rows) y[t * N + row0 + lane] = narrow<TY>((lane ? total[1] : total[0]) + halves[2 * quarter + lane]);
}

template <typename TX, typename TY>
int run(const Fp4Gemv& g, cudaStream_t s) {
  const GemvParams p{g.w, g.w_scales, g.w_scale, g.x_scale, g.ids, g.topk_w, g.err, g.stride, g.top_k, g.E, g.K, g.N};
  auto kernel = g.fmt == TQ_FP4_NV ? fp4_gemv_kernel<TX, TY, TQ_FP4_NV> : fp4_gemv_kernel<TX, TY, TQ_FP4_MX>;
  const size_t smem = static_cast<size_t>(g.K) * 2 + static_cast<size_t>(g.K) / 16 * 4;
  return launch_pdl(kernel, dim3((g.N + 127) / 128 * 16, static_cast<unsigned>(g.n)), dim3(kThreads), smem, s,
                    static_cast<const TX*>(g.x), p, static_cast<TY*>(g.y));
}

template <typename TX>
int run_to(const Fp4Gemv& g, cudaStream_t s) {
  return g.y_type == TQ_FP32 ? run<TX, float>(g, s)
         : g.y_type == TQ_BF16 ? run<TX, __nv_bfloat16>(g, s)
                               : run<TX, __half>(g, s);
}

}  // namespace

int launch_fp4_gemv(const Fp4Gemv& g, cudaStream_t s) {
  const int st = g.x_type == TQ_FP32 ? run_to<float>(g, s)
                 : g.x_type == TQ_BF16 ? run_to<__nv_bfloat16>(g, s)
                                       : run_to<__half>(g, s);
  if (st == TQ_OK) count_launch(kCntFp4Gemv);
  return st;
}

}  // namespace tq
