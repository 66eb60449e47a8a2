// Matrix products with few activation rows: y[t] = W x[t] for up to 8 or 16 rows of x
// that share a matrix, bound by the reading of W.
//
// A warp multiplies 16 weight rows (gated: 16 of the gate and 16 of the up
// projection) with all the activation rows, K 128 bytes at a time, by m16n8
// MMAs whose operands come straight from global memory: the order of K inside a sum
// is free, so a lane takes 16 consecutive bytes of a weight row and of an activation
// row and gives them to the MMAs four bytes at a time, both in the same order.  No
// shared memory and no conversion on the way; tensor memory and its 128-row tiles
// would mean a pipeline set up for 16 KB of weights.  The MMA is not the bound: 8
// rows a pass are far below its rate at the memory's.
//
// The eight warps of a block split K by blocks of 128 bytes and add up through
// shared memory in a fixed order; a block's warps have up to four such blocks each
// in flight.
//
// 8-bit products: 128 bytes are a scale block, whose partial sums are scaled into
// fp32 registers.
#include <cuda_runtime.h>

#include <algorithm>

#include "tq_device.cuh"
#include "tq_internal.h"
#include "tq_types.cuh"

namespace tq {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kRows = 16;          // weight rows per block
constexpr int kStepBytes = 128;    // of a row per step
// Steps in flight per warp: 64 registers of weights.
template <int kParts>
constexpr int kAheadOf = 4 / kParts;

enum Kind { kFp8 = 0, kBf16 = 1, kFp16 = 2 };

__device__ __forceinline__ uint4 load_stream(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// c[16][8] += a[16][32 bytes of K] b[8][the same]^T
template <int kKind>
__device__ __forceinline__ void mma16x8(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
#define TQ_MMA(shape, types)                                                                                     \
  asm volatile("mma.sync.aligned." shape ".row.col.f32." types ".f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, " \
               "{%0, %1, %2, %3};"                                                                              \
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])                                                  \
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1))
  if constexpr (kKind == kFp8)
    TQ_MMA("m16n8k32", "e4m3.e4m3");
  else if constexpr (kKind == kBf16)
    TQ_MMA("m16n8k16", "bf16.bf16");
  else
    TQ_MMA("m16n8k16", "f16.f16");
#undef TQ_MMA
}

template <bool kFirst, typename T>
__device__ __forceinline__ T& either(T& a, T& b) {
  if constexpr (kFirst)
    return a;
  else
    return b;
}

// kParts: matrices of 16 rows per warp (2 gated); kTiles: groups of 8 activation rows.
template <int kKind, int kParts, int kTiles>
__global__ void __launch_bounds__(kThreads, 2) few_rows_kernel(const FewRows p) {
  constexpr int kCols = 8 * kTiles, kAhead = kAheadOf<kParts>;
  __shared__ float sums[kWarps][kParts][kRows][kCols];
  __shared__ int x_row[kCols], y_row[kCols];
  __shared__ int expert;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int tile = blockIdx.y;
  if (p.num_tiles && tile >= *p.num_tiles) return;
  // the unit's activation rows: of a tile map's tile, of one pair, or consecutive
  if (threadIdx.x < kCols) {
    const int c = threadIdx.x;
    int e = 0, slot0 = tile * kCols, rows = p.M - slot0, xr = -1, yr = -1;
    if (p.tiles) {
      e = __ldg(p.tiles + 3 * tile);
      slot0 = __ldg(p.tiles + 3 * tile + 1);
      rows = __ldg(p.tiles + 3 * tile + 2);
    } else if (p.ids) {
      slot0 = tile;
      rows = 1;
      e = __ldg(p.ids + tile);
    }
    if (e < 0 || e >= p.E || slot0 < 0 || rows > p.M - slot0) {
      if (c == 0) record_error(p.err, TQ_ERR_INVALID_ARG, kWhereFewRows);
      e = -1;
    } else if (c < rows) {
      const int slot = slot0 + c;
      const int pair = p.sorted_pairs ? __ldg(p.sorted_pairs + slot) : slot;
      if (pair >= 0 && pair < p.M) {
        xr = p.gather ? pair / p.top_k : slot;
        yr = p.scatter ? pair : slot;
      } else {
        record_error(p.err, TQ_ERR_INVALID_ARG, kWhereFewRows);
      }
    }
    x_row[c] = xr;
    y_row[c] = yr;
    if (c == 0) expert = e;
  }
  __syncthreads();
  const int e = expert;
  if (e < 0) return;

  const int row0 = blockIdx.x * kRows;
  const long long row_bytes = p.row_bytes;
  const uint8_t* w[kParts][2];   // this lane's two rows of each part
  bool in[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = row0 + g + 8 * h;
    in[h] = r < p.N;
#pragma unroll
    for (int a = 0; a < kParts; ++a)
      w[a][h] = p.w + (static_cast<long long>(e) * kParts * p.N + a * p.N + min(r, p.N - 1)) * row_bytes + 16 * q;
  }
  const uint8_t* x[kTiles];
  bool has[kTiles];
#pragma unroll
  for (int t = 0; t < kTiles; ++t) {
    const int xr = x_row[8 * t + g];
    has[t] = xr >= 0;
    x[t] = p.x + max(xr, 0) * p.x_stride + 16 * q;
  }
  // the scales of a lane's two columns of sums, and of the weights' rows
  const float* sx[kTiles][2];
  const float* sw[kParts];
  if constexpr (kKind == kFp8) {
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
#pragma unroll
      for (int i = 0; i < 2; ++i) sx[t][i] = p.x_scales + static_cast<long long>(max(x_row[8 * t + 2 * q + i], 0)) * p.steps;
    }
#pragma unroll
    for (int a = 0; a < kParts; ++a)
      sw[a] = p.w_scales + (static_cast<long long>(e) * p.w_blocks + (a * p.N + row0) / 128) * p.steps;
  }

  float sum[kParts][kTiles][4] = {};
  for (int k0 = warp; k0 < p.steps; k0 += kWarps * kAhead) {
    uint4 wv[kAhead][kParts][2][2];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int k = k0 + i * kWarps;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int at = k * kStepBytes + 64 * j;
        const bool there = k < p.steps && at + 16 * q < row_bytes;
#pragma unroll
        for (int a = 0; a < kParts; ++a) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            wv[i][a][h][j] = make_uint4(0u, 0u, 0u, 0u);
            if (there && in[h]) wv[i][a][h][j] = load_stream(w[a][h] + at);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int k = k0 + i * kWarps;
      if (k >= p.steps) break;
      float part[kParts][kTiles][4];
      if constexpr (kKind == kFp8) {
#pragma unroll
        for (int a = 0; a < kParts; ++a)
#pragma unroll
          for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int c = 0; c < 4; ++c) part[a][t][c] = 0.f;
      }
      auto& to = either<kKind == kFp8>(part, sum);
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int at = k * kStepBytes + 64 * j;
          uint4 xv = make_uint4(0u, 0u, 0u, 0u);
          if (has[t] && at + 16 * q < row_bytes) xv = __ldg(reinterpret_cast<const uint4*>(x[t] + at));
#pragma unroll
          for (int a = 0; a < kParts; ++a) {
            const uint4 lo = wv[i][a][0][j], hi = wv[i][a][1][j];
            mma16x8<kKind>(to[a][t], lo.x, hi.x, lo.y, hi.y, xv.x, xv.y);
            mma16x8<kKind>(to[a][t], lo.z, hi.z, lo.w, hi.w, xv.z, xv.w);
          }
        }
      }
      if constexpr (kKind == kFp8) {
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          const float s0 = __ldg(sx[t][0] + k), s1 = __ldg(sx[t][1] + k);
#pragma unroll
          for (int a = 0; a < kParts; ++a) {
            const float f = __ldg(sw[a] + k);
            sum[a][t][0] = fmaf(part[a][t][0], s0 * f, sum[a][t][0]);
            sum[a][t][1] = fmaf(part[a][t][1], s1 * f, sum[a][t][1]);
            sum[a][t][2] = fmaf(part[a][t][2], s0 * f, sum[a][t][2]);
            sum[a][t][3] = fmaf(part[a][t][3], s1 * f, sum[a][t][3]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int a = 0; a < kParts; ++a) {
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<float2*>(&sums[warp][a][g + 8 * h][8 * t + 2 * q]) =
            make_float2(sum[a][t][2 * h], sum[a][t][2 * h + 1]);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kRows * kCols; i += kThreads) {
    const int r = i % kRows, c = i / kRows;
    const long long to = y_row[c];
    if (to < 0 || row0 + r >= p.N) continue;
    float v[kParts];
#pragma unroll
    for (int a = 0; a < kParts; ++a) {
      v[a] = 0.f;
#pragma unroll
      for (int s = 0; s < kWarps; ++s) v[a] += sums[s][a][r][c];
    }
    float out = v[0];
    if constexpr (kParts == 2) {
      if (p.gate_up) {
        p.gate_up[to * 2 * p.N + row0 + r] = v[0];
        p.gate_up[(to * 2 + 1) * p.N + row0 + r] = v[1];
      }
      out = v[0] / (1.f + expf(-v[0])) * v[1];
    }
    const long long at = to * p.N + row0 + r;
    if (!p.y) continue;
    if (p.y_type == TQ_FP32)
      static_cast<float*>(p.y)[at] = out;
    else if (p.y_type == TQ_BF16)
      static_cast<__nv_bfloat16*>(p.y)[at] = narrow<__nv_bfloat16>(out);
    else
      static_cast<__half*>(p.y)[at] = narrow<__half>(out);
  }
}

template <int kKind, int kParts>
int run(const FewRows& p, int cols, unsigned units, cudaStream_t s) {
  const dim3 grid((p.N + kRows - 1) / kRows, units);
  return cols == 8 ? launch_pdl(few_rows_kernel<kKind, kParts, 1>, grid, dim3(kThreads), 0, s, p)
                   : launch_pdl(few_rows_kernel<kKind, kParts, 2>, grid, dim3(kThreads), 0, s, p);
}

}  // namespace

int launch_few_rows(const FewRows& p, int type, bool gated, int cols, int64_t units, cudaStream_t s) {
  if (units < 1 || units > 65535 || (cols != 8 && cols != 16)) return TQ_ERR_INVALID_ARG;
  const unsigned u = static_cast<unsigned>(units);
  const int st = type == kFewRowsFp8 ? run<kFp8, 1>(p, cols, u, s)
                 : type == TQ_BF16   ? (gated ? run<kBf16, 2>(p, cols, u, s) : run<kBf16, 1>(p, cols, u, s))
                                     : (gated ? run<kFp16, 2>(p, cols, u, s) : run<kFp16, 1>(p, cols, u, s));
  if (st == TQ_OK) count_launch(kCntFewRows);
  return st;
}

}  // namespace tq
