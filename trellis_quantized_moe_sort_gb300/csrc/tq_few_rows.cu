// Matrix products with few activation rows: y[t] = W x[t] for up to 8 or 16 rows of x
// at a time, of one matrix or of the experts of a few tokens, bound by the reading of W.
//
// A warp multiplies 16 weight rows (gated: 8 of the gate and 8 of the up projection)
// with all the activation rows, K 128 bytes at a time, by m16n8 MMAs whose operands
// come as they are in memory: the order of K inside a sum is free, so a lane takes
// 16 consecutive bytes of a weight row and of an activation row and gives them to the
// MMAs four bytes at a time, both in the same order.  A lane's weights wait for it in
// shared memory (asynchronous copies that it alone reads back: six steps ahead and no
// barrier; in registers four were the most).  Tensor memory and its 128-row tiles would
// mean a pipeline set up for 16 KB of weights.  The MMA is not the bound: 8 rows a pass
// are far below its rate at the memory's.
//
// The eight warps of a block split K by blocks of 128 bytes and add up through
// shared memory in a fixed order.  Blocks walk their share of the units (a group of
// rows x 16 weight rows), each warp with its next blocks of weights under way, across
// units too.  A step costs about 200 instructions of a warp (the 8-bit MMAs are
// expanded into conversions and 16-bit ones), and a unit of 32 steps gives a warp four
// between two barriers.  Measured, six experts of one token, 8 bits: gated 4096 -> 2 x
// 2048 24 us (100 MB, 62% of the measured copy rate, 45% of the issue slots; 1536 units on
// 304 blocks), 2048 -> 4096 weighted and added 20 us (50 MB, 38%: a unit a block, so its
// start and its last sums show).  From where experts share tokens on the tensor-memory
// tiles are faster (16 tokens of top-6 of 256, 4096 -> 2048: 150 us here, 132 there).
//
// A single token's experts are the segments of one unit: the sums of each are added,
// weighted, to the token's, and its product is this one launch.  (The weight does not
// multiply a scale: the two scales' product is in fp32's range, one scale's with the
// router's weight need not be.)
//
// 8-bit products: 128 bytes are a scale block, whose partial sums are scaled into
// fp32 registers.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "tq_device.cuh"
#include "tq_internal.h"
#include "tq_types.cuh"

namespace tq {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kRows = 16;          // weight rows per unit
constexpr int kStepBytes = 128;    // of a row per step

constexpr int kAhead = 6;          // steps of weights in flight per warp
constexpr int kLaneBytes = 64;     // of a step: 16 rows x 128 bytes over a warp
constexpr int kRingBytes = kAhead * kThreads * kLaneBytes;

enum Kind { kFp8 = 0, kBf16 = 1, kFp16 = 2 };

// Copies 16 bytes (or, with `bytes` 0, zeros), 4 bytes, to shared memory in this
// thread's current group of copies.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 read16(uint32_t src) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(src) : "memory");
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

// The matrix of a unit's segment; -1 when out of range.
__device__ __forceinline__ int matrix_at(const FewRows& p, int tile, int segment) {
  const int e = p.ids ? __ldg(p.ids + static_cast<long long>(tile) * p.segments + segment) : 0;
  return e >= 0 && e < p.E ? e : -1;
}

// A place in the walk over units, their segments and this warp's steps: k = warp, warp +
// 8, ... of a unit's segments laid end to end.
template <bool kSegments>
struct Place {
  unsigned unit;
  int tile, block, segment, k;
  __device__ __forceinline__ void start(const FewRows& p, int warp) {
    segment = 0;
    k = warp;
    settle(p);
  }
  __device__ __forceinline__ bool settle(const FewRows& p) {
    bool moved = false;
    if constexpr (kSegments) {
      while (k >= p.steps && segment < p.segments) {
        k -= p.steps;
        ++segment;
        moved = true;
      }
    }
    return moved;
  }
  __device__ __forceinline__ void next_unit(const FewRows& p, int row_blocks, int warp) {
    ++unit;
    if (++block == row_blocks) {
      block = 0;
      ++tile;
    }
    start(p, warp);
  }
  __device__ __forceinline__ bool past_unit(const FewRows& p) const { return kSegments ? segment >= p.segments : k >= p.steps; }
};

// kTiles: groups of 8 activation rows; kSegments: a token's experts one after another.
template <int kKind, bool kGated, int kTiles, bool kSegments>
__global__ void __launch_bounds__(kThreads, 2) few_rows_kernel(const FewRows p, const int row_blocks, const unsigned units) {
  constexpr int kCols = 8 * kTiles, kFeatures = kGated ? kRows / 2 : kRows;
  extern __shared__ uint4 ring[];   // [kAhead][warps][4][lanes]: a lane's own bytes, read back by it alone
  __shared__ float scale_ring[kAhead][kWarps][2];
  __shared__ float sums[2][kWarps][kRows][kCols];
  if (!p.only_x) {
    pdl_wait();
    pdl_trigger();
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, q = lane & 3;
  const long long row_bytes = p.row_bytes;
  // this block's units, neighbours
  const unsigned each = units / gridDim.x, more = units % gridDim.x;
  const unsigned u0 = each * blockIdx.x + min(blockIdx.x, more), u1 = u0 + each + (blockIdx.x < more ? 1u : 0u);

  // Weights: the place that is loaded next, kAhead steps before its use.
  Place<kSegments> here;
  here.unit = u0;
  here.tile = static_cast<int>(u0 / row_blocks);
  here.block = static_cast<int>(u0 - static_cast<unsigned>(here.tile) * row_blocks);
  here.start(p, warp);
  const bool idle = here.past_unit(p);   // a warp without a step in a unit only joins its sums
  Place<kSegments> ahead = here;
  // This lane's two rows of the step that is loaded next, and the scales of one (gated:
  // of the first lane the gate's, of the others the up projection's).  Rows past the
  // matrix repeat its last: nothing of theirs is stored.
  const uint8_t* w[2];
  const float* sw = nullptr;
  auto aim = [&] {
    const int e = max(matrix_at(p, ahead.tile, ahead.segment), 0), first = ahead.block * kFeatures;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int f = min(first + g + (kGated ? 0 : 8 * h), p.N - 1);
      w[h] = p.w + ((kGated ? (2ll * e + h) * p.N : static_cast<long long>(e) * p.N) + f) * row_bytes +
             static_cast<long long>(ahead.k) * kStepBytes + 16 * q;
    }
    if (kKind == kFp8)
      sw = p.w_scales + (static_cast<long long>(e) * p.w_blocks + (first + (kGated && lane ? p.N : 0)) / 128) * p.steps +
           ahead.k;
  };
  const int full_steps = static_cast<int>(row_bytes / kStepBytes), tail = static_cast<int>(row_bytes % kStepBytes);
  const uint32_t mine = smem_u32(ring) + static_cast<uint32_t>(warp * 32 * kLaneBytes + lane * 16);
  auto load = [&](int slot) {
    if (!idle && ahead.unit < u1) {
      const uint32_t dst = mine + static_cast<uint32_t>(slot * kThreads * kLaneBytes);
      if (ahead.k < full_steps) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          copy16(dst + 1024 * h, w[h]);
          copy16(dst + 1024 * h + 512, w[h] + 64);
        }
      } else {   // the last bytes of the rows, zeros behind them
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          copy16(dst + 1024 * h, w[h], 16 * q < tail ? 16 : 0);
          copy16(dst + 1024 * h + 512, 64 + 16 * q < tail ? w[h] + 64 : w[h], 64 + 16 * q < tail ? 16 : 0);
        }
      }
      if (kKind == kFp8 && lane <= (kGated ? 1 : 0)) copy4(smem_u32(&scale_ring[slot][warp][lane]), sw);
      ahead.k += kWarps;
      w[0] += kWarps * kStepBytes;
      w[1] += kWarps * kStepBytes;
      sw += kWarps;
      bool moved = ahead.settle(p);
      if (ahead.past_unit(p)) {
        ahead.next_unit(p, row_blocks, warp);
        moved = ahead.unit < u1;
      }
      if (moved) aim();
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (!idle) aim();
#pragma unroll 1
  for (int i = 0; i < kAhead; ++i) load(i);
  if (p.only_x) {
    pdl_wait();
    pdl_trigger();
  }

  // The unit that is multiplied.  Column g (+ 8 c) is this lane's: its rows of x and of
  // the output, -1 for none.
  int x_row[kTiles], y_row[kTiles];
  const uint8_t* x[kTiles];     // of the step that is loaded next
  const float* sx[kTiles][2];   // and the scales of this lane's two columns of sums
  float weight = 1.f;           // of the segment
  auto enter_tile = [&] {
#pragma unroll
    for (int c = 0; c < kTiles; ++c) {
      // the rows of one matrix lie together; a pair's, or a token's, is alone
      const int row = p.ids ? (8 * c + g == 0 ? here.tile : p.M) : here.tile * kCols + 8 * c + g;
      y_row[c] = row < p.M ? row : -1;
      x_row[c] = y_row[c] >= 0 && p.gather ? row / p.top_k : y_row[c];
    }
  };
  auto enter_segment = [&] {
    const int e = matrix_at(p, here.tile, here.segment);
    if (e < 0 && here.block == 0 && lane == 0) record_error(p.err, TQ_ERR_INVALID_ARG, kWhereFewRows);
    if (kSegments) weight = __ldg(p.topk_w + static_cast<long long>(here.tile) * p.segments + here.segment);
#pragma unroll
    for (int c = 0; c < kTiles; ++c) {
      // a unit of segments has one row of x for all, or one for each
      const int row = kSegments && !p.gather && x_row[c] >= 0 ? x_row[c] * p.segments + here.segment : x_row[c];
      x[c] = p.x + max(row, 0) * p.x_stride + static_cast<long long>(here.k) * kStepBytes + 16 * q;
      if constexpr (kKind == kFp8) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          sx[c][i] = p.x_scales + here.k +
                     static_cast<long long>(max(__shfl_sync(0xffffffffu, row, 4 * (2 * q + i)), 0)) * p.steps;
      }
    }
    return e >= 0;
  };
  // x of a step, loaded a step ahead inside a segment
  struct Step {
    uint4 v[kTiles][2];
    float s0[kTiles], s1[kTiles];
  };
  auto load_x = [&](Step& to, int k) {
#pragma unroll
    for (int c = 0; c < kTiles; ++c) {
      const uint4* const src = reinterpret_cast<const uint4*>(x[c]);
      if (x_row[c] < 0) {
        // nothing of the column is stored
      } else if (k < full_steps) {
        to.v[c][0] = __ldg(src);
        to.v[c][1] = __ldg(src + 4);
      } else {
        to.v[c][0] = to.v[c][1] = make_uint4(0u, 0u, 0u, 0u);
        if (16 * q < tail) to.v[c][0] = __ldg(src);
        if (64 + 16 * q < tail) to.v[c][1] = __ldg(src + 4);
      }
      x[c] += kWarps * kStepBytes;
      if constexpr (kKind == kFp8) {
        to.s0[c] = __ldg(sx[c][0]);
        to.s1[c] = __ldg(sx[c][1]);
        sx[c][0] += kWarps;
        sx[c][1] += kWarps;
      }
    }
  };
  enter_tile();
  bool live = false;
  Step steps[2] = {};
  if (!idle) {
    live = enter_segment();
    load_x(steps[0], here.k);
  }

  float sum[kTiles][4] = {};
  float total[kTiles][4] = {};   // of the segments before the present one, weighted
  auto end_segment = [&] {
#pragma unroll
    for (int c = 0; c < kTiles; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (live) total[c][j] = fmaf(sum[c][j], weight, total[c][j]);
        sum[c][j] = 0.f;
      }
  };
  int buffer = 0, slot = 0;
  const int per_unit = (p.steps - warp + kWarps - 1) / kWarps;   // steps of this warp, without segments
  // One step, its x in `now`; false after the last.
  auto turn = [&](const Step& now, Step& next) {
    if (!idle) {
      if (here.k + kWarps < p.steps) load_x(next, here.k + kWarps);
      asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
      __syncwarp();
      const uint32_t src = mine + static_cast<uint32_t>(slot * kThreads * kLaneBytes);
      const float w0 = kKind == kFp8 ? scale_ring[slot][warp][0] : 0.f;
      const float w1 = kKind == kFp8 && kGated ? scale_ring[slot][warp][1] : w0;
      if (live) {
        float part[kTiles][4];
        if constexpr (kKind == kFp8) {
#pragma unroll
          for (int c = 0; c < kTiles; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) part[c][j] = 0.f;
        }
        auto& to = either<kKind == kFp8>(part, sum);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint4 lo = read16(src + 512 * j), hi = read16(src + 512 * (2 + j));
#pragma unroll
          for (int c = 0; c < kTiles; ++c) {
            const uint4 v = now.v[c][j];
            mma16x8<kKind>(to[c], lo.x, hi.x, lo.y, hi.y, v.x, v.y);
            mma16x8<kKind>(to[c], lo.z, hi.z, lo.w, hi.w, v.z, v.w);
          }
        }
        if constexpr (kKind == kFp8) {
#pragma unroll
          for (int c = 0; c < kTiles; ++c) {
            sum[c][0] = fmaf(part[c][0], now.s0[c] * w0, sum[c][0]);
            sum[c][1] = fmaf(part[c][1], now.s1[c] * w0, sum[c][1]);
            sum[c][2] = fmaf(part[c][2], now.s0[c] * w1, sum[c][2]);
            sum[c][3] = fmaf(part[c][3], now.s1[c] * w1, sum[c][3]);
          }
        }
      }
      __syncwarp();   // every lane has its scales
      load(slot);
      if (++slot == kAhead) slot = 0;
      here.k += kWarps;
      const bool moved = here.settle(p);
      if (kSegments && moved) end_segment();
      if (!here.past_unit(p)) {
        if (moved) {
          live = enter_segment();
          load_x(next, here.k);
        }
        return true;
      }
    }
    // the unit's end: its sums, and the next one
#pragma unroll
    for (int c = 0; c < kTiles; ++c) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        *reinterpret_cast<float2*>(&sums[buffer][warp][g + 8 * h][8 * c + 2 * q]) =
            kSegments ? make_float2(total[c][2 * h], total[c][2 * h + 1]) : make_float2(sum[c][2 * h], sum[c][2 * h + 1]);
        sum[c][2 * h] = sum[c][2 * h + 1] = total[c][2 * h] = total[c][2 * h + 1] = 0.f;
      }
    }
    __syncthreads();   // (a buffer is written again after the next unit's barrier)
    if (threadIdx.x < kFeatures * kCols) {
      static_assert(kFeatures * kCols <= kThreads && kFeatures * kCols % 32 == 0, "one result a thread, whole warps");
      const int r = threadIdx.x % kFeatures, c = threadIdx.x / kFeatures;   // a warp's columns are of the same eight
      int row = y_row[0];
      if (kTiles > 1 && c >= 8) row = y_row[kTiles - 1];
      const long long to = __shfl_sync(0xffffffffu, row, 4 * (c % 8));
      const int f = here.block * kFeatures + r;
      if (to >= 0 && f < p.N) {
        float v[2] = {0.f, 0.f};
#pragma unroll
        for (int s = 0; s < kWarps; ++s) {
          v[0] += sums[buffer][s][r][c];
          if (kGated) v[1] += sums[buffer][s][r + (kGated ? 8 : 0)][c];
        }
        float out = v[0];
        if constexpr (kGated) {
          if (p.gate_up) {
            p.gate_up[to * 2 * p.N + f] = v[0];
            p.gate_up[(to * 2 + 1) * p.N + f] = v[1];
          }
          out = silu(v[0]) * v[1];
        }
        const long long at = to * p.N + f;
        if (!p.y) {
        } else if (p.y_type == TQ_FP32) {
          static_cast<float*>(p.y)[at] = out;
        } else if (p.y_type == TQ_BF16) {
          static_cast<__nv_bfloat16*>(p.y)[at] = narrow<__nv_bfloat16>(out);
        } else {
          static_cast<__half*>(p.y)[at] = narrow<__half>(out);
        }
      }
    }
    buffer ^= 1;
    const int tile = here.tile;
    here.next_unit(p, row_blocks, warp);
    if (here.unit >= u1) return false;
    if (here.tile != tile) enter_tile();
    if (!idle) {
      if (kSegments || here.tile != tile) {
        live = enter_segment();
      } else {   // the same rows from their start
#pragma unroll
        for (int c = 0; c < kTiles; ++c) {
          x[c] -= static_cast<long long>(per_unit) * (kWarps * kStepBytes);
          if constexpr (kKind == kFp8) {
            sx[c][0] -= per_unit * kWarps;
            sx[c][1] -= per_unit * kWarps;
          }
        }
      }
      load_x(next, here.k);
    }
    return true;
  };
  while (turn(steps[0], steps[1]) && turn(steps[1], steps[0])) {
  }
}

template <int kKind, bool kGated, int kTiles, bool kSegments>
int run(const FewRows& p, int tiles, cudaStream_t s) {
  const int features = kGated ? kRows / 2 : kRows, row_blocks = (p.N + features - 1) / features;
  const long long units = static_cast<long long>(tiles) * row_blocks;
  if (units >= (1ll << 31)) return TQ_ERR_INVALID_ARG;
  const dim3 grid(static_cast<unsigned>(std::min<long long>(units, 2ll * sm_count())));
  auto kernel = few_rows_kernel<kKind, kGated, kTiles, kSegments>;
  static std::atomic<uint64_t> allowed{0};   // bit d: device d
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) {
    cudaGetLastError();
    return TQ_ERR_CUDA;
  }
  const uint64_t bit = 1ull << (device & 63);
  if (!(allowed.load() & bit)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes) != cudaSuccess) {
      cudaGetLastError();
      return TQ_ERR_CUDA;
    }
    allowed.fetch_or(bit);
  }
  return launch_pdl(kernel, grid, dim3(kThreads), kRingBytes, s, p, row_blocks, static_cast<unsigned>(units));
}
template <int kKind, bool kGated>
int run_rows(const FewRows& p, cudaStream_t s) {
  return p.M <= 8 ? run<kKind, kGated, 1, false>(p, 1, s) : run<kKind, kGated, 2, false>(p, (p.M + 15) / 16, s);
}

}  // namespace

int launch_few_rows(const FewRows& p, int type, cudaStream_t s) {
  int st;
  if (type == kFewRowsFp8)
    st = p.topk_w ? run<kFp8, false, 1, true>(p, p.M, s)
         : p.ids  ? run<kFp8, true, 1, false>(p, p.M, s)
                  : run_rows<kFp8, false>(p, s);
  else
    st = type == TQ_BF16 ? run_rows<kBf16, true>(p, s) : run_rows<kFp16, true>(p, s);
  if (st == TQ_OK) count_launch(kCntFewRows);
  return st;
}

}  // namespace tq
