// Product of 4-bit microscaled weights and activations on the block-scaled
// tensor-core path of sm_103a: D = W X^T with W rows as the MMA's M and
// activation rows as its N, for one matrix (linear) or for the experts of a
// tile map.
//
// A unit is (m-tile of up to tile_m activation rows) x (128 weight rows, or 256
// over a pair of CTAs), or a split of its K range.  Persistent CTAs, one per SM,
// walk the units.  Two warps load, one the weights' side and one the
// activations', per step of 256 values a 128 x 128-byte box of codes and the
// tile's rows of codes (both 128-byte swizzled) and the operands' block scales
// (contiguous in the tiled layout); a third moves the scales to tensor memory
// (32 x 128-bit copies, which tcgen05 orders before the MMAs issued after them)
// and issues up to four MMAs of K = 64; eight epilogue warps drain the fp32
// accumulator.  The accumulators alternate so that a unit's drain overlaps the
// next unit's steps.
//
// Weights are the MMA's M so that few rows cost few columns, not a padded 128.
// A pair (m-tiles of 128 rows and more) halves the activations that an SM
// stages and the MMAs that are issued.
//
// Outputs: per pair in fp32, part[split][pair][N] (plain stores, one writer
// each, summed in a fixed order by the combine: results do not depend on the
// schedule), or, for a linear without splits, y itself.
//
// Bound: memory, where the experts' weights are read for few rows each: 92-96 us
// for the 587 MB of 136 MX experts 4096 -> 2048 (32 tokens of top-6, 6.1-6.4 TB/s),
// 75 us for 333 MB read and 75 MB written (2048 tokens on 64 NV experts; the
// tensor pipe is busy 30% of it), 271 us for 1.2 GB read and 0.4 GB written
// (8192 tokens on 256).  A linear of many rows is bound by the units' fixed parts
// (first copies, last drain) beside MMAs of 4 x T / 2 cycles a step: 21.9 us for
// 3001 rows 2048 -> 4099, staging included.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "tq_fp4.cuh"
#include "tq_internal.h"

namespace tq {
namespace {

constexpr int kRows = 128;              // weight rows per unit (MMA M)
constexpr int kRowBytes = kFp4Step / 2; // a step of one row: one 128-byte swizzle row
constexpr int kWBytes = kRows * kRowBytes;
constexpr int kMaxStages = 12;
constexpr int kMaxAcc = 4;
constexpr int kWarpLoadW = 0, kWarpMma = 1, kWarpEpi0 = 2, kEpiWarps = 8;   // epilogue: two warps per lane quarter
constexpr int kWarpLoadX = kWarpEpi0 + kEpiWarps;
constexpr int kThreads = 32 * (kWarpLoadX + 1);
constexpr int kSmemLimit = 232448;
constexpr int kNumBars = 2 * kMaxStages + 2 * kMaxAcc + 1;

struct GemmParams {
  const int32_t* sorted_pairs;   // nullptr: the pair of a slot is the slot
  const int32_t* tiles;          // nullptr: tile i = rows [i * tile_m, ...) of expert 0
  const int32_t* num_tiles;
  const float* x_scale;
  const float* w_scale;
  void* y;                       // [P][N], or fp32 [splits][P][N]
  int scaled;                    // by x_scale and w_scale: y is the result, not partial sums
  int y_words;                   // each row of y starts on a multiple of four bytes
  int* err;
  long long cap, split_stride;
  int P, E, K, N, tile_m;
  int row_blocks, steps, splits;
  int n_max;                     // tile_m rounded up to 16
  int stages, accs, acc_cols;
  int sf_col, tmem_cols;
  int x_bytes, x_sf_bytes, stage_bytes;
  uint32_t off_bar, off_rows;
};

struct Ring {
  int at = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void advance(int n) {
    if (++at == n) {
      at = 0;
      phase ^= 1u;
    }
  }
};

struct Unit {
  int tile, e, slot0, rows, rb, k0, k1, split;
  bool ok;
};

// Unit u of this CTA: a pair of CTAs takes neighbouring row blocks of the same
// m-tile (the second of them past the matrix where their number is odd: its
// loads read what follows and its output rows do not exist).
template <bool kPair>
__device__ __forceinline__ Unit unit_at(const GemmParams& p, long long u, int num_tiles, int rank) {
  Unit t;
  const int groups = kPair ? (p.row_blocks + 1) / 2 : p.row_blocks;
  t.rb = static_cast<int>(u % groups);
  if (kPair) t.rb = 2 * t.rb + rank;
  u /= groups;
  t.tile = static_cast<int>(u % num_tiles);
  t.split = static_cast<int>(u / num_tiles);
  t.k0 = static_cast<int>(static_cast<long long>(p.steps) * t.split / p.splits);
  t.k1 = static_cast<int>(static_cast<long long>(p.steps) * (t.split + 1) / p.splits);
  if (p.tiles) {
    const int32_t* const entry = p.tiles + 3ll * t.tile;
    t.e = __ldg(entry);
    t.slot0 = __ldg(entry + 1);
    t.rows = __ldg(entry + 2);
  } else {
    t.e = 0;
    t.slot0 = t.tile * p.tile_m;
    t.rows = min(p.tile_m, p.P - t.slot0);
  }
  t.ok = t.e >= 0 && t.e < p.E && t.rows >= 1 && t.rows <= p.tile_m && t.slot0 >= 0 && t.slot0 <= p.P - t.rows;
  return t;
}

// Instruction descriptor of the block-scaled kinds: E2M1 x E2M1, both K-major,
// M x N (M = 256 over a pair), scales E4M3 (NV) or E8M0 (MX); the scales of the
// MMA start at byte `sf` of their 32-bit columns.
template <int kFmt, bool kPair>
__device__ __forceinline__ uint32_t idesc_fp4(uint32_t n, uint32_t sf) {
  return (sf << 4)                                        // B scale id
         | (1u << 7)                                      // A: E2M1
         | (1u << 10)                                     // B: E2M1
         | ((n >> 3) << 17)                               // N / 8
         | ((kFmt == TQ_FP4_MX ? 1u : 0u) << 23)          // scale type: E8M0 or E4M3
         | (((kPair ? 2 * kRows : kRows) >> 4) << 24)     // M / 16
         | (sf << 29);                                    // A scale id
}

#define TQ_FP4_MMA(group, kind)                                                                              \
  asm volatile(                                                                                             \
      "{\n\t.reg .pred p;\n\t"                                                                             \
      "setp.ne.b32 p, %6, 0;\n\t"                                                                           \
      "tcgen05.mma.cta_group::" group ".kind::" kind " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),      \
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)                                        \
      : "memory")
template <int kFmt, bool kPair>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        uint32_t accumulate) {
  if constexpr (kFmt == TQ_FP4_NV && kPair) {
    TQ_FP4_MMA("2", "mxf4nvf4.block_scale.scale_vec::4X");
  } else if constexpr (kFmt == TQ_FP4_NV) {
    TQ_FP4_MMA("1", "mxf4nvf4.block_scale.scale_vec::4X");
  } else if constexpr (kPair) {
    TQ_FP4_MMA("2", "mxf4.block_scale.scale_vec::2X");
  } else {
    TQ_FP4_MMA("1", "mxf4.block_scale.scale_vec::2X");
  }
}
#undef TQ_FP4_MMA

// Shared-memory descriptors from an address in units of 16 bytes: a K-major
// operand in 128-byte swizzled rows (8-row groups 1024 bytes apart), and a
// 512-byte scale tile (32 x 128 bits, 8-row groups of 128 bytes).
__device__ __forceinline__ uint64_t desc_sw128(uint32_t at) {
  return static_cast<uint64_t>(at) | static_cast<uint64_t>(1) << 16 | static_cast<uint64_t>(1024 >> 4) << 32 |
         static_cast<uint64_t>(1) << 46 | static_cast<uint64_t>(2) << 61;
}
__device__ __forceinline__ uint64_t scale_desc(uint32_t at) {
  return static_cast<uint64_t>(at) | static_cast<uint64_t>(1) << 16 | static_cast<uint64_t>(128 >> 4) << 32 |
         static_cast<uint64_t>(1) << 46;
}
// Copies a scale tile to four tensor-memory columns, replicated over the four
// lane quarters; a pair's copy does so in both CTAs, each from its own shared
// memory.
template <bool kPair>
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc) {
  if constexpr (kPair)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

// A 2-D box whose bytes count on the pair's first CTA's barrier (`bar`, an
// address of the cluster's shared memory).
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* m, int32_t x, int32_t y,
                                                 uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
template <bool kPair>
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* m, int32_t x, int32_t y, uint32_t bar) {
  if constexpr (kPair)
    tma_load_2d_pair(dst, m, x, y, bar);
  else
    tma_load_2d(dst, m, x, y, bar);
}

// Arrives on the barrier (of both CTAs of a pair) once every MMA issued so far
// has completed.
template <bool kPair>
__device__ __forceinline__ void commit(uint32_t bar) {
  if constexpr (kPair)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
  else
    mma_commit(bar);
}

// The same on a barrier of this CTA alone.
template <bool kPair>
__device__ __forceinline__ void commit_own(uint32_t bar) {
  if constexpr (kPair)
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
  else
    mma_commit(bar);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// The address in the cluster's shared memory of CTA `rank`'s `addr`.
__device__ __forceinline__ uint32_t of_cta(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <bool kPair>
__device__ __forceinline__ void alloc_columns(uint32_t dst, uint32_t columns) {
  if constexpr (kPair) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    tmem_alloc(dst, columns);
  }
}
template <bool kPair>
__device__ __forceinline__ void free_columns(uint32_t tmem, uint32_t columns) {
  if constexpr (kPair)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(columns) : "memory");
  else
    tmem_dealloc(tmem, columns);
}

// The output rows of 16 columns.
__device__ __forceinline__ void read_rows(const int* p, int (&row)[16]) {
#pragma unroll
  for (int j = 0; j < 16; j += 4) {
    const int4 r = *reinterpret_cast<const int4*>(p + j);
    row[j] = r.x;
    row[j + 1] = r.y;
    row[j + 2] = r.z;
    row[j + 3] = r.w;
  }
}

// take(values, column) for every second 16 columns of this warp's
// accumulator rows, from the `half`-th on, the next ones in flight meanwhile.
// (Two blocks a turn and no more: unrolled over the whole tile the addresses
// spill.)
template <typename Take>
__device__ __forceinline__ void drain(uint32_t src, int rows, int half, Take&& take) {
  uint32_t v[2][16];
  const int first = 16 * half;
  if (first < rows) tmem_ld16(src + first, v[0]);
#pragma unroll 1
  for (int c = first; c < rows; c += 64) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = c + 32 * i;
      if (at >= rows) break;
      tmem_wait_ld();
      if (at + 32 < rows) tmem_ld16(src + at + 32, v[(i + 1) & 1]);
      take(v[i], at);
    }
  }
}

// out[row][f] = alpha * D, to the rows of a list.
__device__ __forceinline__ void store_scattered(float* out, int N, uint32_t src, int rows, int half, const int* rows_out,
                                                int f, float alpha) {
  const bool in = f < N;
  drain(src, rows, half, [&](const uint32_t (&v)[16], int at) {
    int row[16];
    read_rows(rows_out + at, row);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      if (row[j] >= 0 && in) out[static_cast<size_t>(row[j]) * N + f] = __uint_as_float(v[j]) * alpha;
    }
  });
}

// Neighbouring lanes exchange their values of two rows: the even one returns its
// column and the next of the first row, the odd one those of the second.
template <typename T>
__device__ __forceinline__ uint32_t two_of_a_row(uint32_t first, uint32_t second, bool odd, float alpha) {
  const uint32_t give = odd ? first : second, keep = odd ? second : first;
  const uint32_t got = __shfl_xor_sync(0xffffffffu, give, 1);
  const T two[2] = {narrow<T>(__uint_as_float(odd ? got : keep) * alpha),
                    narrow<T>(__uint_as_float(odd ? keep : got) * alpha)};
  uint32_t bits;
  memcpy(&bits, two, 4);
  return bits;
}

// y[row0 + c][f] = alpha * D[c], rounded once: consecutive rows.  16-bit types
// with words on word boundaries: neighbouring lanes exchange so that each stores
// two rows of one column.  (Row addresses by one addition each: from a list in
// shared memory, as the scattered rows' are, 3001 rows 2048 -> 4099 took 27.6 us
// and not 21.9.  Turning blocks in shared memory for stores of 256 bytes a row
// gained nothing: the tensor path and the copies need its rate.)
template <typename T>
__device__ __forceinline__ void store_rows(T* y, bool by_two, int N, long long row0, uint32_t src, int rows, int half,
                                           int f, float alpha) {
  const bool odd = f & 1, in = by_two ? (f & ~1) < N : f < N;
  drain(src, rows, half, [&](const uint32_t (&v)[16], int at) {
    T* const out = y + (row0 + at) * N + f;
    if (sizeof(T) == 2 && by_two) {
#pragma unroll
      for (int j = 0; j < 16; j += 2) {
        const uint32_t bits = two_of_a_row<T>(v[j], v[j + 1], odd, alpha);
        const int c = odd ? j + 1 : j;
        if (in && at + c < rows) *reinterpret_cast<uint32_t*>(out + static_cast<long long>(c) * N - odd) = bits;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        if (in && at + j < rows) out[static_cast<long long>(j) * N] = narrow<T>(__uint_as_float(v[j]) * alpha);
      }
    }
  });
}

template <int kFmt, bool kPair, typename TOut>
__global__ void __launch_bounds__(kThreads, 1)
fp4_gemm_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                const __grid_constant__ CUtensorMap tm_ws, const __grid_constant__ CUtensorMap tm_xs,
                const GemmParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (base - raw);
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  constexpr int kSfStep = fp4_scale_step_bytes(kFmt);   // per 128 rows and step
  constexpr int kSfTiles = kSfStep / 512;               // scale tiles per step (4 NV, 2 MX)
  const int rank = kPair ? static_cast<int>(cluster_rank()) : 0;
  const bool first = rank == 0;   // of the pair: the barriers that the MMA waits for are its

  const uint32_t bar_full = base + p.off_bar;
  const uint32_t bar_empty = bar_full + 8 * kMaxStages;
  const uint32_t bar_accfull = bar_empty + 8 * kMaxStages;
  const uint32_t bar_accempty = bar_accfull + 8 * kMaxAcc;
  const uint32_t bar_drain = bar_accempty + 8 * kMaxAcc;
  uint32_t* const tmem_holder = reinterpret_cast<uint32_t*>(gbase + p.off_bar + 8 * kNumBars);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(bar_full + 8 * s, 2);
      mbar_init(bar_empty + 8 * s, 1);
    }
    for (int a = 0; a < p.accs; ++a) {
      mbar_init(bar_accfull + 8 * a, 1);
      mbar_init(bar_accempty + 8 * a, (kPair ? 2 : 1) * kEpiWarps);
    }
    mbar_init(bar_drain, 1);
    *abort_flag = 0;
    mbar_fence_init();
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_x);
    tma_prefetch_desc(&tm_ws);
    tma_prefetch_desc(&tm_xs);
  }
  if (warp == kWarpLoadW) alloc_columns<kPair>(smem_u32(tmem_holder), static_cast<uint32_t>(p.tmem_cols));
  tc_fence_before();
  __syncthreads();
  if (kPair) cluster_sync();   // both CTAs' barriers are ready
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_holder);
  pdl_wait();   // the tile map, the staged activations

  const int num_tiles = p.tiles ? static_cast<int>(min(static_cast<long long>(*p.num_tiles), p.cap))
                                : static_cast<int>(p.cap);
  const long long units =
      static_cast<long long>(num_tiles) * (kPair ? (p.row_blocks + 1) / 2 : p.row_blocks) * p.splits;
  const int unit0 = kPair ? blockIdx.x / 2 : blockIdx.x, unit_step = kPair ? gridDim.x / 2 : gridDim.x;
  // in registers: read through the parameter they would be fetched again after
  // every asm with a memory clobber
  const int stages = p.stages, accs = p.accs, stage_bytes = p.stage_bytes, x_bytes = p.x_bytes;
  int* const err = p.err;

  if (warp == kWarpLoadW || warp == kWarpLoadX) {
    // Two warps load, one thread each: the weights' codes and scales, and the
    // activations'.  (One thread for both took about 500 cycles a step, as long
    // as the step's MMAs.)
    if (elect_one()) {
      const bool is_w = warp == kWarpLoadW;
      // bytes of a step that count on the barrier: both CTAs' in a pair, which
      // splits the tile's rows; each CTA holds all of their scales
      const uint32_t bytes = static_cast<uint32_t>(is_w ? kWBytes + kSfStep : x_bytes + p.x_sf_bytes) * (kPair ? 2 : 1);
      const uint32_t to_codes = is_w ? 0u : kWBytes;
      const uint32_t to_scales = static_cast<uint32_t>(kWBytes + x_bytes + (is_w ? 0 : kSfStep));
      const bool two_groups = !is_w && p.x_sf_bytes > kSfStep;
      const CUtensorMap* const map = is_w ? &tm_w : &tm_x;
      const CUtensorMap* const scale_map = is_w ? &tm_ws : &tm_xs;
      constexpr int kSfRows = kSfStep / 128;   // 128-byte rows of the scale maps per step
      const int x_groups = p.x_sf_bytes / kSfStep, group = p.steps * kSfRows;
      const uint32_t full0 = kPair ? of_cta(bar_full, 0) : bar_full;
      Ring ring;
      long long issued = 0;
      bool ok = true, ready = false;
      for (long long u = unit0; ok && u < units; u += unit_step) {
        const Unit t = unit_at<kPair>(p, u, num_tiles, rank);
        if (!t.ok) {
          if (is_w && first) record_error(err, TQ_ERR_INVALID_ARG, kWhereFp4Load);
          continue;
        }
        const int half = kPair ? rank * (((t.rows + 15) & ~15) / 2) : 0;
        const int row = is_w ? t.e * p.N + t.rb * kRows : t.slot0 + half;
        int sf = t.k0 * kSfRows + (is_w ? t.e * p.row_blocks + t.rb : t.tile * x_groups) * group;
        for (int k = t.k0; k < t.k1; ++k) {
          if (!ready &&
              !mbar_wait_short(bar_empty + 8 * ring.at, ring.phase ^ 1u, abort_flag, err, kWhereFp4Load)) {
            ok = false;
            break;
          }
          const uint32_t full = full0 + 8 * ring.at;
          const uint32_t dst = base + static_cast<uint32_t>(ring.at * stage_bytes);
          if (first) mbar_arrive_expect_tx(bar_full + 8 * ring.at, bytes);
          load_box<kPair>(dst + to_codes, map, k * kRowBytes, row, full);
          load_box<kPair>(dst + to_scales, scale_map, 0, sf, full);
          if (two_groups) load_box<kPair>(dst + to_scales + kSfStep, scale_map, 0, sf + group, full);
          sf += kSfRows;
          ++issued;
          ring.advance(stages);
          ready = mbar_test(bar_empty + 8 * ring.at, ring.phase ^ 1u);
        }
      }
      // Before the CTA exits, every copy issued has landed (of a pair: in both
      // CTAs, counted on the first's barriers) and, in the second CTA, every
      // arrival that the MMAs owe its barriers.
      const uint32_t bars = first ? bar_full : bar_empty;
      const long long pending = min(issued, static_cast<long long>(stages));
      for (long long i = 1; i <= pending; ++i) {
        int st = ring.at - static_cast<int>(i);
        uint32_t ph = ring.phase;
        if (st < 0) {
          st += stages;
          ph ^= 1u;
        }
        const uint64_t t0 = globaltimer();
        while (!mbar_try_wait(bars + 8 * st, ph)) {
          if (globaltimer() - t0 > kWaitTimeoutNs) {
            record_error(err, TQ_ERR_DEVICE_TIMEOUT, kWhereFp4Teardown);
            break;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == kWarpMma && !first) {
    // the first CTA of the pair issues for both
  } else if (warp == kWarpMma) {
    // The whole warp walks the steps, so that stage addresses and descriptors
    // stay in uniform registers; one elected thread issues.  A wait that gives
    // up raises the abort flag, which ends the walk at the unit's end.
    const uint32_t sfa = tmem + static_cast<uint32_t>(p.sf_col);
    const uint32_t sfb = sfa + 4 * kSfTiles;
    // A stage's operands are at fixed distances from its start: one running
    // 16-byte address serves the low words of the three descriptors, whose high
    // words never change.
    const uint32_t desc0 = (base & 0x3FFFFu) >> 4;
    const uint32_t desc_stage = static_cast<uint32_t>(stage_bytes) / 16, desc_sf = static_cast<uint32_t>(kWBytes + x_bytes) / 16;
    const uint32_t bar_end = bar_full + 8 * stages;
    uint32_t desc = desc0, bar = bar_full, phase = 0;
    bool ready = false;
    const bool leader = elect_one();
    Ring acc;
    for (long long u = unit0; u < units; u += unit_step) {
      const Unit t = unit_at<kPair>(p, u, num_tiles, rank);
      if (!t.ok) continue;
      const uint32_t n_mma = static_cast<uint32_t>((t.rows + 15) & ~15);
      const bool wide = n_mma > 128;
      const uint32_t idesc = idesc_fp4<kFmt, kPair>(n_mma, 0), idesc_odd = idesc_fp4<kFmt, kPair>(n_mma, 2);
      mbar_wait_short(bar_accempty + 8 * acc.at, acc.phase ^ 1u, abort_flag, err, kWhereFp4Mma);
      tc_fence_after();
      const uint32_t d = tmem + static_cast<uint32_t>(acc.at * p.acc_cols);
      for (int k = t.k0; k < t.k1; ++k) {
        if (!ready) mbar_wait_short(bar, phase, abort_flag, err, kWhereFp4Mma);
        const uint32_t this_bar = bar, this_desc = desc;
        desc += desc_stage;
        bar += 8;
        if (bar == bar_end) {
          desc = desc0;
          bar = bar_full;
          phase ^= 1u;
        }
        // the next stage's barrier is asked while this stage's work is issued
        ready = mbar_test(bar, phase);
        if (leader) {
          const uint64_t w_desc = desc_sw128(this_desc), x_desc = desc_sw128(this_desc + kWBytes / 16);
          const uint64_t s_desc = scale_desc(this_desc + desc_sf);
#pragma unroll
          for (int i = 0; i < kSfTiles; ++i) {
            copy_scales<kPair>(sfa + 4 * i, s_desc + 32 * i);
            // row group r of the tile's scales: columns 4r .. 4r + 3 of its block group
            copy_scales<kPair>(sfb + 8 * i, s_desc + kSfStep / 16 + 32 * i);
            if (wide) copy_scales<kPair>(sfb + 8 * i + 4, s_desc + 2 * kSfStep / 16 + 32 * i);
          }
          // values past K are zeros with finite scales: always four MMAs
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            constexpr int kPer = 4 / kSfTiles;   // MMAs per scale tile
            mma_fp4<kFmt, kPair>(d, w_desc + 2 * i, x_desc + 2 * i, (kPer == 2 && (i & 1)) ? idesc_odd : idesc,
                          sfa + 4 * (i / kPer), sfb + 8 * (i / kPer), (k != t.k0 || i != 0) ? 1u : 0u);
          }
          commit<kPair>(this_bar + 8 * kMaxStages);   // the stage's empty barrier
          if (k == t.k1 - 1) commit<kPair>(bar_accfull + 8 * acc.at);
        }
      }
      acc.advance(accs);
      if (*abort_flag) break;
    }
    __syncwarp();
    if (elect_one()) {   // every MMA issued has completed before teardown
      commit_own<kPair>(bar_drain);
      const uint64_t t0 = globaltimer();
      while (!mbar_try_wait(bar_drain, 0)) {
        if (globaltimer() - t0 > kWaitTimeoutNs) {
          record_error(err, TQ_ERR_DEVICE_TIMEOUT, kWhereFp4Teardown);
          break;
        }
      }
    }
    __syncwarp();
  } else {
    // Lane l of quarter q holds weight row 32 q + l of every column.
    const int q = warp & 3, half = (warp - kWarpEpi0) >> 2;
    // The output row of each column of an experts' tile is kept in shared memory
    // (read back four at a time, the same for all lanes), -1 for none.
    int* const rows_out = reinterpret_cast<int*>(gbase + p.off_rows) + 256 * (warp - kWarpEpi0);
    Ring acc;
    for (long long u = unit0; u < units; u += unit_step) {
      const Unit t = unit_at<kPair>(p, u, num_tiles, rank);
      if (!t.ok) continue;
      if (p.sorted_pairs) {
        __syncwarp();   // the last unit's rows have been read
        for (int col = lane; col < ((t.rows + 15) & ~15); col += 32) {
          int pair = -1;
          if (col < t.rows) {
            pair = __ldg(p.sorted_pairs + t.slot0 + col);
            if (pair < 0 || pair >= p.P) {
              record_error(err, TQ_ERR_INVALID_ARG, kWhereFp4Epilogue);
              pair = -1;
            }
          }
          rows_out[col] = pair;
        }
        __syncwarp();
      }
      if (!mbar_wait_short(bar_accfull + 8 * acc.at, acc.phase, abort_flag, err, kWhereFp4Epilogue)) break;
      tc_fence_after();
      const uint32_t src = tmem + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(acc.at * p.acc_cols);
      const int f = t.rb * kRows + 32 * q + lane;
      TOut* out = static_cast<TOut*>(p.y);
      float alpha = 1.f;
      if (p.scaled)
        alpha = (p.x_scale ? __ldg(p.x_scale) : 1.f) * (p.w_scale ? __ldg(p.w_scale + t.e) : 1.f);
      else
        out += static_cast<size_t>(t.split) * p.split_stride;
      if (sizeof(TOut) == 4 && p.sorted_pairs)   // experts' partial sums
        store_scattered(reinterpret_cast<float*>(out), p.N, src, t.rows, half, rows_out, f, alpha);
      else
        store_rows(out, p.y_words, p.N, t.slot0, src, t.rows, half, f, alpha);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (kPair && !first)
          cluster_arrive(of_cta(bar_accempty + 8 * acc.at, 0));
        else
          mbar_arrive(bar_accempty + 8 * acc.at);
      }
      acc.advance(accs);
    }
  }

  pdl_trigger();
  tc_fence_before();
  __syncthreads();
  if (kPair) cluster_sync();   // neither CTA's memory is needed by the other any more
  if (warp == kWarpLoadW) {
    tc_fence_after();
    free_columns<kPair>(tmem, static_cast<uint32_t>(p.tmem_cols));
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// Codes as a 2-D tensor of bytes, boxes of one step x `box_rows`
// (swizzled), or scales in the tiled layout as rows of 128 bytes.
bool encode_bytes(CUtensorMap* m, const uint8_t* bytes, int64_t rows, int row_bytes, int box_rows, bool swizzle) {
  auto encode = encoder();
  if (!encode) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(row_bytes), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(row_bytes)};
  const cuuint32_t box[2] = {kRowBytes, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(bytes), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

using GemmKernel = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, GemmParams);

// The kernel of an output type, allowed its shared memory on the current device
// (once for each; nullptr where that fails).
template <typename TOut>
static GemmKernel kernel_for(int fmt, bool pair) {
  static std::atomic<uint64_t> allowed[4];   // bit d: device d
  GemmKernel const kernel =
      fmt == TQ_FP4_NV ? (pair ? fp4_gemm_kernel<TQ_FP4_NV, true, TOut> : fp4_gemm_kernel<TQ_FP4_NV, false, TOut>)
                       : (pair ? fp4_gemm_kernel<TQ_FP4_MX, true, TOut> : fp4_gemm_kernel<TQ_FP4_MX, false, TOut>);
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) {
    cudaGetLastError();
    return nullptr;
  }
  std::atomic<uint64_t>& done = allowed[2 * (fmt == TQ_FP4_NV) + pair];
  const uint64_t bit = 1ull << (device & 63);
  if (!(done.load() & bit)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit) != cudaSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    done.fetch_or(bit);
  }
  return kernel;
}

int launch_fp4_gemm(const Fp4Gemm& g, cudaStream_t s) {
  GemmParams p{};
  p.sorted_pairs = g.sorted_pairs;
  p.tiles = g.tiles;
  p.num_tiles = g.num_tiles;
  p.x_scale = g.x_scale;
  p.w_scale = g.w_scale;
  p.y = g.y ? g.y : g.part;
  p.scaled = g.y != nullptr;
  p.y_words = g.N % 2 == 0 && (reinterpret_cast<uintptr_t>(g.y) & 3u) == 0;
  p.err = g.err;
  p.cap = g.cap;
  p.split_stride = static_cast<long long>(g.P) * g.N;
  p.P = static_cast<int>(g.P);
  p.E = g.E;
  p.K = g.K;
  p.N = g.N;
  p.tile_m = g.tile_m;
  p.row_blocks = (g.N + kRows - 1) / kRows;
  p.steps = fp4_steps(g.K);
  p.splits = g.splits;
  p.n_max = (g.tile_m + 15) & ~15;

  const int sf_step = fp4_scale_step_bytes(g.fmt);
  const int x_groups = (p.n_max + 127) / 128;
  const bool pair = fp4_takes_pairs(g.tile_m);
  p.x_bytes = (pair ? p.n_max / 2 : p.n_max) * kRowBytes;
  p.x_sf_bytes = x_groups * sf_step;
  p.stage_bytes = kWBytes + p.x_bytes + sf_step + p.x_sf_bytes;
  const int type = g.y ? g.y_type : TQ_FP32;
  const int bar_bytes = (8 * kNumBars + 16 + 15) / 16 * 16;
  const int rows_bytes = g.sorted_pairs ? kEpiWarps * 256 * 4 : 0;
  p.stages = std::min(kMaxStages, (kSmemLimit - 1024 - bar_bytes - rows_bytes) / p.stage_bytes);
  p.off_bar = static_cast<uint32_t>(p.stages * p.stage_bytes);
  p.off_rows = p.off_bar + bar_bytes;
  // one CTA (and one tensor-memory allocation) per SM
  const int smem = std::max(1024 + p.stages * p.stage_bytes + bar_bytes + rows_bytes, 120 * 1024);

  // Tensor memory: accumulators, then the scales of one step (4 columns per
  // scale tile of the weights, 8 of the activations).
  const int sf_cols = fp4_scale_columns(g.fmt);
  p.acc_cols = p.n_max;
  p.accs = std::min(kMaxAcc, (512 - sf_cols) / p.acc_cols);
  p.sf_col = p.accs * p.acc_cols;
  p.tmem_cols = 32;
  while (p.tmem_cols < p.sf_col + sf_cols) p.tmem_cols <<= 1;

  CUtensorMap tm_w, tm_x, tm_ws, tm_xs;
  const int64_t w_groups = static_cast<int64_t>(g.E) * p.row_blocks, x_tiles = g.cap * x_groups;
  const int sf_rows = sf_step / 128;
  if (!encode_bytes(&tm_w, g.w, static_cast<int64_t>(g.E) * g.N, g.K / 2, kRows, true) ||
      !encode_bytes(&tm_x, g.x, g.P, g.K / 2, pair ? p.n_max / 2 : p.n_max, true) ||
      !encode_bytes(&tm_ws, g.w_scales, w_groups * p.steps * sf_rows, 128, sf_rows, false) ||
      !encode_bytes(&tm_xs, g.x_scales, x_tiles * p.steps * sf_rows, 128, sf_rows, false))
    return TQ_ERR_INVALID_ARG;
  const GemmKernel kernel = type == TQ_FP32   ? kernel_for<float>(g.fmt, pair)
                            : type == TQ_BF16 ? kernel_for<__nv_bfloat16>(g.fmt, pair)
                                              : kernel_for<__half>(g.fmt, pair);
  if (!kernel) return TQ_ERR_CUDA;
  const long long units = g.cap * (pair ? (p.row_blocks + 1) / 2 : p.row_blocks) * p.splits;
  const int width = pair ? 2 : 1;
  const int grid = width * static_cast<int>(std::max<long long>(1, std::min<long long>(units, sm_count() / width)));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = width;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pair ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kernel, tm_w, tm_x, tm_ws, tm_xs, p) != cudaSuccess) {
    cudaGetLastError();
    return TQ_ERR_LAUNCH;
  }
  count_launch(kCntFp4Gemm);
  return TQ_OK;
}

}  // namespace tq
