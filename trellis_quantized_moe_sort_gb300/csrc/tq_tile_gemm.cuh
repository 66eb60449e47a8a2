// Matrix product D = A B^T on the tensor cores of sm_103a, activation rows as the
// MMA's M: the frame of the 8-bit block-scaled products and of the 16-bit gated
// projection with its gradients.
//
// A unit is 128 rows of A (256 over a pair of CTAs) x 2 kCols columns, or a split
// of its K range.  Persistent CTAs, one per SM, walk the units.  One warp loads A
// and one B, per step of 128 bytes along K, in 128-byte swizzled boxes; a third
// issues four MMAs a step; eight epilogue warps drain tensor memory, lane = row,
// two warps (kCols columns each) per 32 rows.  Warps 0-3 load A, load B, issue MMAs and
// load A's gathered rows; 4-11 are the epilogue.
//
// 8-bit products: a step is one block of 128 values, whose two scales multiply its
// partial sums.  Each step accumulates into an accumulator of its own; the epilogue
// adds scale * partial into fp32 registers while the next step is multiplied.  With
// rows as lanes the scale of a step is one register of each thread; with columns
// holding the activation rows it would be a shared-memory read per column and step,
// on the port that feeds the MMAs.  The registers of 256 columns need the uneven
// register split of setmaxnreg.  Measured: 8192 rows 4096 -> 4096 116 us (2.4 PFLOP/s),
// the tensor pipe at 55%: a step of 256 x 256 takes 980 cycles where its MMAs take 512,
// the copies and the hand-over of accumulators alone 865, and the epilogue's reads of
// tensor memory and additions stand out by the rest.  Sixteen epilogue warps of 64 sums
// took 134 us where these eight of 128 take 121.
//
// 16-bit products accumulate their whole K range in tensor memory.  Their operands
// may be stored with K as the slow axis (kAMn, kBMn: the gradients' transposed
// reads), as boxes of 64 columns x 64 rows of K.  Measured, 8192 rows 4096 -> 2 x 2048:
// forward with gate and up kept 155 us (79% of the tensor pipe), grad_x 143 (85%) and
// grad_w 165 (76%: its 256 units are four rounds of 76 pairs, the last a third full), at
// 1.74 to 1.80 GHz under the power limit.
//
// A pair shares one MMA of 256 rows and halves B: 32 KB a CTA and step for 128 x 256
// results, in place of 48.  Experts' rows fill tiles of 128 better than of 256 and go by
// CTAs alone.  Every copy fills its own CTA's shared memory: tensor maps hold the caller's
// addresses, and a copy to several CTAs at once may only read this GPU's own memory.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>

#include "tq_device.cuh"
#include "tq_fp8.cuh"
#include "tq_internal.h"
#include "tq_types.cuh"

namespace tq {
namespace tile {

constexpr int kRows = 128;                    // rows of A per CTA
constexpr int kStepBytes = 128;               // of a row and step: one swizzle row
constexpr int kABytes = kRows * kStepBytes;
constexpr int kMaxStages = 12, kMaxAcc = 8;
constexpr int kThreads = 384;
constexpr int kWarpA = 0, kWarpB = 1, kWarpMma = 2, kWarpA2 = 3, kWarpEpi0 = 4, kEpiWarps = 8;
constexpr int kSmemLimit = 232448;
constexpr int kNumBars = 2 * kMaxStages + 2 * kMaxAcc + 1;
constexpr int kPitch = 33;                    // floats per row of an epilogue warp's 32 x 32 turning block
constexpr int kTurnBytes = kEpiWarps * 32 * kPitch * 4;
constexpr int kListBytes = kRows * 4;         // rows of A that a CTA gathers
constexpr int kTopBytes = 2 * 2 * kRows * 4;  // two buffers of both column halves' largest magnitudes

// 128 fp32 sums a thread beside the accumulator columns in flight: 128 threads give
// up registers to 256, 128 x 40 + 256 x 232 = 384 x 168, which the launch has to have.
constexpr bool splits_registers(bool k8, int cols) { return k8 && cols == 128; }
constexpr int kLaunchRegisters = 168;

enum Epilogue {
  kStore = 0,     // y[row][column], or partial sums, one fp32 matrix per split
  kGated8 = 1,    // h = silu(gate) * up, kept in 8 bits with its scales
  kGated16 = 2,   // the same in 16 bits, and gate and up in fp32 if asked
};

struct Params {
  // units
  const int32_t* tiles;         // {e, slot0, rows}, or nullptr: tile i = rows [i * tile_m, ...) of matrix 0
  const int32_t* num_tiles;
  const int32_t* sorted_pairs;  // with tiles: the pair of a slot
  int gather;                   // (not by pairs) A's row of a slot is token pair / top_k, else the slot
  int scatter;                  // the output row of a slot is its pair, else the slot
  long long cap, split_stride, y_ld;   // y_ld: values between rows of y
  int M, E, N, tile_m, top_k;   // M: slots, or rows of A; N: columns (of h, when gated)
  int col_blocks, steps, splits;
  // scales of 8-bit operands
  const float* a_scales;        // [rows of A][steps]
  const float* b_scales;        // [E][b_blocks][steps]
  int b_blocks;
  // output
  void* y;
  int y_type, type;             // type: of 16-bit operands
  int aligned;                  // rows of y start on multiples of 16 bytes
  float* gate_up;               // [M][2 N], or nullptr
  uint8_t* codes;               // kGated8: [M][N], scales [M][N / 128]
  float* scales;
  int* err;
  int stages, accs, tmem_cols;
  uint32_t off_bar, off_list, off_top, off_turn;
};

// kind::f8f6f4 (E4M3 x E4M3) or kind::f16, fp32 accumulators; mn: the operand's K is
// its slow axis.
template <bool k8>
__device__ __forceinline__ uint32_t instruction(int type, uint32_t m, uint32_t n, bool a_mn, bool b_mn) {
  const uint32_t f = k8 ? 0u : (type == TQ_BF16 ? 1u : 0u);
  return (1u << 4) | (f << 7) | (f << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((n >> 3) << 17) |
         ((m >> 4) << 24);
}

#define TQ_TILE_MMA(group, kind)                                                                                   \
  asm volatile(                                                                                                   \
      "{\n\t.reg .pred p;\n\t"                                                                                   \
      "setp.ne.b32 p, %4, 0;\n\t"                                                                                 \
      "tcgen05.mma.cta_group::" group ".kind::" kind " [%0], %1, %2, %3, p;\n\t}" ::"r"(d),                        \
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)                                                                 \
      : "memory")
template <bool k8, bool kPair>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (k8 && kPair) {
    TQ_TILE_MMA("2", "f8f6f4");
  } else if constexpr (k8) {
    TQ_TILE_MMA("1", "f8f6f4");
  } else if constexpr (kPair) {
    TQ_TILE_MMA("2", "f16");
  } else {
    TQ_TILE_MMA("1", "f16");
  }
}
#undef TQ_TILE_MMA

inline PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    cudaGetLastError();
    return static_cast<PFN_cuTensorMapEncodeTiled_v12000>(nullptr);
  }();
  return fn;
}

// `rows` rows of `width` values (1 or 2 bytes), `stride` bytes apart, taken as
// swizzled boxes of 128 bytes x box_rows.
inline bool encode(CUtensorMap* m, const void* data, int value_bytes, int64_t width, int64_t rows, int64_t stride,
                   int box_rows) {
  const auto fn = encoder();
  if (!fn) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(kStepBytes / value_bytes), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t each[2] = {1, 1};
  // 16-bit patterns are copied as they are: zeros past the edges in any type
  return fn(m, value_bytes == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2,
            const_cast<void*>(data), dims, strides, box, each, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Descriptor of a 128-byte swizzled operand from an address in units of 16 bytes.
// K along the rows: 8-row groups 1024 bytes apart.  K across them (kMn): rows of 64
// values of one K, 8 K 1024 bytes apart, the next 64 values a box of 64 K (8192
// bytes) on.
template <bool kMn>
__device__ __forceinline__ uint64_t operand(uint32_t at) {
  return static_cast<uint64_t>(at) | static_cast<uint64_t>(kMn ? 8192 >> 4 : 1) << 16 |
         static_cast<uint64_t>(1024 >> 4) << 32 | static_cast<uint64_t>(1) << 46 | static_cast<uint64_t>(2) << 61;
}

// Copies whose bytes count on a barrier of the pair's first CTA (an address of the
// cluster's shared memory), or on this CTA's.
template <bool kPair>
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* m, int32_t x, int32_t y, uint32_t bar) {
  if constexpr (kPair)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    tma_load_2d(dst, m, x, y, bar);
}
// Arrives on the barrier (of both CTAs of a pair) once every MMA issued so far has
// completed.
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
__device__ __forceinline__ uint32_t of_cta(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_arrive(uint32_t bar) {
  // No memory of this thread is handed over, only tensor memory that it has read: the
  // cluster-wide release, which waits for the thread's outstanding accesses, would cost
  // more than a step (8192 rows 4096 -> 4096: 237 us, and 129 without it).
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
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
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
// (a.x, a.y) + (p.x, p.y) * f, each rounded once, in one instruction.
__device__ __forceinline__ void add_scaled(float2& a, uint32_t p0, uint32_t p1, float f) {
  asm("{\n\t.reg .b64 a, p, f;\n\t"
      "mov.b64 a, {%0, %1};\n\tmov.b64 p, {%2, %3};\n\tmov.b64 f, {%4, %4};\n\t"
      "fma.rn.f32x2 a, p, f, a;\n\t"
      "mov.b64 {%0, %1}, a;\n\t}"
      : "+f"(a.x), "+f"(a.y)
      : "r"(p0), "r"(p1), "f"(f));
}

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
  int e, slot0, rows, cb, k0, k1, split;
  bool ok;
};

__device__ __forceinline__ Unit unit_at(const Params& p, unsigned u, unsigned num_tiles) {
  Unit t;
  const unsigned row = u / static_cast<unsigned>(p.col_blocks);
  t.cb = static_cast<int>(u - row * p.col_blocks);
  int tile = static_cast<int>(row);
  t.split = 0;
  t.k0 = 0;
  t.k1 = p.steps;
  if (p.splits > 1) {
    t.split = static_cast<int>(row / num_tiles);
    tile = static_cast<int>(row - t.split * num_tiles);
    t.k0 = static_cast<int>(static_cast<long long>(p.steps) * t.split / p.splits);
    t.k1 = static_cast<int>(static_cast<long long>(p.steps) * (t.split + 1) / p.splits);
  }
  if (p.tiles) {
    const int32_t* const entry = p.tiles + 3ll * tile;
    t.e = __ldg(entry);
    t.slot0 = __ldg(entry + 1);
    t.rows = __ldg(entry + 2);
  } else {
    t.e = 0;
    t.slot0 = tile * p.tile_m;
    t.rows = min(p.tile_m, p.M - t.slot0);
  }
  t.ok = t.e >= 0 && t.e < p.E && t.rows >= 1 && t.rows <= p.tile_m && t.slot0 >= 0 && t.slot0 <= p.M - t.rows;
  return t;
}

// The pair of a slot; -1 (and an error) for an entry out of range.
__device__ __forceinline__ int pair_of(const Params& p, int slot, int where) {
  const int pair = __ldg(p.sorted_pairs + slot);
  if (pair >= 0 && pair < p.M) return pair;
  record_error(p.err, TQ_ERR_INVALID_ARG, where);
  return -1;
}

// Copies of four rows that a tile's gathered rows take, and how many of `n` copies a warp
// takes: `share` from the lead-th of every eight.
__device__ __forceinline__ int gathered(int rows) { return (min(kRows, rows) + 3) / 4; }
__device__ __forceinline__ int shared_copies(int n, int lead, int share) {
  return n / 8 * share + max(0, min(share, n % 8 - lead));
}

// Output rows of a warp's 32: of lane l, `row`, < 0: none; where they are first + l * step
// for l < live, step is not 0.
struct Rows {
  long long row, first;
  int step, live;
};
// kCount values of this lane's row to columns [col, col + kCount) of y, those below N.
// A lane's own stores would be 32 rows' sectors an instruction (128 x 256 results a CTA:
// 4000 cycles), so the warp turns blocks of 32 rows x 128 bytes in shared memory and
// stores whole lines of them, 16 bytes a lane.  Rows that do not start on 16-byte
// boundaries are turned by single values, 32 columns at a time.
template <typename T, int kCount>
__device__ __forceinline__ void store_columns(T* y, const float (&v)[kCount], const Rows& rows, int col, int N, long long ld,
                                              bool aligned, uint8_t* turn, int lane) {
  const long long row = rows.row;
  constexpr int kVec = 16 / static_cast<int>(sizeof(T)), kLine = 8 * kVec;   // values of 16 and of 128 bytes
  constexpr int kBlock = kLine < kCount ? kLine : kCount, kParts = kBlock / kVec;
  if (aligned) {
    constexpr int kRowsOnce = 32 / kParts;
#pragma unroll
    for (int b = 0; b < kCount; b += kBlock) {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kParts; ++i) {
        T t[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) t[j] = narrow<T>(v[b + i * kVec + j]);
        uint4 o;
        memcpy(&o, t, 16);
        // neighbouring rows start in different banks
        *reinterpret_cast<uint4*>(turn + 128 * lane + 16 * (i ^ (lane & 7))) = o;
      }
      __syncwarp();
      const int part = lane % kParts, at = col + b + part * kVec;
#pragma unroll
      for (int r0 = 0; r0 < 32; r0 += kRowsOnce) {
        const int r = r0 + lane / kParts;
        const long long to = __shfl_sync(0xffffffffu, row, r);
        const uint4 o = *reinterpret_cast<const uint4*>(turn + 128 * r + 16 * (part ^ (r & 7)));
        if (to >= 0 && at < N) *reinterpret_cast<uint4*>(y + to * ld + at) = o;   // ld is a multiple of kVec
      }
    }
    return;
  }
  float* const floats = reinterpret_cast<float*>(turn);
  constexpr int kWide = kCount < 32 ? kCount : 32;
#pragma unroll
  for (int b = 0; b < kCount; b += kWide) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kWide; ++i) floats[lane * kPitch + i] = v[b + i];
    __syncwarp();
    const bool in = col + b + lane < N && lane < kWide;
    if (rows.step) {
      // an addition a row, where the lookup of each took 12 instructions (3001 rows 2048 ->
      // 4099: 59 us with it)
      T* to = y + rows.first * ld + col + b + lane;
      const long long next = rows.step * ld;
#pragma unroll 8
      for (int r = 0; r < rows.live; ++r, to += next) {
        if (in) *to = narrow<T>(floats[r * kPitch + lane]);
      }
      continue;
    }
#pragma unroll 4
    for (int r = 0; r < 32; ++r) {
      const long long to = __shfl_sync(0xffffffffu, row, r);
      if (to >= 0 && in) y[to * ld + col + b + lane] = narrow<T>(floats[r * kPitch + lane]);
    }
  }
}
template <int kCount>
__device__ __forceinline__ void store_typed(void* y, int type, const float (&v)[kCount], const Rows& row, int col, int N,
                                            long long ld, bool aligned, uint8_t* turn, int lane) {
  if (type == TQ_FP32)
    store_columns(static_cast<float*>(y), v, row, col, N, ld, aligned, turn, lane);
  else if (type == TQ_BF16)
    store_columns(static_cast<__nv_bfloat16*>(y), v, row, col, N, ld, aligned, turn, lane);
  else
    store_columns(static_cast<__half*>(y), v, row, col, N, ld, aligned, turn, lane);
}

template <bool k8, bool kPair, int kCols, bool kAMn, bool kBMn, int kEpi>
__global__ void __launch_bounds__(kThreads, 1)
tile_gemm_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b, const Params p) {
  static_assert(kCols == 128 || kCols == 64 || kCols == 32, "");
  static_assert(!k8 || (!kAMn && !kBMn), "8-bit operands keep K along their rows");
  static_assert(kEpi != kGated8 || (k8 && kCols == 128), "a block of h is one unit's columns");
  static_assert(kEpi == kStore || kCols >= 64, "");
  static_assert(k8 || kCols >= 64, "16-bit sums are read 64 columns at a time");
  static_assert(!kBMn || kCols >= 64, "");
  constexpr bool kGated = kEpi != kStore, kSplitRegisters = splits_registers(k8, kCols);
  constexpr int kN = 2 * kCols;                                   // the MMA's N
  constexpr int kBBytes = (kPair ? kCols : kN) * kStepBytes;      // of B per CTA and step
  constexpr int kStageBytes = kABytes + kBBytes;
  constexpr int kStepValues = k8 ? 128 : 64;
  constexpr int kBoxRows = kBMn ? 64 : kCols;                     // columns of D per box of B
  constexpr int kBBoxes = (kPair ? kCols : kN) / kBoxRows;
  constexpr int kABoxes = kAMn ? kRows / 64 : 1;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (base - raw);
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int rank = kPair ? static_cast<int>(cluster_rank()) : 0;
  const bool first = rank == 0;   // of a pair: the barriers that the MMA waits for are its
  const bool gather = !kPair && p.gather;

  const uint32_t bar_full = base + p.off_bar;
  const uint32_t bar_empty = bar_full + 8 * kMaxStages;
  const uint32_t bar_accfull = bar_empty + 8 * kMaxStages;
  const uint32_t bar_accempty = bar_accfull + 8 * kMaxAcc;
  const uint32_t bar_drain = bar_accempty + 8 * kMaxAcc;
  uint32_t* const tmem_holder = reinterpret_cast<uint32_t*>(gbase + p.off_bar + 8 * kNumBars);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(bar_full + 8 * s, gather ? 3 : 2);
      mbar_init(bar_empty + 8 * s, 1);
    }
    for (int a = 0; a < p.accs; ++a) {
      mbar_init(bar_accfull + 8 * a, 1);
      mbar_init(bar_accempty + 8 * a, (kPair ? 2 : 1) * kEpiWarps);
    }
    mbar_init(bar_drain, 1);
    *abort_flag = 0;
    mbar_fence_init();
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_b);
  }
  if (warp == kWarpA) alloc_columns<kPair>(smem_u32(tmem_holder), static_cast<uint32_t>(p.tmem_cols));
  tc_fence_before();
  __syncthreads();
  if (kPair) cluster_sync();   // both CTAs' barriers are ready
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_holder);
  pdl_wait();

  const int num_tiles = p.tiles ? static_cast<int>(max(0ll, min(static_cast<long long>(*p.num_tiles), p.cap)))
                                : static_cast<int>(p.cap);
  const unsigned units = num_tiles * p.col_blocks * p.splits;   // (the host keeps them below 2^31)
  constexpr int kCtas = kPair ? 2 : 1;
  const unsigned unit0 = blockIdx.x / kCtas, unit_step = gridDim.x / kCtas;
  const int stages = p.stages, accs = p.accs;
  int* const err = p.err;

  if (warp < kWarpEpi0) {
    if constexpr (kSplitRegisters) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp != kWarpMma && (warp != kWarpA2 || gather)) {
      // The whole warp walks the steps, so that addresses stay in uniform registers;
      // one elected thread issues (a loop that only it walks takes about 100 cycles a
      // copy).  Gathered rows come four to a copy, and a copy takes about 80 cycles of a
      // warp: three warps share them, in every eight copies three, two (beside B's box)
      // and three, none for the rows past the tile, whose results are not stored (8192
      // tokens of top-6 of 256, 4096 -> 2048, in pairs of CTAs: 1113 us by one warp, 744 by
      // two, 716 so).
      const bool is_b = warp == kWarpB;
      const int lead = is_b ? 3 : warp == kWarpA ? 0 : 5, share = is_b ? 2 : 3;
      int* const list = reinterpret_cast<int*>(gbase + p.off_list);
      const uint32_t full0 = kPair ? of_cta(bar_full, 0) : bar_full;
      const bool leader = elect_one();
      Ring ring;
      long long issued = 0;
      bool ok = true, ready = false;
      for (unsigned u = unit0; ok && u < units; u += unit_step) {
        const Unit t = unit_at(p, u, num_tiles);
        if (!t.ok) {
          if (is_b && first && leader) record_error(err, TQ_ERR_INVALID_ARG, kWhereTileLoad);
          continue;
        }
        const int row0 = t.slot0 + rank * kRows;
        // a tile's copies of four gathered rows, and the bytes of this warp's copies (of a pair,
        // whose rows lie together: in both CTAs)
        const int copies = gathered(t.rows);
        uint32_t bytes = static_cast<uint32_t>(is_b ? kBBytes : 0) * (kPair ? 2 : 1);
        if (gather) {
          bytes += 4 * kStepBytes * shared_copies(copies, lead, share);
          __syncwarp();
          for (int i = lane; i < 16 * share; i += 32) {
            const int in = 32 * (i / (4 * share)) + 4 * lead + i % (4 * share);   // row of the tile
            const int pair = __ldg(p.sorted_pairs + t.slot0 + min(in, t.rows - 1));
            list[in] = pair >= 0 && pair < p.M ? pair / p.top_k : 0;   // the epilogue reports and skips a bad pair
          }
          __syncwarp();
        } else if (!is_b) {
          bytes = kABytes * (kPair ? 2 : 1);
        }
        // column of D of this CTA's first box, and the second's distance from it
        const int col = t.cb * (kGated ? kCols : kN);
        const int second = kGated ? p.N : kCols;
        const int b_row = (kBMn ? 0 : t.e * (kGated ? 2 * p.N : p.N)) + col;
        for (int k = t.k0; k < t.k1; ++k) {
          if (!ready && !mbar_wait_short(bar_empty + 8 * ring.at, ring.phase ^ 1u, abort_flag, err, kWhereTileLoad)) {
            ok = false;
            break;
          }
          const uint32_t full = full0 + 8 * ring.at;
          const uint32_t dst = base + static_cast<uint32_t>(ring.at * kStageBytes);
          const int at = k * kStepValues;
          if (leader) {
            if (first) mbar_arrive_expect_tx(bar_full + 8 * ring.at, bytes);
            if (is_b) {
#pragma unroll
              for (int i = 0; i < kBBoxes; ++i) {
                const int c = (kPair ? rank * kCols : 0) + i * kBoxRows;   // column of the MMA's N
                const int row = kGated ? b_row + (c >= kCols ? second : 0) + c % kCols : b_row + c;
                load_box<kPair>(dst + kABytes + i * kBoxRows * kStepBytes, &tm_b, kBMn ? row : at, kBMn ? at : row, full);
              }
            }
            if (gather) {
#pragma unroll
              for (int j = 0; j < kRows / 4; j += 8) {
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                  const int c = j + lead + i;
                  if (i < share && c < copies) {
                    const int4 rows = *reinterpret_cast<const int4*>(list + 4 * c);
                    tma_gather4_2d(dst + 4 * c * kStepBytes, &tm_a, at, rows.x, rows.y, rows.z, rows.w, full);
                  }
                }
              }
            } else if (!is_b) {
#pragma unroll
              for (int i = 0; i < kABoxes; ++i)
                load_box<kPair>(dst + i * 8192, &tm_a, kAMn ? row0 + 64 * i : at, kAMn ? at : row0, full);
            }
          }
          ++issued;
          ring.advance(stages);
          ready = mbar_test(bar_empty + 8 * ring.at, ring.phase ^ 1u);
        }
        ok = __all_sync(0xffffffffu, ok);
      }
      if (leader) {
        // Before the CTA exits, every copy issued has landed (of a pair: in both
        // CTAs, counted on the first's barriers) and every arrival that the MMAs owe its
        // barriers; the empty ones, whose MMAs waited for the copies, tell both.
        const long long pending = min(issued, static_cast<long long>(stages));
        for (long long i = 1; i <= pending; ++i) {
          int st = ring.at - static_cast<int>(i);
          uint32_t ph = ring.phase;
          if (st < 0) {
            st += stages;
            ph ^= 1u;
          }
          const uint64_t t0 = globaltimer();
          while (!mbar_try_wait(bar_empty + 8 * st, ph)) {
            if (globaltimer() - t0 > kWaitTimeoutNs) {
              record_error(err, TQ_ERR_DEVICE_TIMEOUT, kWhereTileTeardown);
              break;
            }
          }
        }
      }
      __syncwarp();
    } else if (warp == kWarpMma && first) {
      // The whole warp walks the steps, so that addresses stay in uniform registers;
      // one elected thread issues.
      const uint32_t idesc = instruction<k8>(p.type, kPair ? 2 * kRows : kRows, kN, kAMn, kBMn);
      const uint32_t desc0 = (base & 0x3FFFFu) >> 4, bar_end = bar_full + 8 * stages;
      uint32_t desc = desc0, bar = bar_full, phase = 0;
      bool ready = false;
      const bool leader = elect_one();
      Ring acc;
      for (unsigned u = unit0; u < units; u += unit_step) {
        const Unit t = unit_at(p, u, num_tiles);
        if (!t.ok) continue;
        for (int k = t.k0; k < t.k1; ++k) {
          if (k8 || k == t.k0) {
            mbar_wait_short(bar_accempty + 8 * acc.at, acc.phase ^ 1u, abort_flag, err, kWhereTileMma);
            tc_fence_after();
          }
          const uint32_t d = tmem + static_cast<uint32_t>(acc.at * kN);
          if (!ready) mbar_wait_short(bar, phase, abort_flag, err, kWhereTileMma);
          const uint32_t this_bar = bar, this_desc = desc;
          desc += kStageBytes / 16;
          bar += 8;
          if (bar == bar_end) {
            desc = desc0;
            bar = bar_full;
            phase ^= 1u;
          }
          ready = mbar_test(bar, phase);
          const bool last = k8 || k == t.k1 - 1;
          if (leader) {
            const uint64_t a = operand<kAMn>(this_desc), b = operand<kBMn>(this_desc + kABytes / 16);
            // K of an MMA: 32 bytes along a row, or 16 rows of 128
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mma<k8, kPair>(d, a + i * (kAMn ? 128 : 2), b + i * (kBMn ? 128 : 2), idesc,
                             (i != 0 || (!k8 && k != t.k0)) ? 1u : 0u);
            commit<kPair>(this_bar + 8 * kMaxStages);   // the stage's empty barrier
            if (last) commit<kPair>(bar_accfull + 8 * acc.at);
          }
          if (last) acc.advance(accs);
          if (*abort_flag) break;
        }
        if (*abort_flag) break;
      }
      __syncwarp();
      if (elect_one()) {   // every MMA issued has completed before teardown
        commit_own<kPair>(bar_drain);
        const uint64_t t0 = globaltimer();
        while (!mbar_try_wait(bar_drain, 0)) {
          if (globaltimer() - t0 > kWaitTimeoutNs) {
            record_error(err, TQ_ERR_DEVICE_TIMEOUT, kWhereTileTeardown);
            break;
          }
        }
      }
      __syncwarp();
    }
  } else {
    if constexpr (kSplitRegisters) asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    const int q = warp & 3, half = (warp - kWarpEpi0) >> 2;
    uint8_t* const turn = gbase + p.off_turn + (warp - kWarpEpi0) * (32 * kPitch * 4);
    float* const tops = reinterpret_cast<float*>(gbase + p.off_top);
    // Column of D's tile of this thread's 32-column chunk c: its half of the columns,
    // or its half of the gate's and then of the up projection's.
    auto chunk_at = [&](int c) {
      return kGated ? (c < kCols / 64 ? half * (kCols / 2) + 32 * c : kCols + half * (kCols / 2) + 32 * c - kCols / 2)
                    : half * kCols + 32 * c;
    };
    int parity = 0;
    Ring acc;
    for (unsigned u = unit0; u < units; u += unit_step) {
      const Unit t = unit_at(p, u, num_tiles);
      if (!t.ok) continue;
      const int in_tile = rank * kRows + 32 * q + lane;
      const int slot = t.slot0 + min(in_tile, t.rows - 1);
      int pair = slot;
      if (gather || p.scatter) pair = pair_of(p, slot, kWhereTileEpilogue);
      const bool live = in_tile < t.rows && pair >= 0;
      const int first_row = t.slot0 + rank * kRows + 32 * q;
      const Rows out_row{!live ? -1 : p.scatter ? pair : slot, first_row, p.scatter ? 0 : 1,
                         max(0, min(32, t.slot0 + t.rows - first_row))};
      bool ok = true;
      if constexpr (k8) {
        const int a_row = gather ? max(pair, 0) / p.top_k : slot;
        const float* sa = p.a_scales + static_cast<long long>(a_row) * p.steps + t.k0;
        // the blocks of this thread's columns; past the matrix the last one (nothing of it is stored)
        const int col = t.cb * (kGated ? kCols : kN);
        const int last_block = (kGated ? p.N / 128 : p.b_blocks) - 1;
        const int b0 = min((kGated ? col : col + half * kCols) / 128, last_block);
        const float* sb = p.b_scales + (static_cast<long long>(t.e) * p.b_blocks + b0) * p.steps + t.k0;
        const float* sc = kGated ? sb + static_cast<long long>(p.N / 128) * p.steps : sb;
        float2 sum[kCols / 2];
#pragma unroll
        for (int i = 0; i < kCols / 2; ++i) sum[i] = make_float2(0.f, 0.f);
        // The scales are read two steps ahead: a read that misses L1, which has little room
        // beside the stages, takes longer than a step.
        float na = __ldg(sa), nb = __ldg(sb), nc = kGated ? __ldg(sc) : 0.f;
        int ahead = t.k1 - t.k0 > 1 ? 1 : 0;
        float ma = __ldg(sa + ahead), mb = __ldg(sb + ahead), mc = kGated ? __ldg(sc + ahead) : 0.f;
        for (int k = t.k0; k < t.k1; ++k) {
          const float f0 = na * nb, f1 = kGated ? na * nc : f0;
          na = ma;
          nb = mb;
          nc = mc;
          if (k + 2 < t.k1) {
            ++ahead;
            ma = __ldg(sa + ahead);
            mb = __ldg(sb + ahead);
            if (kGated) mc = __ldg(sc + ahead);
          }
          ok = mbar_wait_short(bar_accfull + 8 * acc.at, acc.phase, abort_flag, err, kWhereTileEpilogue);
          if (!ok) break;
          tc_fence_after();
          const uint32_t src = tmem + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(acc.at * kN);
          uint32_t v[2][32];
          constexpr int kChunks = kCols / 32;
          tmem_ld32(src + chunk_at(0), v[0]);
          if (kChunks > 1) tmem_ld32(src + chunk_at(1), v[1]);
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            if (c % 2 == 0) {
              tmem_wait_ld();
              if (c + 2 >= kChunks) {
                // read: the accumulator may be written again
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                  if (kPair && !first)
                    cluster_arrive(of_cta(bar_accempty + 8 * acc.at, 0));
                  else
                    mbar_arrive(bar_accempty + 8 * acc.at);
                }
              }
            }
            const float f = kGated && c >= kCols / 64 ? f1 : f0;
#pragma unroll
            for (int i = 0; i < 16; ++i) add_scaled(sum[16 * c + i], v[c & 1][2 * i], v[c & 1][2 * i + 1], f);
            if (c + 2 < kChunks) tmem_ld32(src + chunk_at(c + 2), v[c & 1]);
          }
          acc.advance(accs);
        }
        if constexpr (kEpi == kGated8) {
          // (A warp whose wait gave up walks on, its waits answered by the abort flag,
          // so that its partner's barrier below is always met.)
          // h of 64 columns a thread; the other 64 of the block are the other half's
          float h[64], top = 0.f;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            h[2 * i] = silu(sum[i].x) * sum[32 + i].x;
            h[2 * i + 1] = silu(sum[i].y) * sum[32 + i].y;
          }
          top = fp8_top<64>(h);
          float* const mine = tops + (2 * parity + half) * kRows + 32 * q + lane;
          *mine = top;
          asm volatile("bar.sync %0, 64;" ::"r"(1 + q) : "memory");
          top = fmaxf(top, tops[(2 * parity + (half ^ 1)) * kRows + 32 * q + lane]);
          parity ^= 1;
          if (live && ok && col < p.N) {
            const Fp8Scale s(top);
            uint8_t* const out = p.codes + static_cast<long long>(slot) * p.N + col + 64 * half;
#pragma unroll
            for (int i = 0; i < 64; i += 16) *reinterpret_cast<uint4*>(out + i) = fp8_codes16(h + i, s);
            if (half == 0) p.scales[static_cast<long long>(slot) * (p.N / 128) + t.cb] = s.s;
          }
        } else {
          if (!ok) break;
          const size_t width = p.y_type == TQ_FP32 ? 4 : 2;
          uint8_t* const y = static_cast<uint8_t*>(p.y) + static_cast<size_t>(t.split) * p.split_stride * width;
          constexpr int kCount = kCols < 64 ? kCols : 64;
#pragma unroll
          for (int c = 0; c < kCols; c += kCount) {
            float v[kCount];
#pragma unroll
            for (int i = 0; i < kCount / 2; ++i) {
              v[2 * i] = sum[c / 2 + i].x;
              v[2 * i + 1] = sum[c / 2 + i].y;
            }
            store_typed(y, p.y_type, v, out_row, col + half * kCols + c, p.N, p.y_ld, p.aligned, turn, lane);
          }
        }
      } else {
        ok = mbar_wait_short(bar_accfull + 8 * acc.at, acc.phase, abort_flag, err, kWhereTileEpilogue);
        if (!ok) break;
        tc_fence_after();
        const uint32_t src = tmem + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(acc.at * kN);
        const int col = t.cb * (kGated ? kCols : kN);
        if constexpr (kGated) {
#pragma unroll
          for (int c = 0; c < kCols / 64; ++c) {
            uint32_t g[32], up[32];
            tmem_ld32(src + chunk_at(c), g);
            tmem_ld32(src + chunk_at(c + kCols / 64), up);
            tmem_wait_ld();
            const int at = col + half * (kCols / 2) + 32 * c;
            float v[32];
            if (p.gate_up) {
              // rows of 2 N values: the gate's below N, then the up projection's
              float* const gu = p.gate_up;
              const Rows gate_row{out_row.row < 0 ? -1 : 2 * out_row.row, 2 * out_row.first, 2, out_row.live};
              const Rows up_row{out_row.row < 0 ? -1 : 2 * out_row.row + 1, 2 * out_row.first + 1, 2, out_row.live};
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(g[i]);
              store_columns(gu, v, gate_row, at, p.N, p.N, p.N % 4 == 0, turn, lane);
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(up[i]);
              store_columns(gu, v, up_row, at, p.N, p.N, p.N % 4 == 0, turn, lane);
            }
            if (p.y) {
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = silu(__uint_as_float(g[i])) * __uint_as_float(up[i]);
              store_typed(p.y, p.y_type, v, out_row, at, p.N, p.y_ld, p.aligned, turn, lane);
            }
          }
        } else {
          const size_t width = p.y_type == TQ_FP32 ? 4 : 2;
          uint8_t* const y = static_cast<uint8_t*>(p.y) + static_cast<size_t>(t.split) * p.split_stride * width;
#pragma unroll
          for (int c = 0; c < kCols / 64; ++c) {
            uint32_t v[2][32];
            tmem_ld32(src + half * kCols + 64 * c, v[0]);
            tmem_ld32(src + half * kCols + 64 * c + 32, v[1]);
            tmem_wait_ld();
            float f[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) f[i] = __uint_as_float(v[i / 32][i % 32]);
            store_typed(y, p.y_type, f, out_row, col + half * kCols + 64 * c, p.N, p.y_ld, p.aligned, turn, lane);
          }
        }
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
  }

  pdl_trigger();
  tc_fence_before();
  __syncthreads();
  if (kPair) cluster_sync();   // neither CTA's memory is needed by the other any more
  if (warp == kWarpA) {
    tc_fence_after();
    free_columns<kPair>(tmem, static_cast<uint32_t>(p.tmem_cols));
  }
}

// Launches one variant; `units` bounds the units of a launch whose tile map is on the
// device.  Stages, accumulators and shared memory are filled in here.
template <bool k8, bool kPair, int kCols, bool kAMn, bool kBMn, int kEpi>
int launch(Params p, const CUtensorMap& a, const CUtensorMap& b, long long units, cudaStream_t s) {
  constexpr int kCtas = kPair ? 2 : 1;
  auto kernel = tile_gemm_kernel<k8, kPair, kCols, kAMn, kBMn, kEpi>;
  static std::atomic<uint64_t> allowed{0};   // bit d: device d
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) {
    cudaGetLastError();
    return TQ_ERR_CUDA;
  }
  const uint64_t bit = 1ull << (device & 63);
  if (!(allowed.load() & bit)) {
    cudaFuncAttributes attr;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit) != cudaSuccess ||
        cudaFuncGetAttributes(&attr, kernel) != cudaSuccess) {
      cudaGetLastError();
      return TQ_ERR_CUDA;
    }
    // with fewer registers at launch the split would wait for ever
    if (splits_registers(k8, kCols) && attr.numRegs < kLaunchRegisters) return TQ_ERR_UNSUPPORTED_ARCH;
    allowed.fetch_or(bit);
  }
  constexpr int kStageBytes = kABytes + (kPair ? kCols : 2 * kCols) * kStepBytes;
  constexpr int kBarBytes = (8 * kNumBars + 16 + 15) / 16 * 16;
  constexpr int kFixed = kBarBytes + kListBytes + (kEpi == kGated8 ? kTopBytes : kTurnBytes);
  p.stages = std::min(kMaxStages, (kSmemLimit - 1024 - kFixed) / kStageBytes);
  p.accs = std::min(kMaxAcc, 512 / (2 * kCols));
  p.tmem_cols = 512;
  p.off_bar = static_cast<uint32_t>(p.stages * kStageBytes);
  p.off_list = p.off_bar + kBarBytes;
  p.off_top = p.off_turn = p.off_list + kListBytes;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  // one CTA (and one tensor-memory allocation) per SM
  cfg.dynamicSmemBytes = std::max(1024 + p.stages * kStageBytes + kFixed, 120 * 1024);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCtas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (units >= (1ll << 31)) return TQ_ERR_INVALID_ARG;
  cfg.gridDim = dim3(kCtas * static_cast<int>(std::max<long long>(1, std::min<long long>(units, sm_count() / kCtas))));
  if (cudaLaunchKernelEx(&cfg, kernel, a, b, p) != cudaSuccess) {
    cudaGetLastError();
    return TQ_ERR_LAUNCH;
  }
  return TQ_OK;
}

}  // namespace tile
}  // namespace tq
