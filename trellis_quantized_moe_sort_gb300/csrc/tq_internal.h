// Host-side internals shared by the library's translation units.
#pragma once
#include <cstdint>
#include <initializer_list>
#include <cuda_runtime.h>

#include "tqmoe.h"

namespace tq {

// Device address of the current device's error word (int[2]: code, where),
// or nullptr with *status set on failure.
int* error_word(int* status);

// Checks (and on first use takes) the arch witness for the current device.
// Refuses during capture of `stream` if the witness has not been cached yet.
int require_sm103(cudaStream_t stream);

// Converts the last launch error into a status and clears it.
int launch_status();

enum Counter {
  kCntRoute = 0, kCntTileMap, kCntGrouped, kCntGemv, kCntCombine, kCntGather, kCntRouter, kCntDequant,
  kCntRouteTileMap, kCntClear, kCntSwiglu,
  // from here on only in tq_launch_counts_all
  kCntRouterScored, kCntRouterScoredBackward, kCntFp4Quantize, kCntFp4Dequantize, kCntFp4TileScales, kCntFp4Stage,
  kCntFp4Gemm, kCntFp4Combine, kCntFp4Swiglu, kCntFp4Gemv, kCntNorm, kCntNormBackward, kCntNormWeight, kCntFp8Quantize,
  kCntFp8Dequantize, kCntFp8Gemm, kCntFewRows, kCntGatedGemm, kCntSwigluSum, kCntSwigluGrad, kCntNum
};
static_assert(kCntRouterScored == TQ_NUM_LAUNCH_COUNTERS, "counter layout of tq_launch_counts");
static_assert(kCntNum == TQ_NUM_ALL_LAUNCH_COUNTERS, "counter layout of tq_launch_counts_all");
void count_launch(Counter c);

// Number of SMs of the current device (cached per device).
int sm_count();

// Launches `kernel` with programmatic stream serialization: it may begin while
// the previous kernel on the stream finishes, so it must call pdl_wait()
// before touching anything that kernel writes.  Returns the launch status.
template <typename... KArgs, typename... Args>
int launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...) != cudaSuccess) {
    cudaGetLastError();
    return TQ_ERR_LAUNCH;
  }
  return TQ_OK;
}

// Kernel launchers (defined in their own translation units).  Arguments are
// validated by the caller; these only configure and launch.
int launch_route(const int32_t* topk_ids, int P, int E, int32_t* counts, int32_t* offsets,
                 int32_t* sorted_pairs, int* err, cudaStream_t s);
int launch_tile_map(const int32_t* offsets, int E, int tile_m, int32_t* tiles, int32_t* num_tiles,
                    int64_t cap, int* err, cudaStream_t s);
int launch_combine(const float* y32, uint16_t* y, int64_t count, cudaStream_t s);
// y[0 .. count) = 0 (fp32), as a programmatic dependent of the previous kernel.
int launch_clear(float* y, int64_t count, cudaStream_t s);
int launch_router(const float* logits, int n, int E, int top_k, int32_t* ids, float* w, cudaStream_t s);
int launch_gather(const uint16_t* x, const int32_t* sorted_pairs, int P, int top_k, int K,
                  uint16_t* x_sorted, int* err, cudaStream_t s);
// Route and tile map in one launch, also clearing y32[0 .. y32_count) (in
// extra blocks of the same launch, or by a separate memset when y32 is not
// 16-byte aligned or y32_count % 4 != 0).
// With slot_of (device, [P]) the sort also writes its inverse: slot_of[p] =
// the sorted slot of pair p, -1 for a pair whose expert is out of range; with
// tile_first ([E]) the first m-tile of every expert.
int launch_route_tile_map(const int32_t* topk_ids, int P, int E, int tile_m, int32_t* counts, int32_t* offsets,
                          int32_t* sorted_pairs, int32_t* tiles, int32_t* num_tiles, int64_t cap, int* err,
                          cudaStream_t s, float* y32 = nullptr, int64_t y32_count = 0,
                          int32_t* slot_of = nullptr, int32_t* tile_first = nullptr);
// x_sorted[slot_of[t * top_k + j]] = x[t]: the pair-sorted copy written in
// token order (each row of x read once); slot -1 is skipped.
int launch_gather_tokens(const uint16_t* x, const int32_t* slot_of, int64_t n, int top_k, int K, uint16_t* x_sorted,
                         cudaStream_t s);
// x: token rows [n][K], gathered by sorted pair inside the kernel; or, with
// x_pair_sorted, the pair-sorted rows [n*top_k][K] (row = sorted slot).
int launch_grouped(const uint16_t* x, const uint8_t* packed, const uint16_t* lut, int L,
                   const int32_t* sorted_pairs, const float* topk_w, const int32_t* tiles,
                   const int32_t* num_tiles, int64_t cap, int64_t n, int top_k, int E, int K, int N,
                   int tile_m, float* y32, int* err, cudaStream_t s, int pair_out = 0,
                   const uint16_t* dense_w = nullptr, bool pdl = false, bool store_out = false,
                   bool x_pair_sorted = false);
// Materializes weights: out[i] = bf16(W_{e_i}) [N][K] for slot i < m, e_i =
// expert_ids[i] (or i when expert_ids is null); a slot whose expert has
// counts[e_i] == 0 (when counts is given) or e_i < 0 is skipped.
int launch_dequant(const uint8_t* packed, const uint16_t* lut, int L, const int32_t* expert_ids,
                   const int32_t* counts, int m, int E, int N, int K, uint16_t* out, int* err, cudaStream_t s);

// True when the whole-product calls let the grouped kernel gather the token
// rows itself (kernel m-tile <= TQ_GATHER_MAX_TILE_M); above it they copy the
// rows into pair-sorted order first (tq_gather_rows), which is faster there.
inline bool gathers_in_kernel(int kernel_tile_m) { return kernel_tile_m <= TQ_GATHER_MAX_TILE_M; }

// The scratch regions of tq_moe_forward inside a caller workspace (layout of
// tq_moe_workspace_size: counts, offsets, sorted pairs, tiles, num_tiles, y32,
// then x_sorted [P][K] only when the kernel m-tile does not gather in the
// kernel, each 256-byte aligned); `end` is the first byte after them.
struct MoeScratch {
  int32_t* counts;
  int32_t* offsets;
  int32_t* sorted_pairs;
  int32_t* tiles;
  int32_t* num_tiles;
  float* y32;
  uint16_t* x_sorted;   // nullptr when the kernel gathers
  int32_t* slot_of;     // pair -> sorted slot, with x_sorted
  uint8_t* end;
};
MoeScratch carve_moe_scratch(void* workspace, int64_t n, int top_k, int E, int K, int N, int64_t cap,
                             int kernel_tile_m);

// tile_m of the whole-product calls: 1..256 for both the arm selection and the
// kernel, or TQ_TILE_NATIVE (the kernel's native tile or TQ_TILE_M from the
// environment, the pages' TILE_M for the selection).  Returns false on an
// invalid value.
bool resolve_tile(int64_t n, int top_k, int E, int tile_m, int* kernel_tile, int* gate_tile);
int launch_swiglu(const float* gate_up, int64_t P, int I, uint16_t* h, cudaStream_t s);
// pair_in: x holds one row per pair (x[pair]) instead of per token;
// pair_out: out[pair][row] = the row's dot product (plain store, no router
// weight) instead of y32[token][row] += w * dot; y_tok (x per token, neither
// pair_in nor pair_out): y_tok[token][row] = bf16(sum_j w_j dot_j) written
// once per element, y32 unused.  Launched as a programmatic dependent of the
// previous kernel; early_prologue: that kernel writes none of x, topk_ids,
// the LUT or packed, so the kernel stages them (and loads its first row)
// before waiting for it.
int launch_gemv(const uint16_t* x, const uint8_t* packed, const uint16_t* lut, int L,
                const int32_t* topk_ids, const float* topk_w, int64_t n, int top_k, int E, int K,
                int N, float* y32, int* err, cudaStream_t s, int pair_in = 0, int pair_out = 0,
                bool early_prologue = false, uint16_t* y_tok = nullptr);
// Arguments of the scored router, validated by the entry points.
struct RouterArgs {
  int64_t n, stride;   // stride: elements between rows of logits
  const float* bias;
  int E, top_k, score, groups, top_groups, renorm;
  float scale;
};

// 4-bit operators (layouts: include/tqmoe.h, tq_fp4.cuh).
int launch_fp4_quantize(const void* x, int type, int64_t stride, int64_t n, int K, int fmt, const float* scale,
                        uint8_t* packed, uint8_t* scales, cudaStream_t s);
int launch_fp4_dequantize(const uint8_t* packed, const uint8_t* scales, int64_t n, int K, int fmt, const float* scale,
                          void* out, int type, cudaStream_t s);
int launch_fp4_tile_scales(const uint8_t* scales, int E, int N, int K, int fmt, uint8_t* tiled, cudaStream_t s);
// Where the staged row of a pair goes: the sort's inverse and, per expert, its
// first slot and first m-tile.  All nullptr: row r is slot r of tile r / tile_m.
struct Fp4Slots {
  const int32_t* ids;
  const int32_t* slot_of;
  const int32_t* offsets;
  const int32_t* tile_first;
};
// Activations quantised into the product's layout: codes xq [slots][K/2] and
// tiled scales xs [tiles].
int launch_fp4_stage(const void* x, int type, int64_t stride, int64_t n, int K, int fmt, const float* scale, int top_k,
                     const Fp4Slots& slots, int tile_m, uint8_t* xq,
                     uint8_t* xs, cudaStream_t s);
// The same for h = silu(gate) * up of every pair, gate and up from the partial
// sums part[split][pair][2I] times x_scale * w_scale[expert].
int launch_fp4_stage_swiglu(const float* part, int64_t split_stride, int splits, const float* x_scale,
                            const float* w_scale, int64_t P, int E, int I, int fmt, const float* h_scale,
                            const Fp4Slots& slots, int tile_m, uint8_t* hq, uint8_t* hs, cudaStream_t s);
// Partial sums part[split][row], rows part_ld >= N values apart.
int launch_fp4_combine(const float* part, int64_t part_ld, int64_t split_stride, int splits, const int32_t* ids, const float* topk_w,
                       const float* x_scale, const float* w_scale, int64_t n, int top_k, int E, int N, void* y,
                       int type, cudaStream_t s);
struct Fp4Gemm {
  int fmt;
  const uint8_t* w;           // codes [E][N][K/2]
  const uint8_t* w_scales;    // tiled
  const float* w_scale;       // [E] or nullptr
  const uint8_t* x;           // codes [P][K/2]
  const uint8_t* x_scales;    // tiled per m-tile
  const float* x_scale;       // [1] or nullptr
  const int32_t* sorted_pairs;   // nullptr with tiles: one matrix, row = slot
  const int32_t* tiles;
  const int32_t* num_tiles;
  int64_t cap;                // capacity of tiles, or the number of m-tiles
  int64_t P;                  // activation rows
  int E, K, N, tile_m, splits;
  float* part;                // [splits][P][N] fp32, when y is nullptr
  void* y;                    // [P][N] of y_type, scaled; splits == 1
  int y_type;
  int* err;
};
// y[t] = sum_j topk_w[t][j] W_{ids[t][j]} x[t] (ids nullptr: one matrix) in
// one launch, x quantised inside; n < 65536, K <= kFp4GemvMaxK.
struct Fp4Gemv {
  int fmt;
  const uint8_t* w;
  const uint8_t* w_scales;    // tiled
  const float* w_scale;
  const void* x;
  int x_type;
  int64_t stride;
  const float* x_scale;
  const int32_t* ids;
  const float* topk_w;
  int64_t n;
  int top_k, E, K, N;
  void* y;
  int y_type;
  int* err;
};
constexpr int kFp4GemvMaxK = 16384;   // x in shared memory, 2.25 bytes a value
int launch_fp4_gemv(const Fp4Gemv& g, cudaStream_t s);
// Pairs of CTAs (two SMs sharing one MMA of 256 weight rows, each holding half
// of the activation rows) from 128 rows per m-tile on: a CTA then takes in 36 KB
// a step for 128 x 224 results in place of 51 (experts, 8192 tokens: 460 -> 424
// us).  At 64 rows the pairs are no faster, and their second CTA idles where
// there are few weight rows.
inline bool fp4_takes_pairs(int tile_m) { return tile_m >= 128; }
int launch_fp4_gemm(const Fp4Gemm& g, cudaStream_t s);

// Whether two buffers share bytes (a null or an empty one shares none).
inline bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
  return a && b && a_bytes > 0 && b_bytes > 0 && p < q + static_cast<uintptr_t>(b_bytes) &&
         q < p + static_cast<uintptr_t>(a_bytes);
}
struct Span {
  const void* p;
  int64_t bytes;
};
// Whether an output shares bytes with another or with an input.
inline bool outputs_overlap(std::initializer_list<Span> outputs, std::initializer_list<Span> inputs) {
  for (const Span* o = outputs.begin(); o != outputs.end(); ++o) {
    for (const Span* other = o + 1; other != outputs.end(); ++other)
      if (overlap(o->p, o->bytes, other->p, other->bytes)) return true;
    for (const Span& in : inputs)
      if (overlap(o->p, o->bytes, in.p, in.bytes)) return true;
  }
  return false;
}
// Bytes from the first to the last value of `n` rows, `stride` values apart.
inline int64_t row_bytes(int64_t n, int64_t stride, int64_t width, int64_t size) {
  return n > 0 ? ((n - 1) * stride + width) * size : 0;
}

// The norm and its gradient (tq_norm.cu).  Rows of the outputs are dense.
struct NormArgs {
  const void *x, *residual, *weight;
  void *residual_out, *y;
  float* rstd;
  uint8_t* codes;
  float* scales;
  long long x_stride, residual_stride, n;
  int K, w_type;
  float eps;
};
struct NormGradArgs {
  const void *grad_y, *x, *weight, *grad_residual;
  const float* rstd;
  void* grad_x;
  float* part;   // [blocks][K] shares of grad_weight, or nullptr
  long long grad_y_stride, x_stride, grad_residual_stride, n;
  int K, w_type;
};

// 8-bit block-scaled values (tq_fp8.cuh).
int launch_fp8_quantize_rows(const void* x, int type, int64_t stride, int64_t n, int K, uint8_t* codes, float* scales,
                             cudaStream_t s);
int launch_fp8_quantize_blocks(const void* x, int type, int64_t stride, int E, int N, int K, uint8_t* codes,
                               float* scales, cudaStream_t s);
int launch_fp8_dequantize(const uint8_t* codes, const float* scales, int E, int64_t N, int K, int rows_per_block,
                          void* out, int type, cudaStream_t s);

// Product of 8-bit rows with 8-bit matrices on the tensor cores (tq_tile_gemm.cuh).
struct Fp8Gemm {
  const uint8_t* x;             // codes [x_rows][K]
  const float* x_scales;        // [x_rows][K / 128]
  int64_t x_rows;
  const uint8_t* w;             // codes [E][N][K], gated [E][2 N][K]
  const float* w_scales;        // [E][N / 128][K / 128]
  const int32_t *sorted_pairs, *tiles, *num_tiles;   // nullptr: one matrix, row = slot
  int64_t cap;                  // capacity of tiles, or the number of m-tiles
  int64_t M;                    // slots
  int top_k, E, K, N;
  bool gather;                  // x holds token rows
  bool scatter;                 // output rows are pairs, else slots
  bool gated;                   // h in codes and scales, else y
  int tile_m;                   // 128, or 256: pairs of CTAs (one matrix alone)
  int cols;                     // half the columns of a unit: 128, 64 or 32 (128 in pairs and gated)
  int splits;                   // y is fp32 [splits][M][N]
  void* y;
  int64_t y_ld;                 // values between rows of y, >= N
  int y_type;
  uint8_t* codes;
  float* scales;
  int* err;
};
int launch_fp8_gemm(const Fp8Gemm& g, cudaStream_t s);

// Product of 16-bit matrices, D[M][N] = A B^T over K (tq_tile_gemm.cuh): gated; plain
// (cols 64); or with b_mn.
struct GemmF16 {
  int type;
  const void* a;                // [M][K], or [K][M] with a_mn
  int64_t a_stride;
  const void* b;                // [N][K] (gated: [2 N][K]), or [K][N] with b_mn
  int64_t b_stride;
  int64_t M, N, K;
  bool a_mn, b_mn, gated;       // a_mn only with b_mn, gated with neither
  int tile_m, cols, splits;
  void* y;                      // [M][N] of y_type, or fp32 [splits][M][N]
  int y_type;
  float* gate_up;               // gated: fp32 [M][2 N], or nullptr
  int* err;
};
int launch_gemm_f16(const GemmF16& g, cudaStream_t s);

// Products with few activation rows (tq_few_rows.cu): of one matrix (8 bits, or 16
// gated), of pairs (ids; 8 bits gated), or of tokens (ids and topk_w; 8 bits).
struct FewRows {
  const uint8_t* w;             // [E][N] rows, gated [2 N]
  const uint8_t* x;
  const float *w_scales, *x_scales;   // 8 bits
  const int32_t* ids;           // [M][segments]
  const float* topk_w;          // [M][segments]: y[m] = sum over segments of topk_w * W_ids x
  long long row_bytes, x_stride;   // bytes: of a row of w; between rows of x
  int M;                        // output rows
  int E, N, top_k, steps, w_blocks;
  int segments;                 // 1 but for tokens
  int gather;                   // x holds a row per top_k output rows (pairs), per output row (tokens); else the segments' rows
  void* y;                      // [M][N] of y_type
  int y_type;
  float* gate_up;               // gated: fp32 [M][2 N], or nullptr
  // The launch before this one writes x and its scales and nothing else that this one
  // reads, and lets it start only after its own wait: weights are read before waiting.
  int only_x;
  int* err;
};
constexpr int kFewRowsFp8 = -1;   // `type` of the 8-bit products
int launch_few_rows(const FewRows& p, int type, cudaStream_t s);

// TQ_FORCE_ARM (auto|gemv|grouped|measured) applied to an automatic pin.
int env_pin(int pin);

}  // namespace tq
