// C entry points of the 8-bit operators: argument checks, workspace layout and the
// launch chains of the products.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "tq_fp8.cuh"
#include "tq_internal.h"
#include "tq_tiling.h"

namespace tq {
namespace {

// Values between rows of partial sums: their stores and loads are vectors of four for any
// N (4803 tokens of top-6 of 256, 512 -> 777: 184 us with N values, 103 so).
int64_t part_ld(int64_t N) { return (N + 3) / 4 * 4; }
size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
constexpr size_t kNoWorkspace = 256;   // reported where none is used; a null workspace will do
// Rows of pairs and of weights: 32-bit coordinates with room for a tile past the end.
constexpr int64_t kMaxIndex = (static_cast<int64_t>(1) << 31) - 1024;

bool bad_k(int K) { return K < 16 || K % 16 != 0 || K >= kMaxIndex; }
int blocks_of(int K) { return (K - 1) / kFp8Block + 1; }
// Values whose bytes, up to 16 splits of fp32 partial sums, would not fit a size_t.
bool bad_output(int64_t rows, int64_t N) { return static_cast<double>(rows) * static_cast<double>(N) >= 0x1p57; }
bool bad_matrix(int64_t E, int K, int64_t N) { return bad_k(K) || N < 1 || E * N >= kMaxIndex; }
bool bad_moe_shape(int64_t n, int top_k, int E) {
  return E < 1 || E > 1024 || top_k < 1 || top_k > E || top_k > 32 || n < 0 || n >= kMaxIndex ||
         n * top_k >= kMaxIndex;
}
bool bad_blocking(int rows_per_block) { return rows_per_block != 1 && rows_per_block != kFp8Block; }
// What codes and scales of E matrices of n rows of K take, in blocks of `rows` x 128.
int64_t scale_bytes(int64_t E, int64_t n, int K, int rows) { return 4 * E * ((n + rows - 1) / rows) * blocks_of(K); }
int64_t y_bytes(int64_t n, int64_t N, int y_type) { return n * N * static_cast<int64_t>(type_size(y_type)); }
bool bad_workspace(const void* p, size_t bytes, size_t need) { return !p || bytes < need || !aligned(p, 256); }

// Takes 256-byte aligned regions from a buffer, or only counts their bytes.
struct Carver {
  uint8_t* base;
  size_t used = 0;
  template <typename T>
  T* take(size_t count) {
    T* p = base ? reinterpret_cast<T*>(base + used) : nullptr;
    used += align256(std::max<size_t>(count, 1) * sizeof(T));
    return p;
  }
};

struct LinearPlan {
  bool few;
  TileChoice tile;
  float* part;   // nullptr without splits
  size_t bytes;
};
LinearPlan plan_linear(void* base, int64_t n, int K, int N) {
  LinearPlan l{};
  l.bytes = kNoWorkspace;
  l.tile = choose_tile(true, static_cast<double>(std::max<int64_t>(n, 1)), 1.0, blocks_of(K), N, false, TileRows::kOne,
                       false, true);
  l.few = few_rows_cost(n, static_cast<double>(N) * K, true) < l.tile.cost;
  if (!l.few && l.tile.splits > 1) {
    Carver c{static_cast<uint8_t*>(base)};
    l.part = c.take<float>(static_cast<size_t>(l.tile.splits) * n * part_ld(N));
    l.bytes = c.used;
  }
  return l;
}

// How the experts' products go: a token's pairs one after another, without a sort, or in
// the tensor-core tiles of sorted pairs.
enum Arm { kTokens, kTiles };
struct MoePlan {
  Arm arm;
  int tile_m;
  int64_t cap, P;
};
// A token's pairs read their weights each, at the rate of the few-rows kernel and some
// time for each of its units; sorted pairs read every woken expert's once, after a sort and
// before a combine.  Fitted, in us, to 140 sizes from 256 -> 256 to 4096 -> 2048, of 1 to 256
// tokens on 1, 8, 64 and 256 experts, of products and MLPs each: by this rule the slower
// arm is taken for few sizes and by at most 35% (6 us; 0.5% behind the best on the average;
// where only tokens whose experts nobody shares went by themselves, 21% behind, and up to
// 2.8 times).  Of top-6 of 256, 4096 -> 2048: 4, 8, 16 and 32 tokens 54, 89, 150 and 276 us
// by themselves, 67, 100, 132 and 216 in tiles; top-2 of 8, 512 -> 1024, 8, 32 and 128
// tokens 11, 18 and 44, and 20 in tiles.
// `bytes`: of an expert's weights; `units`: of the few-rows products.
MoePlan plan_arm(int64_t n, int top_k, int E, bool mlp, double bytes, double units) {
  MoePlan m;
  m.P = n * top_k;
  const double mean = n ? tq_pairs_per_woken_expert(n, top_k, E) : 1.0, P = static_cast<double>(m.P);
  const double tokens = mlp ? 12.7 + 0.162e-6 * P * bytes + 1.75e-3 * units : 9.5 + 0.188e-6 * P * bytes + 1.13e-3 * units;
  const double tiles = (mlp ? 28.1 : 21.1) + (mlp ? 0.221e-6 : 0.213e-6) * P / mean * bytes;   // P / mean: experts woken
  m.arm = tokens < tiles ? kTokens : kTiles;
  m.tile_m = 128;
  m.cap = std::max<int64_t>(1, tq_tile_map_capacity(n, top_k, E, m.tile_m));
  return m;
}
double typical_rows(int64_t n, int top_k, int E) {
  const double mean = n ? tq_pairs_per_woken_expert(n, top_k, E) : 1.0;
  return mean + 2.0 * std::sqrt(mean);
}
TileChoice moe_tile(int64_t n, int top_k, int E, int steps, int N, bool gated, TileRows kind) {
  if (n == 0) return {128, 128, 1, 0.0};
  const double mean = tq_pairs_per_woken_expert(n, top_k, E);
  return choose_tile(true, typical_rows(n, top_k, E), n * top_k / mean, steps, N, gated, kind, !gated, !gated);
}

struct Routed {
  int32_t *counts, *offsets, *sorted_pairs, *tiles, *num_tiles;
};
Routed carve_routed(Carver& c, const MoePlan& m, int E) {
  Routed r{};
  if (m.arm == kTokens) return r;
  r.counts = c.take<int32_t>(E);
  r.offsets = c.take<int32_t>(E + 1);
  r.sorted_pairs = c.take<int32_t>(m.P);
  r.tiles = c.take<int32_t>(3 * m.cap);
  r.num_tiles = c.take<int32_t>(1);
  return r;
}
int route_pairs(const MoePlan& m, const Routed& r, const int32_t* ids, int E, int* err, cudaStream_t s) {
  if (m.arm == kTokens) return TQ_OK;
  return launch_route_tile_map(ids, static_cast<int>(m.P), E, m.tile_m, r.counts, r.offsets, r.sorted_pairs, r.tiles,
                               r.num_tiles, m.cap, err, s);
}

struct ProductPlan {
  MoePlan m;
  TileChoice tile;
  Routed routed;
  float* part;
  size_t bytes;
};
ProductPlan plan_moe(void* base, int64_t n, int top_k, int E, int K, int N) {
  ProductPlan p{};
  p.m = plan_arm(n, top_k, E, false, static_cast<double>(N) * K, static_cast<double>(n) * ((N - 1) / 16 + 1));
  if (p.m.arm == kTiles) p.tile = moe_tile(n, top_k, E, blocks_of(K), N, false, TileRows::kGathered);
  Carver c{static_cast<uint8_t*>(base)};
  p.routed = carve_routed(c, p.m, E);
  p.part = p.m.arm == kTokens ? nullptr : c.take<float>(static_cast<size_t>(p.tile.splits) * p.m.P * part_ld(N));
  p.bytes = std::max(c.used, kNoWorkspace);
  return p;
}

struct MlpPlan {
  MoePlan m;
  TileChoice gu, down;
  Routed routed;
  float *h32, *part;   // h32: of tokens by themselves
  uint8_t* h;
  float* h_scales;
  size_t bytes;
};
MlpPlan plan_mlp(void* base, int64_t n, int top_k, int E, int H, int I) {
  MlpPlan p{};
  p.m = plan_arm(n, top_k, E, true, 3.0 * H * I, static_cast<double>(n) * (top_k * (I / 8.0) + H / 16.0));
  if (p.m.arm == kTiles) {   // one tile map for both products
    p.gu = moe_tile(n, top_k, E, blocks_of(H), I, true, TileRows::kGathered);
    p.down = moe_tile(n, top_k, E, blocks_of(I), H, false, TileRows::kSlots);
  }
  Carver c{static_cast<uint8_t*>(base)};
  p.routed = carve_routed(c, p.m, E);
  p.h32 = p.m.arm == kTiles ? nullptr : c.take<float>(static_cast<size_t>(p.m.P) * I);
  p.h = c.take<uint8_t>(static_cast<size_t>(p.m.P) * I);
  p.h_scales = c.take<float>(static_cast<size_t>(p.m.P) * (I / kFp8Block));
  if (p.m.arm != kTokens) p.part = c.take<float>(static_cast<size_t>(p.down.splits) * p.m.P * H);
  p.bytes = c.used;
  return p;
}

struct Operand {
  const uint8_t* codes;
  const float* scales;
};

// What the few-rows products have in common: w [E][N (gated 2 N)][K].
FewRows few_rows(Operand x, Operand w, int64_t M, int top_k, int E, int K, int N, bool gated, void* y, int y_type, int* err) {
  FewRows f{};
  f.w = w.codes;
  f.x = x.codes;
  f.w_scales = w.scales;
  f.x_scales = x.scales;
  f.row_bytes = f.x_stride = K;
  f.M = static_cast<int>(M);
  f.E = E;
  f.N = N;
  f.top_k = top_k;
  f.steps = blocks_of(K);
  f.w_blocks = ((gated ? 2 * N : N) + kFp8Block - 1) / kFp8Block;
  f.segments = 1;
  f.y = y;
  f.y_type = y_type;
  f.err = err;
  return f;
}
// y[t] = sum_j topk_w[t][j] W x, in one launch: x the token's row, or its pairs' rows.
int token_product(FewRows f, const int32_t* ids, const float* topk_w, bool gather, cudaStream_t s) {
  f.ids = ids;
  f.topk_w = topk_w;
  f.segments = f.top_k;
  f.top_k = 1;
  f.gather = gather;
  return launch_few_rows(f, kFewRowsFp8, s);
}

// The product of sorted pairs to partial sums by pair, its rows gathered from the
// tokens or in slot order.
int sorted_product(const MoePlan& m, const Routed& r, Operand x, int64_t x_rows, bool gather, Operand w, int top_k, int E,
                   int K, int N, TileChoice tile, float* part, int* err, cudaStream_t s) {
  Fp8Gemm g{x.codes, x.scales, x_rows, w.codes, w.scales, r.sorted_pairs, r.tiles, r.num_tiles, m.cap, m.P, top_k, E,
            K, N, gather, true, false, m.tile_m, tile.cols, tile.splits, part, part_ld(N),
            TQ_FP32, nullptr, nullptr, err};
  return launch_fp8_gemm(g, s);
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" {

int tq_fp8_quantize(const void* x, int x_type, int64_t x_stride, int E, int64_t n, int K, int rows_per_block,
                    uint8_t* codes, float* scales, tq_stream_t stream) {
  if (E < 0 || n < 0 || n >= kMaxIndex || E * n >= kMaxIndex || bad_k(K) || bad_type(x_type) ||
      bad_blocking(rows_per_block) || x_stride < K || (rows_per_block != 1 && E > 65535))
    return TQ_ERR_INVALID_ARG;
  const int64_t rows = E * n;
  if (bad_output(rows, x_stride) || (x_stride % 16 * static_cast<int64_t>(type_size(x_type))) % 16 != 0)
    return TQ_ERR_INVALID_ARG;
  if (rows > 0 && (!x || !codes || !scales || !aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 4)))
    return TQ_ERR_INVALID_ARG;
  if (rows_per_block != 1 && (n + kFp8Block - 1) / kFp8Block > 65535) return TQ_ERR_INVALID_ARG;
  if (outputs_overlap({{codes, rows * K}, {scales, scale_bytes(E, n, K, rows_per_block)}},
                      {{x, row_bytes(rows, x_stride, K, static_cast<int64_t>(type_size(x_type)))}}))
    return TQ_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int rc = require_sm103(s);
  if (rc != TQ_OK || rows == 0) return rc;
  return rows_per_block == 1
             ? launch_fp8_quantize_rows(x, x_type, x_stride, rows, K, codes, scales, s)
             : launch_fp8_quantize_blocks(x, x_type, x_stride, E, static_cast<int>(n), K, codes, scales, s);
}

int tq_fp8_dequantize(const uint8_t* codes, const float* scales, int E, int64_t n, int K, int rows_per_block, void* out,
                      int out_type, tq_stream_t stream) {
  if (E < 0 || n < 0 || n >= kMaxIndex || E * n >= kMaxIndex || bad_k(K) || bad_type(out_type) ||
      bad_blocking(rows_per_block) || bad_output(E * n, K))
    return TQ_ERR_INVALID_ARG;
  if (E * n > 0 && (!codes || !scales || !out || !aligned(codes, 16) || !aligned(scales, 4) || !aligned(out, 16) ||
                    outputs_overlap({{out, y_bytes(E * n, K, out_type)}},
                                    {{codes, E * n * K}, {scales, scale_bytes(E, n, K, rows_per_block)}})))
    return TQ_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int rc = require_sm103(s);
  if (rc != TQ_OK || E * n == 0) return rc;
  return launch_fp8_dequantize(codes, scales, E, n, K, rows_per_block, out, out_type, s);
}

size_t tq_fp8_linear_workspace_size(int64_t n, int K, int N) {
  if (n < 0 || n >= kMaxIndex || bad_matrix(1, K, N) || bad_output(n, N)) return 0;
  return plan_linear(nullptr, n, K, N).bytes;
}

int tq_fp8_linear(const uint8_t* x, const float* x_scales, const uint8_t* w, const float* w_scales, int64_t n, int K,
                  int N, void* workspace, size_t workspace_bytes, void* y, int y_type, tq_stream_t stream) {
  if (n < 0 || n >= kMaxIndex || bad_matrix(1, K, N) || bad_output(n, N) || bad_type(y_type)) return TQ_ERR_INVALID_ARG;
  if (n > 0 && (!x || !x_scales || !w || !w_scales || !y || !aligned(x, 16) || !aligned(w, 16) || !aligned(x_scales, 4) ||
                !aligned(w_scales, 4) || !aligned(y, type_size(y_type))))
    return TQ_ERR_INVALID_ARG;
  const LinearPlan l = plan_linear(workspace, n, K, N);
  const bool splits = !l.few && l.tile.splits > 1;
  if (n > 0 && splits && bad_workspace(workspace, workspace_bytes, l.bytes)) return TQ_ERR_WORKSPACE;
  if (n > 0 && outputs_overlap({{y, y_bytes(n, N, y_type)}, {splits ? workspace : nullptr, static_cast<int64_t>(l.bytes)}},
                               {{x, n * K}, {x_scales, scale_bytes(1, n, K, 1)}, {w, static_cast<int64_t>(N) * K},
                                {w_scales, scale_bytes(1, N, K, kFp8Block)}}))
    return TQ_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int rc = require_sm103(s);
  if (rc != TQ_OK || n == 0) return rc;
  int* err = error_word(&rc);
  if (!err) return rc;
  if (l.few)
    return launch_few_rows(few_rows({x, x_scales}, {w, w_scales}, n, 1, 1, K, N, false, y, y_type, err), kFewRowsFp8, s);
  Fp8Gemm g{x, x_scales, n, w, w_scales, nullptr, nullptr, nullptr, (n + l.tile.tile_m - 1) / l.tile.tile_m, n, 1, 1, K, N,
            false, false, false, l.tile.tile_m, l.tile.cols, l.tile.splits, splits ? l.part : y,
            splits ? part_ld(N) : N, splits ? TQ_FP32 : y_type, nullptr, nullptr, err};
  rc = launch_fp8_gemm(g, s);
  if (rc != TQ_OK || !splits) return rc;
  return launch_fp4_combine(l.part, part_ld(N), n * part_ld(N), l.tile.splits, nullptr, nullptr, nullptr, nullptr, n, 1,
                            1, N, y, y_type, s);
}

size_t tq_fp8_moe_workspace_size(int64_t n, int top_k, int E, int K, int N) {
  if (bad_moe_shape(n, top_k, E) || bad_matrix(E, K, N) || bad_output(n * top_k, N)) return 0;
  return plan_moe(nullptr, n, top_k, E, K, N).bytes;
}

int tq_fp8_moe_forward(const uint8_t* x, const float* x_scales, const uint8_t* w, const float* w_scales,
                       const int32_t* topk_ids, const float* topk_w, int64_t n, int top_k, int E, int K, int N,
                       void* workspace, size_t workspace_bytes, void* y, int y_type, tq_stream_t stream) {
  if (bad_moe_shape(n, top_k, E) || bad_matrix(E, K, N) || bad_output(n * top_k, N) || bad_type(y_type))
    return TQ_ERR_INVALID_ARG;
  if (n > 0 && (!x || !x_scales || !w || !w_scales || !topk_ids || !topk_w || !y || !aligned(x, 16) || !aligned(w, 16) ||
                !aligned(x_scales, 4) || !aligned(w_scales, 4) || !aligned(y, type_size(y_type))))
    return TQ_ERR_INVALID_ARG;
  const ProductPlan p = plan_moe(workspace, n, top_k, E, K, N);
  if (n > 0 && p.m.arm != kTokens && bad_workspace(workspace, workspace_bytes, p.bytes)) return TQ_ERR_WORKSPACE;
  if (n > 0 &&
      outputs_overlap({{y, y_bytes(n, N, y_type)}, {p.m.arm != kTokens ? workspace : nullptr, static_cast<int64_t>(p.bytes)}},
                      {{x, n * K}, {x_scales, scale_bytes(1, n, K, 1)}, {w, static_cast<int64_t>(E) * N * K},
                       {w_scales, scale_bytes(E, N, K, kFp8Block)}, {topk_ids, 4 * n * top_k}, {topk_w, 4 * n * top_k}}))
    return TQ_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int rc = require_sm103(s);
  if (rc != TQ_OK || n == 0) return rc;
  int* err = error_word(&rc);
  if (!err) return rc;
  if (p.m.arm == kTokens)
    return token_product(few_rows({x, x_scales}, {w, w_scales}, n, top_k, E, K, N, false, y, y_type, err), topk_ids, topk_w,
                         true, s);
  rc = route_pairs(p.m, p.routed, topk_ids, E, err, s);
  if (rc != TQ_OK) return rc;
  rc = sorted_product(p.m, p.routed, {x, x_scales}, n, true, {w, w_scales}, top_k, E, K, N, p.tile, p.part, err, s);
  if (rc != TQ_OK) return rc;
  return launch_fp4_combine(p.part, part_ld(N), p.m.P * part_ld(N), p.tile.splits, topk_ids, topk_w, nullptr, nullptr, n,
                            top_k, E, N, y, y_type, s);
}

size_t tq_fp8_moe_mlp_workspace_size(int64_t n, int top_k, int E, int H, int I) {
  if (bad_moe_shape(n, top_k, E) || I < 1 || I > (1 << 29) || I % kFp8Block != 0 || bad_matrix(E, H, 2ll * I) ||
      bad_matrix(E, I, H) || bad_output(n * top_k, 2ll * I) || bad_output(n * top_k, H))
    return 0;
  return plan_mlp(nullptr, n, top_k, E, H, I).bytes;
}

int tq_fp8_moe_mlp_forward(const uint8_t* x, const float* x_scales, const uint8_t* w_gu, const float* gu_scales,
                           const uint8_t* w_down, const float* down_scales, const int32_t* topk_ids,
                           const float* topk_w, int64_t n, int top_k, int E, int H, int I, void* workspace,
                           size_t workspace_bytes, void* y, int y_type, tq_stream_t stream) {
  if (tq_fp8_moe_mlp_workspace_size(n, top_k, E, H, I) == 0 || bad_type(y_type)) return TQ_ERR_INVALID_ARG;
  if (n > 0 && (!x || !x_scales || !w_gu || !gu_scales || !w_down || !down_scales || !topk_ids || !topk_w || !y ||
                !aligned(x, 16) || !aligned(w_gu, 16) || !aligned(w_down, 16) || !aligned(x_scales, 4) ||
                !aligned(gu_scales, 4) || !aligned(down_scales, 4) || !aligned(y, type_size(y_type))))
    return TQ_ERR_INVALID_ARG;
  const MlpPlan p = plan_mlp(workspace, n, top_k, E, H, I);
  if (n > 0 && bad_workspace(workspace, workspace_bytes, p.bytes)) return TQ_ERR_WORKSPACE;
  if (n > 0 &&
      outputs_overlap({{y, y_bytes(n, H, y_type)}, {workspace, static_cast<int64_t>(p.bytes)}},
                      {{x, n * H}, {x_scales, scale_bytes(1, n, H, 1)}, {w_gu, 2ll * E * I * H},
                       {gu_scales, scale_bytes(E, 2ll * I, H, kFp8Block)}, {w_down, static_cast<int64_t>(E) * H * I},
                       {down_scales, scale_bytes(E, H, I, kFp8Block)}, {topk_ids, 4 * n * top_k},
                       {topk_w, 4 * n * top_k}}))
    return TQ_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int rc = require_sm103(s);
  if (rc != TQ_OK || n == 0) return rc;
  int* err = error_word(&rc);
  if (!err) return rc;
  const MoePlan& m = p.m;
  const Routed& r = p.routed;
  rc = route_pairs(m, r, topk_ids, E, err, s);
  if (rc != TQ_OK) return rc;
  if (m.arm == kTiles) {
    Fp8Gemm g{x, x_scales, n, w_gu, gu_scales, r.sorted_pairs, r.tiles, r.num_tiles, m.cap, m.P, top_k, E, H, I, true,
              false, true, m.tile_m, p.gu.cols, 1, nullptr, I, TQ_FP32, p.h, p.h_scales, err};
    rc = launch_fp8_gemm(g, s);
  } else {
    FewRows f = few_rows({x, x_scales}, {w_gu, gu_scales}, m.P, top_k, E, H, I, true, p.h32, TQ_FP32, err);
    f.gather = 1;
    f.ids = topk_ids;
    rc = launch_few_rows(f, kFewRowsFp8, s);
    if (rc == TQ_OK) rc = launch_fp8_quantize_rows(p.h32, TQ_FP32, I, m.P, I, p.h, p.h_scales, s);
    if (rc != TQ_OK) return rc;
    f = few_rows({p.h, p.h_scales}, {w_down, down_scales}, n, top_k, E, I, H, false, y, y_type, err);
    f.only_x = 1;
    return token_product(f, topk_ids, topk_w, false, s);
  }
  if (rc != TQ_OK) return rc;
  rc = sorted_product(m, r, {p.h, p.h_scales}, m.P, false, {w_down, down_scales}, top_k, E, I, H, p.down, p.part, err, s);
  if (rc != TQ_OK) return rc;
  return launch_fp4_combine(p.part, H, m.P * H, p.down.splits, topk_ids, topk_w, nullptr, nullptr, n, top_k, E, H, y,
                            y_type, s);
}

}  // extern "C"
