// C entry points of the 4-bit operators: argument checks, workspace layout and
// the launch chains of the products.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "tq_fp4.cuh"
#include "tq_internal.h"

namespace tq {
namespace {

size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool bad_format(int fmt) { return fmt != TQ_FP4_NV && fmt != TQ_FP4_MX; }
constexpr size_t kNoWorkspace = 256;   // reported where none is used; a null workspace will do
// Rows of pairs and of weights: 32-bit coordinates with room for a tile past the end.
constexpr int64_t kMaxIndex = (static_cast<int64_t>(1) << 31) - 1024;

// Rows of fp4 values: K a multiple of 32.  (A row's K / 2 bytes of codes fit the
// 32-bit coordinates of the copies.)
bool bad_k(int K) { return K < 32 || K % 32 != 0; }

// Rows per m-tile and K splits of a tensor-core product, by the time that the
// kernel's parts take (cycles of an SM; the pair kernel's for two of them):
//   a step of 256 values   the MMAs, 4 x T / 2 and a seventh more, the issue of
//                          one step (360), or the step's bytes at 72 a clock
//   a unit                 2500 beside its steps; its drain of 14 a column runs
//                          beside the next unit's (at 22, 4000 rows 512 -> 2048
//                          took 16.9 us for 15.4, 6000 rows 1024 -> 4096 32.4 for
//                          31.1, 2000 rows 1024 -> 1024 8.9 against 9.9)
//   the launch             about 4000 until the first MMA
//   weights                from memory at 3400 bytes a clock over the chip
//   splits                 their partial sums written and read again at 3000
//                          bytes a clock, and the combine's launch (5000),
//                          which the experts' product has in any case
// `rows` a matrix, `matrices` of them.  T is a multiple of 16 up to the most of
// which tensor memory holds two accumulators beside a step's scales: 224 (NV, 48
// columns of scales) or 240 (MX, 24).  Experts take as few m-tiles as hold their
// rows: another reads the matrix again.
// Measured against m-tiles of a power of two or 224 and splits by the units
// alone (us): linear 4096 -> 4096, 500 rows 22.3 -> 12.2; 4096 -> 2048, 1500 rows
// 32.7 -> 15.6; 512 -> 256, 4000 rows 17.6 -> 10.3 when it came in (now 11.7,
// 15.0 and 9.1).
struct Tiling {
  int tile_m, splits;
};
Tiling search_tiling(double rows, double matrices, int K, int N, int fmt, bool experts) {
  const int steps = fp4_steps(K), blocks = (N + 127) / 128, sms = sm_count();
  const double sf = fp4_scale_step_bytes(fmt);
  const double weights = matrices * N * (K / 2.0 + K / fp4_block(fmt)) / 3400.0;
  Tiling best{16, 1};
  double best_cost = 1e300;
  const int most = (512 - fp4_scale_columns(fmt)) / 2 / 16 * 16;
  const int fewest = experts ? static_cast<int>(std::ceil(rows / most)) : 0;   // m-tiles of a matrix
  for (int T = 16; T <= most; T += 16) {
    if (experts && std::ceil(rows / T) > fewest) continue;
    const bool pair = fp4_takes_pairs(T);
    const double tiles = matrices * std::ceil(rows / T);
    const double units = tiles * (pair ? (blocks + 1) / 2 : blocks);
    const int slots = pair ? sms / 2 : sms;
    const double bytes = 128.0 * 128 + sf + 128.0 * (pair ? T / 2 : T) + sf * ((T + 127) / 128);
    const double step = std::max({360.0, 2.3 * T, bytes / 72.0});
    for (int s = 1; s <= std::min(8, steps); ++s) {
      const double unit = std::max(((steps + s - 1) / s) * step + 2500.0, 14.0 * T);
      double cost = 4000.0 + std::max(std::ceil(units * s / slots) * unit, weights) + 14.0 * T;
      if (s > 1 || experts) cost += 5000.0 + 8.0 * s * rows * matrices * N / 3000.0;
      if (cost < best_cost * 0.99) {
        best = {T, s};
        best_cost = cost;
      }
    }
  }
  return best;
}
// The search takes about 2 us, so a thread keeps the answers of the sizes it has
// met last (a pure function of them and of the device's SM count).
Tiling choose_tiling(double rows, double matrices, int K, int N, int fmt, bool experts) {
  struct Entry {
    double rows, matrices;
    int K, N, fmt, experts, sms;
    Tiling tiling;
  };
  constexpr int kEntries = 64;
  static thread_local Entry kept[kEntries];
  const int sms = sm_count();
  const uint64_t mix = (static_cast<uint64_t>(rows * 16.0) * 0x9E3779B97F4A7C15ull) ^
                       (static_cast<uint64_t>(K) * 0xC2B2AE3D27D4EB4Full) ^ (static_cast<uint64_t>(N) * 0x165667B19E3779F9ull);
  Entry& e = kept[(mix >> 40) % kEntries];
  if (!(e.sms == sms && e.rows == rows && e.matrices == matrices && e.K == K && e.N == N && e.fmt == fmt &&
        e.experts == experts))
    e = {rows, matrices, K, N, fmt, experts, sms, search_tiling(rows, matrices, K, N, fmt, experts)};
  return e.tiling;
}
// The rows that most experts stay below: their expectation and two standard
// deviations of an even routing.
Tiling moe_tiling(int64_t n, int top_k, int E, int K, int N, int fmt) {
  if (n == 0) return {16, 1};
  const double mean = tq_pairs_per_woken_expert(n, top_k, E);
  return choose_tiling(mean + 2.0 * std::sqrt(mean), n * top_k / mean, K, N, fmt, true);
}

// Whether a product takes the one-launch GEMV, which reads a matrix once per
// activation row, or the tensor-core chain (three or four launches), which
// reads it once per m-tile.  In us, fitted in CUDA graphs: the GEMV 2 and, per
// row and 2048 weight rows, 0.85 (its blocks, each quantising the row) and 0.93
// per 4096 values of each of top_k matrices; the chain 7 (linear) or 15 (experts)
// and 0.75 per 2048 x 4096 matrix.  At 2048 x 4096 the GEMV took 3.8, 5.6, 8.7,
// 15.8 for 1, 2, 4, 8 rows of a linear and 10.4, 17.6, 29.3, 55.0 for 1, 2, 4, 8
// tokens of top-6 of 256, the chain 7.9, 7.7, 7.8, 7.9 and 21.9, 26.1, 35.1, 53.1.
// Held against both arms at 14 other sizes (linears 256 -> 256 to 8192 -> 8192,
// experts 256 -> 256 to 4096 -> 4096 of 8 to 256, 1 to 32 rows each): the arm that
// it takes is the slower one in 5 of 84 cases, by 8% at most (256 -> 256, 32 tokens
// of top-6 of 64: 15.6 for the chain's 14.4; linear 4096 -> 4096, 2 rows: 8.2 for
// the GEMV's 7.8).
bool takes_gemv(int64_t n, int top_k, double matrices, double chain_us, int K, int N) {
  if (n > 64 || K > kFp4GemvMaxK) return false;
  const double rows = N / 2048.0, values = K / 4096.0;
  return 2.0 + n * rows * (0.85 + 0.93 * top_k * values) <= chain_us + 0.75 * rows * values * matrices;
}
bool linear_gemv(int64_t n, int K, int N) { return takes_gemv(n, 1, 1.0, 7.0, K, N); }
bool moe_gemv(int64_t n, int top_k, int E, int K, int N) {
  return n > 0 && takes_gemv(n, top_k, n * top_k / tq_pairs_per_woken_expert(n, top_k, E), 15.0, K, N);
}

size_t staged_scale_bytes(int64_t tiles, int tile_m, int K, int fmt) {
  return static_cast<size_t>(tiles) * ((tile_m + 127) / 128) * fp4_steps(K) * fp4_scale_step_bytes(fmt);
}

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

struct Routed {
  int32_t *counts, *offsets, *sorted_pairs, *slot_of, *tiles, *num_tiles, *tile_first;
};
Routed carve_routed(Carver& c, int64_t P, int E, int64_t cap) {
  Routed r;
  r.counts = c.take<int32_t>(E);
  r.offsets = c.take<int32_t>(E + 1);
  r.sorted_pairs = c.take<int32_t>(P);
  r.slot_of = c.take<int32_t>(P);
  r.tiles = c.take<int32_t>(3 * cap);
  r.num_tiles = c.take<int32_t>(1);
  r.tile_first = c.take<int32_t>(E);
  return r;
}

struct Staged {
  uint8_t *codes, *scales;
};
Staged carve_staged(Carver& c, int64_t P, int64_t tiles, int tile_m, int K, int fmt) {
  Staged s;
  s.codes = c.take<uint8_t>(static_cast<size_t>(P) * (K / 2));
  s.scales = c.take<uint8_t>(staged_scale_bytes(tiles, tile_m, K, fmt));
  return s;
}

bool bad_moe_shape(int64_t n, int top_k, int E) {
  return E < 1 || E > 1024 || top_k < 1 || top_k > E || top_k > 32 || n < 0 || n >= kMaxIndex ||
         n * top_k >= kMaxIndex;
}
bool bad_matrix(int E, int K, int N) { return bad_k(K) || N < 1 || static_cast<int64_t>(E) * N >= kMaxIndex; }

// Values whose bytes, up to 8 splits of fp32 partial sums, would not fit a size_t.
bool bad_output(int64_t rows, int64_t N) { return static_cast<double>(rows) * static_cast<double>(N) >= 0x1p58; }

bool bad_rows(const void* x, int type, int64_t stride, int64_t n, int K) {
  return bad_type(type) || stride < K || (stride % 16 * static_cast<int64_t>(type_size(type))) % 16 != 0 ||
         (n > 1 && bad_output(n, stride)) || (n > 0 && (!x || !aligned(x, 16)));
}

struct MoePlan {
  int tile_m, splits;
  int64_t cap, P;
  Routed routed;
  Staged staged;
  float* part;
  size_t bytes;
};
MoePlan plan_moe(void* base, int64_t n, int top_k, int E, int K, int N, int fmt) {
  MoePlan m;
  const Tiling tiling = moe_tiling(n, top_k, E, K, N, fmt);
  m.tile_m = tiling.tile_m;
  m.splits = tiling.splits;
  m.P = n * top_k;
  m.cap = std::max<int64_t>(1, tq_tile_map_capacity(n, top_k, E, m.tile_m));
  Carver c{static_cast<uint8_t*>(base)};
  m.routed = carve_routed(c, m.P, E, m.cap);
  m.staged = carve_staged(c, m.P, m.cap, m.tile_m, K, fmt);
  m.part = c.take<float>(static_cast<size_t>(m.splits) * m.P * N);
  m.bytes = c.used;
  return m;
}

struct LinearPlan {
  int tile_m, splits;
  int64_t tiles;
  Staged staged;
  float* part;   // nullptr without splits
  size_t bytes;
};
LinearPlan plan_linear(void* base, int64_t n, int K, int N, int fmt) {
  LinearPlan l;
  const Tiling tiling = choose_tiling(static_cast<double>(n), 1.0, K, N, fmt, false);
  l.tile_m = tiling.tile_m;
  l.splits = tiling.splits;
  l.tiles = std::max<int64_t>(1, (n + l.tile_m - 1) / l.tile_m);
  Carver c{static_cast<uint8_t*>(base)};
  l.staged = carve_staged(c, n, l.tiles, l.tile_m, K, fmt);
  l.part = l.splits > 1 ? c.take<float>(static_cast<size_t>(l.splits) * n * N) : nullptr;
  l.bytes = c.used;
  return l;
}

struct MlpPlan {
  int tile_m, splits_gu, splits_down;
  int64_t cap, P;
  Routed routed;
  Staged x, h;
  float *gate_up, *down;
  size_t bytes;
};
MlpPlan plan_mlp(void* base, int64_t n, int top_k, int E, int H, int I, int fmt) {
  MlpPlan m;
  // one tile map for both products, by the gate and up product; the down product's
  // splits are those of a search over m-tiles of its own (any number gives the sum)
  const Tiling gu = moe_tiling(n, top_k, E, H, 2 * I, fmt), down = moe_tiling(n, top_k, E, I, H, fmt);
  m.tile_m = gu.tile_m;
  m.splits_gu = gu.splits;
  m.splits_down = down.splits;
  m.P = n * top_k;
  m.cap = std::max<int64_t>(1, tq_tile_map_capacity(n, top_k, E, m.tile_m));
  Carver c{static_cast<uint8_t*>(base)};
  m.routed = carve_routed(c, m.P, E, m.cap);
  m.x = carve_staged(c, m.P, m.cap, m.tile_m, H, fmt);
  m.h = carve_staged(c, m.P, m.cap, m.tile_m, I, fmt);
  m.gate_up = c.take<float>(static_cast<size_t>(m.splits_gu) * m.P * 2 * I);
  m.down = c.take<float>(static_cast<size_t>(m.splits_down) * m.P * H);
  m.bytes = c.used;
  return m;
}

bool bad_workspace(const void* p, size_t bytes, size_t need) { return !p || bytes < need || !aligned(p, 256); }

int route_pairs(const Routed& r, const int32_t* ids, int64_t P, int E, int tile_m, int64_t cap, int* err,
                cudaStream_t s) {
  return launch_route_tile_map(ids, static_cast<int>(P), E, tile_m, r.counts, r.offsets, r.sorted_pairs, r.tiles,
                               r.num_tiles, cap, err, s, nullptr, 0, r.slot_of, r.tile_first);
}

Fp4Slots slots_of(const Routed& r, const int32_t* ids) { return {ids, r.slot_of, r.offsets, r.tile_first}; }

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" {

int tq_fp4_quantize(const void* x, int x_type, int64_t x_stride, int64_t n, int K, int fmt, const float* global_scale,
                    uint8_t* packed, uint8_t* scales, tq_stream_t stream) {
  if (n < 0 || bad_k(K) || bad_output(n, K) || bad_format(fmt) || (fmt == TQ_FP4_MX && global_scale))
    return TQ_ERR_INVALID_ARG;
  if (bad_rows(x, x_type, x_stride, n, K)) return TQ_ERR_INVALID_ARG;
  if (n > 0 && (!packed || !scales || !aligned(packed, 8))) return TQ_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int rc = require_sm103(s);
  if (rc != TQ_OK || n == 0) return rc;
  return launch_fp4_quantize(x, x_type, x_stride, n, K, fmt, global_scale, packed, scales, s);
}

int tq_fp4_dequantize(const uint8_t* packed, const uint8_t* scales, int64_t n, int K, int fmt,
                      const float* global_scale, void* out, int out_type, tq_stream_t stream) {
  if (n < 0 || bad_k(K) || bad_output(n, K) || bad_format(fmt) || bad_type(out_type) ||
      (fmt == TQ_FP4_MX && global_scale))
    return TQ_ERR_INVALID_ARG;
  if (n > 0 && (!packed || !scales || !out || !aligned(packed, 8) || !aligned(out, 16))) return TQ_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int rc = require_sm103(s);
  if (rc != TQ_OK || n == 0) return rc;
  return launch_fp4_dequantize(packed, scales, n, K, fmt, global_scale, out, out_type, s);
}

size_t tq_fp4_tiled_scales_size(int E, int N, int K, int fmt) {
  if (E < 1 || bad_matrix(E, K, N) || bad_output(static_cast<int64_t>(E) * (N + 127ll), K) || bad_format(fmt)) return 0;
  return static_cast<size_t>(E) * ((N + 127) / 128) * fp4_steps(K) * fp4_scale_step_bytes(fmt);
}

int tq_fp4_tile_scales(const uint8_t* scales, int E, int N, int K, int fmt, uint8_t* tiled, tq_stream_t stream) {
  if (tq_fp4_tiled_scales_size(E, N, K, fmt) == 0 || !scales || !tiled || !aligned(tiled, 16))
    return TQ_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int rc = require_sm103(s);
  if (rc != TQ_OK) return rc;
  return launch_fp4_tile_scales(scales, E, N, K, fmt, tiled, s);
}

size_t tq_fp4_linear_workspace_size(int64_t n, int K, int N, int fmt) {
  if (n < 0 || n >= kMaxIndex || bad_matrix(1, K, N) || bad_output(n, N) || bad_format(fmt)) return 0;
  return linear_gemv(n, K, N) ? kNoWorkspace : plan_linear(nullptr, n, K, N, fmt).bytes;
}

int tq_fp4_linear(const void* x, int x_type, int64_t x_stride, const uint8_t* packed, const uint8_t* tiled_scales,
                  int fmt, const float* w_scale, const float* x_scale, int64_t n, int K, int N, void* workspace,
                  size_t workspace_bytes, void* y, int y_type, tq_stream_t stream) {
  if (n < 0 || n >= kMaxIndex || bad_matrix(1, K, N) || bad_output(n, N) || bad_format(fmt) || bad_type(y_type) ||
      bad_rows(x, x_type, x_stride, n, K) || (fmt == TQ_FP4_MX && (w_scale || x_scale)))
    return TQ_ERR_INVALID_ARG;
  if (n > 0 && (!packed || !tiled_scales || !y || !aligned(packed, 16) || !aligned(tiled_scales, 16) ||
                !aligned(y, type_size(y_type))))
    return TQ_ERR_INVALID_ARG;
  const bool gemv = linear_gemv(n, K, N);
  const LinearPlan l = plan_linear(workspace, n, K, N, fmt);
  if (n > 0 && !gemv && bad_workspace(workspace, workspace_bytes, l.bytes)) return TQ_ERR_WORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int rc = require_sm103(s);
  if (rc != TQ_OK || n == 0) return rc;
  int* err = error_word(&rc);
  if (!err) return rc;
  if (gemv) {
    const Fp4Gemv v{fmt, packed, tiled_scales, w_scale, x, x_type, x_stride, x_scale, nullptr, nullptr, n, 1, 1, K, N,
                    y, y_type, err};
    return launch_fp4_gemv(v, s);
  }
  rc = launch_fp4_stage(x, x_type, x_stride, n, K, fmt, x_scale, 1, Fp4Slots{}, l.tile_m, l.staged.codes, l.staged.scales, s);
  if (rc != TQ_OK) return rc;
  Fp4Gemm g{fmt, packed, tiled_scales, w_scale, l.staged.codes, l.staged.scales, x_scale, nullptr, nullptr, nullptr,
            l.tiles, n, 1, K, N, l.tile_m, l.splits, l.part, l.splits > 1 ? nullptr : y, y_type, err};
  rc = launch_fp4_gemm(g, s);
  if (rc != TQ_OK || l.splits == 1) return rc;
  return launch_fp4_combine(l.part, n * N, l.splits, nullptr, nullptr, x_scale, w_scale, n, 1, 1, N, y, y_type, s);
}

size_t tq_fp4_moe_workspace_size(int64_t n, int top_k, int E, int K, int N, int fmt) {
  if (bad_moe_shape(n, top_k, E) || bad_matrix(E, K, N) || bad_output(n * top_k, N) || bad_format(fmt)) return 0;
  return moe_gemv(n, top_k, E, K, N) ? kNoWorkspace : plan_moe(nullptr, n, top_k, E, K, N, fmt).bytes;
}

int tq_fp4_moe_forward(const void* x, int x_type, int64_t x_stride, const uint8_t* packed, const uint8_t* tiled_scales,
                       int fmt, const float* w_scale, const float* x_scale, const int32_t* topk_ids,
                       const float* topk_w, int64_t n, int top_k, int E, int K, int N, void* workspace,
                       size_t workspace_bytes, void* y, int y_type, tq_stream_t stream) {
  if (bad_moe_shape(n, top_k, E) || bad_matrix(E, K, N) || bad_output(n * top_k, N) || bad_format(fmt) ||
      bad_type(y_type) || bad_rows(x, x_type, x_stride, n, K) || (fmt == TQ_FP4_MX && (w_scale || x_scale)))
    return TQ_ERR_INVALID_ARG;
  if (n > 0 && (!packed || !tiled_scales || !topk_ids || !topk_w || !y || !aligned(packed, 16) ||
                !aligned(tiled_scales, 16) || !aligned(y, type_size(y_type))))
    return TQ_ERR_INVALID_ARG;
  const bool gemv = moe_gemv(n, top_k, E, K, N);
  const MoePlan m = plan_moe(workspace, n, top_k, E, K, N, fmt);
  if (n > 0 && !gemv && bad_workspace(workspace, workspace_bytes, m.bytes)) return TQ_ERR_WORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int rc = require_sm103(s);
  if (rc != TQ_OK || n == 0) return rc;
  int* err = error_word(&rc);
  if (!err) return rc;
  if (gemv) {
    const Fp4Gemv v{fmt, packed, tiled_scales, w_scale, x, x_type, x_stride, x_scale, topk_ids, topk_w, n, top_k, E, K,
                    N, y, y_type, err};
    return launch_fp4_gemv(v, s);
  }
  rc = route_pairs(m.routed, topk_ids, m.P, E, m.tile_m, m.cap, err, s);
  if (rc == TQ_OK)
    rc = launch_fp4_stage(x, x_type, x_stride, n, K, fmt, x_scale, top_k, slots_of(m.routed, topk_ids), m.tile_m,
                          m.staged.codes, m.staged.scales, s);
  if (rc != TQ_OK) return rc;
  Fp4Gemm g{fmt, packed, tiled_scales, w_scale, m.staged.codes, m.staged.scales, x_scale, m.routed.sorted_pairs,
            m.routed.tiles, m.routed.num_tiles, m.cap, m.P, E, K, N, m.tile_m, m.splits, m.part, nullptr, y_type, err};
  rc = launch_fp4_gemm(g, s);
  if (rc != TQ_OK) return rc;
  return launch_fp4_combine(m.part, m.P * N, m.splits, topk_ids, topk_w, x_scale, w_scale, n, top_k, E, N, y, y_type,
                            s);
}

size_t tq_fp4_moe_mlp_workspace_size(int64_t n, int top_k, int E, int H, int I, int fmt) {
  if (bad_moe_shape(n, top_k, E) || I < 1 || I > (1 << 29) || bad_matrix(E, H, 2 * I) || bad_matrix(E, I, H) ||
      bad_output(n * top_k, 2ll * I) || bad_output(n * top_k, H) || bad_format(fmt))
    return 0;
  return plan_mlp(nullptr, n, top_k, E, H, I, fmt).bytes;
}

int tq_fp4_moe_mlp_forward(const void* x, int x_type, int64_t x_stride, const uint8_t* packed_gu,
                           const uint8_t* tiled_gu, const float* gu_scale, const uint8_t* packed_down,
                           const uint8_t* tiled_down, const float* down_scale, int fmt, const float* x_scale,
                           const float* h_scale, const int32_t* topk_ids, const float* topk_w, int64_t n, int top_k,
                           int E, int H, int I, void* workspace, size_t workspace_bytes, void* y, int y_type,
                           tq_stream_t stream) {
  if (tq_fp4_moe_mlp_workspace_size(n, top_k, E, H, I, fmt) == 0 || bad_type(y_type) ||
      bad_rows(x, x_type, x_stride, n, H) || (fmt == TQ_FP4_MX && (gu_scale || down_scale || x_scale || h_scale)))
    return TQ_ERR_INVALID_ARG;
  if (n > 0 && (!packed_gu || !tiled_gu || !packed_down || !tiled_down || !topk_ids || !topk_w || !y ||
                !aligned(packed_gu, 16) || !aligned(tiled_gu, 16) || !aligned(packed_down, 16) ||
                !aligned(tiled_down, 16) || !aligned(y, type_size(y_type))))
    return TQ_ERR_INVALID_ARG;
  const MlpPlan m = plan_mlp(workspace, n, top_k, E, H, I, fmt);
  if (n > 0 && bad_workspace(workspace, workspace_bytes, m.bytes)) return TQ_ERR_WORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int rc = require_sm103(s);
  if (rc != TQ_OK || n == 0) return rc;
  int* err = error_word(&rc);
  if (!err) return rc;
  const Routed& r = m.routed;
  rc = route_pairs(r, topk_ids, m.P, E, m.tile_m, m.cap, err, s);
  if (rc == TQ_OK)
    rc = launch_fp4_stage(x, x_type, x_stride, n, H, fmt, x_scale, top_k, slots_of(r, topk_ids), m.tile_m, m.x.codes, m.x.scales, s);
  if (rc != TQ_OK) return rc;
  Fp4Gemm gu{fmt, packed_gu, tiled_gu, gu_scale, m.x.codes, m.x.scales, x_scale, r.sorted_pairs, r.tiles, r.num_tiles,
             m.cap, m.P, E, H, 2 * I, m.tile_m, m.splits_gu, m.gate_up, nullptr, y_type, err};
  rc = launch_fp4_gemm(gu, s);
  if (rc == TQ_OK)
    rc = launch_fp4_stage_swiglu(m.gate_up, m.P * 2 * I, m.splits_gu, x_scale, gu_scale, m.P, E, I, fmt, h_scale,
                                 slots_of(r, topk_ids), m.tile_m, m.h.codes, m.h.scales, s);
  if (rc != TQ_OK) return rc;
  Fp4Gemm down{fmt, packed_down, tiled_down, down_scale, m.h.codes, m.h.scales, h_scale, r.sorted_pairs, r.tiles,
               r.num_tiles, m.cap, m.P, E, I, H, m.tile_m, m.splits_down, m.down, nullptr, y_type, err};
  rc = launch_fp4_gemm(down, s);
  if (rc != TQ_OK) return rc;
  return launch_fp4_combine(m.down, m.P * H, m.splits_down, topk_ids, topk_w, h_scale, down_scale, n, top_k, E, H, y,
                            y_type, s);
}

}  // extern "C"
