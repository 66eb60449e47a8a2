// Product of 8-bit block-scaled rows with 8-bit matrices (one, or the experts of a
// tile map), and the SwiGLU experts' gate and up projections with h kept in 8 bits:
// variants of tq_tile_gemm.cuh.
#include "tq_tile_gemm.cuh"

namespace tq {
int launch_fp8_gemm(const Fp8Gemm& g, cudaStream_t s) {
  using namespace tile;
  if ((g.gated || g.tile_m > kRows) && g.cols != 128) return TQ_ERR_INVALID_ARG;
  Params p{};
  const bool pair = g.tile_m > kRows;
  p.tiles = g.tiles;
  p.num_tiles = g.num_tiles;
  p.sorted_pairs = g.sorted_pairs;
  p.gather = g.gather;
  p.scatter = g.scatter;
  p.cap = g.cap;
  p.split_stride = static_cast<long long>(g.M) * g.y_ld;
  p.y_ld = g.y_ld;
  p.M = static_cast<int>(g.M);
  p.E = g.E;
  p.N = g.N;
  p.tile_m = g.tile_m;
  p.top_k = g.top_k;
  p.steps = (g.K + kFp8Block - 1) / kFp8Block;
  p.splits = g.splits;
  const int columns = g.gated ? g.cols : 2 * g.cols;
  p.col_blocks = (g.N + columns - 1) / columns;
  p.a_scales = g.x_scales;
  p.b_scales = g.w_scales;
  p.b_blocks = ((g.gated ? 2 * g.N : g.N) + kFp8Block - 1) / kFp8Block;
  p.y = g.y;
  p.y_type = g.y_type;
  const int64_t size = g.y_type == TQ_FP32 ? 4 : 2;
  p.aligned = g.y_ld * size % 16 == 0 && (reinterpret_cast<uintptr_t>(g.y) & 15u) == 0;
  p.codes = g.codes;
  p.scales = g.scales;
  p.err = g.err;
  CUtensorMap a, b;
  const int64_t w_rows = static_cast<int64_t>(g.E) * (g.gated ? 2 : 1) * g.N;
  if (!encode(&a, g.x, 1, g.K, g.x_rows, g.K, g.gather ? 1 : kRows) ||
      !encode(&b, g.w, 1, g.K, w_rows, g.K, g.cols))
    return TQ_ERR_INVALID_ARG;
  const long long units = g.cap * p.col_blocks * g.splits;
  int st;
  if (g.gated)
    st = launch<true, false, 128, false, false, kGated8>(p, a, b, units, s);
  else
    st = pair            ? launch<true, true, 128, false, false, kStore>(p, a, b, units, s)
         : g.cols == 128 ? launch<true, false, 128, false, false, kStore>(p, a, b, units, s)
         : g.cols == 64  ? launch<true, false, 64, false, false, kStore>(p, a, b, units, s)
                         : launch<true, false, 32, false, false, kStore>(p, a, b, units, s);
  if (st == TQ_OK) count_launch(kCntFp8Gemm);
  return st;
}

}  // namespace tq
