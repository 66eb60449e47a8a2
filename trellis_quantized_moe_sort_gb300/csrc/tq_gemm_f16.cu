// Product of 16-bit matrices on the tensor cores: the gated projection and its
// gradients, variants of tq_tile_gemm.cuh.
#include "tq_tile_gemm.cuh"

namespace tq {

int launch_gemm_f16(const GemmF16& g, cudaStream_t s) {
  using namespace tile;
  Params p{};
  const bool pair = g.tile_m > kRows;
  p.cap = (g.M + g.tile_m - 1) / g.tile_m;
  p.split_stride = g.M * g.N;
  p.y_ld = g.N;
  p.M = static_cast<int>(g.M);
  p.E = 1;
  p.N = static_cast<int>(g.N);
  p.tile_m = g.tile_m;
  p.top_k = 1;
  p.steps = static_cast<int>((g.K + 63) / 64);
  p.splits = g.splits;
  const int columns = g.gated ? g.cols : 2 * g.cols;
  p.col_blocks = static_cast<int>((g.N + columns - 1) / columns);
  p.y = g.y;
  p.y_type = g.y_type;
  p.type = g.type;
  const int64_t size = g.y_type == TQ_FP32 ? 4 : 2;
  p.aligned = g.N * size % 16 == 0 && (reinterpret_cast<uintptr_t>(g.y) & 15u) == 0;
  p.gate_up = g.gate_up;
  p.err = g.err;
  CUtensorMap a, b;
  if (!(g.a_mn ? encode(&a, g.a, 2, g.M, g.K, 2 * g.a_stride, 64) : encode(&a, g.a, 2, g.K, g.M, 2 * g.a_stride, kRows)) ||
      !(g.b_mn ? encode(&b, g.b, 2, g.N, g.K, 2 * g.b_stride, 64)
               : encode(&b, g.b, 2, g.K, g.gated ? 2 * g.N : g.N, 2 * g.b_stride, g.cols)))
    return TQ_ERR_INVALID_ARG;
  const long long units = p.cap * p.col_blocks * g.splits;
  int st;
  if (g.gated)
    st = pair            ? launch<false, true, 128, false, false, kGated16>(p, a, b, units, s)
         : g.cols == 128 ? launch<false, false, 128, false, false, kGated16>(p, a, b, units, s)
                         : launch<false, false, 64, false, false, kGated16>(p, a, b, units, s);
  else if (!g.b_mn)
    st = launch<false, false, 64, false, false, kStore>(p, a, b, units, s);
  else if (g.a_mn)
    st = pair            ? launch<false, true, 128, true, true, kStore>(p, a, b, units, s)
         : g.cols == 128 ? launch<false, false, 128, true, true, kStore>(p, a, b, units, s)
                         : launch<false, false, 64, true, true, kStore>(p, a, b, units, s);
  else
    st = pair            ? launch<false, true, 128, false, true, kStore>(p, a, b, units, s)
         : g.cols == 128 ? launch<false, false, 128, false, true, kStore>(p, a, b, units, s)
                         : launch<false, false, 64, false, true, kStore>(p, a, b, units, s);
  if (st == TQ_OK) count_launch(kCntGatedGemm);
  return st;
}

}  // namespace tq
