// Which variant of tq_tile_gemm.cuh a product takes.
#pragma once
#include <algorithm>
#include <cmath>

#include "tq_internal.h"

namespace tq {

struct TileChoice {
  int tile_m;   // 128, or 256: a pair of CTAs
  bool quad;    // two pairs share the rows of A
  int cols;     // half the columns of a unit
  int splits;
};

// By the time that the parts take (cycles of an SM; a pair's for two of them): a
// step's MMAs, 4 cycles a column and row of 128, or its bytes at 72 a clock; a unit's
// first copies and last drain; the matrices from memory at 3400 bytes a clock over
// the chip; the partial sums of splits (and of experts' pairs, `partial`) written and
// read again at 3000 bytes a clock, and the launch that adds them up.  `rows` rows for
// each of `matrices` matrices; N columns, of h when gated (no splits: the activation
// needs whole sums).
// Two pairs that share their rows halve the copies of gathered rows, which bound a pair
// (8192 tokens of top-6 of 256, 4096 -> 2048: 716 us by pairs, 640 so); where rows come
// in whole boxes they gain less than the SMs that clusters of four leave idle (a linear
// of 8192 rows 4096 -> 4096: 122 us by pairs, 133 so).
inline TileChoice choose_tile(double rows, double matrices, int steps, int64_t N, bool gated, bool gather, bool partial,
                              bool takes_splits) {
  struct Variant {
    int tile_m, cols;
    double step;
  };
  static constexpr Variant kVariants[] = {{256, 128, 560}, {128, 128, 690}, {128, 64, 460}, {128, 32, 345}};
  const int sms = sm_count();
  const double weights = matrices * N * (gated ? 2 : 1) * steps * 128.0 / 3400.0;
  TileChoice best{128, false, 128, 1};
  double best_cost = 1e300;
  for (const Variant& v : kVariants) {
    if (gated && v.cols < 64) continue;
    const bool pair = v.tile_m > 128;
    const double tiles = matrices * std::ceil(rows / v.tile_m);
    const double units = tiles * std::ceil(static_cast<double>(N) / (gated ? v.cols : 2 * v.cols));
    const int slots = pair ? sms / 2 : sms;
    for (int s = 1; s <= (takes_splits ? std::min(16, steps) : 1); ++s) {
      const double unit = ((steps + s - 1) / s) * v.step + 2000.0;
      double cost = 4000.0 + std::max(std::ceil(units * s / slots) * unit, weights);
      if (s > 1 || partial) cost += 5000.0 + 8.0 * s * rows * matrices * N / 3000.0;
      if (cost < best_cost * 0.99) {
        best = {v.tile_m, pair && gather, v.cols, s};
        best_cost = cost;
      }
    }
  }
  return best;
}

}  // namespace tq
