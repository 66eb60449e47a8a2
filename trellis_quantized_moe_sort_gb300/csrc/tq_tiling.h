// Which variant of tq_tile_gemm.cuh a product takes.
#pragma once
#include <algorithm>
#include <cmath>

#include "tq_internal.h"

namespace tq {

struct TileChoice {
  int tile_m;   // 128, or 256: a pair of CTAs
  int cols;     // half the columns of a unit
  int splits;
  double cost;
};

// What the rows of a product are: of one matrix; token rows of experts, gathered; or
// experts' slots, which lie together.
enum class TileRows { kOne, kGathered, kSlots };

// By the time that the parts take (cycles of an SM; of two where they work together): a
// step, by its bytes at 50 a clock, its MMAs and the way of an accumulator to the
// epilogue and back; with the copies of gathered rows, `gathered` for a full tile and 24
// less for each copy of four rows that it lacks; a unit's first copies, last
// drain and stores; the matrices from memory at 3400 bytes a clock over the chip; the
// partial sums of splits (and of experts' pairs, `partial`) written and read again at
// 3000 bytes a clock, and the launch that adds them up.  `rows` rows for each of
// `matrices` matrices; N columns, of h when gated (no splits: the activation needs whole
// sums).
// Measured: 8192 rows 4096 -> 4096 of one matrix 130 us by pairs (its quantising
// included), 142 by CTAs alone.  Experts 4096 -> 2048, of 128, 64 and 32 columns a half:
// 256 rows for each of 76 213, 340 and 639 us, 96 for each of 152 260, 292 and 535; 512
// tokens of top-6 of 256 351, 357 and 588.
inline TileChoice choose_tile(bool k8, double rows, double matrices, int steps, int64_t N, bool gated, TileRows kind,
                              bool partial, bool takes_splits, int only_cols = 0) {
  struct Variant {
    int tile_m;
    int cols;
    double step, gathered, step16;
  };
  static constexpr Variant kVariants[] = {{256, 128, 980, 0, 740},
                                          {128, 128, 1000, 1440, 980},
                                          {128, 64, 660, 1180, 660},
                                          {128, 32, 500, 1120, 0}};
  const int sms = sm_count();
  const double weights = matrices * N * (gated ? 2 : 1) * steps * 128.0 / 3400.0;
  TileChoice best{128, 128, 1, 1e300};
  for (const Variant& v : kVariants) {
    if ((kind != TileRows::kOne && v.tile_m > 128) || (!k8 && v.step16 == 0)) continue;
    if (gated && v.cols < (k8 ? 128 : 64)) continue;   // (in 8 bits a block of h is one unit's columns)
    if (only_cols && (v.cols != only_cols || v.tile_m > 128)) continue;
    const int together = v.tile_m > 128 ? 2 : 1;
    const double tiles = matrices * std::ceil(rows / v.tile_m);
    const double columns = gated ? v.cols : 2 * v.cols;
    const double units = tiles * std::ceil(static_cast<double>(N) / columns);
    const double copies = std::ceil(rows / std::ceil(rows / v.tile_m) / 4.0);   // of a tile
    const double step = !k8                          ? v.step16
                        : kind == TileRows::kGathered ? std::max(v.step, v.gathered - 24.0 * (32.0 - copies))
                                                      : v.step;
    for (int s = 1; s <= (takes_splits ? std::min(16, steps) : 1); ++s) {
      const double unit = ((steps + s - 1) / s) * step + 24.0 * v.cols + 1500.0;
      double cost = 4000.0 + std::max(std::ceil(units * s / (sms / together)) * unit, weights);
      if (s > 1 || partial) cost += 9000.0 + 8.0 * s * rows * matrices * N / 3000.0;
      if (cost < best.cost * 0.99) best = {v.tile_m, v.cols, s, cost};
    }
  }
  return best;
}

// The same measure of the few-rows kernel, `bytes` of weights: 8 rows a pass, or 16 a
// pass with twice the work.  Measured in 8 bits, 8, 16 and 32 rows: 4096 -> 2048 4.5, 6.2
// and 7.9 us (tiles 9.5, 9.7, 9.4), 4096 -> 8192 11.5, 15.9 and 25.7 (13.5, 17.5, 12.8); in
// 16 bits gated 4096 -> 2 x 2048 9.0, 10.7 and 16.4 (tiles with K split 13.4), 1024 -> 2 x
// 512 2.8, 3.3 and 3.4 (12.8).
inline double few_rows_cost(int64_t n, double bytes, bool k8) {
  if (n > 256) return 1e300;
  const double pass = n <= 8 ? (k8 ? 0.26 : 0.20) : (k8 ? 0.37 : 0.24) * static_cast<double>((n + 15) / 16);
  return 1900.0 * (2.3 + pass * bytes * 1e-6);   // us per MB; cycles
}

}  // namespace tq
