"""Every variant of the tile product that a size chooses is one that is built."""
import itertools
import os
import shutil
import subprocess

import pytest

from trellis_quantized_moe_sort_gb300 import build

PROGRAM = r"""
#include <cstdio>
#include "tq_tiling.h"
namespace tq { int sm_count() { return 152; } }
int main() {
  int k8, kind, gated, steps, splits, only;
  double rows, matrices;
  long long N;
  while (scanf("%d %d %d %lf %lf %d %lld %d %d", &k8, &kind, &gated, &rows, &matrices, &steps, &N, &splits, &only) == 9) {
    const tq::TileChoice t = tq::choose_tile(k8, rows, matrices, steps, N, gated, static_cast<tq::TileRows>(kind), splits,
                                             splits, only);
    printf("%d %d %d\n", t.tile_m, t.cols, t.splits);
  }
}
"""
ONE, GATHERED, SLOTS = 0, 1, 2
# (8 bits, rows, gated, splits allowed, only these columns) -> (tile_m, cols)
BUILT = {
    (1, ONE, 0, 1, 0): {(256, 128), (128, 128), (128, 64), (128, 32)},
    (1, GATHERED, 0, 1, 0): {(128, 128), (128, 64), (128, 32)},
    (1, SLOTS, 0, 1, 0): {(128, 128), (128, 64), (128, 32)},
    (1, GATHERED, 1, 0, 0): {(128, 128)},
    (0, ONE, 1, 0, 0): {(256, 128), (128, 128), (128, 64)},
    (0, ONE, 0, 1, 0): {(256, 128), (128, 128), (128, 64)},
    (0, ONE, 0, 1, 64): {(128, 64)},
}


def test_choices_are_built_variants(tmp_path):
    if not shutil.which("g++"):
        pytest.skip("no g++")
    source, program = tmp_path / "choice.cc", tmp_path / "choice"
    source.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", build.CSRC, "-I", build.INCLUDE,
                    "-I", os.path.join(build.cuda_home(), "include"), str(source), "-o", str(program)], check=True)
    asked, built = [], []
    for (k8, kind, gated, splits, only), variants in BUILT.items():
        for rows, matrices, steps, N in itertools.product((1, 3, 17, 64, 127, 129, 300, 2048, 8191), (1, 8, 136),
                                                          (1, 2, 8, 33, 128), (8, 128, 256, 777, 2048, 16384)):
            if kind == ONE and matrices > 1:
                continue
            asked.append((k8, kind, gated, rows, matrices, steps, N, splits, only))
            built.append(variants)
    out = subprocess.run([str(program)], input="\n".join(" ".join(map(str, a)) for a in asked), capture_output=True,
                         text=True, check=True).stdout.split("\n")[:-1]
    assert len(out) == len(asked)
    for a, line, variants in zip(asked, out, built):
        tile_m, cols, splits = map(int, line.split())
        assert (tile_m, cols) in variants, (a, line)
        assert splits == 1 or (a[7] and splits <= min(16, a[5])), (a, line)
