"""Outputs and workspaces of the norm, the 8-bit operators and the gated projection that
share memory with what is read, or with each other, are refused before any device work.

The addresses are stand-ins that no call reaches: without a device a call that is not
refused ends with the missing device."""
import itertools

import pytest
import torch

INVALID, WORKSPACE = -1, -8

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="a call that is not refused would run")


@pytest.fixture(scope="module")
def lib():
    from trellis_quantized_moe_sort_gb300 import build
    build.build()
    import trellis_quantized_moe_sort_gb300 as tq
    return tq.lib()


class Call:
    """A call whose buffers, [name: (bytes, is written)], lie far apart unless moved; pairs that
    may start at one address, and pairs that may overlap in any way."""

    def __init__(self, call, buffers, same_start=(), any_way=()):
        self.call, self.buffers, self.same_start, self.any_way = call, buffers, same_start, any_way
        self.at = {name: (i + 1) << 34 for i, name in enumerate(buffers)}

    def check(self):
        assert self.call(self.at) not in (0, INVALID, WORKSPACE)
        for a, b in itertools.permutations(self.buffers, 2):
            (a_bytes, a_out), (b_bytes, b_out) = self.buffers[a], self.buffers[b]
            assert a_bytes > 0
            if not (a_out or b_out) or (a, b) in self.any_way or (b, a) in self.any_way:
                continue
            # b ends where a starts; b's last 256 bytes lie over a's first (a buffer of fewer: all of it)
            over = (self.at[a] - b_bytes) // 256 * 256 + 256
            if over + b_bytes > self.at[a]:
                assert self._moved(b, over) == INVALID, (a, b)
            assert self._moved(b, (self.at[a] - b_bytes) // 256 * 256) not in (0, INVALID, WORKSPACE), (a, b)
            same = self._moved(b, self.at[a])
            if (a, b) in self.same_start or (b, a) in self.same_start:
                assert same not in (0, INVALID, WORKSPACE), (a, b)
            else:
                assert same == INVALID, (a, b)

    def _moved(self, name, at):
        return self.call({**self.at, name: at})


def test_norm(lib):
    n, K = 40, 512
    row, blocks = 2 * n * K, n * 4 * 4
    Call(lambda a: lib.tq_rms_norm(a["x"], 1, K, a["res"], K, a["w"], 0, 1e-6, n, K, a["r"], a["y"], a["rstd"], a["codes"],
                                   a["scales"], None),
         dict(x=(row, 0), res=(row, 0), w=(4 * K, 0), r=(row, 1), y=(row, 1), rstd=(4 * n, 1), codes=(n * K, 1),
              scales=(blocks, 1)),
         same_start=[("x", "r"), ("x", "y"), ("res", "r"), ("res", "y")]).check()
    work = lib.tq_rms_norm_backward_workspace_size(n, K)
    Call(lambda a: lib.tq_rms_norm_backward(a["dy"], K, a["x"], 1, K, a["w"], 0, a["rstd"], a["g"], K, n, K, a["work"], work,
                                            a["gx"], a["gw"], None),
         dict(dy=(row, 0), x=(row, 0), w=(4 * K, 0), rstd=(4 * n, 0), g=(row, 0), work=(work, 1), gx=(row, 1), gw=(4 * K, 1)),
         same_start=[("dy", "gx"), ("x", "gx"), ("g", "gx")]).check()


@pytest.mark.parametrize("rows", (1, 128))
def test_quantize(lib, rows):
    E, n, K = 3, 200, 400
    codes, scales = E * n * K, 4 * E * -(-n // rows) * 4
    Call(lambda a: lib.tq_fp8_quantize(a["x"], 1, K, E, n, K, rows, a["codes"], a["scales"], None),
         dict(x=(2 * codes, 0), codes=(codes, 1), scales=(scales, 1))).check()
    Call(lambda a: lib.tq_fp8_dequantize(a["codes"], a["scales"], E, n, K, rows, a["out"], 1, None),
         dict(codes=(codes, 0), scales=(scales, 0), out=(2 * codes, 1))).check()


def _scales(E, N, K):
    return 4 * E * -(-N // 128) * -(-K // 128)


@pytest.mark.parametrize("n,N", [(2, 300), (8000, 4096)])   # few rows, tiles
def test_linear(lib, n, N):
    K = 4096
    work = lib.tq_fp8_linear_workspace_size(n, K, N)
    assert work == 256   # (K is split on a device alone)
    Call(lambda a: lib.tq_fp8_linear(a["x"], a["xs"], a["w"], a["ws"], n, K, N, None, 0, a["y"], 1, None),
         dict(x=(n * K, 0), xs=(4 * n * K // 128, 0), w=(N * K, 0), ws=(_scales(1, N, K), 0), y=(2 * n * N, 1))).check()


@pytest.mark.parametrize("n", (2, 4000))   # tokens by themselves, sorted tiles
def test_experts(lib, n):
    E, k, K, N, H, I = 8, 2, 400, 300, 400, 256
    work = lib.tq_fp8_moe_workspace_size(n, k, E, K, N)
    buffers = dict(x=(n * K, 0), xs=(4 * n * 4, 0), w=(E * N * K, 0), ws=(_scales(E, N, K), 0), ids=(4 * n * k, 0),
                   tw=(4 * n * k, 0), y=(2 * n * N, 1))
    if work > 256:
        buffers["work"] = (work, 1)
    assert ("work" in buffers) == (n == 4000)
    Call(lambda a: lib.tq_fp8_moe_forward(a["x"], a["xs"], a["w"], a["ws"], a["ids"], a["tw"], n, k, E, K, N, a.get("work"),
                                          work, a["y"], 1, None), buffers).check()
    work = lib.tq_fp8_moe_mlp_workspace_size(n, k, E, H, I)
    Call(lambda a: lib.tq_fp8_moe_mlp_forward(a["x"], a["xs"], a["gu"], a["gus"], a["d"], a["ds"], a["ids"], a["tw"], n, k, E,
                                              H, I, a["work"], work, a["y"], 1, None),
         dict(x=(n * H, 0), xs=(4 * n * 4, 0), gu=(E * 2 * I * H, 0), gus=(_scales(E, 2 * I, H), 0), d=(E * H * I, 0),
              ds=(_scales(E, H, I), 0), ids=(4 * n * k, 0), tw=(4 * n * k, 0), work=(work, 1), y=(2 * n * H, 1))).check()


@pytest.mark.parametrize("n,H,I", [(4, 512, 256), (4000, 512, 256)])   # few rows, tiles
def test_gated(lib, n, H, I):
    work = lib.tq_swiglu_linear_workspace_size(n, H, I)
    assert work == 256
    Call(lambda a: lib.tq_swiglu_linear(a["x"], 1, H, a["w"], n, H, I, None, 0, a["h"], a["gu"], None),
         dict(x=(2 * n * H, 0), w=(4 * I * H, 0), h=(2 * n * I, 1), gu=(8 * n * I, 1))).check()
    work = lib.tq_swiglu_linear_backward_workspace_size(n, H, I, 1)
    Call(lambda a: lib.tq_swiglu_linear_backward(a["x"], 1, H, a["w"], a["gu"], a["gh"], n, H, I, a["work"], work, a["gx"],
                                                 a["gw"], None),
         dict(x=(2 * n * H, 0), w=(4 * I * H, 0), gu=(8 * n * I, 0), gh=(2 * n * I, 0), work=(work, 1), gx=(2 * n * H, 1),
              gw=(4 * I * H, 1)),
         any_way=[("gx", "gu"), ("gx", "gh"), ("gw", "gu"), ("gw", "gh")]).check()
