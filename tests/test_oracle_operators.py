"""The definitions in oracle/moe_operators.py held to facts stated apart from
them: E2M1 and E4M3 as lists of values, the tie rule, small router rows worked
out by hand, the router's gradient against differences."""
import numpy as np
import pytest

import oracle.moe_operators as M


def test_e4m3_values_and_bytes():
    every = [M.dequantize(np.array([[0x02] + [0] * 7], np.uint8), np.array([[b]], np.uint8), "nv")[0, 0] for b in range(127)]
    assert every[0] == 0.0 and every[1] == 2.0 ** -9 and every[8] == 2.0 ** -6 and every[126] == 448.0
    assert all(a < b for a, b in zip(every, every[1:]))
    v = np.array(every)
    assert np.array_equal(M.e4m3(v), v)
    assert np.array_equal(M.e4m3_byte(v), np.arange(127))
    mid = (v[:-1] + v[1:]) / 2
    even = np.where(np.arange(126) % 2 == 0, v[:-1], v[1:])
    assert np.array_equal(M.e4m3(mid), even)
    assert np.array_equal(M.e4m3(mid * (1 + 1e-12)), v[1:]) and np.array_equal(M.e4m3(mid * (1 - 1e-12)), v[:-1])
    assert M.e4m3(1e9) == 448.0


def test_e2m1_nearest_ties_to_even():
    # scale 1: a block whose largest value is 6
    x = np.zeros((1, 32))
    x[0, 0] = 6.0
    x[0, 1:15] = [0.25, 0.26, 0.75, 0.74, 1.25, 1.26, 1.75, 1.74, 2.5, 2.51, 3.5, 3.49, 5.0, 5.01]
    want = [6.0, 0.0, 0.5, 1.0, 0.5, 1.0, 1.5, 2.0, 1.5, 2.0, 3.0, 4.0, 3.0, 4.0, 6.0]
    for sign in (1.0, -1.0):
        code, byte, values = M.quantize(sign * x, "nv")
        assert byte[0, 0] == 0x38 and np.array_equal(values[0, :15], sign * np.array(want))
        code, byte, values = M.quantize(sign * x, "mx")
        assert byte[0, 0] == 127 and np.array_equal(values[0, :15], sign * np.array(want))


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_quantize_special_blocks(fmt):
    B = M.BLOCK[fmt]
    x = np.zeros((1, 6 * 32))
    x[0, 32] = np.nan
    x[0, 64], x[0, 65] = np.inf, 1.0
    x[0, 96] = -3.0
    x[0, 128] = 2.0 ** -149
    code, byte, values = M.quantize(x, fmt)
    assert np.isfinite(values).all()
    assert not values[0, :64].any()
    # an infinity is the largest finite number, which saturates
    assert values[0, 64] == (2688.0 if fmt == "nv" else 6.0 * 2.0 ** 125) and values[0, 65] == 0.0
    assert values[0, 96] == (-3.0 if fmt == "mx" else -6.0 * 0.5)
    assert values[0, 128] == 0.0
    assert np.array_equal(M.dequantize(M.pack(code), byte, fmt), values)
    assert byte.shape == (1, 192 // B)


def test_router_by_hand():
    x = np.log(np.array([[1.0, 2.0, 4.0, 8.0, 1.0, 8.0]]))
    ids, w, _ = M.router(x, 3, score="softmax", renormalize=False)
    assert ids.tolist() == [[3, 5, 2]] and np.allclose(w * 24, [[8, 8, 4]])
    ids, w, _ = M.router(x, 3, score="softmax", renormalize=True, scale=2.0)
    assert np.allclose(w, [[0.8, 0.8, 0.4]])
    # the bias moves the choice and not the weight
    ids, w, _ = M.router(x, 2, score="softmax", bias=[1, 0, 0, 0, 0, 0], renormalize=False)
    assert ids.tolist() == [[0, 3]] and np.allclose(w * 24, [[1, 8]])
    # groups (0,1) (2,3) (4,5): 3, 12 and 9 of 24; the best one holds 2 and 3
    ids, w, _ = M.router(x, 2, score="softmax", groups=3, top_groups=1, renormalize=False)
    assert ids.tolist() == [[3, 2]]
    # sigmoid of 0 is 1/2; masked logits come last, with weight 0; an empty row has none
    y = np.array([[0.0, -np.inf, np.nan, 0.0], [-np.inf, np.nan, np.inf, -np.inf]])
    ids, w, _ = M.router(y, 3)
    assert ids.tolist() == [[0, 3, 1], [0, 1, 2]] and np.allclose(w, [[0.5, 0.5, 0.0], [0, 0, 0]])


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_router_gradient_is_the_slope(score, renormalize):
    rng = np.random.default_rng(7)
    x = rng.standard_normal((3, 9))
    x[1, 4] = -np.inf
    ids, w, _ = M.router(x, 4, score=score, renormalize=renormalize)
    live = w != 0
    g = rng.standard_normal((3, 4))
    got = M.router_backward(x, ids, live, g, score, renormalize, 1.5)
    h = 1e-5
    for t in range(3):
        for e in range(9):
            if not np.isfinite(x[t, e]):
                assert got[t, e] == 0
                continue
            up, down = x.copy(), x.copy()
            up[t, e] += h
            down[t, e] -= h
            f = [(M.router_weights(v, ids, live, score, renormalize, 1.5) * g).sum() for v in (up, down)]
            assert abs((f[0] - f[1]) / (2 * h) - got[t, e]) < 1e-8    # h^2 times third derivatives below 10
