"""The plain definitions of the norm, the 8-bit blocks and the gated projection
against properties and differences."""
import numpy as np
import torch

import oracle.block_operators as B


def test_code_values_are_the_grid():
    v = B.code_value(np.arange(256))
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v, t, equal_nan=True)
    finite = v[np.isfinite(v)]
    assert np.array_equal(B.e4m3(finite), finite)
    mid = (np.sort(np.unique(finite))[1:] + np.sort(np.unique(finite))[:-1]) / 2
    want = torch.from_numpy(mid).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(B.e4m3(mid), want)
    assert B.e4m3(1e30) == 448.0 and B.e4m3(-1e30) == -448.0 and np.isnan(B.e4m3(np.nan))


def test_quantize_blocks():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((130, 144)).astype(np.float32)
    for rows in (1, 128):
        q, s = B.quantize(x, rows)
        assert s.shape == (-(-130 // rows), 2)
        assert np.abs(B.values(q, s, rows) - x).max() <= np.abs(x).max() / 16
        assert np.abs(q[:rows, :128]).max() == 448.0


def _difference(f, x, d, h=1e-6):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


def test_gradients_are_differences():
    rng = np.random.default_rng(2)
    r, w, dy, dr = rng.standard_normal((4, 3, 10))[:, :, :10]
    w = w[0]
    dx, dw = B.rms_norm_grad(dy, r, w, 0.1, dr)
    at = rng.standard_normal(r.shape)
    got = _difference(lambda z: (B.rms_norm(z, w, 0.1)[0] * dy + z * dr).sum(), r, at)
    assert abs(got - (dx * at).sum()) < 1e-7
    at = rng.standard_normal(w.shape)
    assert abs(_difference(lambda z: (B.rms_norm(r, z, 0.1)[0] * dy).sum(), w, at) - (dw * at).sum()) < 1e-7

    x, wgu, dh = rng.standard_normal((5, 8)), rng.standard_normal((12, 8)), rng.standard_normal((5, 6))
    gx, gw, _ = B.gated_grad(x, wgu, dh)
    at = rng.standard_normal(x.shape)
    assert abs(_difference(lambda z: (B.gated(z, wgu)[0] * dh).sum(), x, at) - (gx * at).sum()) < 1e-6
    at = rng.standard_normal(wgu.shape)
    assert abs(_difference(lambda z: (B.gated(x, z)[0] * dh).sum(), wgu, at) - (gw * at).sum()) < 1e-6
