"""Plain fp64 definitions of the RMS norm, the 8-bit block-scaled operators and the
gated projection, for the tests.  Nothing here is shared with the library or its
binding."""
import numpy as np

BLOCK = 128
MOST = 448.0
FP32_MOST = float(np.finfo(np.float32).max)


# ------------------------------------------------------------------ 8 bits

def e4m3(v):
    """The nearest E4M3 value (ties to even, saturating; NaN stays)."""
    v = np.asarray(v, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        a = np.minimum(np.abs(v), MOST)
        _, e = np.frexp(a)
        step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
        return np.copysign(np.minimum(np.round(a / step) * step, MOST), v)


def code_value(byte):
    """The value of E4M3 codes."""
    byte = np.asarray(byte, dtype=np.uint8).astype(np.int64)
    e, m = (byte >> 3) & 15, byte & 7
    v = np.where(e > 0, np.ldexp(1.0 + m / 8.0, e - 7), np.ldexp(m / 8.0, -6))
    v = np.where((byte & 127) == 127, np.nan, v)
    return np.where(byte & 128, -v, v)


def quantize(x, rows=1):
    """(E4M3 values [n, K], scales [n / rows, K / 128]) of fp32 numbers x in blocks of
    rows x 128.  The scale and the quotients are rounded to fp32."""
    x = np.asarray(x, dtype=np.float64)
    n, K = x.shape
    nb, kb = -(-n // rows), -(-K // BLOCK)
    q, s = np.zeros((n, K)), np.zeros((nb, kb))
    for i in range(nb):
        for j in range(kb):
            at = np.s_[i * rows:(i + 1) * rows, j * BLOCK:(j + 1) * BLOCK]
            b = x[at]
            top = np.abs(np.where(np.isnan(b), 0.0, b)).max()
            s[i, j] = np.float32(np.float32(min(top, FP32_MOST)) / np.float32(MOST))
            with np.errstate(all="ignore"):
                q[at] = e4m3((b.astype(np.float32) / np.float32(s[i, j])).astype(np.float64)) if s[i, j] > 0 else b * 0.0
    return q, s


def values(q, s, rows=1):
    """Values of E4M3 values and scales, [.., n, K]."""
    n, K = q.shape[-2:]
    wide = np.repeat(np.repeat(s, rows, -2)[..., :n, :], BLOCK, -1)[..., :K]
    return q * wide


# ------------------------------------------------------------------ norm

def rms_norm(r, weight=None, eps=1e-6):
    """(y, rstd [n, 1]) of normed rows r."""
    r = np.asarray(r, dtype=np.float64)
    rstd = 1.0 / np.sqrt((r * r).mean(-1, keepdims=True) + eps)
    return r * rstd * (1.0 if weight is None else np.asarray(weight, dtype=np.float64)), rstd


def rms_norm_grad(grad_y, r, weight=None, eps=1e-6, grad_r=None):
    """(grad_x, grad_weight)."""
    dy, r = np.asarray(grad_y, dtype=np.float64), np.asarray(r, dtype=np.float64)
    _, rstd = rms_norm(r, None, eps)
    a = dy * (1.0 if weight is None else np.asarray(weight, dtype=np.float64))
    dx = rstd * (a - r * rstd ** 2 * (a * r).mean(-1, keepdims=True))
    return dx + (0.0 if grad_r is None else np.asarray(grad_r, dtype=np.float64)), (dy * r * rstd).sum(0)


# ------------------------------------------------------------------ gated

def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def silu(x):
    return x * sigmoid(x)


def gated(x, w_gu):
    """(h, gate, up)."""
    gu = np.asarray(x, dtype=np.float64) @ np.asarray(w_gu, dtype=np.float64).T
    gate, up = np.split(gu, 2, -1)
    return silu(gate) * up, gate, up


def gated_grad(x, w_gu, grad_h):
    """(grad_x, grad_w_gu, d)."""
    _, gate, up = gated(x, w_gu)
    dh = np.asarray(grad_h, dtype=np.float64)
    s = sigmoid(gate)
    d = np.concatenate((dh * up * s * (1.0 + gate * (1.0 - s)), dh * gate * s), -1)
    return d @ np.asarray(w_gu, dtype=np.float64), d.T @ np.asarray(x, dtype=np.float64), d
