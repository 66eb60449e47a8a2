"""Plain numpy fp64 definitions of the scored router and of the 4-bit
microscaled operators, for the tests.  Nothing here is shared with the library
or its binding."""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = {"nv": 16, "mx": 32}


# ------------------------------------------------------------------ router

def scores(logits, score):
    """fp64 scores [n, E]; a logit that is not finite has score 0."""
    x = np.asarray(logits, dtype=np.float64)
    ok = np.isfinite(x)
    x = np.where(ok, x, 0.0)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return np.where(ok, 1.0 / (1.0 + np.exp(-x)), 0.0), ok
    out = np.zeros_like(x)
    for t in range(x.shape[0]):
        if ok[t].any():
            v = np.exp(x[t] - x[t][ok[t]].max()) * ok[t]
            out[t] = v / v.sum()
    return out, ok


def router(logits, top_k, score="sigmoid", bias=None, groups=1, top_groups=1, renormalize=True, scale=1.0):
    """(ids [n, top_k], weights [n, top_k], gap [n]): gap is the smallest
    distance, other than 0, between two values whose order decides the row."""
    s, ok = scores(logits, score)
    n, E = s.shape
    c = s if bias is None else s + np.asarray(bias, dtype=np.float64)
    c = np.where(ok & ~np.isnan(c), c, -np.inf)
    size = E // groups
    ids = np.zeros((n, top_k), dtype=np.int32)
    w = np.zeros((n, top_k))
    gap = np.full(n, np.inf)

    def closest(values):
        """Smallest positive step down a sorted list."""
        with np.errstate(invalid="ignore"):
            d = -np.diff(values)
        return d[d > 0].min() if (d > 0).any() else np.inf

    for t in range(n):
        key = c[t].copy()
        if groups > 1:
            value = np.zeros(groups)
            for g in range(groups):
                two = np.sort(key[g * size:(g + 1) * size])[::-1][:2]
                value[g] = two.sum() if not np.isnan(two.sum()) else -np.inf
            order = sorted(range(groups), key=lambda g: (-value[g], g))
            # which group is the last to stay decides
            gap[t] = min(gap[t], closest(value[order][top_groups - 1:top_groups + 1]))
            for g in order[top_groups:]:
                key[g * size:(g + 1) * size] = -np.inf
        order = sorted(range(E), key=lambda e: (-key[e], e))
        # the order of the chosen, and the first that is not
        gap[t] = min(gap[t], closest(key[order][:top_k + 1]))
        ids[t] = order[:top_k]
        w[t] = np.where(key[ids[t]] > -np.inf, s[t, ids[t]], 0.0)
        if renormalize:
            total = w[t].sum()
            w[t] = w[t] / total if total > 0 else 0.0
    return ids, w * scale, gap


def router_weights(logits, ids, live, score, renormalize, scale):
    """Weights of a fixed choice (for differences): `live` marks real choices."""
    s, _ = scores(logits, score)
    w = np.take_along_axis(s, ids.astype(np.int64), 1) * live
    if renormalize:
        total = w.sum(1, keepdims=True)
        w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    return w * scale


def router_backward(logits, ids, live, grad_w, score, renormalize, scale):
    """Gradient of the logits from the formula."""
    s, _ = scores(logits, score)
    i = ids.astype(np.int64)
    p = np.take_along_axis(s, i, 1) * live
    g = np.asarray(grad_w, dtype=np.float64) * live * scale
    if renormalize:
        total = p.sum(1, keepdims=True)
        safe = np.where(total > 0, total, 1.0)
        g = np.where(total > 0, (g - (g * p).sum(1, keepdims=True) / safe) / safe, 0.0) * live
    dp = np.zeros_like(s)
    np.put_along_axis(dp, i, g, 1)
    if score == "sigmoid":
        return dp * s * (1.0 - s)
    return s * (dp - (g * p).sum(1, keepdims=True))


# ------------------------------------------------------------------ 4-bit values

def e4m3(v):
    """Nearest E4M3 value (ties to even), saturating at 448."""
    v = np.minimum(np.asarray(v, dtype=np.float64), 448.0)
    e = np.maximum(np.floor(np.log2(np.maximum(v, 2.0 ** -30))), -6.0)
    step = np.exp2(e - 3.0)
    return np.minimum(np.round(v / step) * step, 448.0)


def e4m3_byte(v):
    v = np.asarray(v, dtype=np.float64)
    e = np.floor(np.log2(np.maximum(v, 2.0 ** -30)))
    normal = ((e + 7).astype(int) << 3) + np.round((v / np.exp2(e) - 1.0) * 8).astype(int)
    return np.where(v < 2.0 ** -6, np.round(v * 2.0 ** 9).astype(int), normal).astype(np.uint8)


def quantize(x, fmt, g=1.0):
    """(codes [n, K] with the sign in bit 3, scale bytes [n, K/B], values [n, K])."""
    B = BLOCK[fmt]
    x = np.asarray(x, dtype=np.float64)
    n, K = x.shape
    big = float(np.finfo(np.float32).max)
    v = np.where(np.isnan(x), 0.0, np.clip(x, -big, big)).reshape(n, K // B, B)
    top = np.abs(v).max(-1)
    if fmt == "nv":
        s = e4m3(top / (6.0 * g))
        byte = e4m3_byte(s)
        d = s * g
    else:
        e = np.where(top > 0, np.floor(np.log2(np.where(top > 0, top, 1.0))) - 2.0, -127.0)
        e = np.clip(e, -127.0, 127.0)
        byte = (e + 127).astype(np.uint8)
        d = np.exp2(e)
    q = np.abs(v) / np.where(d > 0, d, 1.0)[..., None]
    # nearest grid value (saturating), the even code on a tie
    q = np.minimum(q, 8.0)
    dist = np.abs(q[..., None] - E2M1)
    code = dist.argmin(-1)
    up = np.minimum(code + 1, 7)
    tie = (np.take_along_axis(dist, code[..., None], -1) == np.take_along_axis(dist, up[..., None], -1))[..., 0]
    code = np.where(tie & (up != code) & (code % 2 == 1), up, code)
    values = np.where(d[..., None] > 0, E2M1[code] * np.sign(v) * d[..., None], 0.0)
    code = np.where(d[..., None] > 0, code | (np.signbit(v).astype(int) << 3), 0)
    return code.reshape(n, K).astype(np.uint8), byte, values.reshape(n, K)


def pack(code):
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def dequantize(packed, byte, fmt, g=1.0):
    """fp64 values of packed codes [..., K/2] and scale bytes [..., K/B]."""
    code = np.stack((packed & 15, packed >> 4), -1).reshape(*packed.shape[:-1], -1)
    v = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    b = byte.astype(np.float64)
    if fmt == "nv":
        e, m = np.floor(b / 8), b % 8
        s = np.where(e > 0, (1 + m / 8) * np.exp2(e - 7), m / 8 * 2.0 ** -6) * g
    else:
        s = np.exp2(b - 127.0)
    return v * np.repeat(s, BLOCK[fmt], -1)


def tile_scales(byte, fmt):
    """Row-major scale bytes [E, N, K/B] in the products' tiled layout (1-D), by its formula."""
    E, N, kb = byte.shape
    step = 256 // BLOCK[fmt]
    rows, blocks = -(-N // 128) * 128, -(-kb // step) * step
    out = np.zeros((E, rows // 128, blocks // 4, 512), dtype=np.uint8)
    for r in range(N):
        for b in range(kb):
            out[:, r // 128, b // 4, (r % 32) * 16 + (r % 128 // 32) * 4 + b % 4] = byte[:, r, b]
    return out.reshape(-1)


def moe(xq, ids, w, matrices):
    """(y, sum of magnitudes): y_t = sum_j w_tj W_e x_t; ids out of range add nothing."""
    n, k = ids.shape
    E, N, _ = matrices.shape
    y, mag = np.zeros((n, N)), np.zeros((n, N))
    for t in range(n):
        for j in range(k):
            e = ids[t, j]
            if 0 <= e < E:
                y[t] += float(w[t, j]) * (matrices[e] @ xq[t])
                mag[t] += abs(float(w[t, j])) * (np.abs(matrices[e]) @ np.abs(xq[t]))
    return y, mag
