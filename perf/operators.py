"""Cases that time and compare the routing, quantisation and 4-bit product operators.

Each case stands for a call of a served (or, for the router's gradient, trained)
mixture-of-experts layer.  `run` computes it either from elementary torch
operations in 32 bits (own = False) or by the calls a user makes (own = True).

Definitions, shared by the plain forms below and by `exact`:

router    s = sigmoid(x) or softmax(x) over the E experts; a logit that is not
          finite has score 0 and is never chosen before a finite one.  Choice
          goes by c = s + bias: the experts fall into `groups` equal groups, a
          group's score is the sum of its two largest c, the best `top_groups`
          groups stay, and the top_k largest c among them are taken (ties to
          the lower index).  Weights are the s of the chosen, divided by their
          sum when renormalised, times `scale`.
quantise  blocks along a row share a scale.  "nv": 16 values, scale
          e4m3(max|x| / (6 g)), g one 32-bit scale for the whole tensor; "mx":
          32 values, scale 2^(floor(log2 max|x|) - 2).  A value is kept as the
          nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 (ties to even, saturating),
          with its sign, of x / (scale g).
products  y = W x with both sides so quantised (the weights before the call,
          the activations in it), and for experts y_t = sum_j w_tj W_e(t,j) x_t.
"""
import math

import torch

own = False

BLOCK = {"nv": 16, "mx": 32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
TYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
SIZES = {"float32": 4, "bfloat16": 2, "float16": 2}


# ------------------------------------------------------------------ cases

def _router(name, n, E, k, score, groups, top_groups, bias, renorm, scale, dtype, grad=False):
    return {"name": name, "kind": "router_grad" if grad else "router", "n": n, "E": E, "k": k, "score": score,
            "groups": groups, "top_groups": top_groups, "bias": bias, "renorm": renorm, "scale": scale,
            "dtype": dtype}


def listed():
    return [
        # one token of a decode step: nothing but latency
        _router("route 1 token", 1, 256, 6, "sigmoid", 8, 4, True, True, 2.5, "float32"),
        # a prefill batch through the grouped, bias-balanced router
        _router("route 8192 tokens", 8192, 256, 6, "sigmoid", 8, 4, True, True, 2.5, "float32"),
        # softmax scores over a count of experts that is no power of two, bf16 logits
        _router("route 1001 softmax of 160", 1001, 160, 6, "softmax", 1, 1, True, False, 1.0, "bfloat16"),
        # the router's gradient in a training step, dense through the softmax
        _router("route gradient softmax", 8192, 256, 6, "softmax", 1, 1, False, True, 1.0, "float32", True),
        # the same through sigmoid scores: only the chosen experts have one
        _router("route gradient sigmoid", 683, 256, 8, "sigmoid", 8, 4, True, True, 2.5, "bfloat16", True),
        # a decode batch's activations, quantised and read back
        {"name": "quantise 32 rows mx", "kind": "quantise", "n": 32, "K": 4096, "fmt": "mx", "dtype": "bfloat16"},
        # a prefill batch's activations
        {"name": "quantise 8192 rows nv", "kind": "quantise", "n": 8192, "K": 4096, "fmt": "nv", "dtype": "bfloat16"},
        # a shared expert's projection at a decode step
        {"name": "linear 1 row", "kind": "linear", "n": 1, "K": 4096, "N": 2048, "fmt": "nv", "dtype": "bfloat16"},
        # the same in a prefill, a ragged batch and an output width that fills no tile
        {"name": "linear 3001 rows mx", "kind": "linear", "n": 3001, "K": 2048, "N": 4099, "fmt": "mx",
         "dtype": "bfloat16"},
        # routed experts: a single token, a decode batch, a prefill
        {"name": "experts 1 token", "kind": "experts", "n": 1, "E": 256, "k": 6, "K": 4096, "N": 2048, "fmt": "nv",
         "dtype": "bfloat16"},
        {"name": "experts 32 tokens", "kind": "experts", "n": 32, "E": 256, "k": 6, "K": 4096, "N": 2048,
         "fmt": "mx", "dtype": "bfloat16"},
        {"name": "experts 8192 tokens", "kind": "experts", "n": 8192, "E": 256, "k": 6, "K": 4096, "N": 2048,
         "fmt": "nv", "dtype": "bfloat16"},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, most):
    """A row length: a power of two, or an odd multiple of 32."""
    if rng.random() < 0.5:
        return 1 << rng.randint(8, int(math.log2(most)))
    return 32 * (_spread(rng, 8, most // 32 - 1) | 1)


def draw(rng):
    kind = rng.choice(("router", "router", "router_grad", "quantise", "linear", "experts", "experts"))
    dtype = rng.choice(("float32", "bfloat16", "float16"))
    if kind in ("router", "router_grad"):
        groups = rng.choice((1, 1, 4, 8))
        E = groups * rng.randint(2, 512 // groups)
        top_groups = rng.randint((groups + 1) // 2, groups)
        k = rng.randint(1, min(16, top_groups * (E // groups)))
        n = _spread(rng, 1, 8192)
        return {"kind": kind, "n": n if n < 64 else n | 1, "E": E, "k": k, "score": rng.choice(("sigmoid", "softmax")),
                "groups": groups, "top_groups": top_groups, "bias": rng.random() < 0.6,
                "renorm": rng.random() < 0.6, "scale": rng.choice((1.0, 2.5)), "dtype": dtype}
    fmt = rng.choice(("nv", "mx"))
    if kind == "quantise":
        n = _spread(rng, 1, 8191)
        return {"kind": kind, "n": n if n < 64 else n | 1, "K": _width(rng, 4096), "fmt": fmt, "dtype": dtype}
    n = _spread(rng, 1, 8191)
    n = n if n < 64 else n | 1
    K = _width(rng, 4096)
    N = rng.choice((256, 2048, 4096, 2 * rng.randint(64, 2048) + 1))
    if kind == "linear":
        return {"kind": kind, "n": n, "K": K, "N": N, "fmt": fmt, "dtype": dtype}
    E, k = rng.choice(((8, 2), (64, 6), (256, 6), (256, 8), (160, 6)))
    N = rng.choice((256, 2048, 2 * rng.randint(64, 1023) + 1))
    return {"kind": kind, "n": min(n, 8192 * 6 // k), "E": E, "k": k, "K": K, "N": N, "fmt": fmt, "dtype": dtype}


# ------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activations(n, K, dtype, g):
    """Rows as a norm leaves them: unit spread, some channels several times larger."""
    channel = torch.exp(0.5 * torch.randn(K, device="cuda", generator=g))
    return (torch.randn((n, K), device="cuda", generator=g) * channel).to(dtype)


def _weights(E, N, K, fmt, g):
    """E matrices N(0, 1/K), quantised: packed bytes, block scales row by row and in
    the 128-row tiles the product reads, and one 32-bit scale per matrix ("nv")."""
    B = BLOCK[fmt]
    packed = torch.empty((E, N, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((E, N, K // B), dtype=torch.uint8, device="cuda")
    w_scale = torch.empty(E, dtype=torch.float32, device="cuda") if fmt == "nv" else None
    for e in range(E):
        w = torch.randn((N, K), device="cuda", generator=g) * (1.0 / math.sqrt(K))
        gs = None
        if fmt == "nv":
            gs = w_scale[e:e + 1]
            gs.copy_(w.abs().max() / (6.0 * 448.0))
        code, byte, _ = _quantise(w, fmt, gs)
        packed[e] = code[:, 0::2] | (code[:, 1::2] << 4)
        scales[e] = byte
    return packed, scales, _tiles(scales, fmt), w_scale


def _tiles(scales, fmt):
    """Block scales [E, N, K/B] as tiles of 128 rows x 4 blocks of 512 bytes, byte
    (row % 32) * 16 + (row / 32) * 4 + block, rows padded to 128 and columns to
    256 values with zeros."""
    E, N, kb = scales.shape
    step = 256 // BLOCK[fmt]
    full = torch.zeros((E, -(-N // 128) * 128, -(-kb // step) * step), dtype=torch.uint8, device=scales.device)
    full[:, :N, :kb] = scales
    full = full.view(E, full.shape[1] // 128, 4, 32, full.shape[2] // 4, 4)
    return full.permute(0, 1, 4, 3, 2, 5).contiguous()


def _x_scale(fmt):
    # what calibration gives for the largest activation that it saw
    return torch.full((1,), 11.37 / (6.0 * 448.0), dtype=torch.float32, device="cuda") if fmt == "nv" else None


def _logits(n, E, dtype, g):
    popular = 0.3 * torch.randn(E, device="cuda", generator=g)
    return (torch.randn((n, E), device="cuda", generator=g) + popular).to(dtype)


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    if case["kind"] in ("router", "router_grad"):
        s["logits"] = _logits(case["n"], case["E"], TYPES[case["dtype"]], g)
        s["bias"] = 0.05 * torch.randn(case["E"], device="cuda", generator=g) if case["bias"] else None
        if case["kind"] == "router_grad":
            s["ids"], s["w"] = _route(s)
            s["grad_w"] = torch.randn((case["n"], case["k"]), device="cuda", generator=g)
        return s
    s["x"] = _activations(case["n"], case["K"], TYPES[case["dtype"]], g)
    s["x_scale"] = _x_scale(case["fmt"])
    if case["kind"] == "quantise":
        return s
    E = case.get("E", 1)
    s["packed"], s["scales"], s["tiles"], s["w_scale"] = _weights(E, case["N"], case["K"], case["fmt"], g)
    if case["kind"] == "experts":
        s["ids"], s["w"] = _route({"logits": _logits(case["n"], E, torch.float32, g), "bias": None, "score": "softmax",
                                   "k": case["k"], "groups": 1, "top_groups": 1, "renorm": True, "scale": 1.0})
    else:
        s["packed"], s["scales"], s["tiles"] = s["packed"][0], s["scales"][0], s["tiles"][0]
    return s


# ------------------------------------------------------------------ plain forms

def _pairwise(t):
    """The sum over the last axis as a balanced tree of neighbours (a power of two of them)."""
    return t[..., 0] if t.shape[-1] == 1 else _pairwise(t[..., 0::2] + t[..., 1::2])


def _scores(logits, score):
    x = logits.float()
    ok = torch.isfinite(x)
    if score == "sigmoid":
        return torch.where(ok, 1.0 / (1.0 + torch.exp(-x)), 0.0), ok
    x = torch.where(ok, x, -math.inf)
    top = x.max(-1, keepdim=True).values
    e = torch.where(ok, torch.exp(x - top), 0.0)
    E = e.shape[-1]
    total = _pairwise(torch.nn.functional.pad(e, (0, (1 << (E - 1).bit_length()) - E)))[..., None]
    return torch.where(ok, e / total, 0.0), ok


def _route(s):
    score, ok = _scores(s["logits"], s["score"])
    c = score if s["bias"] is None else score + s["bias"]
    c = torch.where(ok & (c == c), c, -math.inf)
    if s["groups"] > 1:
        n, E = c.shape
        size = E // s["groups"]
        grouped = c.view(n, s["groups"], size)
        value = torch.sort(grouped, dim=-1, descending=True).values[..., :2].sum(-1)
        value = torch.where(value == value, value, -math.inf)
        best = torch.sort(value, dim=-1, descending=True, stable=True).indices[:, : s["top_groups"]]
        keep = torch.zeros_like(value, dtype=torch.bool).scatter_(1, best, True)
        c = torch.where(keep[..., None], grouped, -math.inf).view(n, E)
    value, ids = torch.sort(c, dim=-1, descending=True, stable=True)
    value, ids = value[:, : s["k"]], ids[:, : s["k"]]
    w = torch.where(value > -math.inf, score.gather(1, ids), 0.0)
    if s["renorm"]:
        total = w.sum(-1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return ids.to(torch.int32), w * s["scale"]


def _route_grad(s):
    score, ok = _scores(s["logits"], s["score"])
    ids = s["ids"].long()
    live = s["w"] != 0
    p = torch.where(live, score.gather(1, ids), 0.0)
    grad = torch.where(live, s["grad_w"], 0.0) * s["scale"]
    if s["renorm"]:
        total = p.sum(-1, keepdim=True)
        grad = torch.where(total > 0, (grad - (grad * p).sum(-1, keepdim=True) / total) / total, 0.0)
        grad = torch.where(live, grad, 0.0)
    if s["score"] == "sigmoid":
        out = torch.zeros_like(score).scatter_(1, ids, grad * p * (1.0 - p))
    else:
        dense = torch.zeros_like(score).scatter_(1, ids, grad)
        out = score * (dense - (grad * p).sum(-1, keepdim=True))
    return out.to(s["logits"].dtype)


def _code(a):
    """The E2M1 code (0 to 7) of magnitudes a: the nearest value, ties to even."""
    return ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))


def _power_of_two(byte):
    """2^(byte - 127) in 32 bits, from its bits: byte is the biased exponent (0 is half of the smallest normal number)."""
    b = byte.int()
    return torch.where(b > 0, b << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _quantise(x, fmt, scale):
    """Codes [n, K] with the sign in bit 3, scale bytes [n, K/B] and the scales in 32 bits."""
    B = BLOCK[fmt]
    n, K = x.shape
    x = torch.nan_to_num(x.float(), nan=0.0).view(n, K // B, B)
    top = x.abs().amax(-1)
    if fmt == "nv":
        g = 1.0 if scale is None else scale
        e4m3 = torch.clamp(top / (6.0 * g), max=448.0).to(torch.float8_e4m3fn)
        byte, value = e4m3.view(torch.uint8), e4m3.float()
        d = value * g
    else:
        exponent = torch.clamp(torch.frexp(top).exponent - 3, -127, 127)
        exponent = torch.where(top > 0, exponent, -127)
        byte = (exponent + 127).to(torch.uint8)
        d = value = _power_of_two(byte)
    q = x / d[..., None]
    code = torch.where(d[..., None] > 0, _code(q.abs()) | (torch.signbit(q).to(torch.uint8) << 3), 0)
    return code.to(torch.uint8).view(n, K), byte, value


def _values(code):
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=code.device)
    return table[code.int()]


def _dequantised(x, fmt, scale):
    code, _, value = _quantise(x, fmt, scale)
    n, K = code.shape
    v = _values(code).view(n, K // BLOCK[fmt], BLOCK[fmt]) * value[..., None]
    return (v if scale is None else v * scale).view(n, K)


def _scale_values(byte, fmt):
    return byte.view(torch.float8_e4m3fn).float() if fmt == "nv" else _power_of_two(byte)


def _weight_values(packed, scales, fmt, w_scale):
    """Matrices [.., N, K] in 32 bits."""
    pair = torch.stack((packed & 15, packed >> 4), -1)
    v = _values(pair).view(*scales.shape, BLOCK[fmt])
    s = _scale_values(scales, fmt)
    if w_scale is not None:
        s = s * w_scale.view(*w_scale.shape, *(1,) * (s.dim() - w_scale.dim()))
    v.mul_(s[..., None])
    return v.view(*packed.shape[:-1], packed.shape[-1] * 2)


def _experts(s):
    x = _dequantised(s["x"], s["fmt"], s["x_scale"])
    n, k = s["ids"].shape
    flat = s["ids"].reshape(-1).long()
    if n * k <= s["E"]:
        # few pairs: the matrices of each pair
        ws = None if s["w_scale"] is None else s["w_scale"][flat]
        m = _weight_values(s["packed"][flat], s["scales"][flat], s["fmt"], ws)
        y = torch.matmul(m, x.repeat_interleave(k, 0)[..., None])[..., 0]
    else:
        # many: each expert's rows side by side, padded to the fullest expert's count
        order = torch.argsort(flat, stable=True)
        counts = torch.bincount(flat, minlength=s["E"])
        first = torch.cumsum(counts, 0) - counts
        place = torch.arange(n * k, device=flat.device) - first[flat[order]]
        rows = torch.zeros((s["E"], int(counts.max()), x.shape[1]), device=x.device)
        rows[flat[order], place] = x[order // k]
        out = torch.matmul(rows, _weight_values(s["packed"], s["scales"], s["fmt"], s["w_scale"]).transpose(1, 2))
        y = torch.empty((n * k, out.shape[2]), device=x.device)
        y[order] = out[flat[order], place]
    return (y.view(n, k, -1) * s["w"][..., None]).sum(1).to(s["x"].dtype)


def _plain(s):
    kind = s["kind"]
    if kind == "router":
        ids, w = _route(s)
        return {"ids": ids, "w": w}
    if kind == "router_grad":
        return {"grad_logits": _route_grad(s)}
    if kind == "quantise":
        return {"values": _dequantised(s["x"], s["fmt"], s["x_scale"]).to(torch.bfloat16)}
    if kind == "linear":
        w = _weight_values(s["packed"], s["scales"], s["fmt"], s["w_scale"])
        return {"y": (_dequantised(s["x"], s["fmt"], s["x_scale"]) @ w.t()).to(s["x"].dtype)}
    return {"y": _experts(s)}


# ------------------------------------------------------------------ the framework's calls

def _own(s):
    import trellis_quantized_moe_sort_gb300 as tq

    kind = s["kind"]
    if kind in ("router", "router_grad"):
        score = tq.SCORE_SIGMOID if s["score"] == "sigmoid" else tq.SCORE_SOFTMAX
        if kind == "router":
            ids, w = tq.tq_router_scored(s["logits"], s["k"], score=score, bias=s["bias"], groups=s["groups"],
                                         top_groups=s["top_groups"], renormalize=s["renorm"], scale=s["scale"])
            return {"ids": ids, "w": w}
        return {"grad_logits": tq.tq_router_scored_backward(s["logits"], s["ids"], s["w"], s["grad_w"], score=score,
                                                            renormalize=s["renorm"], scale=s["scale"])}
    fmt = tq.FP4_NV if s["fmt"] == "nv" else tq.FP4_MX
    if kind == "quantise":
        packed, scales = tq.tq_fp4_quantize(s["x"], fmt=fmt, global_scale=s["x_scale"])
        return {"values": tq.tq_fp4_dequantize(packed, scales, fmt=fmt, global_scale=s["x_scale"],
                                               dtype=torch.bfloat16)}
    if kind == "linear":
        return {"y": tq.tq_fp4_linear(s["x"], s["packed"], s["tiles"], fmt=fmt, w_scale=s["w_scale"],
                                      x_scale=s["x_scale"])}
    return {"y": tq.tq_fp4_moe_forward(s["x"], s["packed"], s["tiles"], s["ids"], s["w"], fmt=fmt,
                                       w_scale=s["w_scale"], x_scale=s["x_scale"])}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ work

def work(case):
    size = SIZES[case["dtype"]]
    n = case["n"]
    if case["kind"] == "router":
        E, k = case["E"], case["k"]
        return {"bytes": n * E * size + n * k * 8 + (4 * E if case["bias"] else 0), "flops": 8 * n * E}
    if case["kind"] == "router_grad":
        E, k = case["E"], case["k"]
        read = n * E * size if case["score"] == "softmax" else n * k * size
        return {"bytes": read + n * E * size + n * k * 12, "flops": 8 * n * E}
    K, B = case["K"], BLOCK[case["fmt"]]
    held = K // 2 + K // B
    if case["kind"] == "quantise":
        return {"bytes": n * (K * size + 2 * held + 2 * K), "flops": 4 * n * K}
    N = case["N"]
    if case["kind"] == "linear":
        return {"bytes": n * K * size + N * held + n * N * size, "flops": 2 * n * N * K}
    E, k = case["E"], case["k"]
    woken = E * (1.0 - (1.0 - k / E) ** n)
    return {"bytes": n * K * size + woken * N * held + n * k * 8 + n * N * size, "flops": 2 * n * k * N * K}


# ------------------------------------------------------------------ 64 bits

def _exact_scores(logits, score):
    x = logits.double()
    x = torch.where(torch.isfinite(x), x, -math.inf)
    return torch.sigmoid(x) if score == "sigmoid" else torch.nan_to_num(torch.softmax(x, -1))


def _exact_grid(a):
    """Nearest E2M1 magnitude by distance: twice the mantissa step below 2, then 1, then 2."""
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0)).double()
    return torch.clamp(torch.round(a / step) * step, max=6.0)


def _exact_power(k):
    """2^k in 64 bits, from its bits."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def _exact_quantised(x, fmt, scale):
    B = BLOCK[fmt]
    n, K = x.shape
    v = x.double().reshape(n, K // B, B)
    top = v.abs().amax(-1, keepdim=True)
    if fmt == "nv":
        g = scale.double()
        t = torch.clamp(top / (6.0 * g), max=448.0)
        # e4m3: 3 mantissa bits, the smallest step 2^-9
        step = _exact_power(torch.clamp(torch.frexp(t).exponent - 1, min=-6) - 3)
        d = torch.clamp(torch.round(t / step) * step, max=448.0) * g
    else:
        d = _exact_power(torch.clamp(torch.frexp(top).exponent - 1 - 2, min=-127))
    safe = torch.where(d > 0, d, 1.0)
    q = _exact_grid(v.abs() / safe) * torch.sign(v)
    return torch.where(d > 0, q * safe, 0.0).reshape(n, K)


def _exact_matrix(packed, scales, fmt, w_scale):
    low, high = (packed & 15).double(), (packed >> 4).double()
    c = torch.stack((low, high), -1).reshape(packed.shape[0], -1)
    mag = c % 8
    e, m = torch.floor(mag / 2), mag % 2
    v = torch.where(e > 0, (1.0 + m / 2) * _exact_power(e - 1.0), m / 2)
    v = torch.where(c >= 8, -v, v)
    b = scales.double()
    if fmt == "nv":
        be, bm = torch.floor(b / 8), b % 8
        s = torch.where(be > 0, (1.0 + bm / 8) * _exact_power(be - 7.0), bm / 8 * 2.0 ** -6)
        s = s * w_scale.double()
    else:
        s = _exact_power(b - 127.0)
    return v * s.repeat_interleave(BLOCK[fmt], 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "router":
        p = _exact_scores(s["logits"], case["score"])
        c = p if s["bias"] is None else p + s["bias"].double()
        n, E = p.shape
        G = case["groups"]
        if G > 1:
            size = E // G
            value = torch.topk(c.view(n, G, size), min(2, size), -1).values.sum(-1)
            bound = torch.topk(value, case["top_groups"], -1).values[:, -1:]
            c = torch.where((value >= bound).repeat_interleave(size, 1), c, -1e300)
        w = p.gather(1, torch.topk(c, case["k"], -1).indices)
        if case["renorm"]:
            w = w / w.sum(-1, keepdim=True)
        return {"ids": None, "w": w * case["scale"]}
    if case["kind"] == "router_grad":
        x = s["logits"].double().requires_grad_(True)
        p = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, -1)
        w = p.gather(1, s["ids"].long())
        if case["renorm"]:
            w = w / w.sum(-1, keepdim=True)
        return {"grad_logits": torch.autograd.grad((w * case["scale"] * s["grad_w"].double()).sum(), x)[0]}
    x = _exact_quantised(s["x"], case["fmt"], s["x_scale"])
    if case["kind"] == "quantise":
        return {"values": x}
    if case["kind"] == "linear":
        return {"y": x @ _exact_matrix(s["packed"], s["scales"], case["fmt"], s["w_scale"]).t()}
    y = torch.zeros((case["n"], case["N"]), dtype=torch.float64, device=x.device)
    for e in range(case["E"]):
        t, j = torch.nonzero(s["ids"] == e, as_tuple=True)
        if t.numel():
            m = _exact_matrix(s["packed"][e], s["scales"][e], case["fmt"],
                              None if s["w_scale"] is None else s["w_scale"][e])
            y.index_add_(0, t, (x[t] @ m.t()) * s["w"][t, j].double()[:, None])
    return {"y": y}
