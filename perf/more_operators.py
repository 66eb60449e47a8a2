"""Cases that time and compare the norm, the 8-bit block-scaled products and the gated projection.

Each case stands for a call of a served (or, for the gradients, trained)
mixture-of-experts layer.  `run` computes it either from elementary torch
operations in 32 bits (own = False) or by the calls a user makes (own = True).

Definitions, shared by the plain forms below and by `exact`:

norm      r = x + residual, rounded to x's type and kept; rstd = 1 / sqrt(mean(r^2) + eps);
          y = r rstd w.  Kept in 8 bits where the next product reads it so, else in x's type.
          Its gradient: with a = grad_y w, grad_x = rstd (a - r rstd^2 mean(a r)) + grad_r
          and grad_w = sum over rows of grad_y r rstd.
8 bits    128 values of a row (activations) or 128 x 128 of a matrix (weights) share a scale
          s = max|x| / 448, rounded to 32 bits; a value is kept as e4m3(x / s), the quotient
          rounded to 32 bits first (16-bit values often fall on a border of the e4m3 grid).
products  y = W x with both sides so kept (the weights before the call), for experts
          y_t = sum_j w_tj W_e(t,j) x_t, and for SwiGLU experts
          h = silu(Wg x) * (Wu x) per pair, kept in 8 bits, y_t = sum_j w_tj Wd h_tj.
gated     h = silu(x Wg^T) * (x Wu^T), one 16-bit matrix Wg over Wu, and its gradients.
"""
import math

import torch

own = False

BLOCK = 128
MOST = 448.0   # the largest e4m3 value
EPS = 1e-6
TYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
SIZES = {"float32": 4, "bfloat16": 2, "float16": 2}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token between two blocks of a decode step: nothing but latency
        {"name": "norm 1 token", "kind": "norm", "n": 1, "K": 4096, "dtype": "bfloat16"},
        # the same over a prefill batch
        {"name": "norm 8192 rows", "kind": "norm", "n": 8192, "K": 4096, "dtype": "bfloat16"},
        # a training step's norm, forward and backward, a ragged batch
        {"name": "norm training 4095 rows", "kind": "norm_train", "n": 4095, "K": 4096, "dtype": "bfloat16"},
        # a shared expert's or an attention projection at a decode step
        {"name": "linear 1 row", "kind": "linear", "n": 1, "K": 4096, "N": 2048, "dtype": "bfloat16"},
        # a ragged batch and an output width that fills no tile
        {"name": "linear 3001 rows", "kind": "linear", "n": 3001, "K": 2048, "N": 4099, "dtype": "bfloat16"},
        # a prefill batch
        {"name": "linear 8192 rows", "kind": "linear", "n": 8192, "K": 4096, "N": 4096, "dtype": "bfloat16"},
        # routed experts: a decode batch, a prefill
        {"name": "experts 32 tokens", "kind": "experts", "n": 32, "E": 256, "k": 6, "K": 4096, "N": 2048,
         "dtype": "bfloat16"},
        {"name": "experts 8192 tokens", "kind": "experts", "n": 8192, "E": 256, "k": 6, "K": 4096, "N": 2048,
         "dtype": "bfloat16"},
        # SwiGLU experts: a single token, a prefill
        {"name": "expert MLP 1 token", "kind": "mlp", "n": 1, "E": 64, "k": 6, "H": 4096, "I": 2048,
         "dtype": "bfloat16"},
        {"name": "expert MLP 2048 tokens", "kind": "mlp", "n": 2048, "E": 64, "k": 6, "H": 4096, "I": 2048,
         "dtype": "bfloat16"},
        # a shared expert's gated projection in 16 bits at a decode batch
        {"name": "gated 16 rows", "kind": "gated", "n": 16, "H": 4096, "I": 2048, "dtype": "bfloat16"},
        # the same in a training step, forward and backward
        {"name": "gated training 8192 rows", "kind": "gated_train", "n": 8192, "H": 4096, "I": 2048,
         "dtype": "bfloat16"},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, most, unit):
    """A row length: a power of two, or an odd multiple of `unit`."""
    if rng.random() < 0.5:
        return 1 << rng.randint(8, int(math.log2(most)))
    return unit * (_spread(rng, 256 // unit, most // unit - 1) | 1)


def draw(rng):
    kind = rng.choice(("norm", "norm_train", "linear", "linear", "experts", "experts", "mlp", "gated", "gated_train"))
    n = _spread(rng, 1, 8191)
    n = n if n < 64 else n | 1
    if kind == "norm":
        return {"kind": kind, "n": n, "K": _width(rng, 8192, 16), "dtype": rng.choice(tuple(TYPES))}
    if kind == "norm_train":
        return {"kind": kind, "n": n, "K": _width(rng, 8192, 1), "dtype": rng.choice(tuple(TYPES))}
    if kind in ("gated", "gated_train"):
        return {"kind": kind, "n": n, "H": _width(rng, 4096, 8), "I": _width(rng, 2048, 8),
                "dtype": rng.choice(("bfloat16", "float16"))}
    dtype = rng.choice(tuple(TYPES))
    if kind == "linear":
        return {"kind": kind, "n": n, "K": _width(rng, 4096, 16),
                "N": rng.choice((256, 2048, 4096, 2 * rng.randint(64, 2048) + 1)), "dtype": dtype}
    if kind == "experts":
        E, k = rng.choice(((8, 2), (64, 6), (256, 6), (256, 8), (160, 6)))
        return {"kind": kind, "n": min(n, 8192 * 6 // k), "E": E, "k": k, "K": _width(rng, 4096, 16),
                "N": rng.choice((256, 2048, 2 * rng.randint(64, 1023) + 1)), "dtype": dtype}
    # 16-bit results alone: a value of h next to a border of its 8 bits falls to either side by the last bits of a sum
    E, k = rng.choice(((8, 2), (64, 6), (64, 4), (32, 3)))
    return {"kind": kind, "n": min(n, 2048), "E": E, "k": k, "H": _width(rng, 4096, 16),
            "I": 128 * rng.randint(1, 16), "dtype": rng.choice(("bfloat16", "float16"))}


# ------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activations(n, K, dtype, g):
    """Rows as a norm leaves them: unit spread, some channels several times larger."""
    channel = torch.exp(0.5 * torch.randn(K, device="cuda", generator=g))
    return (torch.randn((n, K), device="cuda", generator=g) * channel).to(dtype)


def _weights(E, N, K, g):
    """E matrices N(0, 1/K) in 8 bits: values [E, N, K] and scales [E, N / 128, K / 128]."""
    codes = torch.empty((E, N, K), dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty((E, -(-N // BLOCK), -(-K // BLOCK)), dtype=torch.float32, device="cuda")
    for e in range(E):
        w = torch.randn((N, K), device="cuda", generator=g) * (1.0 / math.sqrt(K))
        codes[e], scales[e] = _quantise(w, BLOCK)
    return codes, scales


def _routed(n, E, k, g):
    """The k best of E by their logits, some experts more popular, and their softmax weights."""
    popular = 0.3 * torch.randn(E, device="cuda", generator=g)
    value, ids = torch.sort(torch.randn((n, E), device="cuda", generator=g) + popular, dim=-1, descending=True)
    e = torch.exp(value[:, :k] - value[:, :1])
    return ids[:, :k].to(torch.int32).contiguous(), e / e.sum(-1, keepdim=True)


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    kind, n, dtype = case["kind"], case["n"], TYPES[case["dtype"]]
    if kind in ("norm", "norm_train"):
        K = case["K"]
        s["x"] = torch.randn((n, K), device="cuda", generator=g).to(dtype)
        s["residual"] = (3.0 * _activations(n, K, torch.float32, g)).to(dtype)
        s["weight"] = 1.0 + 0.1 * torch.randn(K, device="cuda", generator=g)
        if kind == "norm_train":
            s["grad_y"] = torch.randn((n, K), device="cuda", generator=g).to(dtype)
            s["grad_r"] = torch.randn((n, K), device="cuda", generator=g).to(dtype)
        return s
    if kind in ("gated", "gated_train"):
        H, I = case["H"], case["I"]
        s["x"] = _activations(n, H, dtype, g)
        s["w_gu"] = (torch.randn((2 * I, H), device="cuda", generator=g) * (1.0 / math.sqrt(H))).to(dtype)
        if kind == "gated_train":
            s["grad_h"] = torch.randn((n, I), device="cuda", generator=g).to(dtype)
        return s
    if kind == "mlp":
        s["x"] = _activations(n, case["H"], dtype, g)
        s["w_gu"], s["gu_scales"] = _weights(case["E"], 2 * case["I"], case["H"], g)
        s["w_down"], s["down_scales"] = _weights(case["E"], case["H"], case["I"], g)
    else:
        s["x"] = _activations(n, case["K"], dtype, g)
        s["w"], s["w_scales"] = _weights(case.get("E", 1), case["N"], case["K"], g)
        if kind == "linear":
            s["w"], s["w_scales"] = s["w"][0], s["w_scales"][0]
            return s
    s["ids"], s["topk_w"] = _routed(n, case["E"], case["k"], g)
    return s


# ------------------------------------------------------------------ plain forms

def _quantise(x, rows):
    """x [n, K] in blocks of `rows` x 128: e4m3 values [n, K] and scales [n / rows, K / 128]."""
    n, K = x.shape
    nb, kb = -(-n // rows), -(-K // BLOCK)
    v = torch.nn.functional.pad(x.float(), (0, kb * BLOCK - K, 0, nb * rows - n)).view(nb, rows, kb, BLOCK)
    top = v.abs().amax((1, 3), keepdim=True)
    s = top / torch.full_like(top, MOST)
    q = torch.where(s > 0, v / s, 0.0).to(torch.float8_e4m3fn)
    return q.view(nb * rows, kb * BLOCK)[:n, :K].contiguous(), s.view(nb, kb)


def _values(codes, scales, rows):
    """[.., n, K] in 32 bits."""
    n, K = codes.shape[-2:]
    wide = scales.repeat_interleave(rows, -2)[..., :n, :].repeat_interleave(BLOCK, -1)[..., :K]
    return codes.float().mul_(wide)


def _norm(s):
    r = (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
    v = r.float()
    # a row's sum of squares in 64 bits: codes go by y, next to a border by its last bit
    rstd = torch.rsqrt((v.double() ** 2).mean(-1, keepdim=True) + EPS).float()
    return r, v, rstd, v * rstd * s["weight"]


def _norm_grad(s, v, rstd):
    dy = s["grad_y"].float()
    a = dy * s["weight"]
    grad_x = rstd * (a - v * rstd * rstd * (a * v).mean(-1, keepdim=True)) + s["grad_r"].float()
    # over thousands of rows: in 64 bits
    return grad_x.to(s["x"].dtype), (dy * (v * rstd)).double().sum(0).float()


def _padded(rows, ids, E):
    """rows [P, K], one a pair, side by side for each expert, and where each pair went."""
    flat = ids.reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    counts = torch.bincount(flat, minlength=E)
    first = torch.cumsum(counts, 0) - counts
    place = torch.arange(flat.numel(), device=flat.device) - first[flat[order]]
    side = torch.zeros((E, int(counts.max()), rows.shape[1]), device=rows.device)
    side[flat[order], place] = rows[order]
    return side, (flat[order], place, order)


def _product(rows, ids, w, w_scales):
    """W_e rows of each pair, [P, N]."""
    E = w.shape[0]
    flat = ids.reshape(-1).long()
    if flat.numel() <= E:
        # few pairs: the matrices of each pair
        return torch.matmul(_values(w[flat], w_scales[flat], BLOCK), rows[..., None])[..., 0]
    side, (e, place, order) = _padded(rows, ids, E)
    out = torch.matmul(side, _values(w, w_scales, BLOCK).transpose(1, 2))
    y = torch.empty((flat.numel(), out.shape[2]), device=rows.device)
    y[order] = out[e, place]
    return y


def _silu(g):
    return g / (1.0 + torch.exp(-g))


def _plain(s):
    kind = s["kind"]
    dtype = s["x"].dtype
    if kind == "norm":
        r, _, _, y = _norm(s)
        codes, scales = _quantise(y, 1)
        return {"codes": codes, "scales": scales, "r": r}
    if kind == "norm_train":
        r, v, rstd, y = _norm(s)
        grad_x, grad_w = _norm_grad(s, v, rstd)
        return {"y": y.to(dtype), "r": r, "grad_x": grad_x, "grad_w": grad_w}
    if kind in ("gated", "gated_train"):
        x, w = s["x"].float(), s["w_gu"].float()
        g, u = (x @ w.t()).chunk(2, -1)
        h = (_silu(g) * u).to(dtype)
        if kind == "gated":
            return {"h": h}
        dh = s["grad_h"].float()
        sig = 1.0 / (1.0 + torch.exp(-g))
        d = torch.cat((dh * u * sig * (1.0 + g * (1.0 - sig)), dh * g * sig), -1)
        return {"h": h, "grad_x": (d @ w).to(dtype), "grad_w": (d.t() @ x).to(dtype)}
    x = _values(*_quantise(s["x"], 1), 1)
    if kind == "linear":
        return {"y": (x @ _values(s["w"], s["w_scales"], BLOCK).t()).to(dtype)}
    n, k = s["ids"].shape
    rows = x.repeat_interleave(k, 0)
    if kind == "experts":
        y = _product(rows, s["ids"], s["w"], s["w_scales"])
    else:
        g, u = _product(rows, s["ids"], s["w_gu"], s["gu_scales"]).chunk(2, -1)
        h = _values(*_quantise(_silu(g) * u, 1), 1)
        y = _product(h, s["ids"], s["w_down"], s["down_scales"])
    return {"y": (y.view(n, k, -1) * s["topk_w"][..., None]).sum(1).to(dtype)}


# ------------------------------------------------------------------ the framework's calls

def _own(s):
    import trellis_quantized_moe_sort_gb300 as tq

    kind = s["kind"]
    if kind == "norm":
        codes, scales, r = tq.tq_rms_norm_fp8(s["x"], s["weight"], eps=EPS, residual=s["residual"])
        return {"codes": codes, "scales": scales, "r": r}
    if kind == "norm_train":
        y, r, rstd = tq.tq_rms_norm(s["x"], s["weight"], eps=EPS, residual=s["residual"])
        grad_x, grad_w = tq.tq_rms_norm_backward(s["grad_y"], r, s["weight"], rstd, grad_residual=s["grad_r"])
        return {"y": y, "r": r, "grad_x": grad_x, "grad_w": grad_w}
    if kind == "gated":
        return {"h": tq.tq_swiglu_linear(s["x"], s["w_gu"])}
    if kind == "gated_train":
        gate_up = torch.empty((s["n"], 2 * s["I"]), dtype=torch.float32, device=s["x"].device)
        h = tq.tq_swiglu_linear(s["x"], s["w_gu"], gate_up=gate_up)
        grad_x, grad_w = tq.tq_swiglu_linear_backward(s["x"], s["w_gu"], s["grad_h"], gate_up=gate_up)
        return {"h": h, "grad_x": grad_x, "grad_w": grad_w}
    xq, x_scales = tq.tq_fp8_quantize(s["x"])
    dtype = s["x"].dtype
    if kind == "linear":
        return {"y": tq.tq_fp8_linear(xq, x_scales, s["w"], s["w_scales"], dtype=dtype)}
    if kind == "experts":
        return {"y": tq.tq_fp8_moe_forward(xq, x_scales, s["w"], s["w_scales"], s["ids"], s["topk_w"], dtype=dtype)}
    return {"y": tq.tq_fp8_moe_mlp_forward(xq, x_scales, s["w_gu"], s["gu_scales"], s["w_down"], s["down_scales"],
                                           s["ids"], s["topk_w"], dtype=dtype)}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ work

def work(case):
    size, n, kind = SIZES[case["dtype"]], case["n"], case["kind"]
    if kind == "norm":
        K = case["K"]
        return {"bytes": n * (3 * K * size + K + 4 * -(-K // BLOCK)) + 4 * K, "flops": 8 * n * K}
    if kind == "norm_train":
        # x, residual, grad_y and grad_r in, y, r and grad_x out
        K = case["K"]
        return {"bytes": 7 * n * K * size + 8 * K, "flops": 18 * n * K}
    if kind in ("gated", "gated_train"):
        H, I = case["H"], case["I"]
        once = 2 * n * H * 2 * I
        if kind == "gated":
            return {"bytes": (n * H + 2 * I * H + n * I) * size, "flops": once}
        return {"bytes": (2 * n * H + 4 * I * H + 2 * n * I) * size, "flops": 3 * once}
    if kind == "linear":
        K, N = case["K"], case["N"]
        held = N * K + 4 * -(-N // BLOCK) * -(-K // BLOCK)
        return {"bytes": n * K * size + held + n * N * size, "flops": 2 * n * N * K}
    E, k = case["E"], case["k"]
    woken = E * (1.0 - (1.0 - k / E) ** n)
    if kind == "experts":
        K, N = case["K"], case["N"]
        return {"bytes": n * K * size + woken * N * K + n * k * 8 + n * N * size, "flops": 2 * n * k * N * K}
    H, I = case["H"], case["I"]
    return {"bytes": 2 * n * H * size + woken * 3 * H * I + n * k * 8, "flops": 6 * n * k * H * I}


# ------------------------------------------------------------------ 64 bits

def _e4m3(a):
    """The nearest e4m3 value (3 mantissa bits, the smallest step 2^-9), ties to even, in 64 bits."""
    exponent = torch.clamp(torch.frexp(a).exponent - 1, min=-6)
    step = torch.ldexp(torch.ones_like(a), exponent - 3)
    return torch.clamp(torch.round(a / step) * step, -MOST, MOST)


def _exact_blocks(x):
    """e4m3 values and scales of rows in blocks of 128, in 64 bits but for the two roundings that the format has."""
    parts = [x[:, i:i + BLOCK] for i in range(0, x.shape[1], BLOCK)]
    scales = torch.stack([p.abs().max(-1).values / MOST for p in parts], -1).float().double()
    codes = [_e4m3((p / torch.clamp(scales[:, i:i + 1], min=1e-300)).float().double()) for i, p in enumerate(parts)]
    return torch.cat(codes, -1), scales


def _exact_rows(x):
    codes, scales = _exact_blocks(x.double())
    return codes * scales.repeat_interleave(BLOCK, 1)[:, :x.shape[1]]


def _exact_matrix(codes, scales):
    N, K = codes.shape
    row, column = torch.arange(N, device=codes.device) // BLOCK, torch.arange(K, device=codes.device) // BLOCK
    return codes.double() * scales.double()[row][:, column]


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind in ("norm", "norm_train"):
        r = (s["x"].double() + s["residual"].double()).to(s["x"].dtype).double()
        if kind == "norm_train":
            r = r.requires_grad_(True)
        w = s["weight"].double().requires_grad_(True)
        y = r / torch.sqrt(r.square().mean(-1, keepdim=True) + EPS) * w
        if kind == "norm":
            codes, scales = _exact_blocks(y.detach())
            return {"codes": codes, "scales": scales, "r": r}
        grad_r, grad_w = torch.autograd.grad((y * s["grad_y"].double()).sum(), (r, w))
        return {"y": y.detach(), "r": r.detach(), "grad_x": grad_r + s["grad_r"].double(), "grad_w": grad_w}
    if kind in ("gated", "gated_train"):
        x, w = s["x"].double().requires_grad_(True), s["w_gu"].double().requires_grad_(True)
        I = case["I"]
        h = torch.nn.functional.silu(x @ w[:I].t()) * (x @ w[I:].t())
        if kind == "gated":
            return {"h": h.detach()}
        grad_x, grad_w = torch.autograd.grad((h * s["grad_h"].double()).sum(), (x, w))
        return {"h": h.detach(), "grad_x": grad_x, "grad_w": grad_w}
    x = _exact_rows(s["x"])
    if kind == "linear":
        return {"y": x @ _exact_matrix(s["w"], s["w_scales"]).t()}
    y = torch.zeros((case["n"], case["N"] if kind == "experts" else case["H"]), dtype=torch.float64, device=x.device)
    for e in range(case["E"]):
        t, j = torch.nonzero(s["ids"] == e, as_tuple=True)
        if not t.numel():
            continue
        if kind == "experts":
            out = x[t] @ _exact_matrix(s["w"][e], s["w_scales"][e]).t()
        else:
            gu = x[t] @ _exact_matrix(s["w_gu"][e], s["gu_scales"][e]).t()
            h = torch.nn.functional.silu(gu[:, :case["I"]]) * gu[:, case["I"]:]
            out = _exact_rows(h) @ _exact_matrix(s["w_down"][e], s["down_scales"][e]).t()
        y.index_add_(0, t, out * s["topk_w"][t, j].double()[:, None])
    return {"y": y}
