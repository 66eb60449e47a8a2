"""The scored router and its gradient against the fp64 definition.

Choices are compared exactly on every row whose deciding values are further
apart than fp32 can confuse (2e-6, against scores and sums of at most a few
units whose rounding is below 12 ulp, 7.2e-7); exact ties are kept in, and go to
the lower index.  Weights: expf 2 ulp, the sum's tree 10 roundings, three more
operations, twice over with renormalisation: below 2e-6 relative."""
import numpy as np
import pytest
import torch

import oracle.moe_operators as M
import trellis_quantized_moe_sort_gb300 as tq
from gpu_util import check_no_device_error

pytestmark = pytest.mark.gpu
SCORE = {"sigmoid": tq.SCORE_SIGMOID, "softmax": tq.SCORE_SOFTMAX}
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from trellis_quantized_moe_sort_gb300 import build
    build.build()
    tq.tq_init(0)


def _logits(rng, n, E, dtype="fp32", coarse=False):
    x = rng.standard_normal((n, E)).astype(np.float32)
    if coarse:
        x = np.round(x * 4) / 4      # many exact ties
    return torch.from_numpy(x).to(DTYPES[dtype])


def _check_forward(logits, top_k, score="sigmoid", bias=None, groups=1, top_groups=1, renormalize=True, scale=1.0,
                   most_unclear=0.02):
    ids, w = tq.tq_router_scored(logits.cuda(), top_k, score=SCORE[score],
                                 bias=None if bias is None else torch.from_numpy(bias).cuda(), groups=groups,
                                 top_groups=top_groups, renormalize=renormalize, scale=scale)
    check_no_device_error()
    want_ids, want_w, gap = M.router(logits.float().numpy(), top_k, score, bias, groups, top_groups, renormalize, scale)
    clear = gap > 2e-6
    assert (~clear).mean() <= most_unclear
    ids, w = ids.cpu().numpy(), w.cpu().numpy().astype(np.float64)
    assert np.array_equal(ids[clear], want_ids[clear])
    assert np.allclose(w[clear], want_w[clear], rtol=2e-6, atol=1e-37)
    return ids, w


@pytest.mark.parametrize("n,E,k,groups,top_groups", [
    (1, 1, 1, 1, 1), (1, 256, 6, 8, 4), (2, 2, 2, 2, 2), (3, 8, 2, 4, 2), (5, 7, 7, 1, 1), (37, 31, 5, 1, 1),
    (33, 33, 4, 3, 2), (65, 160, 6, 5, 3), (129, 256, 8, 8, 4), (64, 250, 6, 10, 3), (17, 384, 16, 32, 9),
    (9, 512, 32, 16, 16), (11, 1000, 10, 20, 7), (6, 1024, 32, 32, 32), (1000, 64, 6, 8, 3), (13, 96, 4, 32, 5)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", sorted(DTYPES))
def test_forward(n, E, k, groups, top_groups, score, dtype):
    rng = np.random.default_rng([n, E, k, groups])
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    # 16-bit logits are coarse and their scores crowded: rows are left out more often
    _check_forward(_logits(rng, n, E, dtype), k, score, bias, groups, top_groups, True, 2.5, most_unclear=0.35)
    _check_forward(_logits(rng, n, E, dtype), k, score, None, groups, top_groups, False, 1.0, most_unclear=0.35)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups,top_groups", [(1, 1), (8, 3)])
def test_ties_go_to_the_lower_index(score, groups, top_groups):
    rng = np.random.default_rng(5)
    logits = _logits(rng, 300, 64, coarse=True)
    _check_forward(logits, 6, score, None, groups, top_groups)
    _check_forward(torch.zeros(3, 64), 6, score, None, groups, top_groups)
    _check_forward(logits, 6, score, np.full(64, -1.0, np.float32), groups, top_groups)


@pytest.mark.parametrize("E,k,groups,top_groups", [
    (65, 3, 1, 1), (128, 32, 1, 1), (256, 8, 1, 1), (256, 12, 8, 1), (256, 3, 8, 1), (480, 7, 6, 2), (1024, 32, 1, 1)])
@pytest.mark.parametrize("values", [1, 2, 12, 400])
def test_many_equal_candidates(E, k, groups, top_groups, values):
    """From every expert equal (more candidates than a warp has lanes) to a few ties; some rows mostly masked."""
    rng = np.random.default_rng([E, k, values])
    x = rng.integers(0, values, (70, E)).astype(np.float32) / 64
    x[60:][rng.random((10, E)) < 0.97] = -np.inf
    _check_forward(torch.from_numpy(x), k, "sigmoid", None, groups, top_groups, most_unclear=0.05)
    _check_forward(torch.from_numpy(x), k, "softmax", None, groups, top_groups, most_unclear=0.05)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups,top_groups", [(1, 1), (4, 2)])
def test_masked_and_empty_rows(score, groups, top_groups):
    rng = np.random.default_rng(9)
    x = rng.standard_normal((64, 32)).astype(np.float32)
    x[0] = -np.inf                                   # nothing left
    x[1] = np.nan
    x[2, 1:] = -np.inf                               # one left
    x[3, ::2] = np.nan
    x[4, 3] = np.inf                                 # counts as masked
    x[5] = np.finfo(np.float32).min                  # finite: the type's lowest value
    x[6, :30] = np.finfo(np.float32).min
    x[7] = np.finfo(np.float32).max
    x[8, :8] = -np.inf                               # a whole group
    x[9:20][rng.random((11, 32)) < 0.9] = -np.inf    # fewer than top_k left
    ids, w = _check_forward(torch.from_numpy(x), 6, score, None, groups, top_groups, most_unclear=0.0)
    assert np.isfinite(w).all() and not w[:2].any() and (ids >= 0).all() and (ids < 32).all()
    assert w[2, 0] == 1.0 and not w[2, 1:].any()


def test_bias_extremes():
    rng = np.random.default_rng(3)
    logits = _logits(rng, 40, 16)
    bias = np.zeros(16, np.float32)
    bias[3], bias[5], bias[7] = np.inf, -np.inf, np.nan
    ids, w = _check_forward(logits, 13, "sigmoid", bias)
    assert (ids[:, 0] == 3).all() and not np.isin(ids, (5, 7)).any()
    ids, w = _check_forward(logits, 16, "sigmoid", bias)
    assert (ids[:, 14:] == (5, 7)).all() and not w[:, 14:].any()     # fillers


def test_saturated_scores():
    x = torch.tensor([[200.0, 100.0, -200.0, -90.0, 0.0, 89.0], [-200.0] * 6])
    ids, w = tq.tq_router_scored(x.cuda(), 3, score=tq.SCORE_SIGMOID, renormalize=True)
    assert ids.cpu().tolist() == [[0, 1, 5], [0, 1, 2]]
    assert torch.allclose(w.cpu(), torch.tensor([[1 / 3] * 3, [0.0] * 3]))    # no sum: no weights
    ids, w = tq.tq_router_scored(x.cuda(), 2, score=tq.SCORE_SOFTMAX, renormalize=False)
    # exp(-100) is 27 times fp32's smallest subnormal number
    assert w.cpu()[0, 0] == 1.0 and 0.0 < w.cpu()[0, 1] < 4e-44 and torch.allclose(w.cpu()[1], torch.full((2,), 1 / 6))


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("pitch,offset", [(256, 0), (257, 1), (264, 3), (512, 8)])
def test_strided_rows(dtype, pitch, offset):
    rng = np.random.default_rng(11)
    rows = _logits(rng, 70, pitch + offset, dtype).cuda()
    view = rows[:, offset:offset + 200] if pitch < 512 else rows[:, offset:offset + 200].contiguous()[::2]
    a = tq.tq_router_scored(view, 6, groups=4, top_groups=2)
    b = tq.tq_router_scored(view.contiguous(), 6, groups=4, top_groups=2)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    g = torch.randn(view.shape[0], 6, device="cuda")
    a = tq.tq_router_scored_backward(view, *a, g, score=tq.SCORE_SOFTMAX)
    b = tq.tq_router_scored_backward(view.contiguous(), *b, g, score=tq.SCORE_SOFTMAX)
    assert torch.equal(a, b)


def test_rows_do_not_depend_on_the_batch():
    rng = np.random.default_rng(12)
    logits = _logits(rng, 3000, 160).cuda()
    ids, w = tq.tq_router_scored(logits, 6, score=tq.SCORE_SOFTMAX, groups=5, top_groups=3)
    for t in (0, 1, 777, 2999):
        a, b = tq.tq_router_scored(logits[t:t + 1], 6, score=tq.SCORE_SOFTMAX, groups=5, top_groups=3)
        assert torch.equal(a[0], ids[t]) and torch.equal(b[0], w[t])


def test_no_tokens_and_given_outputs():
    ids, w = tq.tq_router_scored(torch.empty(0, 64, device="cuda"), 4)
    assert ids.shape == w.shape == (0, 4)
    logits = torch.randn(10, 64, device="cuda")
    ids, w = torch.full((10, 4), -1, dtype=torch.int32, device="cuda"), torch.zeros(10, 4, device="cuda")
    got = tq.tq_router_scored(logits, 4, topk_ids=ids, topk_w=w)
    assert got[0] is ids and got[1] is w and (ids >= 0).all()
    grad = torch.empty(0, 64, device="cuda")
    assert tq.tq_router_scored_backward(grad, ids[:0], w[:0], w[:0]).shape == (0, 64)


# The formula in fp32: p, its sum and its dot products each a few ulp; values
# cancel in g - dot, so the error is relative to the row's largest terms, not to
# the result.  2^-19 of sum |g| p scale / total covers 32 roundings.
@pytest.mark.parametrize("n,E,k", [(1, 1, 1), (3, 8, 2), (33, 33, 4), (65, 160, 6), (300, 256, 8), (5, 1000, 32),
                                   (9, 31, 31)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("dtype", sorted(DTYPES))
def test_backward(n, E, k, score, renormalize, dtype):
    rng = np.random.default_rng([n, E, k])
    logits = _logits(rng, n, E, dtype)
    if n > 2:
        logits[1, : E // 2] = float("-inf")
        logits[2] = float("nan")
    dev = logits.cuda()
    ids, w = tq.tq_router_scored(dev, k, score=SCORE[score], renormalize=renormalize, scale=2.5)
    g = rng.standard_normal((n, k)).astype(np.float32)
    got = tq.tq_router_scored_backward(dev, ids, w, torch.from_numpy(g).cuda(), score=SCORE[score],
                                       renormalize=renormalize, scale=2.5)
    check_no_device_error()
    assert got.dtype == DTYPES[dtype]
    ids, live = ids.cpu().numpy(), w.cpu().numpy() != 0
    x = logits.float().numpy()
    want = M.router_backward(x, ids, live, g, score, renormalize, 2.5)
    got = got.float().cpu().numpy().astype(np.float64)
    s, _ = M.scores(x, score)
    p = np.take_along_axis(s, ids.astype(np.int64), 1) * live
    size = (np.abs(g) * 2.5 * live).sum(1, keepdims=True)
    if renormalize:
        total = p.sum(1, keepdims=True)
        size = np.divide(size, total, out=np.zeros_like(size), where=total > 0)
    rounding = {"fp32": 0.0, "bf16": 2.0 ** -8, "fp16": 2.0 ** -10}[dtype]
    assert (np.abs(got - want) <= 2.0 ** -19 * size + rounding * np.abs(want) + 6e-8).all()
    unchosen = np.ones_like(s, dtype=bool)
    np.put_along_axis(unchosen, ids.astype(np.int64), ~live, 1)
    if score == "sigmoid":
        assert not got[unchosen].any()
    assert not got[~np.isfinite(x)].any()


def test_backward_is_the_slope_of_the_forward():
    rng = np.random.default_rng(21)
    x = rng.standard_normal((4, 24))
    logits = torch.from_numpy(x.astype(np.float32)).cuda()
    for score in ("sigmoid", "softmax"):
        ids, w = tq.tq_router_scored(logits, 5, score=SCORE[score], renormalize=True, scale=1.5)
        g = rng.standard_normal((4, 5))
        got = tq.tq_router_scored_backward(logits, ids, w, torch.from_numpy(g.astype(np.float32)).cuda(),
                                           score=SCORE[score], renormalize=True, scale=1.5).cpu().numpy()
        i, live, h = ids.cpu().numpy(), np.ones((4, 5)), 1e-5
        for e in range(24):
            up, down = x.astype(np.float32).astype(np.float64), x.astype(np.float32).astype(np.float64)
            up[:, e] += h
            down[:, e] -= h
            f = [(M.router_weights(v, i, live, score, True, 1.5) * g).sum(1) for v in (up, down)]
            assert np.allclose((f[0] - f[1]) / (2 * h), got[:, e], atol=5e-6)


def test_backward_reports_bad_ids_and_writes_the_rest():
    logits = torch.randn(3, 16, device="cuda")
    ids, w = tq.tq_router_scored(logits, 2)
    ids[1, 0], ids[2, 1] = 16, -1
    grad = tq.tq_router_scored_backward(logits, ids, w, torch.ones_like(w))
    torch.cuda.synchronize()
    assert tq.tq_device_error()[0] == -1
    assert torch.isfinite(grad).all()


def test_streams_and_graph():
    logits = torch.randn(500, 256, device="cuda")
    want = tq.tq_router_scored(logits, 6, groups=8, top_groups=4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = tq.tq_router_scored(logits, 6, groups=8, top_groups=4)
    b = tq.tq_router_scored(logits, 6, groups=8, top_groups=4, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = tq.tq_router_scored(logits, 6, groups=8, top_groups=4)
    graph.replay()
    torch.cuda.synchronize()
    for got in (a, b, c):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
