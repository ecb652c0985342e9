"""Routing at the edges of its scores' range."""
import math

import numpy as np
import pytest
import torch

from gpu_util import announce, need_gpu
from oracle import block as ob

pytestmark = pytest.mark.gpu
U = ob.U


@pytest.fixture(scope="module")
def ep():
    need_gpu()
    import combine_top_expert_amd as ep
    return ep


def route(ep, logits, K, bias=None, score="sigmoid", n=1, keep=1, top=2, renorm=True):
    T = logits.shape[0]
    ids = torch.full((T, K), -9, dtype=torch.int32, device="cuda")
    w = torch.full((T, K), math.nan, device="cuda")
    ep.moe_router_group_topk(torch.from_numpy(logits).cuda(), K, ids, w,
                             bias=None if bias is None else torch.from_numpy(bias).cuda(),
                             score=ep.MOE_SCORE_SIGMOID if score == "sigmoid" else ep.MOE_SCORE_SOFTMAX, n_group=n,
                             topk_group=keep, group_top=top, renorm=renorm)
    torch.cuda.synchronize()
    return ids.cpu().numpy(), w.double().cpu().numpy()


def same_choice(ep, rows, K, T=None, **kw):
    """The oracle's ids for `rows`, repeated to a batch of T."""
    at = np.arange(len(rows)) if T is None else np.resize(np.arange(len(rows)), T)
    want, _ = ob.group_topk(rows, K, kw.get("bias"), kw.get("score", "sigmoid"), kw.get("n", 1), kw.get("keep", 1),
                            kw.get("top", 2))
    ids, _ = route(ep, rows[at], K, **kw)
    assert np.array_equal(ids, want[at]), (kw, np.argwhere(ids != want[at])[:4].tolist())
    return want


def saturated_rows(E, rng):
    """Sigmoid logits whose fp64 scores tie (from about 37 on all are 1, from 23
    on neighbouring logits' are), ordinary ones among them, and tiny logits."""
    step = np.float32(2.0 ** -19)                       # neighbouring logits between 16 and 32
    up = (24 + step * rng.permutation(E)).astype(np.float32)
    rows = [np.arange(40, 40 + E), np.arange(40 + E, 40, -1), up, up + 6, 1e-20 * rng.permutation(E),
            15 + 30 * rng.random(E), np.where(rng.random(E) < 0.5, 50 * rng.random(E), rng.standard_normal(E)),
            -1000.0 - rng.permutation(E), np.where(np.arange(E) % 2, 0.0, -1000.0 - rng.permutation(E))]
    rows = np.stack(rows).astype(np.float32)
    rows[5, 1], rows[6, 0] = np.inf, np.inf
    return rows


@pytest.mark.parametrize("E,K,n,keep", [(8, 2, 1, 1), (8, 2, 2, 1), (8, 3, 4, 2), (64, 6, 1, 1), (100, 7, 5, 2), (256, 8, 1, 1),
                                        (256, 8, 8, 4), (384, 12, 2, 1), (1024, 32, 1, 1), (1024, 32, 64, 16)])
def test_route_saturated_sigmoid(ep, E, K, n, keep):
    """One rule with and without groups and bias: scores that fp64 does not tell
    apart tie, and ties go to the lower id."""
    announce("route saturated", E, K, n, keep)
    rng = np.random.default_rng(E + n)
    rows = saturated_rows(E, rng)
    for bias in (None, np.zeros(E, np.float32)):
        for top in (1, 2):
            want = same_choice(ep, rows, K, bias=bias, n=n, keep=keep, top=top)
    if n == 1:
        assert want[0].tolist() == list(range(K))


@pytest.mark.parametrize("E,K,n,keep", [(8, 2, 1, 1), (8, 2, 2, 1), (64, 6, 1, 1), (100, 7, 5, 2), (256, 8, 8, 4), (1024, 32, 1, 1)])
def test_route_softmax_ties(ep, E, K, n, keep):
    """Softmax scores that fp64 does not tell apart: logits that differ by less
    than its step, and those whose scores underflow."""
    announce("route softmax ties", E, K, n, keep)
    rng = np.random.default_rng(E + n)
    rows = np.stack([1e-20 * rng.permutation(E), np.where(np.arange(E) < 2, 3.0, 1e-18 * rng.permutation(E)),
                     np.where(np.arange(E) % 4, -1000.0 - rng.permutation(E), 0.0),
                     np.where(np.arange(E) == 3, 1.0, -2000.0 + rng.permutation(E))]).astype(np.float32)
    for bias in (None, np.zeros(E, np.float32)):
        for top in (1, 2):
            same_choice(ep, rows, K, score="softmax", bias=bias, n=n, keep=keep, top=top)


@pytest.mark.parametrize("E,K,n,keep", [(256, 8, 1, 1), (256, 8, 8, 4), (128, 6, 4, 2), (160, 6, 1, 1)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_rows_far_below_every_score(ep, E, K, n, keep, score):
    """Rows filled with a large negative number that is no mask, biases that tie:
    the lower ids, in large batches as in small ones."""
    announce("route far below", E, K, n, keep, score)
    rng = np.random.default_rng(E)
    rows = np.stack([np.full(E, -3e38), np.full(E, -2.5e38), np.where(rng.random(E) < 0.5, -3e38, -np.inf),
                     rng.standard_normal(E), np.full(E, 3e38)]).astype(np.float32)
    for bias in (np.zeros(E, np.float32), (np.round(rng.standard_normal(E)) / 4).astype(np.float32)):
        for T in (None, 5123):
            same_choice(ep, rows, K, T, bias=bias, score=score, n=n, keep=keep)


@pytest.mark.parametrize("E,T", [(8, None), (256, None), (256, 5123)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("n", [1, 2])
def test_route_scores_below_fp32s_normal_range(ep, E, T, score, n):
    """Scores that fp32 hardware flushes to zero, against biases of their size."""
    announce("route tiny scores", E, T, score, n)
    row, bias = np.full(E, -200.0, np.float32), np.zeros(E, np.float32)
    row[E - 3] = -87.5                                   # sigmoid 1.0e-38, below 2^-126
    bias[1] = 5e-39
    if score == "softmax":
        row[0] = 0.0                                     # its own score is 1 and leaves through the bias
        bias[0] = -2.0
    want = same_choice(ep, row[None], 1, T, score=score, bias=bias, n=n, keep=1, top=1)
    assert want[0, 0] == E - 3


def call_time(fn, calls=20, rounds=5):
    """Microseconds a call, the best of some rounds."""
    best = math.inf
    for _ in range(rounds):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(calls):
            fn()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) * 1e3 / calls)
    return best


def test_route_batches_that_drop_no_live_group(ep):
    """A batch in which every group stays, or in which the dropped groups are all
    masked, or whose rows are padding, costs about what any other does: its
    rows are not decided in fp64."""
    announce("route keeps every live group")
    T, E, K = 65536, 256, 8
    torch.manual_seed(4)
    logits, bias = torch.randn(T, E, device="cuda"), 0.1 * torch.randn(E, device="cuda")
    half = logits.clone()
    half[:, 128:] = -math.inf                            # four of eight groups masked
    none = torch.full_like(logits, -math.inf)
    ids, w = torch.empty(T, K, dtype=torch.int32, device="cuda"), torch.empty(T, K, device="cuda")

    def time(x, keep, score):
        return call_time(lambda: ep.moe_router_group_topk(x, K, ids, w, bias=bias, n_group=8, topk_group=keep, score=score))
    for score in (ep.MOE_SCORE_SIGMOID, ep.MOE_SCORE_SOFTMAX):
        usual = time(logits, 4, score)
        others = {"all stay": time(logits, 8, score), "others masked": time(half, 4, score), "all masked": time(none, 4, score)}
        print(f"[metric] score {score}: 4 of 8 {usual:.1f} us, " + ", ".join(f"{k} {v:.1f}" for k, v in others.items()))
        assert max(others.values()) < 1.75 * usual


@pytest.mark.parametrize("E,K,n,keep", [(256, 8, 8, 8), (128, 6, 4, 4), (160, 6, 5, 5), (256, 8, 8, 6)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_choice_where_no_live_group_is_dropped(ep, E, K, n, keep, score):
    announce("route no live group dropped", E, K, n, keep, score)
    rng = np.random.default_rng(E + keep)
    x = rng.standard_normal((40, E)).astype(np.float32)
    x[30:, (E // n) * (keep // 2):] = -np.inf            # fewer live groups than stay
    x[20:30, rng.random(E) < 0.5] = -np.inf
    x[38:] = -np.inf
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    for top in (1, 2):
        same_choice(ep, x, K, 5123, bias=bias, score=score, n=n, keep=keep, top=top)


def backward(ep, x, ids, dw, score, scale=1.0):
    dl = torch.full(x.shape, math.nan, device="cuda")
    ep.moe_router_group_topk_backward(torch.from_numpy(x).cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(dw).cuda(), dl,
                                      score=score, renorm=False, route_scale=scale)
    torch.cuda.synchronize()
    return dl.double().cpu().numpy()


@pytest.mark.parametrize("E", [8, 64, 100, 256, 1000])
@pytest.mark.parametrize("K", [1, 2, 20])
def test_softmax_gradient_of_confident_routers(ep, E, K):
    """One expert holds all but e^-gap of a row: ds_e - sum_k ds_k s_k loses all
    but that much of its terms.

    Each exponential is off by at most (spread + 3) u of itself (l - max and the
    exponential), so a score and what is left of 1 beside it are within twice
    that, and s_e (ds_e (1 - s_e) - sum over the others of ds_k s_k) within four
    times that of the sum of its terms; four roundings to fp32 and those of
    fp64 (2^-49 of the uncancelled terms) come on top."""
    if K > E:
        pytest.skip("K > E")
    announce("softmax gradient, confident", E, K)
    rng = np.random.default_rng(E + K)
    gaps = np.array([4, 8, 10, 12, 14, 16], np.float32)
    x = (0.3 * rng.standard_normal((30, E))).astype(np.float32)
    top = rng.integers(0, E, 30)
    x[np.arange(30), top] += np.resize(gaps, 30) + math.log(E)
    ids = np.stack([np.concatenate([[t], rng.permutation(np.delete(np.arange(E), t))[:K - 1]]) for t in top]).astype(np.int32)
    dw = (0.5 + rng.random((30, K))).astype(np.float32)
    dw[:6] = 1.0
    if K > 1:
        ids[7, 1] = ids[7, 0]                            # twice, and the two all but cancel
        dw[7, 1] = -dw[7, 0] * np.float32(1 - 2.0 ** -10)
        ids[8, K - 1] = -1
    got = backward(ep, x, ids, dw, ep.MOE_SCORE_SOFTMAX, 2.5)
    worst = 0.0
    for t in range(30):
        e = np.exp(x[t].astype(np.float64) - x[t].max())
        s = e / math.fsum(e)
        d = np.zeros(E)
        for k in range(K):
            if ids[t, k] >= 0:
                d[ids[t, k]] += 2.5 * float(dw[t, k])
        rest = np.array([math.fsum(np.delete(e, i)) for i in range(E)]) / math.fsum(e)      # 1 - s
        cross = np.array([math.fsum(np.delete(d * s, i)) for i in range(E)])
        ref = s * (d * rest - cross)
        size = s * (np.abs(d) * rest + math.fsum(np.abs(d * s)) - np.abs(d * s))
        spread = float(x[t].max() - x[t].min())
        bound = (4 * (spread + 3) + 4) * U * size + 2.0 ** -49 * s * (np.abs(d) + np.abs(d * s).sum()) + 1e-40
        worst = max(worst, float(np.max(np.abs(got[t] - ref) / bound)))
        assert np.all(np.abs(got[t] - ref) <= bound), (t, np.max(np.abs(got[t] - ref) / bound))
    print(f"[metric] softmax gradient {E} {K}: worst error / bound {worst:.3f}")


@pytest.mark.parametrize("K", [2, 8, 15, 16, 17, 20, 32])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_gradient_where_an_expert_occurs_twice(ep, K, score):
    """At every two places of a token's ids, at three, and at all."""
    announce("gradient, expert twice", K, score)
    E = 40
    rng = np.random.default_rng(K)
    pairs = [(i, j) for i in range(K) for j in range(i)] + [()]
    T = len(pairs) + 3
    x = rng.standard_normal((T, E)).astype(np.float32)
    ids = np.stack([rng.permutation(E)[:K] for _ in range(T)]).astype(np.int32)
    for t, at in enumerate(pairs):
        if at:
            ids[t, at[0]] = ids[t, at[1]]
    ids[T - 3, [0, K // 2, K - 1]] = 5
    ids[T - 2] = 7
    ids[T - 1, ::2] = -1                                     # no route is no expert that occurs twice
    dw = rng.standard_normal((T, K)).astype(np.float32)
    ref, mag = ob.group_topk_backward(x, ids, dw, score, False, 2.5)
    got = backward(ep, x, ids, dw, ep.MOE_SCORE_SIGMOID if score == "sigmoid" else ep.MOE_SCORE_SOFTMAX, 2.5)
    assert np.all(np.abs(got - ref) <= 160 * U * mag + 1e-30), np.argwhere(np.abs(got - ref) > 160 * U * mag + 1e-30)[:4].tolist()


@pytest.mark.parametrize("E", [8, 256])
def test_sigmoid_gradient_of_saturated_logits(ep, E):
    """s (1 - s) keeps its digits where s is 1 to fp64: formed in fp64 from one
    exponential, rounded once."""
    announce("sigmoid gradient, saturated", E)
    x = np.resize(np.array([-80, -40, -20, -1, 0, 1, 17, 20, 25, 30, 36, 40, 60, 80], np.float32), (14, E)).astype(np.float32)
    ids = np.stack([np.full(14, 3), np.full(14, 5)], 1).astype(np.int32)
    x[:, 3] = np.array([-80, -40, -20, -1, 0, 1, 17, 20, 25, 30, 36, 40, 60, 80], np.float32)
    dw = np.linspace(0.5, 2.0, 28).reshape(14, 2).astype(np.float32)
    got = backward(ep, x, ids, dw, ep.MOE_SCORE_SIGMOID)
    for t in range(14):
        for k in range(2):
            v = float(x[t, ids[t, k]])
            ref = float(dw[t, k]) / (1 + math.exp(-v)) / (1 + math.exp(v))
            assert abs(got[t, ids[t, k]] - ref) <= (2.0 ** -24 + 2.0 ** -45) * ref + 1e-45, (v, got[t, ids[t, k]], ref)
