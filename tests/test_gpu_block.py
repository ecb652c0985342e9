"""GPU parity of libmoe_block.so against oracle/block.py (float64).

Bounds (u = 2^-24, half a step of fp32; half a step of bf16 is 2^-8, of e4m3
2^-4 of a normal value or 2^-10 of the scale):
* norm: a row's sum of squares is a lane's serial sum of at most 32 terms, a
  6-step wave sum and at most 16 waves: 54 u on r^2, so 27 u on r, with the
  mean, the root, the quotient and the two products below 34 u in all; d_w
  adds one rounding per row of a block (T / 512, rounded up, plus 48 partial
  sums in order).
* routing: the ids are those of exact scores.  A weight is within 64 u of
  itself with sigmoid scores (exp, add, divide, K terms and a 6-step sum,
  divide, scale); softmax adds the rounding of l - max, |l - max| u.
* 4-bit products: the sums of |a w'| (w' what the codes pass through) times
  2^-20 for the matrix instruction and 2 u per accumulation step.
"""
import math

import numpy as np
import pytest
import torch

from gpu_util import announce, need_gpu
from oracle import block as ob

pytestmark = pytest.mark.gpu
U = ob.U
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": U}


@pytest.fixture(scope="module")
def ep():
    need_gpu()
    import combine_top_expert_amd as ep
    return ep


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def inside(got, ref, bound, what):
    assert got.shape == ref.shape and np.all(np.isfinite(got)), what
    worst = float(np.max(np.abs(got - ref) / np.maximum(bound, 1e-300))) if got.size else 0.0
    print(f"[metric] {what}: worst error / bound {worst:.3f}", flush=True)
    assert worst <= 1.0, what


def randn(rng, *shape, dt="f32", scale=1.0):
    return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).to(DT[dt]).cuda()


# ------------------------------------------------------------------ norm

NORM_SIZES = [(1, 8), (3, 128), (5, 384), (7, 520), (33, 1408), (2, 2048), (9, 4096), (4, 4104), (130, 7168), (2, 8200),
              (3, 16384)]


def norm_case(ep, T, H, dt, wdt, res, outs, eps=1e-6, seed=0, x=None):
    rng = np.random.default_rng(H * 7 + T + seed)
    x = randn(rng, T, H, dt=dt) if x is None else x
    r = randn(rng, T, H, dt=dt, scale=3.0) if res else None
    w = (1 + 0.3 * randn(rng, H)).to(DT[wdt])
    h = torch.full_like(x, math.nan) if "h" in outs else None
    y = torch.full_like(x, math.nan) if "y" in outs else None
    y8 = torch.full((T, H), 0x7f, dtype=torch.uint8, device="cuda") if "8" in outs else None
    sc = torch.full((T, H // 128), math.nan, device="cuda") if "8" in outs else None
    ep.moe_add_rms_norm(x, r, w, eps, h, y, y8, sc)
    torch.cuda.synchronize()
    href = x if r is None else (x.float() + r.float()).to(DT[dt])
    return href, w, h, y, y8, sc


def check_norm(href, w, h, y, y8, sc, dt, eps=1e-6, what=""):
    ref, _ = ob.rms_norm(f64(href), f64(w), eps)
    if h is not None:
        assert torch.equal(h.view(torch.uint8), href.view(torch.uint8)), what     # one rounding: the same bits
    if y is not None:
        inside(f64(y), ref, (HALF[dt] + 34 * U) * np.abs(ref) + 1e-40, f"y {what}")
    if y8 is not None:
        T, H = ref.shape
        blocks = ref.reshape(T, H // 128, 128)
        amax = np.maximum(np.abs(blocks).max(axis=2), 1e-4)
        inside(f64(sc), amax / 448, 36 * U * amax / 448, f"scales {what}")
        v = f64(y8.view(torch.float8_e4m3fn)).reshape(blocks.shape) * f64(sc)[..., None]
        half = np.maximum(2.0 ** -4 * np.abs(blocks), 2.0 ** -10 * f64(sc)[..., None])
        inside(v, blocks, half * (1 + 2.0 ** -10) + 40 * U * np.abs(blocks), f"codes {what}")


@pytest.mark.parametrize("T,H", NORM_SIZES)
@pytest.mark.parametrize("dt,wdt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
def test_norm(ep, T, H, dt, wdt):
    for res, outs in ((True, "hy"), (False, "y"), (True, "hy8"), (False, "8"), (True, "h")):
        if "8" in outs and H % 128:
            continue
        announce("norm", T, H, dt, wdt, res, outs)
        check_norm(*norm_case(ep, T, H, dt, wdt, res, outs), dt, what=f"{T}x{H} {dt} {outs}")


@pytest.mark.parametrize("T", [1, 257, 4099])
def test_norm_many_rows(ep, T):
    announce("norm rows", T)
    check_norm(*norm_case(ep, T, 1024, "bf16", "bf16", True, "hy8"), "bf16")


def test_norm_edge_rows(ep):
    """Zero rows, tiny and huge rows, and the residual that cancels x."""
    announce("norm edges")
    x = torch.zeros(6, 256, device="cuda")
    x[1] = 1e-20
    x[2] = 1e15
    x[3, 7] = 1e4
    x[4] = torch.arange(256, device="cuda") - 128.0
    href, w, h, y, y8, sc = norm_case(ep, 6, 256, "f32", "f32", False, "hy8", x=x)
    check_norm(href, w, h, y, y8, sc, "f32")
    assert not y[0].any() and torch.all(sc[0] == torch.tensor(1e-4, device="cuda") / 448)
    # a NaN stays in its own row
    x[5, 3] = math.nan
    _, _, _, y2, _, _ = norm_case(ep, 6, 256, "f32", "f32", False, "hy", x=x)
    assert torch.isnan(y2[5]).all() and torch.equal(y2[:5], y[:5])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_norm_in_place(ep, dt):
    announce("norm in place", dt)
    rng = np.random.default_rng(5)
    x, r = randn(rng, 40, 1408, dt=dt), randn(rng, 40, 1408, dt=dt)
    w = randn(rng, 1408, dt=dt)
    h, y = torch.empty_like(x), torch.empty_like(x)
    ep.moe_add_rms_norm(x, r, w, 1e-5, h, y)
    x2, r2 = x.clone(), r.clone()
    ep.moe_add_rms_norm(x2, r2, w, 1e-5, r2, x2)            # the residual stream in r2, the norm in x2
    assert torch.equal(r2, h) and torch.equal(x2, y)


def norm_bw_case(ep, T, H, dt, wdt, with_dh, eps=1e-6):
    rng = np.random.default_rng(H + 3 * T)
    dy, h, dh = randn(rng, T, H, dt=dt), randn(rng, T, H, dt=dt, scale=2.0), randn(rng, T, H, dt=dt)
    w = (1 + 0.3 * randn(rng, H)).to(DT[wdt])
    dx, dw = torch.full_like(dy, math.nan), torch.full((H,), math.nan, device="cuda")
    ws = torch.full((ep.moe_add_rms_norm_backward_workspace_bytes(T, H),), 0xff, dtype=torch.uint8, device="cuda")
    ep.moe_add_rms_norm_backward(dy, h, w, eps, dx, dw, ws, dh=dh if with_dh else None)
    torch.cuda.synchronize()
    return dy, h, w, dh if with_dh else None, dx, dw, ws


@pytest.mark.parametrize("T,H", NORM_SIZES + [(513, 256), (2050, 384)])
@pytest.mark.parametrize("dt,wdt", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
def test_norm_backward(ep, T, H, dt, wdt):
    for with_dh in (False, True):
        announce("norm backward", T, H, dt, wdt, with_dh)
        dy, h, w, dh, dx, dw, ws = norm_bw_case(ep, T, H, dt, wdt, with_dh)
        rx, rw, mag, wmag = ob.rms_norm_backward(f64(dy), f64(h), f64(w), 1e-6, None if dh is None else f64(dh))
        inside(f64(dx), rx, HALF[dt] * np.abs(rx) + 100 * U * mag + 1e-40, f"dx {T}x{H} {dt}")
        inside(f64(dw), rw, (34 + 96 + 2 * (T // 512 + 1)) * U * wmag + 1e-40, f"dw {T}x{H} {dt}")
        # the same bits again, and with dx over dy
        dw2, dy2 = torch.empty_like(dw), dy.clone()
        ep.moe_add_rms_norm_backward(dy2, h, w, 1e-6, dy2, dw2, ws, dh=dh)
        assert torch.equal(dy2, dx) and torch.equal(dw2, dw)


def test_norm_backward_against_differences(ep):
    announce("norm backward differences")
    rng = np.random.default_rng(9)
    h, w, dy = rng.standard_normal((3, 16)), rng.standard_normal(16), rng.standard_normal((3, 16))
    t = lambda v: torch.from_numpy(v.astype(np.float32)).cuda()                       # noqa: E731
    h, w, dy = (f64(t(v)) for v in (h, w, dy))
    dx, dw = torch.empty(3, 16, device="cuda"), torch.empty(16, device="cuda")
    ws = torch.empty(ep.moe_add_rms_norm_backward_workspace_bytes(3, 16), dtype=torch.uint8, device="cuda")
    ep.moe_add_rms_norm_backward(t(dy), t(h), t(w), 1e-2, dx, dw, ws)
    num = np.zeros((3, 16))
    for i in range(3):
        for j in range(16):
            e = np.zeros((3, 16))
            e[i, j] = 1e-5
            num[i, j] = ((ob.rms_norm(h + e, w, 1e-2)[0] - ob.rms_norm(h - e, w, 1e-2)[0]) * dy).sum() / 2e-5
    assert np.max(np.abs(f64(dx) - num)) < 1e-5


def test_norm_empty_batch(ep):
    announce("norm T = 0")
    x = torch.empty(0, 256, device="cuda")
    dw = torch.full((256,), 5.0, device="cuda")
    ep.moe_add_rms_norm(x, None, torch.ones(256, device="cuda"), 1e-6, None, x.clone())
    ep.moe_add_rms_norm_backward(x, x.clone(), torch.ones(256, device="cuda"), 1e-6, x.clone(), dw,
                                 torch.empty(0, dtype=torch.uint8, device="cuda"))
    assert not dw.any()


# ------------------------------------------------------------------ routing

def route(ep, logits, K, bias=None, score="sigmoid", n=1, keep=1, top=2, renorm=True, scale=1.0):
    T = logits.shape[0]
    ids = torch.full((T, K), -9, dtype=torch.int32, device="cuda")
    w = torch.full((T, K), math.nan, device="cuda")
    b = None if bias is None else torch.from_numpy(bias).cuda()
    ep.moe_router_group_topk(torch.from_numpy(logits).cuda(), K, ids, w, bias=b,
                             score=ep.MOE_SCORE_SIGMOID if score == "sigmoid" else ep.MOE_SCORE_SOFTMAX, n_group=n,
                             topk_group=keep, group_top=top, renorm=renorm, route_scale=scale)
    torch.cuda.synchronize()
    return ids.cpu().numpy(), f64(w)


def check_route(ep, logits, K, bias=None, score="sigmoid", n=1, keep=1, top=2, renorm=True, scale=1.0, what=""):
    ids, w = route(ep, logits, K, bias, score, n, keep, top, renorm, scale)
    rid, rw = ob.group_topk(logits, K, bias, score, n, keep, top, renorm, scale)
    assert np.array_equal(ids, rid), (what, np.argwhere(ids != rid)[:4].tolist())
    live = logits[(logits > ob.MASK_AT) & np.isfinite(logits)]
    spread = float(live.max() - live.min()) if score == "softmax" and live.size else 0.0
    inside(w, rw, (64 + 2 * spread) * U * np.abs(rw) + 1e-30, f"weights {what}")
    return ids


ROUTES = [(8, 1, 1, 1), (8, 8, 1, 1), (64, 6, 8, 3), (100, 7, 5, 2), (256, 8, 8, 4), (256, 8, 1, 1), (160, 6, 8, 3),
          (384, 12, 2, 1), (1000, 16, 10, 4), (1024, 32, 64, 16), (12, 2, 12, 2)]


@pytest.mark.parametrize("E,K,n,keep", ROUTES)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route(ep, E, K, n, keep, score):
    rng = np.random.default_rng(E * 31 + K)
    x = (1.5 * rng.standard_normal((61, E))).astype(np.float32)
    bias = (0.2 * rng.standard_normal(E)).astype(np.float32)
    for b in (None, bias):
        for top in (1, 2):
            for renorm, scale in ((True, 2.5), (False, 1.0)):
                announce("route", E, K, n, keep, score, b is not None, top, renorm)
                check_route(ep, x, K, b, score, n, keep, top, renorm, scale, f"{E} {score}")


@pytest.mark.parametrize("E,K,n,keep", ROUTES)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_masks(ep, E, K, n, keep, score):
    """Masked logits and biases (-inf, the lowest finite fp32 and bf16), rows with fewer than K experts and with none."""
    announce("route masks", E, K, n, keep, score)
    rng = np.random.default_rng(E + 5)
    x = rng.standard_normal((40, E)).astype(np.float32)
    lows = np.array([-np.inf, np.finfo(np.float32).min, float(torch.finfo(torch.bfloat16).min)], np.float32)
    for t in range(30):
        at = rng.random(E) < t / 29
        x[t, at] = lows[rng.integers(0, 3, at.sum())]
    x[38], x[39] = -np.inf, lows[1]
    bias = (0.2 * rng.standard_normal(E)).astype(np.float32)
    for b in (None, bias, np.where(rng.random(E) < 0.5, lows[0], bias).astype(np.float32), np.full(E, -np.inf, np.float32)):
        for top in (1, 2):
            ids = check_route(ep, x, K, b, score, n, keep, top, True, 1.0, f"masks {E} {score}")
            assert np.all(ids[38:] == -1)


@pytest.mark.parametrize("E,K,n,keep", ROUTES)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_ties_and_near_ties(ep, E, K, n, keep, score):
    """Equal logits, and scores a few fp32 steps apart: the order of exact scores, the lower id on a tie."""
    announce("route ties", E, K, n, keep, score)
    rng = np.random.default_rng(E + 6)
    coarse = (np.round(rng.standard_normal((24, E)) * 2) / 2).astype(np.float32)
    near = (0.5 + 3e-7 * rng.integers(-3, 4, (24, E))).astype(np.float32)
    x = np.concatenate([coarse, near, np.zeros((2, E), np.float32)])
    bias = (np.round(rng.standard_normal(E) * 4) / 16).astype(np.float32)
    tiny = (6e-8 * rng.integers(-3, 4, E)).astype(np.float32)
    for b in (None, bias, tiny):
        for top in (1, 2):
            check_route(ep, x, K, b, score, n, keep, top, True, 1.0, f"ties {E} {score}")


def test_route_special_values(ep):
    announce("route special")
    x = np.zeros((4, 16), np.float32)
    x[0, 3], x[0, 5] = np.nan, 2.0
    x[1] = np.nan
    x[2, 4], x[2, 9] = np.inf, 60.0
    x[3, :] = -90.0
    x[3, 2] = -80.0
    for n, keep in ((1, 1), (4, 2)):
        ids, w = route(ep, x, 4, None, "sigmoid", n, keep)
        rid, rw = ob.group_topk(x, 4, None, "sigmoid", n, keep)
        assert np.array_equal(ids[[0, 1, 3]], rid[[0, 1, 3]])
        assert np.array_equal(np.isnan(w), np.isnan(rw))
        ids, w = route(ep, x, 4, None, "softmax", n, keep)
        rid, rw = ob.group_topk(x, 4, None, "softmax", n, keep)
        assert np.array_equal(ids, rid) and np.array_equal(np.isnan(w), np.isnan(rw))
    b = np.zeros(16, np.float32)
    b[7], b[8] = np.inf, np.nan
    ids, _ = route(ep, x, 16, b)
    assert ids[3, 0] == 7 and ids[3, -1] == 8


@pytest.mark.parametrize("T", [1, 4, 5, 8191])
def test_route_many_tokens(ep, T):
    """Every token of a batch against float64 by sorting (the oracle's loop on some)."""
    announce("route tokens", T)
    rng = np.random.default_rng(T)
    x = (1.5 * rng.standard_normal((T, 256))).astype(np.float32)
    bias = (0.1 * rng.standard_normal(256)).astype(np.float32)
    ids, w = route(ep, x, 8, bias, "sigmoid", 8, 4)
    s = 1 / (1 + np.exp(-x.astype(np.float64)))
    c = s + bias
    gs = np.sort(c.reshape(T, 8, 32), axis=2)[:, :, -2:].sum(axis=2)
    kept = np.argsort(-gs, axis=1, kind="stable")[:, :4]
    allowed = np.zeros((T, 8), bool)
    np.put_along_axis(allowed, kept, True, axis=1)
    c = np.where(np.repeat(allowed, 32, axis=1), c, -np.inf)
    assert np.array_equal(ids, np.argsort(-c, axis=1, kind="stable")[:, :8])
    some = np.unique(np.linspace(0, T - 1, 20).astype(int))
    rid, rw = ob.group_topk(x[some], 8, bias, "sigmoid", 8, 4)
    assert np.array_equal(ids[some], rid)
    inside(w[some], rw, 64 * U * rw, "weights")


@pytest.mark.parametrize("E,K,n,keep", [(256, 8, 8, 4), (256, 8, 1, 1), (256, 1, 16, 1), (160, 6, 5, 2), (160, 6, 1, 1), (128, 6, 4, 2),
                                        (96, 3, 3, 2), (128, 8, 16, 9), (192, 8, 4, 2)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_large_batches(ep, E, K, n, keep, score):
    """5123 tokens and more go four to a wave: ordinary rows, masked ones, ties
    and near ties, NaN and infinities, in every place of a wave; the choice is
    that of the oracle, and the tail of the last wave stays unwritten."""
    announce("route large", E, K, n, keep, score)
    rng = np.random.default_rng(E + K + n)
    rows = [1.5 * rng.standard_normal((9, E)), np.round(rng.standard_normal((6, E)) * 2) / 2,
            0.5 + 3e-7 * rng.integers(-3, 4, (6, E)), np.full((1, E), -np.inf), np.zeros((1, E)),
            np.where(rng.random((8, E)) < np.linspace(0.1, 0.99, 8)[:, None], -np.inf, rng.standard_normal((8, E))),
            -30 + 5 * rng.standard_normal((2, E)), 20 + 5 * rng.standard_normal((2, E))]
    x = np.concatenate(rows).astype(np.float32)
    x = np.concatenate([x, x[:4]])
    x[-4, 3], x[-3, 5], x[-2, 1] = np.nan, 90.0, -np.finfo(np.float32).max
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    masked = np.where(rng.random(E) < 0.3, -np.inf, bias).astype(np.float32)
    T = 5123
    big = np.resize(np.arange(len(x)), T)
    for b in (bias, masked, (np.round(bias * 8) / 8).astype(np.float32)):
        for top in (1, 2):
            rid, rw = ob.group_topk(x, K, b, score, n, keep, top, True, 2.0)
            ids, w = route(ep, x[big], K, b, score, n, keep, top, True, 2.0)
            assert np.array_equal(ids, rid[big]), np.argwhere(ids != rid[big])[:4].tolist()
            ok = np.isfinite(rw).all(axis=1)[big]
            assert np.isnan(w[~ok]).any(axis=1).all()
            # softmax: a chosen score's exponent, at most 60 here, and the sum's
            inside(w[ok], rw[big][ok], (64 + (120 if score == "softmax" else 0)) * U * np.abs(rw[big][ok]) + 1e-30, "weights")


@pytest.mark.parametrize("E,K", [(8, 1), (16, 16), (64, 6), (100, 7), (256, 8), (1000, 16), (1024, 32)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_backward(ep, E, K, score):
    rng = np.random.default_rng(E * 3 + K)
    x = (1.5 * rng.standard_normal((45, E))).astype(np.float32)
    x[7, rng.random(E) < 0.7] = -np.inf
    x[8] = -np.inf
    ids, _ = ob.group_topk(x, K, None, score)
    ids[3, K // 2] = -1
    ids[4] = -1
    ids[5, K - 1] = ids[5, 0]                                # the same expert twice
    ids[6, 0] = E + 3                                        # no expert: no route
    dw = rng.standard_normal((45, K)).astype(np.float32)
    for renorm, scale in ((True, 2.5), (False, 1.0)):
        announce("route backward", E, K, score, renorm)
        dl = torch.full((45, E), math.nan, device="cuda")
        ep.moe_router_group_topk_backward(torch.from_numpy(x).cuda(), torch.from_numpy(ids).cuda(),
                                          torch.from_numpy(dw).cuda(), dl,
                                          score=ep.MOE_SCORE_SIGMOID if score == "sigmoid" else ep.MOE_SCORE_SOFTMAX,
                                          renorm=renorm, route_scale=scale)
        ref, mag = ob.group_topk_backward(x, ids, dw, score, renorm, scale)
        inside(f64(dl), ref, 160 * U * mag + 1e-30, f"d_logits {E} {score}")


# ------------------------------------------------------------------ dispatch of FP8 rows

@pytest.mark.parametrize("T,K,H,cap", [(1, 1, 128, 1), (5, 3, 256, 20), (33, 8, 2048, 300), (17, 64, 2176, 1100),
                                       (130, 8, 7168, 200)])
def test_permute_fp8(ep, T, K, H, cap):
    """Bit for bit; -1 and rows past the buffer are skipped, other rows stay."""
    announce("permute fp8", T, K, H, cap)
    rng = np.random.default_rng(T + H)
    x8 = torch.from_numpy(rng.integers(0, 256, (T, H), dtype=np.uint8)).cuda()
    xs = randn(rng, T, H // 128)
    slot = np.full(T * K, -1, np.int32)
    n = min(T * K, cap) * 2 // 3 + 1
    n = min(n, T * K, cap)
    slot[rng.choice(T * K, n, replace=False)] = rng.choice(cap, n, replace=False)
    free = np.nonzero(slot < 0)[0]
    slot[free[::3]] = cap + 5
    slot = slot.reshape(T, K)
    buf = torch.full((cap, H), 0xA5, dtype=torch.uint8, device="cuda")
    bs = torch.full((cap, H // 128), -3.0, device="cuda")
    want, wants = buf.cpu().clone(), bs.cpu().clone()
    ep.moe_permute_fp8(x8, xs, torch.from_numpy(slot).cuda(), buf, bs)
    for t in range(T):
        for k in range(K):
            if 0 <= slot[t, k] < cap:
                want[slot[t, k]], wants[slot[t, k]] = x8[t].cpu(), xs[t].cpu()
    assert torch.equal(buf.cpu(), want) and torch.equal(bs.cpu(), wants)


def test_permute_fp8_is_permute_of_the_norm(ep):
    """norm -> FP8 rows -> moe_permute_fp8 fills what moe_permute makes of the fp32 norm."""
    announce("permute fp8 of norm")
    rng = np.random.default_rng(2)
    x, w = randn(rng, 20, 512), randn(rng, 512)
    y, y8, sc = torch.empty_like(x), torch.empty(20, 512, dtype=torch.uint8, device="cuda"), torch.empty(20, 4, device="cuda")
    ep.moe_add_rms_norm(x, None, w, 1e-6, None, y, y8, sc)
    slot = torch.from_numpy(rng.permutation(40)[:40].astype(np.int32).reshape(20, 2)).cuda()
    a, b = (torch.zeros(40, 512, dtype=torch.uint8, device="cuda") for _ in range(2))
    sa, sb = torch.zeros(40, 4, device="cuda"), torch.zeros(40, 4, device="cuda")
    ep.moe_permute_fp8(y8, sc, slot, a, sa)
    ep.moe_permute(y, slot, b, sb)
    assert torch.equal(a, b) and torch.equal(sa, sb)


# ------------------------------------------------------------------ 4-bit weights

def gemv_case(ep, counts, R, N, K, fmt, group, sdt, act, epi, odt, seed=0):
    """Runs one call; checks every valid row against the oracle and that padding rows keep what they held."""
    L = len(counts)
    rng = np.random.default_rng(N + K + group + seed)
    codes = rng.integers(0, 256, (L, N, K // 2), dtype=np.uint8)
    scales = torch.from_numpy(((0.5 + rng.random((L, N, K // group))) / (4 * math.sqrt(K))).astype(np.float32)).to(DT[sdt])
    counts = np.asarray(counts, np.int32)
    if R:
        offs, cap = np.arange(L + 1, dtype=np.int32) * R, L * R
    else:
        offs = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        cap = int(offs[-1])
    if act == "fp8":
        a = rng.integers(0, 256, (cap, K), dtype=np.uint8)
        a[(a & 0x7f) == 0x7f] = 0
        asc = (0.01 * (0.5 + rng.random((cap, K // 128)))).astype(np.float32)
        av = f64(torch.from_numpy(a).view(torch.float8_e4m3fn)) * np.repeat(asc.astype(np.float64), 128, axis=1)
    else:
        at = torch.from_numpy(rng.standard_normal((cap, K)).astype(np.float32)).to(torch.bfloat16)
        asc, av = None, f64(at)
    pad = np.ones(cap, bool)
    for e in range(L):
        pad[offs[e]:offs[e] + counts[e]] = False
    if act == "fp8":
        a[pad], asc[pad] = 0x7f, math.nan                     # padding rows hold NaN
        ad, asd = torch.from_numpy(a).cuda(), torch.from_numpy(asc).cuda()
    else:
        at[torch.from_numpy(pad)] = math.nan
        ad, asd = at.cuda(), None
    f = ep.MOE_W4_INT4 if fmt == "int4" else ep.MOE_W4_E2M1
    cd, sd = torch.from_numpy(codes).cuda(), scales.cuda()
    pc, ps = torch.empty_like(cd), torch.empty_like(sd)
    ep.moe_pack_w4(cd, sd, f, pc, ps)
    cols = N // 2 if epi == "silu" else N
    out = torch.full((cap, cols), 7.0, dtype=DT[odt], device="cuda")
    ep.moe_grouped_gemv_w4(ad, asd, pc, ps, f, torch.from_numpy(counts).cuda(), torch.from_numpy(offs).cuda(),
                           ep.MOE_EPI_SILU_MUL if epi == "silu" else ep.MOE_EPI_STORE_G, out)
    torch.cuda.synchronize()
    got = f64(out)
    assert np.all(got[pad] == 7.0), "padding rows were written"
    eps = 2.0 ** -20 + 2 * (K // 32 * 2 + K // group + 32) * U
    for e in range(L):
        if counts[e] == 0:
            continue
        rows = slice(offs[e], offs[e] + counts[e])
        g, mag = ob.w4_product(av[rows], codes[e], f64(scales[e]), "int4" if fmt == "int4" else "e2m1")
        b = eps * mag
        if epi == "silu":
            z = ob.silu_mul(g)
            up, gate = g[:, cols:], g[:, :cols]
            b = 1.1 * np.abs(up) * b[:, :cols] + np.abs(gate) * b[:, cols:] + 2.0 ** -18 * np.abs(z) + 1e-30
            g = z
        inside(got[rows], g, b + HALF[odt] * np.abs(g), f"gemv e{e} rows {counts[e]} {N}x{K} {fmt} {group}")
    return out


@pytest.mark.parametrize("fmt", ["int4", "e2m1"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("act", ["bf16", "fp8"])
@pytest.mark.parametrize("sdt", ["f32", "bf16"])
def test_gemv_forms(ep, fmt, group, act, sdt):
    for epi, odt in (("store", "f32"), ("silu", "bf16"), ("store", "bf16"), ("silu", "f32")):
        announce("gemv", fmt, group, act, sdt, epi, odt)
        gemv_case(ep, [1, 0, 5, 16], 16, 256, 640, fmt, group, sdt, act, epi, odt)


@pytest.mark.parametrize("counts,R", [([0], 4), ([0, 0, 0], 0), ([1], 1), ([15, 17, 31, 33], 40), ([63, 64, 65], 70),
                                      ([130, 2, 0, 49], 0), ([200], 0)])
@pytest.mark.parametrize("fmt,act", [("int4", "fp8"), ("e2m1", "bf16"), ("int4", "bf16")])
def test_gemv_row_counts(ep, counts, R, fmt, act):
    announce("gemv rows", counts, R, fmt, act)
    if sum(counts) or R:
        gemv_case(ep, counts, R, 128, 384, fmt, 64, "f32", act, "silu", "f32")
        gemv_case(ep, counts, R, 128, 384, fmt, 128, "f32", act, "store", "f32")


@pytest.mark.parametrize("N,K", [(128, 128), (384, 256), (128, 1408), (1408, 128), (512, 7168), (256, 2176)])
def test_gemv_sizes(ep, N, K):
    for fmt, act, epi in (("int4", "bf16", "store"), ("e2m1", "fp8", "silu")):
        announce("gemv sizes", N, K, fmt)
        gemv_case(ep, [3, 20], 32, N, K, fmt, 128, "f32", act, epi, "f32")


def test_gemv_many_experts(ep):
    announce("gemv L = 1024")
    rng = np.random.default_rng(8)
    gemv_case(ep, rng.integers(0, 4, 1024), 0, 128, 128, "int4", 64, "bf16", "bf16", "store", "f32")


def test_gemv_rows_past_the_buffer(ep):
    """counts that reach past rows_cap are cut there."""
    announce("gemv past the buffer")
    rng = np.random.default_rng(1)
    codes = torch.from_numpy(rng.integers(0, 256, (2, 128, 64), dtype=np.uint8)).cuda()
    sc = torch.ones(2, 128, 1, device="cuda")
    pc, ps = torch.empty_like(codes), torch.empty_like(sc)
    ep.moe_pack_w4(codes, sc, ep.MOE_W4_E2M1, pc, ps)
    a = randn(rng, 8, 128, dt="bf16")
    out, full = torch.zeros(8, 128, device="cuda"), torch.zeros(8, 128, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")               # noqa: E731
    ep.moe_grouped_gemv_w4(a, None, pc, ps, ep.MOE_W4_E2M1, i32(4, 4), i32(0, 4, 8), ep.MOE_EPI_STORE_G, full)
    ep.moe_grouped_gemv_w4(a, None, pc, ps, ep.MOE_W4_E2M1, i32(4, 400), i32(0, 4, 8), ep.MOE_EPI_STORE_G, out)
    assert torch.equal(out, full)


# ------------------------------------------------------------------ streams, graphs

def test_all_operators_in_a_graph(ep):
    """The block's operators captured once, replayed on new contents with eager
    work between the replays: the bits of eager calls."""
    announce("graph")
    rng = np.random.default_rng(12)
    T, H, E, K, L, R, I = 24, 512, 16, 2, 16, 16, 128
    x, res, w = randn(rng, T, H, dt="bf16"), randn(rng, T, H, dt="bf16"), randn(rng, H, dt="bf16")
    h, y = torch.empty_like(x), torch.empty_like(x)
    y8, sc = torch.empty(T, H, dtype=torch.uint8, device="cuda"), torch.empty(T, H // 128, device="cuda")
    logits, bias = randn(rng, T, E), 0.1 * randn(rng, E)
    ids, wt = torch.empty(T, K, dtype=torch.int32, device="cuda"), torch.empty(T, K, device="cuda")
    dl = torch.empty(T, E, device="cuda")
    slot = torch.from_numpy(rng.permutation(L * R)[:T * K].astype(np.int32).reshape(T, K)).cuda()
    buf, bs = torch.zeros(L * R, H, dtype=torch.uint8, device="cuda"), torch.zeros(L * R, H // 128, device="cuda")
    cnt = torch.full((L,), R, dtype=torch.int32, device="cuda")
    off = torch.arange(L + 1, dtype=torch.int32, device="cuda") * R
    codes = torch.from_numpy(rng.integers(0, 256, (L, 2 * I, H // 2), dtype=np.uint8)).cuda()
    s4 = torch.rand(L, 2 * I, H // 32, device="cuda") * 0.05
    pc, ps = torch.empty_like(codes), torch.empty_like(s4)
    zb = torch.zeros(L * R, I, dtype=torch.bfloat16, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty(H, device="cuda")
    ws = torch.empty(ep.moe_add_rms_norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")

    def step():
        ep.moe_add_rms_norm(x, res, w, 1e-6, h, y, y8, sc)
        ep.moe_router_group_topk(logits, K, ids, wt, bias=bias, n_group=4, topk_group=2)
        ep.moe_permute_fp8(y8, sc, slot, buf, bs)
        ep.moe_pack_w4(codes, s4, ep.MOE_W4_INT4, pc, ps)
        ep.moe_grouped_gemv_w4(buf, bs, pc, ps, ep.MOE_W4_INT4, cnt, off, ep.MOE_EPI_SILU_MUL, zb)
        ep.moe_router_group_topk_backward(logits, ids, wt, dl)
        ep.moe_add_rms_norm_backward(y, h, w, 1e-6, dx, dw, ws, dh=res)

    outs = [h, y, y8, sc, ids, wt, buf, bs, zb, dl, dx, dw]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.copy_(randn(rng, T, H, dt="bf16"))
        logits.copy_(randn(rng, T, E))
        for o in outs:
            o.zero_()
        step()
        torch.cuda.synchronize()
        want = [o.clone() for o in outs]
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(outs, want)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), (i, k)


def test_two_streams_at_once(ep):
    """Calls on two streams with their own buffers do not meet."""
    announce("two streams")
    rng = np.random.default_rng(13)
    T, H = 300, 2048
    sets = []
    for _ in range(2):
        dy, h = randn(rng, T, H, dt="bf16"), randn(rng, T, H, dt="bf16")
        sets.append((dy, h, torch.empty_like(dy), torch.empty(H, device="cuda"),
                     torch.empty(ep.moe_add_rms_norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")))
    w = randn(rng, H)
    want = []
    for dy, h, dx, dw, ws in sets:
        ep.moe_add_rms_norm_backward(dy, h, w, 1e-6, dx, dw, ws)
        torch.cuda.synchronize()
        want.append((dx.clone(), dw.clone()))
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        for s, (dy, h, dx, dw, ws) in zip(streams, sets):
            with torch.cuda.stream(s):
                ep.moe_add_rms_norm_backward(dy, h, w, 1e-6, dx, dw, ws)
    torch.cuda.synchronize()
    for (_, _, dx, dw, _), (a, b) in zip(sets, want):
        assert torch.equal(dx, a) and torch.equal(dw, b)
