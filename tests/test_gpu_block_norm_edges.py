"""Rows that hold a NaN or an infinity, and rows of zeros without an epsilon,
through moe_add_rms_norm's FP8 output: what is broken in y stays visible in the
codes and scales."""
import math

import pytest
import torch

from gpu_util import announce, need_gpu

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def ep():
    need_gpu()
    import combine_top_expert_amd as ep
    return ep


def norm8(ep, x, res, w, eps):
    """y, and the codes' values and scales of the same call, in groups of 128."""
    T, H = x.shape
    y = torch.empty_like(x)
    y8 = torch.zeros(T, H, dtype=torch.uint8, device="cuda")
    sc = torch.zeros(T, H // 128, device="cuda")
    ep.moe_add_rms_norm(x, res, w, eps, None, y, y8, sc)
    torch.cuda.synchronize()
    return y, y8, sc


def check_groups(x, res, w, eps, y, y8, sc):
    """In plain fp32: a group with a NaN is NaN in its scale and codes; one whose
    largest magnitude is infinite has an infinite scale, code 0 at its finite
    values and NaN at its infinities.  Either way every element is NaN once it
    is scaled."""
    T, H = x.shape
    h = x if res is None else (x.float() + res.float()).to(x.dtype)
    f = h.float()
    ref = f * (1.0 / ((f * f).mean(1, keepdim=True) + eps).sqrt()) * w.float()
    g = ref.reshape(T, H // 128, 128)
    nan, inf = torch.isnan(g).any(2), torch.isinf(g).any(2)
    bad = nan | inf
    v = y8.view(torch.float8_e4m3fn).float().reshape(g.shape)
    assert torch.equal(torch.isnan(y), torch.isnan(ref))
    assert bool(torch.isnan(sc[nan]).all()) and bool(torch.isnan(v[nan]).all())
    only = inf & ~nan
    assert bool(torch.isinf(sc[only]).all())
    assert torch.equal(torch.isnan(v[only]), torch.isinf(g[only])) and not bool(v[only][~torch.isinf(g[only])].any())
    assert bool(torch.isnan((v * sc[..., None])[bad]).all())
    assert bool(torch.isfinite(sc[~bad]).all()) and bool(torch.isfinite(v[~bad]).all())
    return bad


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", [(8, 128), (8, 384), (8, 7168), (8, 16384), (12000, 1408), (2400, 7168)])
@pytest.mark.parametrize("res", [False, True])
def test_norm_fp8_of_broken_rows(ep, dt, T, H, res):
    announce("norm fp8 broken rows", dt, T, H, res)
    torch.manual_seed(H + T)
    x = torch.randn(T, H, device="cuda").to(DT[dt])
    r = torch.randn(T, H, device="cuda").to(DT[dt]) if res else None
    w = (1 + 0.1 * torch.randn(H, device="cuda")).to(DT[dt])
    _, clean8, cleans = norm8(ep, x, r, w, 1e-6)
    good = torch.ones(T, dtype=torch.bool, device="cuda")
    for t, (c, v) in {1: (5, math.nan), 2: (H - 1, math.inf), 3: (64, -math.inf), T - 1: (17, math.nan)}.items():
        (x if r is None or t % 2 else r)[t, c] = v
        good[t] = False
    y, y8, sc = norm8(ep, x, r, w, 1e-6)
    bad = check_groups(x, r, w, 1e-6, y, y8, sc)
    assert bool(bad[1].all()) and bool(bad[T - 1].all())             # a NaN makes its whole row NaN
    assert bool(bad[2].any()) and bool(bad[3].any())
    assert torch.equal(y8[good], clean8[good]) and torch.equal(sc[good], cleans[good])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_norm_fp8_of_zero_rows_without_epsilon(ep, dt):
    announce("norm fp8 zero rows", dt)
    x = torch.randn(6, 256, device="cuda").to(DT[dt])
    x[2], x[5] = 0, 0
    w = torch.ones(256, device="cuda").to(DT[dt])
    y, y8, sc = norm8(ep, x, None, w, 0.0)
    bad = check_groups(x, None, w, 0.0, y, y8, sc)
    assert bad.any(1).tolist() == [False, False, True, False, False, True] and bool(bad[2].all())


@pytest.mark.parametrize("v", [math.nan, math.inf, -math.inf])
def test_norm_fp8_of_broken_weights(ep, v):
    announce("norm fp8 broken weight", v)
    x = torch.randn(5, 512, device="cuda")
    w = torch.ones(512, device="cuda")
    w[130] = v
    y, y8, sc = norm8(ep, x, None, w, 1e-6)
    bad = check_groups(x, None, w, 1e-6, y, y8, sc)
    assert bad.tolist() == [[False, True, False, False]] * 5
