"""The 4-bit products on activations and scales that are no finite numbers: what
they reach is not finite, and nothing else changes a bit."""
import math

import pytest
import torch

from gpu_util import announce, need_gpu

pytestmark = pytest.mark.gpu
L, R, N, K = 3, 40, 256, 384
COUNTS = [5, 0, 33]


@pytest.fixture(scope="module")
def ep():
    need_gpu()
    import combine_top_expert_amd as ep
    return ep


def setup(ep, fmt, act, group):
    torch.manual_seed(7)
    codes = torch.randint(0, 256, (L, N, K // 2), dtype=torch.uint8, device="cuda")
    scales = 0.01 + 0.01 * torch.rand(L, N, K // group, device="cuda")
    x = torch.randn(L * R, K, device="cuda")
    if act == "fp8":
        a, asc = x.to(torch.float8_e4m3fn), 0.5 + torch.rand(L * R, K // 128, device="cuda")
    else:
        a, asc = x.to(torch.bfloat16), None
    counts = torch.tensor(COUNTS, dtype=torch.int32, device="cuda")
    offsets = torch.arange(L + 1, dtype=torch.int32, device="cuda") * R

    def run(a, asc, scales, epi):
        pc, ps = torch.empty_like(codes), torch.empty_like(scales)
        ep.moe_pack_w4(codes, scales, fmt, pc, ps)
        out = torch.full((L * R, N // 2 if epi == ep.MOE_EPI_SILU_MUL else N), 7.0, device="cuda")
        ep.moe_grouped_gemv_w4(a, asc, pc, ps, fmt, counts, offsets, epi, out)
        torch.cuda.synchronize()
        return out
    return a, asc, scales, run


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("act", ["bf16", "fp8"])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("silu", [False, True])
def test_rows_that_are_not_finite(ep, fmt, act, group, silu):
    announce("gemv broken rows", fmt, act, group, silu)
    epi = ep.MOE_EPI_SILU_MUL if silu else ep.MOE_EPI_STORE_G
    a, asc, scales, run = setup(ep, fmt, act, group)
    clean = run(a, asc, scales, epi)
    rows = [1, 4, 2 * R, 2 * R + 17, 2 * R + 32]            # of experts 0 and 2, in both 16-row halves and past them
    cols = [0, 37, 128, 200, K - 1]
    if act == "bf16":
        values = [math.nan, math.inf, -math.inf, math.nan, math.inf]
        for r, c, v in zip(rows, cols, values):
            a[r, c] = v
    else:
        b = a.view(torch.uint8)
        b[rows[0], cols[0]] = 0x7f
        b[rows[3], cols[3]] = 0xff
        for r, c, v in zip(rows[1:3], cols[1:3], (math.nan, math.inf)):
            asc[r, c // 128] = v
        asc[rows[4], 2] = math.inf
    out = run(a, asc, scales, epi)
    broken = torch.zeros(L * R, dtype=torch.bool, device="cuda")
    broken[rows] = True
    assert not bool(torch.isfinite(out[broken]).any())
    assert torch.equal(out[~broken], clean[~broken])
    if act == "bf16" and fmt == ep.MOE_W4_INT4 or act == "fp8":
        assert bool(torch.isnan(out[rows[0]]).all())
    if act == "bf16" and fmt == ep.MOE_W4_INT4:
        assert bool(torch.isnan(out[broken]).all())


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("act", ["bf16", "fp8"])
@pytest.mark.parametrize("v", [math.nan, math.inf])
def test_weight_scales_that_are_not_finite(ep, fmt, act, v):
    """One scale reaches its own column of its expert's rows."""
    announce("gemv broken scale", fmt, act, v)
    a, asc, scales, run = setup(ep, fmt, act, 64)
    clean = run(a, asc, scales, ep.MOE_EPI_STORE_G)
    scales[2, 129, 3] = v
    out = run(a, asc, scales, ep.MOE_EPI_STORE_G)
    hit = torch.zeros(L * R, N, dtype=torch.bool, device="cuda")
    hit[2 * R:2 * R + COUNTS[2], 129] = True
    assert not bool(torch.isfinite(out[hit]).any())
    assert torch.equal(out[~hit], clean[~hit])
