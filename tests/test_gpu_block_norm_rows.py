"""The norm and its gradients on batches of 32 MB and more, whose kernels read and
write past the caches with one, two or four chunks of 8 columns a lane, and
whose d_weight is reduced over up to 4096 blocks: every row against float64.

Bounds (u = 2^-24): a row's sum of squares is a lane's serial sum of at most 32
terms, a 6-step wave sum and at most 16 waves, 54 u, so 27 u on r and 30 u with
the mean, the root and the quotient; y is two products on: 34 u.  dx: the sum of
h w dy is within 56 u of the sum of its magnitudes, k = that r / H within 88 u,
n k within 120 u, r (w dy - n k) within 153 u of the terms' magnitudes: 160 u.
d_weight: 32 u for dy n, then one addition a row of a block, and the second
pass's serial and final sums.
"""
import math

import pytest
import torch

from gpu_util import announce, need_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": U}
STREAM = 32 << 20                          # bytes of rows from which the kernels change


@pytest.fixture(scope="module")
def ep():
    need_gpu()
    import combine_top_expert_amd as ep
    return ep


def randn(*shape, dt, scale=1.0):
    return (torch.randn(*shape, device="cuda") * scale).to(DT[dt])


def inside(got, ref, bound, what):
    """|got - ref| <= bound everywhere, a block of rows at a time."""
    assert got.shape == ref.shape, what
    worst = ((got.double() - ref).abs() / bound.clamp(min=1e-300)).max()
    assert bool(torch.isfinite(got.float()).all()), what
    print(f"[metric] {what}: worst error / bound {float(worst):.3f}", flush=True)
    assert float(worst) <= 1.0, what


ROWS = [("bf16", 8, 2097171), ("bf16", 512, 32771), ("bf16", 1408, 11927), ("bf16", 2048, 8191), ("bf16", 2056, 8195),
        ("bf16", 4096, 4099), ("bf16", 4104, 4099), ("bf16", 7168, 2347), ("bf16", 8200, 2051), ("bf16", 16384, 1031),
        ("f32", 1408, 5963), ("f32", 4096, 2051), ("f32", 4104, 2049), ("f32", 7168, 1173), ("f32", 16384, 517),
        ("bf16", 4096, 4096), ("bf16", 4096, 4095)]


@pytest.mark.parametrize("dt,H,T", ROWS)
def test_norm_of_large_batches(ep, dt, H, T):
    torch.manual_seed(H + T)
    x, res = randn(T, H, dt=dt), randn(T, H, dt=dt, scale=3.0)
    x[T // 2] = 0                                           # a row of zeros and one that cancels
    res[T // 2] = 0
    res[T - 1] = -x[T - 1]
    wdt = "f32" if H == 7168 else dt
    w = (1 + 0.3 * torch.randn(H, device="cuda")).to(DT[wdt])
    for r, outs in ((res, "hy8"), (None, "y"), (res, "h8"), (None, "8")):
        if "8" in outs and H % 128:
            outs = outs.replace("8", "")
            if not outs:
                continue
        announce("norm", dt, T, H, r is not None, outs)
        h = torch.full_like(x, math.nan) if "h" in outs else None
        y = torch.full_like(x, math.nan) if "y" in outs else None
        y8 = torch.full((T, H), 0x7f, dtype=torch.uint8, device="cuda") if "8" in outs else None
        sc = torch.full((T, H // 128), math.nan, device="cuda") if "8" in outs else None
        ep.moe_add_rms_norm(x, r, w, 1e-6, h, y, y8, sc)
        torch.cuda.synchronize()
        href = x if r is None else (x.float() + r.float()).to(DT[dt])
        if h is not None:
            assert torch.equal(h, href)
        f = href.double()
        ref = f / torch.sqrt((f * f).mean(1, keepdim=True) + 1e-6) * w.double()
        if y is not None:
            inside(y, ref, (HALF[dt] + 34 * U) * ref.abs() + 1e-40, f"y {dt} {T}x{H}")
        if y8 is not None:
            b = ref.reshape(T, H // 128, 128)
            amax = b.abs().amax(2).clamp(min=1e-4)
            inside(sc, amax / 448, 36 * U * amax / 448, f"scales {dt} {T}x{H}")
            v = y8.view(torch.float8_e4m3fn).float().reshape(b.shape).double() * sc.double()[..., None]
            # half a step of e4m3, of a normal value or next to 0
            half = torch.maximum(2.0 ** -4 * b.abs(), 2.0 ** -10 * sc.double()[..., None])
            inside(v, b, half * (1 + 2.0 ** -10) + 40 * U * b.abs(), f"codes {dt} {T}x{H}")
        del f, ref


BACKWARD = [("bf16", "bf16", 512, 65541), ("bf16", "bf16", 256, 131077), ("bf16", "bf16", 8, 2097171), ("bf16", "f32", 1408, 11927),
            ("bf16", "bf16", 4096, 8195), ("bf16", "bf16", 4096, 4099), ("bf16", "bf16", 4104, 4099), ("bf16", "bf16", 7168, 8195),
            ("bf16", "f32", 7168, 2347), ("bf16", "bf16", 16384, 1031), ("f32", "f32", 256, 65541), ("f32", "f32", 1408, 8197),
            ("f32", "bf16", 4096, 2051), ("f32", "f32", 7168, 1173), ("f32", "f32", 8192, 1027), ("f32", "f32", 8200, 1025),
            ("f32", "f32", 16384, 517)]


@pytest.mark.parametrize("dt,wdt,H,T", BACKWARD)
def test_norm_backward_of_large_batches(ep, dt, wdt, H, T):
    torch.manual_seed(H + 3 * T)
    dy, h, dh = randn(T, H, dt=dt), randn(T, H, dt=dt, scale=2.0), randn(T, H, dt=dt)
    assert T * H * dy.element_size() >= STREAM
    w = (1 + 0.3 * torch.randn(H, device="cuda")).to(DT[wdt])
    need = ep.moe_add_rms_norm_backward_workspace_bytes(T, H)
    blocks = need // (4 * H)
    print(f"[metric] {T}x{H} {dt}: {blocks} blocks")
    second = 32 if blocks <= 1024 else 128                  # rows that the second pass adds side by side
    adds = -(-T // blocks) + -(-blocks // second) + second
    f, g = h.double(), dy.double()
    r = 1.0 / torch.sqrt((f * f).mean(1, keepdim=True) + 1e-6)
    n, u = f * r, g * w.double()
    del f
    un = (u * n).mean(1, keepdim=True)
    base = r * (u - n * un)
    size = r * (u.abs() + n.abs() * (u * n).abs().mean(1, keepdim=True))
    wref, wsize = (g * n).sum(0), (g * n).abs().sum(0)
    del n, u, g
    for d in (None, dh):
        announce("norm backward", dt, wdt, T, H, d is not None)
        dx, dw = torch.full_like(dy, math.nan), torch.full((H,), math.nan, device="cuda")
        ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
        ep.moe_add_rms_norm_backward(dy, h, w, 1e-6, dx, dw, ws, dh=d)
        torch.cuda.synchronize()
        ref, mag = (base, size) if d is None else (base + d.double(), size + d.double().abs())
        inside(dx, ref, HALF[dt] * ref.abs() + 160 * U * mag + 1e-40, f"dx {dt} {T}x{H}")
        inside(dw, wref, (32 + adds) * U * wsize + 1e-40, f"dw {dt} {T}x{H}")
        # the same bits again, and over each input
        for name in ("dy", "h", "dh"):
            if name == "dh" and d is None:
                continue
            at = {"dy": dy.clone(), "h": h.clone(), "dh": None if d is None else d.clone()}
            dw2 = torch.empty_like(dw)
            ep.moe_add_rms_norm_backward(at["dy"], at["h"], w, 1e-6, at[name], dw2, ws, dh=at["dh"])
            torch.cuda.synchronize()
            assert torch.equal(at[name], dx) and torch.equal(dw2, dw), name


def test_large_norm_in_place(ep):
    """Residual stream and norm over their inputs past 32 MB."""
    announce("large norm in place")
    torch.manual_seed(1)
    x, r = randn(2347, 7168, dt="bf16"), randn(2347, 7168, dt="bf16")
    w = randn(7168, dt="bf16")
    h, y = torch.empty_like(x), torch.empty_like(x)
    ep.moe_add_rms_norm(x, r, w, 1e-5, h, y)
    x2, r2 = x.clone(), r.clone()
    ep.moe_add_rms_norm(x2, r2, w, 1e-5, r2, x2)
    assert torch.equal(r2, h) and torch.equal(x2, y)
