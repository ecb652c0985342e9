"""Numbers at the ends of MX4's range and broken blocks, through quantisation, the
products and a layer.  A code is one rounding, so bytes are equal; products
against oracle/experts.py within the bounds of test_gpu_experts_mx4.py."""
import math

import numpy as np
import pytest
import torch

from gpu_util import announce, need_gpu
from oracle import experts as ox
from test_gpu_experts_mx4 import gemm_case, u8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ep():
    need_gpu()
    import combine_top_expert_amd as ep
    return ep


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_where_values_become_infinite(ep, dt):
    """From 3.5 * 2^126 on the scale is 2^126 and the code 4 (3.5 is a tie, to the even code) or more: 2^128 and above."""
    announce("quantize_mx4 3.5 * 2^126", dt)
    tops = [3.484375, 3.5, 3.515625, 3.59375, 3.75, 3.984375]      # in bf16 too
    x = torch.zeros(2 * len(tops), 32, dtype=dt)
    for i, t in enumerate(tops):
        x[2 * i, 7], x[2 * i + 1, 31] = t * 2.0 ** 126, -t * 2.0 ** 126
    x = x.cuda()
    codes, scales, values = u8(x.shape[0], 16), u8(x.shape[0], 1), torch.zeros_like(x)
    ep.moe_quantize_mx4(x, codes, scales, values=values)
    ref = ox.quantise(x.double().cpu().numpy())
    assert np.array_equal(codes.cpu().numpy(), ref[0]) and np.array_equal(scales.cpu().numpy(), ref[1])
    finite = values.isfinite().all(1).reshape(-1, 2).all(1).cpu().tolist()
    assert finite == [t < 3.5 for t in tops]
    assert float(values[0, 7]) == 3.0 * 2.0 ** 126                 # 6 * 2^125


@pytest.mark.parametrize("odt", ["bf16", "f32", "mx4"])
@pytest.mark.parametrize("counts,N,K", [([40, 3], 128, 512), ([7], 64, 128), ([2, 130], 192, 640), ([300, 1], 64, 896)])
def test_broken_rows(ep, counts, N, K, odt):
    """Rows as quantisation leaves broken ones: scale 255 and codes of 0."""
    announce("gemm_mx4 broken rows, zero codes", counts, N, K, odt)
    args, *_, pad, cap = gemm_case(ep, counts, 0, N, K)
    a, sa = args[0].clone(), args[1].clone()
    rows = sum(counts)
    where = [(0, 0), (rows // 2, K // 32 - 1), (rows - 1, 3)]
    for q, b in where:
        a[q, 16 * b:16 * b + 16], sa[q, b] = 0, 255
    if odt == "mx4":
        out, sc = u8(cap, N // 4), u8(cap, N // 64)
        ep.moe_grouped_gemm_mx4(a, sa, *args[2:], ep.MOE_EPI_SILU_MUL, out, out_scales=sc)
        broken = sc == 255
    else:
        out = torch.zeros(cap, N, dtype=torch.bfloat16 if odt == "bf16" else torch.float32, device="cuda")
        ep.moe_grouped_gemm_mx4(a, sa, *args[2:], ep.MOE_EPI_STORE_G, out)
        broken = out.isnan()
    assert torch.equal(broken.all(1), broken.any(1))
    assert broken.all(1).nonzero().flatten().tolist() == sorted({q for q, _ in where})


@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("epi,odt", [("store", "bf16"), ("store", "f32"), ("silu", "bf16"), ("silu", "f32"), ("silu", "mx4")])
@pytest.mark.parametrize("K", [128, 256, 384, 512, 640, 896, 1408])
def test_broken_weight_columns(ep, K, epi, odt, zero):
    """A 255 among a weight column's scales: that column is NaN, the others are what they were.  The last expert's last
    16 columns are among them, whose scales end the buffer."""
    announce("gemm_mx4 broken weights", K, epi, odt, zero)
    counts, N = [5, 0, 21], 128
    (a, sa, _, _, counts_d, offsets_d), *_, pad, cap = gemm_case(ep, counts, 0, N, K)
    rng = np.random.default_rng(K)
    w = torch.from_numpy(rng.integers(0, 256, (3, N, K // 2), dtype=np.uint8)).cuda()
    ws = torch.from_numpy(rng.integers(116, 120, (3, N, K // 32), dtype=np.uint8)).cuda()
    broken = {0: [(0, 0), (17, K // 32 - 1)], 2: [(112, 1), (125, 3), (126, K // 32 - 2), (127, K // 32 - 1)]}
    bw, bws = w.clone(), ws.clone()
    for e, at in broken.items():
        for n, b in at:
            bws[e, n, b] = 255
            if zero:
                bw[e, n, 16 * b:16 * b + 16] = 0
    outs = []
    for codes, scales in ((w, ws), (bw, bws)):
        pw, ps = torch.empty_like(w), torch.empty_like(ws)
        ep.moe_pack_mx4(codes, scales, pw, ps)
        cols = N if epi == "store" else N // 4 if odt == "mx4" else N // 2
        dt = torch.uint8 if odt == "mx4" else torch.bfloat16 if odt == "bf16" else torch.float32
        out, sc = torch.zeros(cap, cols, dtype=dt, device="cuda"), u8(cap, N // 64) if odt == "mx4" else None
        ep.moe_grouped_gemm_mx4(a, sa, pw, ps, counts_d, offsets_d, ep.MOE_EPI_STORE_G if epi == "store" else ep.MOE_EPI_SILU_MUL,
                                out, out_scales=sc)
        outs.append((out, sc))
    for e, (first, n) in enumerate(((0, 5), (5, 0), (5, 21))):
        rows = slice(first, first + n)
        bad = sorted({c if epi == "store" else c % (N // 2) for c, _ in broken.get(e, [])})
        if odt == "mx4":                                           # a block of 32 columns shares the NaN
            blocks = sorted({c // 32 for c in bad})
            good = [b for b in range(N // 64) if b not in blocks]
            assert bool((outs[1][1][rows][:, blocks] == 255).all())
            assert torch.equal(outs[1][1][rows][:, good], outs[0][1][rows][:, good])
            part = lambda o: o[rows].reshape(n, N // 64, 16)[:, good]  # noqa: E731
            assert torch.equal(part(outs[1][0]), part(outs[0][0]))
        else:
            nan = outs[1][0][rows].isnan()
            assert not n or nan.all(0).nonzero().flatten().tolist() == bad and torch.equal(nan.all(0), nan.any(0))
            good = [c for c in range(outs[0][0].shape[1]) if c not in bad]
            assert torch.equal(outs[1][0][rows][:, good], outs[0][0][rows][:, good])


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_broken_tokens_stay_alone(ep, act):
    """An infinite and a NaN token through a whole MX4 layer: only their outputs are NaN."""
    announce("mx4 layer, broken tokens", act)
    from combine_top_expert_amd.pipeline import LayerShape, MoELayer
    T, H, I, E, L, K = 40, 384, 256, 8, 8, 2
    dt = torch.float32 if act == "f32" else torch.bfloat16
    g = torch.Generator().manual_seed(4)
    layer = MoELayer(LayerShape(T=T, K=K, E=E, expert_begin=0, L=L, H=H, I=I, R=0, act=act, wdt="mx4"))
    layer.set_weights(*((torch.randn(L, n, k, generator=g) / math.sqrt(k)).to(dt).cuda() for n, k in ((2 * I, H), (H, I))))
    x = torch.randn(T, H, generator=g).to(dt).cuda()
    ids = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)]).int().cuda()
    wt = torch.rand(T, K, generator=g).cuda() + 0.1
    good = layer.forward(x, ids, wt).clone()
    x[5, 100], x[23, 383], x[39, 0] = math.inf, math.nan, -math.inf
    bad = layer.forward(x, ids, wt)
    broken = [5, 23, 39]
    rest = [t for t in range(T) if t not in broken]
    assert bool(bad[broken].isnan().all())
    assert torch.equal(bad[rest], good[rest]) and bool(good.isfinite().all())


def test_scales_of_8_bit_states_at_any_four_bytes(ep):
    announce("adamw, scales 4-byte aligned")
    f8, n = torch.float8_e4m3fn, 1500
    g = torch.Generator(device="cuda").manual_seed(2)
    w, grad = torch.randn(n, generator=g, device="cuda"), torch.randn(n, generator=g, device="cuda")
    results = []
    for off in range(4):
        flat = [torch.zeros(32, device="cuda") for _ in range(2)]
        scales = [t[off:off + 12] for t in flat]
        p, m, v = w.clone(), *(torch.zeros(n, dtype=torch.uint8, device="cuda").view(f8) for _ in range(2))
        for step in (1, 2):
            ep.moe_adamw_step([p], [grad], [m], [v], 1e-2, step, exp_avg_scales=[scales[0]], exp_avg_sq_scales=[scales[1]], seed=5)
        assert not any(bool(t[:off].any()) or bool(t[off + 12:].any()) for t in flat)
        results.append([p, m.view(torch.uint8), v.view(torch.uint8), *scales])
    for r in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, results[0]))
    assert bool(results[0][3].all()) and bool(results[0][4].all())
