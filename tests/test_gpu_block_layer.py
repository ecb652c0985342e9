"""The block's operators run together, as a decode step uses them: residual +
norm -> router logits -> routing -> a layer with 4-bit weights on the norm's FP8
(or bf16) rows, against the float64 oracle.

Every stage is computed from what the GPU's previous stage stored, so that a
bound covers one stage's arithmetic.  With half steps 2^-8 of bf16: Z is within
its products' bound and 2^-8 of itself, which W2 carries into `out` as at most
(2^-8 + eps) |Z| |W2|; y adds the routes' weighted sum and its own rounding.
"""
import math

import numpy as np
import pytest
import torch

from gpu_util import announce, need_gpu
from oracle import block as ob
from oracle import moe

pytestmark = pytest.mark.gpu
U = ob.U


@pytest.fixture(scope="module")
def ep():
    need_gpu()
    import combine_top_expert_amd as ep
    return ep


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


T, H, I, E, L, K, R, GROUP = 48, 512, 256, 32, 16, 4, 24, 64


def weights(rng, sdt):
    out = []
    for n, k in ((2 * I, H), (H, I)):
        codes = torch.from_numpy(rng.integers(0, 256, (L, n, k // 2), dtype=np.uint8)).cuda()
        scales = torch.from_numpy(((0.5 + rng.random((L, n, k // GROUP))) / (3 * math.sqrt(k))).astype(np.float32))
        out += [codes, scales.to(sdt).cuda()]
    return out


def make(ep, wdt, x_fp8, fused=True, seed=0, act="bf16", R=R):
    from combine_top_expert_amd.pipeline import LayerShape, MoELayer
    rng = np.random.default_rng(seed)
    layer = MoELayer(LayerShape(T=T, K=K, E=E, expert_begin=8, L=L, H=H, I=I, R=R, act=act, wdt=wdt, x_fp8=x_fp8),
                     fused=fused)
    w13, s13, w2, s2 = weights(rng, torch.bfloat16)
    layer.set_weights(w13, w2, s13, s2)
    return rng, layer, (w13, s13, w2, s2)


def entrance(ep, rng, pad=3):
    """Norm, logits and routing of T tokens, the last `pad` of them padding."""
    bf = torch.bfloat16
    x, res = (torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(bf).cuda() for _ in range(2))
    w = (1 + 0.1 * torch.from_numpy(rng.standard_normal(H).astype(np.float32))).to(bf).cuda()
    wr = torch.from_numpy((rng.standard_normal((E, H)) / math.sqrt(H)).astype(np.float32)).cuda()
    bias = torch.from_numpy((0.1 * rng.standard_normal(E)).astype(np.float32)).cuda()
    st = dict(x=x, res=res, w=w, wr=wr, bias=bias, h=torch.empty_like(x), y=torch.empty_like(x),
              y8=torch.empty(T, H, dtype=torch.uint8, device="cuda"), sc=torch.empty(T, H // 128, device="cuda"),
              logits=torch.empty(T, E, device="cuda"), ids=torch.empty(T, K, dtype=torch.int32, device="cuda"),
              wt=torch.empty(T, K, device="cuda"), pad=pad)
    return st


def step(ep, st, layer):
    ep.moe_add_rms_norm(st["x"], st["res"], st["w"], 1e-6, st["h"], st["y"], st["y8"], st["sc"])
    torch.mm(st["y"].float(), st["wr"].t(), out=st["logits"])
    if st["pad"]:
        st["logits"][T - st["pad"]:].fill_(-math.inf)
    ep.moe_router_group_topk(st["logits"], K, st["ids"], st["wt"], bias=st["bias"], n_group=8, topk_group=4,
                             route_scale=2.5)
    if layer.shape.x_fp8:
        return layer.forward(st["y8"], st["ids"], st["wt"], x_scales=st["sc"])
    return layer.forward(st["y"], st["ids"], st["wt"])


def check(st, layer, w, fmt):
    w13, s13, w2, s2 = w
    s = layer.shape
    ids, wt = ob.group_topk(st["logits"].cpu().numpy(), K, st["bias"].cpu().numpy(), "sigmoid", 8, 4, 2, True, 2.5)
    assert np.array_equal(st["ids"].cpu().numpy(), ids)
    assert np.max(np.abs(f64(st["wt"]) - wt)) <= 64 * U * 2.5
    if st["pad"]:
        assert np.all(ids[T - st["pad"]:] == -1)
    lay = moe.dispatch_layout(ids, E, s.expert_begin, L, s.R)
    assert np.array_equal(layer.slot_of.cpu().numpy(), lay["slot_of"])
    slot = np.asarray(lay["slot_of"])
    if s.x_fp8:
        rows = f64(st["y8"].view(torch.float8_e4m3fn)) * np.repeat(f64(st["sc"]), 128, axis=1)
    else:
        rows = f64(st["y"])
    z_gpu, out_gpu, y_gpu = f64(layer.z), f64(layer.out), f64(layer.y)
    y, y_mag = np.zeros((T, H)), np.zeros((T, H))
    eps = 2.0 ** -20 + 2 * (H // 32 * 2 + H // GROUP + 32) * U
    half = 2.0 ** -8
    counts = np.zeros(L, int)
    for e in range(L):
        tk = np.argwhere((slot >= e * s.R) & (slot < (e + 1) * s.R))
        counts[e] = len(tk)
        if not len(tk):
            continue
        q = slot[tk[:, 0], tk[:, 1]]
        g, mag = ob.w4_product(rows[tk[:, 0]], w13[e].cpu().numpy(), f64(s13[e]), fmt)
        z, b = ob.silu_mul(g), eps * mag
        zb = 1.1 * np.abs(g[:, I:]) * b[:, :I] + np.abs(g[:, :I]) * b[:, I:] + (half + 2.0 ** -18) * np.abs(z) + 1e-30
        if layer.g is not None:       # the unfused layer stores G in fp32: the same terms
            zb = zb + 2 * U * np.abs(z)
        assert np.all(np.abs(z_gpu[q] - z) <= zb), e
        o, omag = ob.w4_product(z_gpu[q], w2[e].cpu().numpy(), f64(s2[e]), fmt)
        assert np.all(np.abs(out_gpu[q] - o) <= eps * omag + half * np.abs(o)), e
        for (t, k), row in zip(tk, q):
            y[t] += wt[t, k] * out_gpu[row]
            y_mag[t] += abs(wt[t, k]) * np.abs(out_gpu[row])
    assert np.all(np.abs(y_gpu - y) <= 80 * U * y_mag + half * np.abs(y) + 1e-30)
    no_route = (slot < 0).all(axis=1)
    assert no_route.any() and not y_gpu[no_route].any()
    print(f"[metric] rows {counts.sum()} of {L} experts, most {counts.max()}, |y| rms {np.sqrt((y ** 2).mean()):.3f}")
    assert np.sqrt((y ** 2).mean()) > 1e-3


@pytest.mark.parametrize("wdt", ["int4", "fp4"])
@pytest.mark.parametrize("x_fp8", [False, True])
@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("R", [24, 0])
def test_decode_step(ep, wdt, x_fp8, fused, R):
    announce("decode step", wdt, x_fp8, fused, R)
    rng, layer, w = make(ep, wdt, x_fp8, fused, R=R)
    if R == 0:                         # exact-fit: slots are not e * R + s; compare with the capacity layer
        _, other, _ = make(ep, wdt, x_fp8, fused)
        st = entrance(ep, rng)
        y = step(ep, st, layer).clone()
        assert torch.equal(y, step(ep, st, other))
        return
    st = entrance(ep, rng)
    step(ep, st, layer)
    torch.cuda.synchronize()
    check(st, layer, w, "int4" if wdt == "int4" else "e2m1")


def test_bound_and_captured_steps(ep):
    """bind_forward, and the layer captured and replayed on new contents with
    eager work between the replays, give the eager bits."""
    announce("bound and captured 4-bit layer")
    rng, layer, w = make(ep, "int4", True)
    st = entrance(ep, rng)
    y = step(ep, st, layer).clone()
    layer.y.zero_()
    for _, f in layer.bind_forward(st["y8"], st["ids"], st["wt"], x_scales=st["sc"]):
        f()
    assert torch.equal(layer.y, y)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        ep.moe_add_rms_norm(st["x"], st["res"], st["w"], 1e-6, st["h"], st["y"], st["y8"], st["sc"])
        ep.moe_router_group_topk(st["logits"], K, st["ids"], st["wt"], bias=st["bias"], n_group=8, topk_group=4,
                                 route_scale=2.5)
        layer.forward(st["y8"], st["ids"], st["wt"], x_scales=st["sc"])
    for i in range(4):
        st["x"].copy_(torch.randn(T, H, device="cuda"))
        y = step(ep, st, layer).clone()
        layer.y.zero_()
        st["ids"].fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(layer.y, y), i


def test_fp8_rows_into_an_fp8_layer(ep):
    """moe_permute_fp8 in front of the block-FP8 GEMMs: the same y as letting
    the layer quantise the fp32 norm itself."""
    announce("fp8 rows, fp8 weights")
    from combine_top_expert_amd.pipeline import LayerShape, MoELayer
    from workloads import make_workload
    wl = make_workload("decode_fp8_small")
    c = wl.cfg
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()                  # noqa: E731
    x = torch.randn(c.T, c.H, device="cuda")
    n, n8, sc = torch.empty_like(x), torch.empty(c.T, c.H, dtype=torch.uint8, device="cuda"), torch.empty(c.T, c.H // 128, device="cuda")
    ep.moe_add_rms_norm(x, None, torch.ones(c.H, device="cuda"), 1e-6, None, n, n8, sc)
    ys = []
    for x_fp8 in (False, True):
        layer = MoELayer(LayerShape(T=c.T, K=c.K, E=c.E, expert_begin=c.expert_begin, L=c.L, H=c.H, I=c.I, R=c.R,
                                    act="f32", wdt="fp8", x_fp8=x_fp8))
        layer.set_weights(dev(wl.w["w13"]), dev(wl.w["w2"]), dev(wl.w["w13_scales"]), dev(wl.w["w2_scales"]))
        args = (n8, dev(wl.ids), dev(wl.weights), sc) if x_fp8 else (n, dev(wl.ids), dev(wl.weights))
        ys.append(layer.forward(*args).clone())
    assert torch.equal(ys[0], ys[1]) and ys[0].any()


def test_layer_refusals(ep):
    announce("layer refusals")
    from combine_top_expert_amd.pipeline import LayerShape
    kw = dict(T=4, K=2, E=8, expert_begin=0, L=8, H=256, I=128, R=8)
    for bad in (dict(act="bf16", wdt="bf16", x_fp8=True), dict(act="f32", wdt="f32", x_fp8=True),
                dict(act="f32", wdt="int4")):
        with pytest.raises(ValueError):
            LayerShape(**kw, **bad)
    _, layer, _ = make(ep, "int4", True)
    x8, ids, wt = (torch.zeros(T, H, dtype=torch.uint8, device="cuda"), torch.zeros(T, K, dtype=torch.int32, device="cuda"),
                   torch.zeros(T, K, device="cuda"))
    with pytest.raises(ValueError, match="x_scales"):
        layer.forward(x8, ids, wt)
    with pytest.raises(ValueError, match="backward"):
        layer.backward(torch.zeros(T, H, device="cuda"), wt)
    _, layer, _ = make(ep, "int4", False)
    with pytest.raises(ValueError, match="x_scales"):
        layer.forward(torch.zeros(T, H, dtype=torch.bfloat16, device="cuda"), ids, wt, torch.zeros(T, H // 128, device="cuda"))


def test_training_entrance(ep):
    """Forward and backward of norm and routing together: the gradient of a
    loss of the routing weights and the normed rows with respect to x, by the
    operators, against differences of the float64 oracle."""
    announce("training entrance")
    rng = np.random.default_rng(3)
    t, h, e, k = 3, 16, 8, 2
    f = lambda *s: rng.standard_normal(s).astype(np.float32)                          # noqa: E731
    x, w, wr, dwt, dy = f(t, h), f(h), f(e, h) / 4, f(t, k), f(t, h)
    cu = lambda a: torch.from_numpy(a).cuda()                                         # noqa: E731
    xg, wg = cu(x), cu(w)
    y = torch.empty_like(xg)
    ep.moe_add_rms_norm(xg, None, wg, 1e-3, None, y)
    logits = y @ cu(wr).t()
    ids, wt = torch.empty(t, k, dtype=torch.int32, device="cuda"), torch.empty(t, k, device="cuda")
    ep.moe_router_group_topk(logits, k, ids, wt, n_group=2, topk_group=1)
    dl = torch.empty_like(logits)
    ep.moe_router_group_topk_backward(logits, ids, cu(dwt), dl)
    dx, dw = torch.empty_like(xg), torch.empty_like(wg)
    ws = torch.empty(ep.moe_add_rms_norm_backward_workspace_bytes(t, h), dtype=torch.uint8, device="cuda")
    ep.moe_add_rms_norm_backward(cu(dy) + dl @ cu(wr), xg, wg, 1e-3, dx, dw, ws)
    chosen = ids.cpu().numpy()

    def loss(xv, wv):
        n, _ = ob.rms_norm(xv, wv, 1e-3)
        lg = n @ wr.astype(np.float64).T
        total = (n * dy).sum()
        for i in range(t):
            s = np.array(ob.scores(lg[i], "sigmoid"))[chosen[i]]
            total += (s / (s.sum() + 1e-20) * dwt[i]).sum()
        return total
    x64, w64 = x.astype(np.float64), w.astype(np.float64)
    assert np.array_equal(chosen, ob.group_topk((ob.rms_norm(x64, w64, 1e-3)[0] @ wr.astype(np.float64).T).astype(np.float32),
                                                k, None, "sigmoid", 2, 1)[0])
    for i in range(t):
        for j in range(h):
            d = np.zeros((t, h))
            d[i, j] = 1e-5
            assert abs((loss(x64 + d, w64) - loss(x64 - d, w64)) / 2e-5 - float(dx[i, j])) < 2e-5
    for j in range(h):
        d = np.zeros(h)
        d[j] = 1e-5
        assert abs((loss(x64, w64 + d) - loss(x64, w64 - d)) / 2e-5 - float(dw[j])) < 2e-5
