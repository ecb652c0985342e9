"""Weights that set_weights refuses leave the layer as it was: its forward, bound
calls and captured steps run on the weights that it had."""
import math

import pytest
import torch

from gpu_util import announce, need_gpu
from test_gpu_experts_grads import captured

pytestmark = pytest.mark.gpu
T, H, I, E, L, K, R, GROUP = 24, 256, 128, 8, 4, 2, 24, 64


@pytest.fixture(scope="module")
def ep():
    need_gpu()
    import combine_top_expert_amd as ep
    return ep


def weights(wdt, seed):
    """(w13, w2, scales of w13, scales of w2)"""
    g = torch.Generator(device="cuda").manual_seed(seed)
    if wdt in ("bf16", "f32"):
        dt = torch.bfloat16 if wdt == "bf16" else torch.float32
        return (*((torch.randn(L, n, k, generator=g, device="cuda") / math.sqrt(k)).to(dt) for n, k in ((2 * I, H), (H, I))), None, None)
    codes, scales = [], []
    for n, k in ((2 * I, H), (H, I)):
        codes.append(torch.randint(0, 256, (L, n, k // 2), dtype=torch.uint8, generator=g, device="cuda"))
        scales.append(torch.randint(118, 122, (L, n, k // 32), dtype=torch.uint8, generator=g, device="cuda") if wdt == "mx4" else
                      (0.5 + torch.rand(L, n, k // GROUP, generator=g, device="cuda")) / (3 * math.sqrt(k)))
    return (*codes, *scales)


def unaligned(t):
    """A contiguous copy that begins one element behind a 16-byte boundary."""
    flat = torch.empty(t.numel() + 16, dtype=t.dtype, device=t.device)
    v = flat[1:1 + t.numel()].view(t.shape)
    return v.copy_(t)


@pytest.mark.parametrize("bad", [0, 1])
@pytest.mark.parametrize("wdt", ["mx4", "int4", "fp4"])
def test_unaligned_4_bit_weights(ep, wdt, bad):
    announce("unaligned 4-bit weights", wdt, bad)
    check(ep, wdt, bad)


@pytest.mark.parametrize("wdt", ["bf16", "f32"])
def test_unaligned_weights(ep, wdt):
    announce("unaligned weights", wdt)
    check(ep, wdt, 0)


def check(ep, wdt, bad):
    from combine_top_expert_amd.pipeline import LayerShape, MoELayer
    layer = MoELayer(LayerShape(T=T, K=K, E=E, expert_begin=0, L=L, H=H, I=I, R=R, act="f32" if wdt == "f32" else "bf16", wdt=wdt))
    layer.set_weights(*weights(wdt, 0))
    x = torch.randn(T, H, device="cuda").to(torch.float32 if wdt == "f32" else torch.bfloat16)
    ids = torch.randint(0, E, (T, K), dtype=torch.int32, device="cuda")
    wt = torch.rand(T, K, device="cuda")
    want = layer.forward(x, ids, wt).clone()
    assert bool(want.isfinite().all()) and bool(want.any())
    bound = layer.bind_forward(x, ids, wt)
    graph = torch.cuda.CUDAGraph()
    with captured(graph):
        layer.forward(x, ids, wt)
    runs = (lambda: layer.forward(x, ids, wt), lambda: [f() for _, f in bound], graph.replay)

    def as_it_was():
        for run in runs:
            layer.y.zero_()
            run()
            torch.cuda.synchronize()
            assert torch.equal(layer.y, want)

    new = list(weights(wdt, 1))
    new[bad] = unaligned(new[bad])
    with pytest.raises(ep.MoEError):
        layer.set_weights(*new)
    as_it_was()
    if wdt in ("bf16", "f32"):
        return
    # scales of a group that the library does not have, for the second weights only
    if wdt != "mx4":
        new = list(weights(wdt, 1))
        new[3] = new[3][:, :, :1].contiguous()
        new[3] = torch.cat([new[3]] * (I // 16), 2)
        with pytest.raises((ep.MoEError, ValueError)):
            layer.set_weights(*new)
        as_it_was()
    # and what it accepts reaches all of them
    new = weights(wdt, 1)
    layer.set_weights(*new)
    fresh = MoELayer(layer.shape)
    fresh.set_weights(*new)
    want = fresh.forward(x, ids, wt).clone()
    as_it_was()
