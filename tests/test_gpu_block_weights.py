"""New 4-bit weights in a layer that has some already, bound or captured."""
import math

import numpy as np
import pytest
import torch

from gpu_util import announce, need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ep():
    need_gpu()
    import combine_top_expert_amd as ep
    return ep


T, H, I, E, L, K, R, GROUP = 24, 256, 128, 8, 8, 2, 24, 64


def weights(seed):
    rng = np.random.default_rng(seed)
    out = []
    for n, k in ((2 * I, H), (H, I)):
        out.append(torch.from_numpy(rng.integers(0, 256, (L, n, k // 2), dtype=np.uint8)).cuda())
        out.append(torch.from_numpy(((0.5 + rng.random((L, n, k // GROUP))) / (3 * math.sqrt(k))).astype(np.float32)).cuda())
    return out


def make(wdt):
    from combine_top_expert_amd.pipeline import LayerShape, MoELayer
    return MoELayer(LayerShape(T=T, K=K, E=E, expert_begin=0, L=L, H=H, I=I, R=R, act="bf16", wdt=wdt))


@pytest.mark.parametrize("wdt", ["int4", "fp4"])
def test_weight_update_reaches_bound_and_captured_steps(ep, wdt):
    announce("4-bit weight update", wdt)
    layer = make(wdt)
    w13, s13, w2, s2 = weights(0)
    layer.set_weights(w13, w2, s13, s2)
    x = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    ids = torch.randint(0, E, (T, K), dtype=torch.int32, device="cuda")
    wt = torch.rand(T, K, device="cuda")
    first = layer.forward(x, ids, wt).clone()
    bound = layer.bind_forward(x, ids, wt)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward(x, ids, wt)
    held = [t.data_ptr() for pair in layer.w4 for t in pair]
    for seed, stream in ((1, torch.cuda.Stream()), (2, torch.cuda.current_stream())):
        w13, s13, w2, s2 = weights(seed)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            layer.set_weights(w13, w2, s13, s2)
        torch.cuda.synchronize()
        # first where the packed copies are: bound calls and graphs read there
        assert [t.data_ptr() for pair in layer.w4 for t in pair] == held
        fresh = make(wdt)
        fresh.set_weights(w13, w2, s13, s2)
        want = fresh.forward(x, ids, wt).clone()
        assert not torch.equal(want, first)
        for run in (graph.replay, lambda: [f() for _, f in bound], lambda: layer.forward(x, ids, wt)):
            layer.y.zero_()
            run()
            torch.cuda.synchronize()
            assert torch.equal(layer.y, want)


def test_refused_weights_leave_the_layer_as_it_was(ep):
    announce("4-bit weights refused")
    layer = make("int4")
    w13, s13, w2, s2 = weights(0)
    layer.set_weights(w13, w2, s13, s2)
    x = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    ids = torch.randint(0, E, (T, K), dtype=torch.int32, device="cuda")
    wt = torch.rand(T, K, device="cuda")
    want = layer.forward(x, ids, wt).clone()
    with pytest.raises((TypeError, ValueError)):
        layer.set_weights(w13, w2, s13, s2[:, :, :0])          # no scales of W2
    with pytest.raises((TypeError, ValueError)):
        layer.set_weights(w13, w2, s13)
    assert torch.equal(layer.forward(x, ids, wt), want)
    # another scale group: new packed copies
    s13b, s2b = s13.repeat_interleave(2, 2), s2.repeat_interleave(2, 2)
    layer.set_weights(w13, w2, s13b, s2b)
    fresh = make("int4")
    fresh.set_weights(w13, w2, s13b, s2b)
    assert torch.equal(layer.forward(x, ids, wt), fresh.forward(x, ids, wt))
