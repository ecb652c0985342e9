"""MoELayer.step applies the gradients of a backward once: what it refuses, and
that a refused step leaves weights and count as they were."""
import contextlib
import gc
import math

import pytest
import torch

from gpu_util import announce, need_gpu

pytestmark = pytest.mark.gpu
T, H, I, E, L, K, R = 24, 256, 128, 8, 4, 2, 24


@pytest.fixture(scope="module")
def ep():
    need_gpu()
    import combine_top_expert_amd as ep
    return ep


def weights(g):
    r = lambda *s: (torch.randn(*s, generator=g) / math.sqrt(s[-1])).to(torch.bfloat16).cuda()  # noqa: E731
    return r(L, 2 * I, H), r(L, H, I)


@contextlib.contextmanager
def captured(graph):
    """A capture that no garbage collection falls into: an old graph which is destroyed during one ends the process."""
    torch.cuda.synchronize()
    gc.collect()
    gc.disable()
    try:
        with torch.cuda.graph(graph):
            yield
    finally:
        gc.enable()


class Case:
    def __init__(self, seed=0):
        from combine_top_expert_amd.pipeline import LayerShape, MoELayer
        g = self.g = torch.Generator().manual_seed(seed)
        self.layer = MoELayer(LayerShape(T=T, K=K, E=E, expert_begin=2, L=L, H=H, I=I, R=R, act="bf16", wdt="bf16"))
        self.ws = weights(g)
        self.layer.set_weights(*self.ws)
        self.layer.prepare_step(weight_decay=0.1)
        self.x, self.dy = (torch.randn(T, H, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
        self.ids = torch.randint(0, E, (T, K), generator=g, dtype=torch.int32).cuda()
        self.wt = torch.rand(T, K, generator=g).cuda()

    def forward(self):
        self.layer.forward(self.x, self.ids, self.wt)

    def backward(self, **more):
        self.forward()
        self.layer.backward(self.dy, self.wt, **more)

    def everything(self):
        o = self.layer.adamw
        return [t.clone() for t in [*o["weights"], *o["masters"], *o["moments"][0], *o["moments"][1]]], o["number"]

    def refused(self, match="weight_grads", **more):
        held, number = self.everything()
        with pytest.raises(ValueError, match=match):
            self.layer.step(1e-2, **more)
        now, after = self.everything()
        assert number == after and all(torch.equal(a, b) for a, b in zip(held, now))

    def accepted(self, **more):
        held, number = self.everything()
        self.layer.step(1e-2, **more)
        now, after = self.everything()
        assert after == number + 1 and not any(torch.equal(a, b) for a, b in zip(held, now))


def test_second_step(ep):
    announce("step twice after one backward")
    c = Case()
    c.backward()
    c.accepted()
    c.refused()
    c.forward()
    c.refused()                                                    # a forward makes no gradients
    c.backward()
    c.accepted()


def test_backward_without_weight_gradients_after_a_good_one(ep):
    announce("step after a backward without weight gradients")
    c = Case()
    c.backward()
    c.backward(weight_grads=False)
    c.refused()
    c.accepted(reuse_grads=True)                                   # the first backward's, asked for by name
    c.backward(weight_grads=False)
    c.refused()


def test_new_weights(ep):
    announce("step after new weights")
    c = Case()
    c.backward()
    c.layer.set_weights(*weights(c.g))
    c.layer.prepare_step()
    c.refused()
    c.refused(reuse_grads=True)                                    # gradients of other weights are no step's
    c.backward()
    c.accepted()


def test_moments_made_after_the_backward(ep):
    """prepare_step between a backward and its step changes no gradient."""
    announce("prepare_step after a backward")
    c = Case()
    c.backward()
    c.layer.prepare_step()
    c.accepted()


def test_captured_backward(ep):
    """A backward that was only captured has filled nothing yet; what follows a replay says so."""
    announce("eager step after a captured backward")
    c = Case()
    c.forward()
    torch.cuda.synchronize()
    c.layer.backward(c.dy, c.wt, weight_grads=False)               # library set-up outside the capture
    graph = torch.cuda.CUDAGraph()
    with captured(graph):
        c.backward()
    c.refused()
    other = Case()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        c.refused()
        c.accepted(reuse_grads=True)
        other.backward()
        other.accepted()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(c.ws, other.ws))


def test_captured_step(ep):
    """A step captured behind its backward, or alone between eager backwards; one whose captured backward makes no
    weight gradients is refused."""
    announce("captured steps")
    number, lr = torch.ones(1, dtype=torch.int64, device="cuda"), torch.full((1,), 1e-2, device="cuda")
    together, alone, eager = Case(), Case(), Case()
    for c in (together, alone, eager):
        c.backward()
    alone.backward()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    with captured(graphs[0]):
        together.backward()
        together.layer.step(lr, number=number)
    with captured(graphs[1]):
        alone.layer.step(lr, number=number)
    for t in (1, 2, 3):
        number.fill_(t)
        graphs[0].replay()
        alone.backward()
        graphs[1].replay()
        torch.cuda.synchronize()
        eager.backward()
        eager.layer.step(lr, number=number)
        torch.cuda.synchronize()
        for c in (together, alone):
            assert all(torch.equal(a, b) for a, b in zip(c.ws, eager.ws)), t
    refused = Case()
    refused.backward()
    with captured(torch.cuda.CUDAGraph()):
        refused.backward(weight_grads=False)
        with pytest.raises(ValueError, match="weight_grads"):
            refused.layer.step(lr, number=number)


def test_eager_step_after_a_captured_one(ep):
    """What a captured step applies is no eager step's: neither the gradients of its replays nor those before them."""
    announce("eager step after a captured one")
    c = Case()
    c.backward()
    number = torch.ones(1, dtype=torch.int64, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with captured(graph):
        c.backward()
        c.layer.step(1e-2, number=number)
    c.refused(number=1)
    graph.replay()
    torch.cuda.synchronize()
    c.refused(number=2)
    c.backward()
    c.layer.step(1e-2, number=2)
    assert c.layer.adamw["number"] == 2
