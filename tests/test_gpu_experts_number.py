"""MoELayer.step's count of updates, and its masters after weights were written in place."""
import math

import pytest
import torch

from gpu_util import announce, need_gpu
from test_gpu_experts_grads import Case, captured

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ep():
    need_gpu()
    import combine_top_expert_amd as ep
    return ep


def test_number_on_the_device_then_counted(ep):
    """Once the count lives on the device, a step without a number is refused rather than run as update 1."""
    announce("device number, then none")
    c = Case()
    c.backward()
    c.layer.step(1e-2, number=torch.full((1,), 1000, dtype=torch.int64, device="cuda"))
    c.backward()
    c.refused(match="number")
    c.layer.step(1e-2, number=1001)                                # a number sets the count again
    c.backward()
    c.accepted()
    assert c.layer.adamw["number"] == 1002
    c.layer.prepare_step()                                         # new moments, counted from 1
    c.backward()
    c.layer.step(1e-2)
    assert c.layer.adamw["number"] == 1


def test_captured_step_needs_a_device_number(ep):
    """Replays would repeat the update that was counted while capturing."""
    announce("captured step without a number")
    c = Case()
    c.backward()
    with captured(torch.cuda.CUDAGraph()):
        c.x.add_(0.0)
        with pytest.raises(ValueError, match="number"):
            c.layer.step(1e-2)
    assert c.layer.adamw["number"] == 0
    c.accepted()


def test_refresh_masters(ep):
    """Weights written in place: the next step starts from them once the masters are taken again."""
    announce("refresh_masters")
    c = Case()
    c.layer.refresh_masters()
    assert all(torch.equal(m, w.float()) for m, w in zip(c.layer.adamw["masters"], c.ws))
    new = [torch.randn(w.shape, generator=c.g).to(w.dtype).cuda() / math.sqrt(w.shape[-1]) for w in c.ws]
    for w, n in zip(c.ws, new):
        w.copy_(n)
    c.layer.set_weights(*c.ws)
    c.layer.refresh_masters()
    c.layer.refresh_transposed_weights()
    fresh = Case(1)
    fresh.ws = [n.clone() for n in new]
    fresh.layer.set_weights(*fresh.ws)
    fresh.layer.prepare_step(weight_decay=0.1)
    fresh.x, fresh.dy, fresh.ids, fresh.wt = c.x, c.dy, c.ids, c.wt
    for x in (c, fresh):
        x.backward()
        x.layer.step(1e-2)
    assert all(torch.equal(a, b) for a, b in zip(c.ws, fresh.ws))
