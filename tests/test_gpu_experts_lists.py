"""moe_adamw_step refuses a tensor that two of its lists name."""
import pytest
import torch

from gpu_util import announce, need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ep():
    need_gpu()
    import combine_top_expert_amd as ep
    return ep


def test_adamw_refuses_a_tensor_in_two_lists(ep):
    announce("adamw a tensor in two lists")
    t = [torch.ones(64, device="cuda") for _ in range(8)]
    p, g, m, v = t[0:2], t[2:4], t[4:6], t[6:8]
    for bad in ((p, g, m, m), (p, g, m, [v[0], m[1]]), (p, g, p, v), (p, g, m, [p[1], v[1]])):
        with pytest.raises(ValueError, match="same tensor"):
            ep.moe_adamw_step(*bad, 1e-3, 1)
    b16 = [x.bfloat16() for x in p]
    with pytest.raises(ValueError, match="same tensor"):
        ep.moe_adamw_step(b16, g, m, v, 1e-3, 1, masters=[v[0], p[0]])
    f8 = lambda: [torch.zeros(64, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]  # noqa: E731
    s = [torch.zeros(1, device="cuda") for _ in range(4)]
    with pytest.raises(ValueError, match="same tensor"):
        ep.moe_adamw_step(p, g, f8(), f8(), 1e-3, 1, exp_avg_scales=s[:2], exp_avg_sq_scales=s[1:3])
    assert all(bool((x == 1).all()) for x in t)                    # nothing has run
    # gradients are only read: any of them may be anything's copy, and empty tensors are no tensor
    e = torch.empty(0, device="cuda")
    ep.moe_adamw_step([e, *p], [e, g[0], g[0]], [e, *m], [e, *v], 1e-3, 1)
    ep.moe_adamw_step(p, g, f8(), f8(), 1e-3, 1, exp_avg_scales=s[:2], exp_avg_sq_scales=s[2:])
    assert torch.equal(p[0], p[1]) and not bool((p[0] == 1).any())
