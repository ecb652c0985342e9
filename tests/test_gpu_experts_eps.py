"""moe_adamw_step at the ends of eps' range, against oracle/experts.py (float64).

Bounds as in test_gpu_experts_adamw.py: a power of two that the quotient's two
sides are scaled by adds no rounding.  Where eps is so large that the update
leaves fp32's normal range, what is lost is below 2^-126."""
import numpy as np
import pytest
import torch

from gpu_util import announce, need_gpu
from oracle import experts as ox

pytestmark = pytest.mark.gpu
U = ox.U
B, LR, WD = (0.9, 0.95), 1e-2, 0.1


@pytest.fixture(scope="module")
def ep():
    need_gpu()
    import combine_top_expert_amd as ep
    return ep


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


# below fp32's least number, subnormal, at the ends of where the factor is 1, large, past fp32's largest
EPS = [1e-300, 1e-50, 2.0 ** -149, 1e-40, 2.0 ** -126, 2.0 ** -101, 2.0 ** -99, 1e-8, 1.0, 2.0 ** 99, 2.0 ** 101, 3e38, 1e45]


@pytest.mark.parametrize("device", [False, True])
@pytest.mark.parametrize("s8", [False, True])
@pytest.mark.parametrize("eps", EPS)
def test_eps(ep, eps, s8, device):
    announce("adamw eps", eps, s8, device)
    n = 1300
    rng = np.random.default_rng(11)
    mk = lambda v: torch.from_numpy(np.asarray(v, np.float32)).cuda()  # noqa: E731
    w0, g0 = rng.standard_normal(n), rng.standard_normal(n) * 1e-2
    m0, r0 = rng.standard_normal(n) * 1e-2, np.abs(rng.standard_normal(n)) * 1e-2 + 1e-3
    g0[::3] = m0[::3] = r0[::3] = 0.0                              # elements that no gradient has reached
    p, g = mk(w0), mk(g0)
    if s8:
        f8 = torch.float8_e4m3fn
        blocks = (n + 127) // 128
        ms, vs = torch.full((blocks,), 2.0 ** -13, device="cuda"), torch.full((blocks,), 2.0 ** -13, device="cuda")
        m, v = (mk(x * 2.0 ** 13).to(f8) for x in (m0, r0))
        m0, v0 = f64(m) * 2.0 ** -13, (f64(v) * 2.0 ** -13) ** 2
        more = dict(exp_avg_scales=[ms], exp_avg_sq_scales=[vs], seed=3)
    else:
        m, v, more = mk(m0), mk(r0 * r0), {}
        m0, v0 = f64(m), f64(v)
    w0, g0 = f64(p), f64(g)
    lr, step = LR, 7
    if device:
        lr, step = torch.tensor([LR], device="cuda"), torch.tensor([step], dtype=torch.int64, device="cuda")
    ep.moe_adamw_step([p], [g], [m], [v], lr, step, betas=B, eps=eps, weight_decay=WD, **more)
    got = f64(p)
    assert np.all(np.isfinite(got))
    ref, _, _, wm, um, _ = ox.adamw(w0, g0, m0, v0, LR, B, eps, WD, 7)
    # lr as the device holds it is off by half a step of fp32
    bound = U * (6 * wm + 26 * um) + 2.0 ** -126
    worst = float(np.max(np.abs(got - ref) / bound))
    print(f"[metric] eps {eps}: worst error / bound {worst:.3f}", flush=True)
    assert worst <= 1.0
    still = np.zeros(n, bool)
    still[::3] = True
    assert np.all(np.abs(got - w0 * (1 - LR * WD))[still] <= 4 * U * np.abs(w0[still]))


def test_eps_of_zero(ep):
    """0 / 0 where nothing has been learnt, as the formula has it; elsewhere the update without eps."""
    announce("adamw eps 0")
    p, g, m, v = (torch.ones(64, device="cuda") for _ in range(4))
    g[::2] = m[::2] = v[::2] = 0.0
    ep.moe_adamw_step([p], [g], [m], [v], LR, 1, betas=B, eps=0.0, weight_decay=0.0)
    assert bool(p[::2].isnan().all()) and bool(p[1::2].isfinite().all())
