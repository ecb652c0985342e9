"""Calls of more rows than one launch can count the lanes of (2^32): short rows,
so that they fit, checked on both sides of every slice's edge and at the end."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import combine_top_expert_amd as mod
    return mod


def _edges(T, slice_rows):
    """Rows around the slices' edges, the first and the last ones."""
    at = {0, 1, T - 2, T - 1}
    for s in range(slice_rows, T, slice_rows):
        at |= {s - 1, s, s + 1}
    return torch.tensor(sorted(r for r in at if 0 <= r < T), device="cuda")


def test_norm_rows(m):
    T, H, eps = (1 << 26) + 5, 8, 1e-6
    torch.manual_seed(0)
    x = torch.randn(T, H, dtype=torch.bfloat16, device="cuda")
    w = torch.rand(H, dtype=torch.bfloat16, device="cuda") + 0.5
    y = torch.full_like(x, float("nan"))
    m.moe_add_rms_norm(x, None, w, eps, y=y)
    r = _edges(T, 1 << 21)
    h = x[r].double()
    ref = h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * w.double()
    # half a step of bf16, and fp32 sums of 8 terms far below it
    assert ((y[r].double() - ref).abs() <= ref.abs() * (2.0 ** -8 + 2.0 ** -18)).all()
    assert not bool(torch.isnan(y).any())


def test_route_rows(m):
    T, E, K = (1 << 26) + 5, 4, 1
    torch.manual_seed(1)
    logits = torch.randn(T, E, device="cuda")
    ids = torch.full((T, K), -7, dtype=torch.int32, device="cuda")
    wts = torch.full((T, K), float("nan"), device="cuda")
    m.moe_router_group_topk(logits, K, ids, wts, renorm=False)
    best = logits.max(1, keepdim=True).values
    assert bool((ids >= 0).all()) and bool((logits.gather(1, ids.long()) == best).all())
    r = _edges(T, 1 << 25)
    ref = torch.sigmoid(best[r].double())
    assert ((wts[r].double() - ref).abs() <= ref * 2.0 ** -20).all()


def test_route_backward_rows(m):
    T = (1 << 28) + 5
    torch.manual_seed(2)
    logits = torch.randn(T, 1, device="cuda")
    ids = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    dw = torch.randn(T, 1, device="cuda")
    dl = torch.full((T, 1), float("nan"), device="cuda")
    m.moe_router_group_topk_backward(logits, ids, dw, dl, renorm=False)
    r = _edges(T, 1 << 26)
    s = torch.sigmoid(logits[r].double())
    ref = dw[r].double() * s * (1 - s)
    # formed in fp64, rounded once to fp32
    assert ((dl[r].double() - ref).abs() <= ref.abs() * (2.0 ** -24 + 2.0 ** -40)).all()
    assert not bool(torch.isnan(dl).any())


def test_permute_rows(m):
    T, H = (1 << 26) + 5, 128
    x8 = torch.zeros(T, H, dtype=torch.uint8, device="cuda")
    xs = torch.zeros(T, 1, device="cuda")
    slot = torch.full((T, 1), -1, dtype=torch.int32, device="cuda")
    r = _edges(T, 1 << 25)
    n = r.numel()
    x8[r] = torch.arange(1, n + 1, dtype=torch.uint8, device="cuda")[:, None].expand(n, H).contiguous()
    xs[r, 0] = torch.arange(1, n + 1, dtype=torch.float32, device="cuda")
    slot[r, 0] = torch.arange(n, dtype=torch.int32, device="cuda")
    buf = torch.full((n + 1, H), 255, dtype=torch.uint8, device="cuda")
    bs = torch.full((n + 1, 1), -1.0, device="cuda")
    m.moe_permute_fp8(x8, xs, slot, buf, bs)
    assert torch.equal(buf[:n], x8[r]) and torch.equal(bs[:n], xs[r])
    assert bool((buf[n] == 255).all()) and float(bs[n, 0]) == -1.0
