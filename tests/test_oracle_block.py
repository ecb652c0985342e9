"""Pins of oracle/block.py (CPU): torch's float64 autograd, differences, and
closed forms."""
import math

import numpy as np
import pytest
import torch

from oracle import block as ob


def test_norm_closed_forms():
    y, n = ob.rms_norm(np.array([[3.0, -4.0]]), np.array([1.0, 2.0]), 0.0)
    r = 1 / math.sqrt(12.5)
    assert np.allclose(n, [[3 * r, -4 * r]]) and np.allclose(y, [[3 * r, -8 * r]])
    assert np.allclose((n ** 2).mean(1), 1.0)


@pytest.mark.parametrize("with_dh", [False, True])
def test_norm_backward_is_the_gradient(with_dh):
    rng = np.random.default_rng(3)
    h, w, dy, dh = (rng.standard_normal(s) for s in ((5, 24), (24,), (5, 24), (5, 24)))
    th, tw = torch.tensor(h, requires_grad=True), torch.tensor(w, requires_grad=True)
    y = th / ((th ** 2).mean(1, keepdim=True) + 1e-3).sqrt() * tw
    ((y * torch.tensor(dy)).sum() + (th * torch.tensor(dh)).sum() * with_dh).backward()
    dx, dw, _, _ = ob.rms_norm_backward(dy, h, w, 1e-3, dh if with_dh else None)
    assert np.allclose(dx, th.grad.numpy(), atol=1e-12) and np.allclose(dw, tw.grad.numpy(), atol=1e-12)


def test_norm_backward_against_differences():
    rng = np.random.default_rng(4)
    h, w, dy = rng.standard_normal((2, 8)), rng.standard_normal(8), rng.standard_normal((2, 8))
    dx, dw, _, _ = ob.rms_norm_backward(dy, h, w, 1e-2)
    for i in range(8):
        e = np.zeros_like(h)
        e[1, i] = 1e-6
        d = ((ob.rms_norm(h + e, w, 1e-2)[0] - ob.rms_norm(h - e, w, 1e-2)[0]) * dy).sum() / 2e-6
        assert abs(d - dx[1, i]) < 1e-8
        d = ((ob.rms_norm(h, w + e[1], 1e-2)[0] - ob.rms_norm(h, w - e[1], 1e-2)[0]) * dy).sum() / 2e-6
        assert abs(d - dw[i]) < 1e-8


def test_routing_without_groups_is_a_plain_topk():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((20, 24)).astype(np.float32)
    for score in ("sigmoid", "softmax"):
        ids, w = ob.group_topk(x, 5, score=score)
        assert np.array_equal(ids, np.argsort(-x, axis=1, kind="stable")[:, :5])
        assert np.allclose(w.sum(1), 1.0)
    s = torch.softmax(torch.tensor(x, dtype=torch.float64), 1).numpy()
    _, w = ob.group_topk(x, 5, score="softmax", renorm=False, scale=2.0)
    assert np.allclose(w, 2 * -np.sort(-s, axis=1)[:, :5])


def test_routing_groups_by_hand():
    # groups {0,1} {2,3} {4,5}; logits are the sigmoid's inverse of these scores
    s = np.array([[0.9, 0.1, 0.6, 0.6, 0.8, 0.3]])
    x = np.log(s / (1 - s)).astype(np.float32)
    assert ob.group_topk(x, 2, n_group=3, topk_group=1, group_top=1)[0].tolist() == [[0, 1]]
    assert ob.group_topk(x, 2, n_group=3, topk_group=1, group_top=2)[0].tolist() == [[2, 3]]      # 1.2 > 1.1 > 1.0
    assert ob.group_topk(x, 2, n_group=3, topk_group=2, group_top=2)[0].tolist() == [[4, 2]]
    # a bias moves the choice, not the weights
    b = np.array([0, 0, -0.5, 0, 0, 0.25], np.float32)
    ids, w = ob.group_topk(x, 2, bias=b, n_group=3, topk_group=1, group_top=2, renorm=False)
    assert ids.tolist() == [[4, 5]] and np.allclose(w, [[0.8, 0.3]], atol=1e-6)


def test_routing_masks_and_ties():
    x = np.zeros((3, 6), np.float32)
    x[1, [0, 1, 2]] = -np.inf
    x[1, 3] = np.finfo(np.float32).min
    x[2] = -np.inf
    ids, w = ob.group_topk(x, 4)
    assert ids.tolist() == [[0, 1, 2, 3], [4, 5, -1, -1], [-1] * 4]
    assert w.tolist() == [[0.25] * 4, [0.5, 0.5, 0, 0], [0] * 4]
    x = np.array([[np.nan, 1.0, -5.0]], np.float32)
    assert ob.group_topk(x, 3)[0].tolist() == [[1, 2, 0]]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
def test_routing_backward_is_the_gradient(score, renorm):
    rng = np.random.default_rng(6)
    x = rng.standard_normal((7, 12)).astype(np.float32)
    x[0, 3] = -np.inf
    ids, _ = ob.group_topk(x, 3, score=score)
    ids[2, 2] = -1
    ids[3, 1] = ids[3, 0]                                   # the same expert twice
    dw = rng.standard_normal((7, 3))
    l = torch.tensor(x, dtype=torch.float64, requires_grad=True)
    s = torch.sigmoid(l) if score == "sigmoid" else torch.softmax(l, 1)
    w = s.gather(1, torch.tensor(ids).long().clamp(min=0)) * torch.tensor(ids >= 0)
    if renorm:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    (w * 2.5 * torch.tensor(dw)).sum().backward()
    got, _ = ob.group_topk_backward(x, ids, dw, score, renorm, 2.5)
    assert np.allclose(got, np.nan_to_num(l.grad.numpy()), atol=1e-12)


def test_routing_backward_against_differences():
    rng = np.random.default_rng(7)
    x = rng.standard_normal((1, 6)).astype(np.float32)
    dw = rng.standard_normal((1, 3))
    for score in ("sigmoid", "softmax"):
        ids, _ = ob.group_topk(x, 3, score=score)
        got, _ = ob.group_topk_backward(x, ids, dw, score, True, 1.0)

        def loss(v):
            w = np.array(ob.scores(v[0], score))[ids[0]]
            return (w / (w.sum() + 1e-20) * dw[0]).sum()
        for e in range(6):
            d = np.zeros((1, 6))
            d[0, e] = 1e-6
            assert abs((loss(x + d) - loss(x - d)) / 2e-6 - got[0, e]) < 1e-8


def test_w4_values():
    codes = np.array([[0x10, 0xF7, 0x8C]], np.uint8)
    assert ob.w4_values(codes, "int4").tolist() == [[-8, -7, -1, 7, 4, 0]]
    assert ob.w4_values(codes, "e2m1").tolist() == [[0, 0.5, 6, -6, -2, 0]]
    g, _ = ob.w4_product(np.ones((1, 6)), codes, np.array([[2.0, 0.5]]), "int4")     # groups of three columns
    assert g.tolist() == [[2 * -16 + 0.5 * 11]]
