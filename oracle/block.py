"""The block around the MoE share, computed plainly on the CPU in float64:
residual add + RMS norm and its gradients, group-limited routing and its
gradient, and products with 4-bit weights.

TEST INFRASTRUCTURE ONLY (see the package docstring).
"""
from __future__ import annotations

import math

import numpy as np

U = 2.0 ** -24                    # half a step of fp32
MASK_AT = -3.3e38
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


# ------------------------------------------------------------------ norm

def rms_norm(h, w, eps):
    """y and n = h r of h [T,H] (float64)."""
    h = np.asarray(h, np.float64)
    r = 1.0 / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)
    return h * r * np.asarray(w, np.float64), h * r


def rms_norm_backward(dy, h, w, eps, dh=None):
    """dx [T,H], d_w [H] and, for bounds, the sums of the absolute terms of each."""
    dy, h, w = (np.asarray(v, np.float64) for v in (dy, h, w))
    r = 1.0 / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)
    n, u = h * r, dy * w
    dx = r * (u - n * (u * n).mean(axis=1, keepdims=True))
    mag = r * (np.abs(u) + np.abs(n) * np.abs(u * n).mean(axis=1, keepdims=True))
    if dh is not None:
        dx = dx + np.asarray(dh, np.float64)
        mag = mag + np.abs(dh)
    return dx, (dy * n).sum(axis=0), mag, np.abs(dy * n).sum(axis=0)


# ------------------------------------------------------------------ routing

def _sigmoid(v):
    if math.isnan(v):
        return v
    return 1.0 / (1.0 + math.exp(-v)) if v >= -700 else 0.0


def scores(row, score):
    """The scores of one token's logits; masked ones are 0."""
    row = [float(v) for v in row]
    live = [not v <= MASK_AT for v in row]
    if score == "sigmoid":
        return [_sigmoid(v) if ok else 0.0 for v, ok in zip(row, live)]
    known = [v for v, ok in zip(row, live) if ok]
    if not known:
        return [0.0] * len(row)
    if any(math.isnan(v) or v == math.inf for v in known):
        return [math.nan if ok else 0.0 for ok in live]
    m = max(known)
    e = [math.exp(v - m) if ok else 0.0 for v, ok in zip(row, live)]
    total = math.fsum(e)
    return [v / total for v in e]


def _rank(v):
    """Sort key: larger first, NaN after every number."""
    return (1, 0.0) if math.isnan(v) else (0, -v)


def group_topk(logits, K, bias=None, score="sigmoid", n_group=1, topk_group=1, group_top=2, renorm=True, scale=1.0):
    """topk_ids [T,K] and topk_weights [T,K] (float64), token by token."""
    T, E = logits.shape
    size = E // n_group
    ids, weights = np.full((T, K), -1, np.int32), np.zeros((T, K))
    for t in range(T):
        s = scores(logits[t], score)
        c = s if bias is None else [a + float(b) for a, b in zip(s, bias)]
        alive = [e for e in range(E) if not logits[t, e] <= MASK_AT and (bias is None or not bias[e] <= MASK_AT)]
        if n_group > 1:
            rank = []
            for g in range(n_group):
                best = sorted((c[e] for e in alive if e // size == g), key=_rank)[:group_top]
                rank.append((2, 0.0, g) if not best else (*_rank(sum(best)), g))
            kept = {g for _, _, g in sorted(rank)[:topk_group]}
            alive = [e for e in alive if e // size in kept]
        chosen = sorted(alive, key=lambda e: (*_rank(c[e]), e))[:K]
        w = [s[e] for e in chosen]
        total = sum(w) + 1e-20 if renorm else 1.0
        ids[t, :len(chosen)] = chosen
        weights[t, :len(chosen)] = [v / total * scale for v in w]
    return ids, weights


def group_topk_backward(logits, ids, d_weights, score="sigmoid", renorm=True, scale=1.0):
    """d_logits [T,E] and, for bounds, the sums of the absolute terms."""
    T, E = logits.shape
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        s = np.array(scores(logits[t], score))
        ks = [k for k in range(ids.shape[1]) if 0 <= ids[t, k] < E]
        w = {k: s[ids[t, k]] for k in ks}
        d = {k: float(d_weights[t, k]) * scale for k in ks}
        a = {k: abs(v) for k, v in d.items()}
        if renorm:
            total = sum(w.values()) + 1e-20
            mean = sum(d[k] * w[k] for k in ks) / total
            amean = sum(a[k] * w[k] for k in ks) / total
            d = {k: (d[k] - mean) / total for k in ks}
            a = {k: (a[k] + amean) / total for k in ks}
        ds, da = np.zeros(E), np.zeros(E)
        for k in ks:
            ds[ids[t, k]] += d[k]
            da[ids[t, k]] += a[k]
        if score == "sigmoid":
            out[t], mag[t] = ds * s * (1 - s), da * s
        else:
            out[t], mag[t] = s * (ds - (ds * s).sum()), s * (da + (da * s).sum())
    return out, mag


# ------------------------------------------------------------------ 4-bit weights

def w4_values(codes, fmt):
    """codes [..,K/2] uint8 -> values [..,K]: the low nibble is the even column."""
    table = np.array([v - 8.0 for v in range(16)] if fmt == "int4" else E2M1)
    return np.stack([table[codes & 15], table[codes >> 4]], axis=-1).reshape(*codes.shape[:-1], -1)


def w4_product(a, codes, scales, fmt):
    """a [m,K] times one expert's weights (codes [N,K/2], scales [N,K/group])
    -> G [m,N] and the sums of |a| |w'|, w' the largest magnitude that the
    codes' representation passes through (INT4: 31 + 24 steps of the scale)."""
    v = w4_values(codes, fmt)
    s = np.repeat(np.asarray(scales, np.float64), v.shape[1] // scales.shape[1], axis=1)
    a = np.asarray(a, np.float64)
    big = np.full_like(v, 55.0) if fmt == "int4" else np.abs(v)
    return a @ (v * s).T, np.abs(a) @ (big * np.abs(s)).T


def silu_mul(g):
    gate, up = g[:, :g.shape[1] // 2], g[:, g.shape[1] // 2:]
    return gate / (1.0 + np.exp(-gate)) * up
