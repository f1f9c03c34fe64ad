"""Oracle of what stands around the experts in training: the root-mean-square
norm with its gradients, experts with plain weights with theirs, and the
gradients of the weighted combine and of the top-k softmax.

Plain numpy in float64, written from the definitions; experts and tokens go one
by one.
"""
from __future__ import annotations

import numpy as np

from oracle import dense


def rms_norm(r, weight, eps):
    """-> (out [T][H], 1 / rms [T][1])."""
    inv = 1.0 / np.sqrt((r * r).mean(axis=1, keepdims=True) + eps)
    return r * inv * weight, inv


def rms_norm_grad(dout, r, weight, eps, dresidual=0.0):
    """-> (dr, dweight) of sum(dout * out) + sum(dresidual * r)."""
    _, inv = rms_norm(r, weight, eps)
    u = r * inv
    g = dout * weight
    return inv * (g - u * (g * u).mean(axis=1, keepdims=True)) + dresidual, (dout * u).sum(axis=0)


def combine_grad(dout, y, dest_row, w):
    """-> (dy, rows that no dest_row names 0; dw [T][k])."""
    T, k = w.shape
    dy, dw = np.zeros_like(y), np.zeros_like(w)
    for t in range(T):
        for j in range(k):
            r = int(dest_row[t * k + j])
            if 0 <= r < T * k:
                dy[r] = w[t, j] * dout[t]
                dw[t, j] = y[r] @ dout[t]
    return dy, dw


def route_grad(dw, ids, w, E):
    """-> dlogits [T][E]: w = softmax over the kept logits, w_j' = w_j (delta - w_i)."""
    T, k = w.shape
    dl = np.zeros((T, E))
    for t in range(T):
        for j in range(k):
            if 0 <= ids[t, j] < E:
                dl[t, ids[t, j]] += w[t, j] * (dw[t, j] - w[t] @ dw[t])
    return dl


def gathered(x, gather, div):
    """Row gather[r] // div of x for each r, zeros for rows that x does not have."""
    out = np.zeros((len(gather), x.shape[1]))
    for r, g in enumerate(np.asarray(gather, dtype=np.int64)):
        if g >= 0 and g // div < x.shape[0]:
            out[r] = x[g // div]
    return out


def expert_ffn(x, offsets, w1, w2, layout="split", act="silu"):
    """x [rows][H] in expert order -> (out, gate_up, h), rows of no expert 0."""
    rows, E = x.shape[0], w1.shape[0]
    out, gu, h = np.zeros((rows, w2.shape[1])), np.zeros((rows, w1.shape[1])), np.zeros((rows, w2.shape[2]))
    for e in range(E):
        s = slice(int(offsets[e]), int(offsets[e + 1]))
        out[s], gu[s], h[s] = dense.gated_ffn(x[s], w1[e], w2[e], layout, act)
    return out, gu, h


def expert_ffn_grad(dout, x, offsets, w1, w2, layout="split", act="silu"):
    """-> (dx rows, dw1, dw2)."""
    dx, dw1, dw2 = np.zeros_like(x), np.zeros_like(w1), np.zeros_like(w2)
    for e in range(w1.shape[0]):
        s = slice(int(offsets[e]), int(offsets[e + 1]))
        dx[s], dw1[e], dw2[e], _ = dense.gated_ffn_grad(dout[s], x[s], w1[e], w2[e], layout, act)
    return dx, dw1, dw2
