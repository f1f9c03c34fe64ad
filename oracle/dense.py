"""Oracle of the dense operators: the gated feed-forward block with its
gradients, and the projection with per-token low-rank adapters.

Plain numpy in float64, written from the definitions; the adapters go token by
token.
"""
from __future__ import annotations

import numpy as np

SQRT_2_OVER_PI = np.sqrt(2.0 / np.pi)


def gate_act(g, act):
    """The gate's activation: "silu" z / (1 + e^-z), "gelu" its tanh form."""
    g = np.asarray(g, dtype=np.float64)
    if act == "silu":
        return g / (1.0 + np.exp(-g))
    if act == "gelu":
        return 0.5 * g * (1.0 + np.tanh(SQRT_2_OVER_PI * (g + 0.044715 * g ** 3)))
    raise ValueError(act)


def gate_act_derivative(g, act):
    g = np.asarray(g, dtype=np.float64)
    if act == "silu":
        s = 1.0 / (1.0 + np.exp(-g))
        return s + g * s * (1.0 - s)
    t = np.tanh(SQRT_2_OVER_PI * (g + 0.044715 * g ** 3))
    return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * SQRT_2_OVER_PI * (1.0 + 3 * 0.044715 * g ** 2)


def split_gate_up(gu, layout):
    """The gate and up columns of gate_up (or rows of w1, transposed)."""
    n = gu.shape[-1] // 2
    if layout == "split":
        return gu[..., :n], gu[..., n:]
    if layout == "interleaved":
        return gu[..., 0::2], gu[..., 1::2]
    raise ValueError(layout)


def join_gate_up(g, u, layout):
    if layout == "split":
        return np.concatenate([g, u], axis=-1)
    out = np.empty(g.shape[:-1] + (2 * g.shape[-1],))
    out[..., 0::2], out[..., 1::2] = g, u
    return out


def gated_ffn(x, w1, w2, layout="split", act="silu", add=None):
    """-> (out [T][H], gate_up [T][2I], h [T][I])."""
    gu = x @ w1.T
    g, u = split_gate_up(gu, layout)
    h = gate_act(g, act) * u
    out = h @ w2.T
    return (out if add is None else out + add), gu, h


def gated_ffn_grad(dout, x, w1, w2, layout="split", act="silu"):
    """-> (dx, dw1, dw2, d_gate_up) of sum(dout * out)."""
    _, gu, h = gated_ffn(x, w1, w2, layout, act)
    g, u = split_gate_up(gu, layout)
    dh = dout @ w2
    dgu = join_gate_up(dh * u * gate_act_derivative(g, act), dh * gate_act(g, act), layout)
    return dgu @ w1, dgu.T @ x, dout.T @ h, dgu


def adapter_linear(x, w, ids, lora_a, lora_b, scales=None, ranks=None, add=None, epilogue="none", act="silu"):
    """-> (out, y, s): y before the epilogue, s [T][R] the scaled low-rank rows (0 where a token has none)."""
    T, n, R = x.shape[0], lora_a.shape[0], lora_a.shape[1]
    N = lora_b.shape[1]
    y = np.zeros((T, N)) if w is None else x @ w.T
    if add is not None:
        y = y + add
    s = np.zeros((T, R))
    for t in range(T):
        i = int(ids[t])
        if not 0 <= i < n:
            continue
        r = R if ranks is None else min(max(int(ranks[i]), 0), R)
        s[t, :r] = (1.0 if scales is None else float(scales[i])) * (lora_a[i, :r] @ x[t])
        y[t] += lora_b[i, :, :r] @ s[t, :r]
    if epilogue == "none":
        return y, y, s
    g, u = split_gate_up(y, epilogue)
    return gate_act(g, act) * u, y, s
