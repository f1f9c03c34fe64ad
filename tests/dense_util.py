"""Inputs and error bounds shared by the GPU tests of the dense operators.

Bounds.  u(t) = finfo(t).eps / 2 is the largest relative rounding error of
type t.  A sum of n products held in fp32 is off by at most
n * 2^-24 * sum|terms| (any order).  An intermediate rounded to 16 bits
contributes sum_i d_i q_i with independent |d_i| <= u and q_i the terms it
multiplies: by Hoeffding's inequality it exceeds 7 u sqrt(sum q_i^2) with
probability 2 e^-24.5 = 5e-11 per output.  The result's own rounding adds
u |result|.  exp, reciprocal and the gate's other fp32 steps: 2^-18 of the
gate's value (a few ulp, times the argument of exp, up to 16 here).  fp16
results below 2^-14 are off by up to 2^-25 (half a subnormal step).
"""
import numpy as np
import torch

from oracle import dense as od

F32 = 2.0 ** -24
GATE = 2.0 ** -18
DEV = "cuda"


def u(dtype):
    return torch.finfo(dtype).eps / 2


def floor(dtype):
    return 2.0 ** -25 if dtype == torch.float16 else 1e-37


def f64(t):
    return t.detach().double().cpu().numpy()


def normal(shape, scale, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).to(DEV)


def strided(t, pad):
    """The same values in rows `pad` elements apart longer than their length."""
    wide = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=t.device)
    wide[:, : t.shape[1]] = t
    return wide[:, : t.shape[1]]


def hoeff(q2, dtype):
    """7 u sqrt(sum q^2): an operand's 16-bit rounding, seen through a product."""
    return 7 * u(dtype) * np.sqrt(q2)


def assert_within(got, ref, bound, what=""):
    g = f64(got)
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    assert np.isfinite(g).all(), f"{what}: not finite"
    over = np.abs(g - ref) - bound
    at = np.unravel_index(int(np.argmax(over)), over.shape) if over.size else None
    assert not over.size or over[at] <= 0, \
        f"{what}: {g[at]} against {ref[at]} at {at}: off by {abs(g[at] - ref[at]):.3e}, bound {bound[at]:.3e}"


def rounded(ref, err, dtype):
    """Bound of a result of type dtype whose exact value's error is err."""
    return err + u(dtype) * (np.abs(ref) + err) + floor(dtype)


def ffn_bounds(x, w1, w2, layout, act, dtype, out_dtype, add=None):
    """(out, its bound, gate_up, its fp32 error, h, its error before rounding)."""
    out, gu, h = od.gated_ffn(x, w1, w2, layout, act, add)
    e_gu = x.shape[1] * F32 * (np.abs(x) @ np.abs(w1).T)
    (g, up), (eg, eu) = od.split_gate_up(gu, layout), od.split_gate_up(e_gu, layout)
    a, da = od.gate_act(g, act), np.abs(od.gate_act_derivative(g, act))
    e_h = np.abs(up) * (da * eg + eg ** 2) + (np.abs(a) + 1.2 * eg) * eu + GATE * np.abs(h)
    err = (e_h + floor(dtype)) @ np.abs(w2).T + w2.shape[1] * F32 * (np.abs(h) @ np.abs(w2).T) \
        + hoeff(h ** 2 @ (w2 ** 2).T, dtype)
    if add is not None:
        err = err + F32 * (np.abs(out) + np.abs(add))
    return out, rounded(out, err, out_dtype), gu, e_gu, h, e_h


def ffn_grad_bounds(dout, x, w1, w2, layout, act, dtype, save_dtype, dx_dtype, dw_dtype, base1=0.0, base2=0.0):
    """((dx, bound), (dw1, bound), (dw2, bound)); base: what the weight gradients were added to."""
    _, gu, h = od.gated_ffn(x, w1, w2, layout, act)
    dx, dw1, dw2, dgu = od.gated_ffn_grad(dout, x, w1, w2, layout, act)
    e_gu = x.shape[1] * F32 * (np.abs(x) @ np.abs(w1).T)
    save = u(save_dtype) if save_dtype != torch.float32 else F32
    r_gu = save * np.abs(gu) + (floor(save_dtype) if save else 0)   # gate_up's rounding when kept
    (g, up), (eg, eu) = od.split_gate_up(gu, layout), od.split_gate_up(e_gu + r_gu, layout)
    a, da = od.gate_act(g, act), np.abs(od.gate_act_derivative(g, act))
    dh = dout @ w2
    e_dh = dout.shape[1] * F32 * (np.abs(dout) @ np.abs(w2))
    # |act''| <= 1.2 for both activations, |act'| <= 1.2
    e_g = (np.abs(up) + eu) * (da + 1.2 * eg) * e_dh + np.abs(dh) * (eu * da + (np.abs(up) + eu) * 1.2 * eg) \
        + GATE * np.abs(dh * up) * (da + 1)
    e_u = (np.abs(a) + 1.2 * eg) * e_dh + np.abs(dh) * 1.2 * eg + GATE * np.abs(dh * a)
    e_dgu = od.join_gate_up(e_g, e_u, layout) + floor(dtype)
    e_h = np.abs(up) * (da * eg + 1.2 * eg ** 2) + (np.abs(a) + 1.2 * eg) * eu + GATE * np.abs(h) + floor(dtype)
    T, n = dout.shape[0], dgu.shape[1]
    ex = e_dgu @ np.abs(w1) + n * F32 * (np.abs(dgu) @ np.abs(w1)) + hoeff(dgu ** 2 @ w1 ** 2, dtype)
    e1 = e_dgu.T @ np.abs(x) + T * F32 * (np.abs(dgu).T @ np.abs(x)) + hoeff((dgu ** 2).T @ x ** 2, dtype)
    e2 = np.abs(dout).T @ e_h + T * F32 * (np.abs(dout).T @ np.abs(h)) + hoeff((dout ** 2).T @ h ** 2, dtype)
    dw1, dw2 = dw1 + base1, dw2 + base2
    e1, e2 = e1 + F32 * (np.abs(dw1) + np.abs(base1)), e2 + F32 * (np.abs(dw2) + np.abs(base2))
    return ((dx, rounded(dx, ex, dx_dtype)), (dw1, rounded(dw1, e1, dw_dtype)), (dw2, rounded(dw2, e2, dw_dtype)))


def adapter_bounds(x, w, ids, a, b, dtype, out_dtype, scales=None, ranks=None, add=None, epilogue="none",
                   act="silu"):
    """(out, bound)."""
    out, y, s = od.adapter_linear(x, w, ids, a, b, scales, ranks, add, epilogue, act)
    T, K = x.shape
    err = np.zeros_like(y) if w is None else K * F32 * (np.abs(x) @ np.abs(w).T)
    n, R = a.shape[:2]
    for t in range(T):
        i = int(ids[t])
        if 0 <= i < n:
            r = R if ranks is None else min(max(int(ranks[i]), 0), R)
            sc = 1.0 if scales is None else abs(float(scales[i]))
            e_s = sc * (K + 2) * F32 * (np.abs(a[i, :r]) @ np.abs(x[t])) + floor(dtype)
            st = np.abs(s[t, :r])
            err[t] += np.abs(b[i][:, :r]) @ (e_s + (R + 2) * F32 * st) + hoeff(b[i][:, :r] ** 2 @ st ** 2, dtype)
    err += F32 * 4 * (np.abs(y) + (0 if add is None else np.abs(add)) + (0 if w is None else np.abs(x @ w.T)))
    if epilogue != "none":
        (g, up), (eg, eu) = od.split_gate_up(y, epilogue), od.split_gate_up(err, epilogue)
        av, da = np.abs(od.gate_act(g, act)), np.abs(od.gate_act_derivative(g, act))
        err = (np.abs(up) + eu) * (da * eg + 1.2 * eg ** 2) + (av + 1.2 * eg) * eu + GATE * np.abs(out)
    return out, rounded(out, err, out_dtype)
