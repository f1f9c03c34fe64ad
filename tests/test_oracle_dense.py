"""Pins of the dense operators' oracle: closed forms, differences, torch's autograd and brute-force loops."""
import numpy as np
import pytest
import torch

from oracle import dense as od

RNG = np.random.default_rng(11)


def test_activations_against_torch_and_identities():
    g = np.linspace(-12, 12, 2001)
    t = torch.from_numpy(g)
    assert np.allclose(od.gate_act(g, "silu"), torch.nn.functional.silu(t).numpy(), atol=1e-14)
    assert np.allclose(od.gate_act(g, "gelu"), torch.nn.functional.gelu(t, approximate="tanh").numpy(), atol=1e-14)
    # act(z) - act(-z) = z for both
    for act in ("silu", "gelu"):
        assert np.allclose(od.gate_act(g, act) - od.gate_act(-g, act), g, atol=1e-13)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_derivatives_against_differences(act):
    g = np.linspace(-8, 8, 401)
    d = 1e-5
    num = (od.gate_act(g + d, act) - od.gate_act(g - d, act)) / (2 * d)
    # central differences: d^2/6 |act'''| (below 2) + 2^-52 |act| / d
    assert np.abs(num - od.gate_act_derivative(g, act)).max() < 1e-9


@pytest.mark.parametrize("layout", ["split", "interleaved"])
def test_gate_up_round_trip_and_rows(layout):
    gu = RNG.standard_normal((3, 10))
    g, u = od.split_gate_up(gu, layout)
    assert np.array_equal(od.join_gate_up(g, u, layout), gu)
    assert g[0, 1] == (gu[0, 1] if layout == "split" else gu[0, 2])


@pytest.mark.parametrize("layout", ["split", "interleaved"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_ffn_and_gradients_against_autograd_and_differences(layout, act):
    T, H, I = 5, 6, 4
    x, w1, w2 = RNG.standard_normal((T, H)), RNG.standard_normal((2 * I, H)), RNG.standard_normal((H, I))
    dout = RNG.standard_normal((T, H))
    tx, t1, t2 = (torch.from_numpy(a).requires_grad_(True) for a in (x, w1, w2))
    gate, up = (t1[:I], t1[I:]) if layout == "split" else (t1[0::2], t1[1::2])
    f = torch.nn.functional
    a = f.silu(tx @ gate.T) if act == "silu" else f.gelu(tx @ gate.T, approximate="tanh")
    out = (a * (tx @ up.T)) @ t2.T
    ref = torch.autograd.grad(out, (tx, t1, t2), torch.from_numpy(dout))
    got = od.gated_ffn_grad(dout, x, w1, w2, layout, act)
    assert np.allclose(od.gated_ffn(x, w1, w2, layout, act)[0], out.detach().numpy(), atol=1e-12)
    for r, o in zip(ref, got):
        assert np.allclose(o, r.numpy(), atol=1e-11)
    d = 1e-6
    for arr, gr in ((x, got[0]), (w1, got[1]), (w2, got[2])):
        at = tuple(RNG.integers(s) for s in arr.shape)
        keep, v = arr[at], []
        for sgn in (1, -1):
            arr[at] = keep + sgn * d
            v.append((dout * od.gated_ffn(x, w1, w2, layout, act)[0]).sum())
        arr[at] = keep
        assert abs((v[0] - v[1]) / (2 * d) - gr[at]) < 1e-6 * max(1.0, abs(gr[at]))


def test_adapters_against_merged_weights():
    T, K, N, n, R = 9, 8, 6, 3, 4
    x, w = RNG.standard_normal((T, K)), RNG.standard_normal((N, K))
    a, b = RNG.standard_normal((n, R, K)), RNG.standard_normal((n, N, R))
    ids, scales, ranks = np.array([0, 1, 2, -1, 3, 2, 1, 0, 2]), np.array([0.5, 2.0, -1.0]), np.array([4, 1, 9])
    add = RNG.standard_normal((T, N))
    out, _, s = od.adapter_linear(x, w, ids, a, b, scales, ranks, add)
    for t, i in enumerate(ids):
        merged = w.copy()
        if 0 <= i < n:
            r = min(ranks[i], R)
            merged = w + scales[i] * b[i][:, :r] @ a[i][:r]
        assert np.allclose(out[t], x[t] @ merged.T + add[t], atol=1e-12)
    assert not s[3].any() and not s[4].any() and not s[1, 1:].any()
    gated, y, _ = od.adapter_linear(x, w, ids, a, b, scales, ranks, add, epilogue="interleaved", act="gelu")
    assert np.allclose(y, out) and np.allclose(gated, od.gate_act(y[:, 0::2], "gelu") * y[:, 1::2])
    only, _, _ = od.adapter_linear(x, None, ids, a, b, scales, ranks)
    assert np.allclose(only + x @ w.T + add, out)
