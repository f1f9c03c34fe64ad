"""Pins of oracle/train.py: automatic differentiation, differences and closed forms."""
import numpy as np
import pytest
import torch

from oracle import dense, moe
from oracle import train as ot

rng = np.random.default_rng(11)


def test_norm_against_autograd():
    x, w, d, dr = rng.normal(size=(5, 24)), rng.normal(size=24), rng.normal(size=(5, 24)), rng.normal(size=(5, 24))
    tx, tw = torch.from_numpy(x).requires_grad_(), torch.from_numpy(w).requires_grad_()
    ty = torch.nn.functional.rms_norm(tx, (24,), tw, eps=1e-3)
    out, _ = ot.rms_norm(x, w, 1e-3)
    assert np.allclose(out, ty.detach().numpy(), rtol=1e-12)
    (ty * torch.from_numpy(d) + tx * torch.from_numpy(dr)).sum().backward()
    dx, dw = ot.rms_norm_grad(d, x, w, 1e-3, dr)
    assert np.allclose(dx, tx.grad.numpy(), rtol=1e-10, atol=1e-13) and np.allclose(dw, tw.grad.numpy(), rtol=1e-11)


def test_norm_of_a_multiple():
    """The norm does not see a row's size, so its gradient is orthogonal to the row (eps = 0)."""
    x, w, d = rng.normal(size=(3, 16)), rng.normal(size=16), rng.normal(size=(3, 16))
    assert np.allclose(ot.rms_norm(x, w, 0.0)[0], ot.rms_norm(7.5 * x, w, 0.0)[0], rtol=1e-13)
    dx, _ = ot.rms_norm_grad(d, x, w, 0.0)
    assert np.allclose((dx * x).sum(axis=1), 0.0, atol=1e-13)


def test_combine_and_route_against_differences():
    """The derivative of sum(dout * combine(y, route(logits))) by each logit and each row."""
    T, E, k, H = 4, 7, 3, 5
    logits, dout = rng.normal(size=(T, E)), rng.normal(size=(T, H))
    y = rng.normal(size=(T * k, H))
    ids, _ = moe.route(logits, k)
    w = np.exp(np.take_along_axis(logits, ids.astype(np.int64), 1))
    w /= w.sum(axis=1, keepdims=True)
    _, _, dest = moe.permute(ids, E)

    def loss(lg, rows):
        kept = np.exp(np.take_along_axis(lg, ids.astype(np.int64), 1))   # (moe.route takes logits in fp32)
        ww = kept / kept.sum(axis=1, keepdims=True)
        return sum(ww[t, j] * (rows[dest[t * k + j]] @ dout[t]) for t in range(T) for j in range(k))

    dy, dw = ot.combine_grad(dout, y, dest, w)
    dl = ot.route_grad(dw, ids, w, E)
    h = 1e-6
    for t in range(T):
        for e in range(E):
            up, down = logits.copy(), logits.copy()
            up[t, e] += h
            down[t, e] -= h
            assert abs((loss(up, y) - loss(down, y)) / (2 * h) - dl[t, e]) < 1e-8
    for r, c in ((0, 0), (5, 2), (T * k - 1, H - 1)):
        up, down = y.copy(), y.copy()
        up[r, c] += h
        down[r, c] -= h
        assert abs((loss(logits, up) - loss(logits, down)) / (2 * h) - dy[r, c]) < 1e-8


def test_route_grad_of_a_repeated_id_adds_up():
    w, dw = np.array([[0.5, 0.25, 0.25]]), np.array([[1.0, 2.0, -1.0]])
    dl = ot.route_grad(dw, np.array([[2, 1, 2]]), w, 4)
    assert np.allclose(dl, [[0, 0.25 * (2 - 0.75), 0.5 * 0.25 + 0.25 * -1.75, 0]])


@pytest.mark.parametrize("layout,act", [("split", "silu"), ("interleaved", "gelu")])
def test_experts_against_autograd(layout, act):
    E, H, I, offsets = 4, 8, 6, np.array([1, 3, 3, 8, 9])
    x, w1, w2 = rng.normal(size=(11, H)), rng.normal(size=(E, 2 * I, H)), rng.normal(size=(E, H, I))
    d = rng.normal(size=(11, H))
    tx, t1, t2 = (torch.from_numpy(t).requires_grad_() for t in (x, w1, w2))
    total = 0
    for e in range(E):
        s = slice(offsets[e], offsets[e + 1])
        gu = tx[s] @ t1[e].T
        g, u = (gu[:, :I], gu[:, I:]) if layout == "split" else (gu[:, 0::2], gu[:, 1::2])
        a = torch.nn.functional.silu(g) if act == "silu" else torch.nn.functional.gelu(g, approximate="tanh")
        total = total + ((a * u) @ t2[e].T * torch.from_numpy(d[s])).sum()
    total.backward()
    out, gu, h = ot.expert_ffn(x, offsets, w1, w2, layout, act)
    assert np.isclose((out * d).sum(), total.item()) and not out[0].any() and not out[9:].any()
    for got, want in zip(ot.expert_ffn_grad(d, x, offsets, w1, w2, layout, act), (tx, t1, t2)):
        assert np.allclose(got, want.grad.numpy(), rtol=1e-9, atol=1e-11)
    # one expert with every row is the dense block
    one, _, _ = ot.expert_ffn(x, [0, 11], w1[:1], w2[:1], layout, act)
    assert np.allclose(one, dense.gated_ffn(x, w1[0], w2[0], layout, act)[0])


def test_gathered_rows():
    x = rng.normal(size=(3, 2))
    got = ot.gathered(x, [4, 0, -1, 6, 5], 2)
    assert np.array_equal(got, [x[2], x[0], [0, 0], [0, 0], x[2]])
