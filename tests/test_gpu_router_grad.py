"""Gradients of the combine and of the routing against the float64 oracle.

Bounds: dy is one product, then its rounding u = finfo(type).eps / 2; a dot product of H terms in fp32 is off by at
most H * 2^-24 of the sum of magnitudes; dlogits: k products and additions and two more roundings."""
import numpy as np
import pytest
import torch

from oracle import train as ot
from tests import dense_util as du

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("mxfp4_weight_mixture_amd")
BF, HF, F = torch.bfloat16, torch.float16, torch.float32


def _routed(T, E, k, seed):
    g = torch.Generator().manual_seed(seed)
    ids, w = mx.route(torch.randn((T, E), generator=g).to("cuda"), k)
    _, _, dest = mx.permute(ids, E)
    return ids, w, dest


@pytest.mark.parametrize("T,E,k,H", [(1, 1, 1, 8), (1, 8, 8, 64), (3, 16, 6, 520), (40, 9, 2, 1096), (17, 256, 6, 4096),
                                     (5, 896, 16, 7168), (9, 64, 64, 24), (300, 12, 3, 136), (2, 20, 9, 8200)])
@pytest.mark.parametrize("yt,dt", [(BF, BF), (F, HF), (HF, HF), (F, F), (BF, F)])
def test_combine_backward(T, E, k, H, yt, dt):
    ids, w, dest = _routed(T, E, k, T + E)
    dout, y = du.normal((T, H), 1.0, F, 3), du.normal((T * k, H), 1.0, yt, 4)
    dy, dw = mx.combine_backward(dout, y, dest, w, dy_dtype=dt)
    d64, y64, w64 = du.f64(dout), du.f64(y), du.f64(w)
    rdy, rdw = ot.combine_grad(d64, y64, dest.cpu().numpy(), w64)
    du.assert_within(dy, rdy, du.rounded(rdy, du.F32 * np.abs(rdy), dt), "dy")
    mag, _ = ot.combine_grad(np.abs(d64), np.abs(y64), dest.cpu().numpy(), w64)[::-1]
    du.assert_within(dw, rdw, (H + 2) * du.F32 * mag + 1e-37, "dtopk_w")
    a, none = mx.combine_backward(dout, None, dest, w, dy_dtype=dt, dw=False)
    assert none is None and torch.equal(a, dy)
    none, b = mx.combine_backward(dout, y, dest.view(T, k), w, dy=False)
    assert none is None and torch.equal(b, dw)


def test_rows_that_are_not_there():
    T, k, H = 6, 3, 72
    _, w, dest = _routed(T, 5, k, 1)
    dout, y = du.normal((T, H), 1.0, F, 3), du.normal((T * k, H), 1.0, BF, 4)
    full, fw = mx.combine_backward(dout, y, dest, w)
    lost = dest[[2, 7, 11]].long()
    dest[2], dest[7], dest[11] = -1, T * k, 2 ** 31 - 1
    dy = torch.full((T * k, H), 9.0, dtype=BF, device="cuda")
    y[lost] = float("nan")
    got, dw = mx.combine_backward(dout, y, dest, w, dy=dy)
    keep = torch.ones(T * k, dtype=torch.bool)
    keep[lost.cpu()] = False
    assert got is dy and torch.equal(dy[keep], full[keep]) and (dy[~keep] == 9.0).all()
    fw.view(-1)[[2, 7, 11]] = 0.0
    assert torch.equal(dw, fw)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 8, 8), (5, 63, 6), (40, 256, 6), (9, 896, 16), (700, 70, 64),
                                   (2, 1024, 64)])
def test_route_backward(T, E, k):
    ids, w, _ = _routed(T, E, k, T * k)
    dw = du.normal((T, k), 1.0, F, 7)
    got = mx.route_backward(dw, ids, w, E)
    w64, d64, i = du.f64(w), du.f64(dw), ids.cpu().numpy()
    ref = ot.route_grad(d64, i, w64, E)
    err = np.zeros((T, E))
    kept = w64 * ((k + 2) * du.F32 * (w64 * np.abs(d64)).sum(axis=1, keepdims=True) + 3 * du.F32 * np.abs(d64))
    np.put_along_axis(err, i.astype(np.int64), kept, 1)
    du.assert_within(got, ref, err + du.F32 * np.abs(ref) + 1e-37, "dlogits")
    assert (du.f64(got)[err == 0] == 0).all()
    # the kept logits' gradients of a softmax add up to nothing
    assert np.abs(du.f64(got).sum(axis=1)).max() <= kept.sum(axis=1).max() + k * du.F32 * np.abs(ref).sum(axis=1).max()


def test_route_backward_repeated_and_foreign_ids():
    ids = torch.tensor([[2, 1, 2], [-1, 5, 0], [4, 4, 4]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, 0.25, 0.25]] * 3, device="cuda")
    dw = torch.tensor([[1.0, 2.0, -1.0]] * 3, device="cuda")
    got = mx.route_backward(dw, ids, w, 5)
    assert np.array_equal(du.f64(got), ot.route_grad(du.f64(dw), ids.cpu().numpy(), du.f64(w), 5))   # exact in fp32


def test_no_tokens():
    z = lambda *s, dtype=F: torch.zeros(s, dtype=dtype, device="cuda")
    dy, dw = mx.combine_backward(z(0, 64), z(0, 64, dtype=BF), z(0, dtype=torch.int32), z(0, 4))
    assert dy.shape == (0, 64) and dw.shape == (0, 4)
    assert mx.route_backward(dw, z(0, 4, dtype=torch.int32), z(0, 4), 9).shape == (0, 9)


def test_against_differences_of_the_forward_calls():
    """sum(dout * combine(y, route(logits))) by the logits: the library's own forward calls, central differences."""
    T, E, k, H = 5, 12, 4, 48
    logits = du.normal((T, E), 1.0, F, 31)
    dout, y = du.normal((T, H), 1.0, F, 32), du.normal((T * k, H), 1.0, F, 33)
    ids, w = mx.route(logits, k)
    _, _, dest = mx.permute(ids, E)
    dl = mx.route_backward(mx.combine_backward(dout, y, dest, w)[1], ids, w, E)
    h = 2.0 ** -9
    vals = []
    for sgn in (1, -1):
        i2, w2 = mx.route(logits + sgn * h * torch.sign(dl), k)
        assert torch.equal(i2, ids)
        vals.append((mx.combine(y, dest, w2).double() * dout.double()).sum().item())
    want = 2 * h * dl.double().abs().sum().item()
    # third order: h^2 / 6 of a slope whose third derivative is of its own order; fp32's roundings of 240 sums of
    # about 1, 2^-23 each, against a difference of 2^-8 times about 20
    assert abs(vals[0] - vals[1] - want) < 1e-3 * want


def test_side_stream_and_graph():
    T, E, k, H = 40, 64, 6, 1096
    ids, w, dest = _routed(T, E, k, 2)
    dout, y = du.normal((T, H), 1.0, F, 3), du.normal((T * k, H), 1.0, BF, 4)
    def step(stream=None):
        dy, dw = mx.combine_backward(dout, y, dest, w, stream=stream)
        return dy, dw, mx.route_backward(dw, ids, w, E, stream=stream)
    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = step(s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for i in range(3):
        dout.copy_(du.normal((T, H), 1.0, F, 50 + i))
        g.replay()
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, eager))


def test_binding_refusals():
    T, E, k, H = 4, 8, 2, 64
    ids, w, dest = _routed(T, E, k, 2)
    dout, y = du.normal((T, H), 1.0, F, 3), du.normal((T * k, H), 1.0, BF, 4)
    for a, kw, needle in (((dout.to(BF), y, dest, w), {}, "dout"), ((dout, y[:3], dest, w), {}, "y must"),
                          ((dout, y, dest.long(), w), {}, "dest_row"), ((dout, None, dest, w), {}, "needs y"),
                          ((dout, y, dest, w.cpu()), {}, "current device|on cpu"),
                          ((dout, y, dest, w), dict(dy=torch.empty_like(y), dy_dtype=HF), "dy must")):
        with pytest.raises((ValueError, mx.MoeError), match=needle):
            mx.combine_backward(*a, **kw)
    with pytest.raises(ValueError, match="topk_ids"):
        mx.route_backward(w, ids.long(), w, E)
    with pytest.raises(mx.MoeError, match="E = 1025"):
        mx.route_backward(w, ids, w, 1025)
