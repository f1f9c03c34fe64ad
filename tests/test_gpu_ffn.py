"""The gated feed-forward block with 16-bit weights, forward and backward, against the float64 oracle.

Sizes cover one token to several row tiles, widths that no tile divides, one
reduction block and several; tolerances are derived in dense_util."""
import numpy as np
import pytest
import torch

from tests import dense_util as du

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("mxfp4_weight_mixture_amd")
BF, HF, F = torch.bfloat16, torch.float16, torch.float32


def _block(T, H, I, dtype, seed, layout="split", act="silu", x_pad=0):
    x = du.normal((T, H), 1.0, dtype, seed)
    w1, w2 = du.normal((2 * I, H), H ** -0.5, dtype, seed + 1), du.normal((H, I), I ** -0.5, dtype, seed + 2)
    return (du.strided(x, x_pad) if x_pad else x), mx.GatedFFN(w1, w2, layout=layout, act=act)


SIZES = [(1, 8, 8), (1, 512, 256), (2, 1000, 136), (5, 264, 72), (16, 128, 128), (17, 520, 264), (31, 2048, 96),
         (33, 96, 1032), (64, 512, 512), (65, 200, 328), (127, 136, 64), (130, 392, 200), (257, 72, 40),
         (300, 1096, 520)]


@pytest.mark.parametrize("T,H,I", SIZES)
@pytest.mark.parametrize("dtype,layout,act", [(BF, "split", "silu"), (HF, "interleaved", "gelu"),
                                              (HF, "split", "gelu"), (BF, "interleaved", "silu")])
def test_forward(T, H, I, dtype, layout, act):
    x, f = _block(T, H, I, dtype, 100 + T, layout, act)
    ref, bound, gu, e_gu, _, _ = du.ffn_bounds(du.f64(x), du.f64(f.w1), du.f64(f.w2), layout, act, dtype, dtype)
    du.assert_within(f.forward(x), ref, bound, "out")
    out, kept = f.forward(x, save=True)
    du.assert_within(out, ref, bound, "out with save")
    du.assert_within(kept, gu, e_gu + 1e-37, "gate_up")
    _, half = f.forward(x, save="half")
    assert half.dtype == dtype
    du.assert_within(half, gu, du.rounded(gu, e_gu, dtype), "gate_up in 16 bits")


@pytest.mark.parametrize("T", [1, 16, 48, 100, 200])
@pytest.mark.parametrize("out_dtype", [F, BF])
def test_forward_strides_and_add(T, out_dtype):
    H, I = 328, 152
    x, f = _block(T, H, I, BF, 7, x_pad=24)
    add = du.strided(du.normal((T, H), 2.0, out_dtype, 9), 8)
    ref, bound, *_ = du.ffn_bounds(du.f64(x), du.f64(f.w1), du.f64(f.w2), "split", "silu", BF, out_dtype,
                                   add=du.f64(add))
    # `out` inside a larger buffer: what lies around its rows keeps its value
    wide = torch.full((T + 2, H + 16), 3.0, dtype=out_dtype, device="cuda")
    out = wide[1: T + 1, 8: H + 8]
    assert f.forward(x, add=add, out=out) is out
    du.assert_within(out, ref, bound, "out")
    wide[1: T + 1, 8: H + 8] = 3.0
    assert (wide == 3.0).all()
    res = add.clone()
    f.forward(x, add=res, out=res)
    du.assert_within(res, ref, bound, "in place")


def test_no_tokens():
    x, f = _block(0, 64, 32, BF, 3)
    out, gu = f.forward(x, save=True)
    assert out.shape == (0, 64) and gu.shape == (0, 64)
    dx, dw1, dw2 = f.backward(out, x, gu)
    assert dx.shape == (0, 64) and dw1.shape == (64, 64) and not dw1.any() and not dw2.any()
    dw1.fill_(2.0), dw2.fill_(3.0)
    f.backward(out, x, gu, dw1=dw1, dw2=dw2, accumulate=True)
    assert (dw1 == 2.0).all() and (dw2 == 3.0).all()


@pytest.mark.parametrize("T,H,I", [(1, 8, 8), (3, 264, 72), (16, 128, 128), (65, 200, 328), (130, 392, 200),
                                   (257, 72, 40), (300, 1096, 264), (520, 264, 520)])
@pytest.mark.parametrize("dtype,layout,act,save", [(BF, "split", "silu", True), (HF, "interleaved", "gelu", True),
                                                   (HF, "split", "silu", "half"),
                                                   (BF, "interleaved", "gelu", "half")])
def test_backward(T, H, I, dtype, layout, act, save):
    x, f = _block(T, H, I, dtype, 300 + T, layout, act)
    dout = du.normal((T, H), 1.0, dtype, 17)
    _, gu = f.forward(x, save=save)
    refs = du.ffn_grad_bounds(du.f64(dout), du.f64(x), du.f64(f.w1), du.f64(f.w2), layout, act, dtype, gu.dtype,
                              dtype, dtype)
    for got, (ref, bound), name in zip(f.backward(dout, x, gu), refs, ("dx", "dw1", "dw2")):
        du.assert_within(got, ref, bound, name)


@pytest.mark.parametrize("T", [40, 200])
def test_backward_fp32_accumulated_and_parts(T):
    H, I = 264, 136
    x, f = _block(T, H, I, BF, 41, x_pad=8)
    dout = du.strided(du.normal((T, H), 1.0, BF, 42), 16)
    _, gu = f.forward(x, save=True)
    b1, b2 = du.normal((2 * I, H), 3.0, F, 43), du.normal((H, I), 3.0, F, 44)
    refs = du.ffn_grad_bounds(du.f64(dout), du.f64(x), du.f64(f.w1), du.f64(f.w2), "split", "silu", BF, F, F, F,
                              du.f64(b1), du.f64(b2))
    wide = torch.full((T, H + 8), 5.0, device="cuda")
    g1, g2 = b1.clone(), b2.clone()
    got = f.backward(dout, x, gu, dx=wide[:, :H], dw1=g1, dw2=g2, accumulate=True)
    for v, (ref, bound), name in zip(got, refs, ("dx", "dw1", "dw2")):
        du.assert_within(v, ref, bound, name)
    assert (wide[:, H:] == 5.0).all()
    # each part alone is the same part
    dx, n1, n2 = f.backward(dout, x, gu, dw1=False, dw2=None)
    assert n1 is None and n2 is None
    all3 = f.backward(dout, x, gu)
    assert torch.equal(dx, all3[0])
    assert torch.equal(f.backward(dout, x, gu, dx=False, dw2=False)[1], all3[1])
    assert torch.equal(f.backward(dout, x, gu, dx=False, dw1=False)[2], all3[2])


def test_gradients_against_differences():
    """The directional derivative of sum(dout * out), by central differences of the forward kernel in fp32 out."""
    T, H, I = 24, 64, 40
    x, f = _block(T, H, I, HF, 51, "interleaved", "gelu")
    dout = du.normal((T, H), 1.0, HF, 52)
    _, gu = f.forward(x, save=True)
    dx, dw1, dw2 = f.backward(dout, x, gu)
    d = 2.0 ** -4
    for grad, base, at in ((dx, x, "x"), (dw1, f.w1, "w1"), (dw2, f.w2, "w2")):
        step = torch.sign(grad.float()).to(HF) * d * base.float().std().to(HF)
        vals, args = [], {"x": x, "w1": f.w1, "w2": f.w2}
        for sgn in (1, -1):
            a = dict(args)
            a[at] = base + sgn * step
            out = mx.GatedFFN(a["w1"], a["w2"], layout="interleaved", act="gelu").forward(a["x"], out_dtype=F)
            vals.append((out.double() * dout.double()).sum().item())
        moved = ((base + step).double() - (base - step).double())
        want = (grad.double() * moved).sum().item()
        # second-order remainder: the step is 1/16 of the values' spread, so its cube is 2.4e-4 of them;
        # the slope along the gradient's signs is a sum of magnitudes, far above fp16's 2^-11 roundings
        assert abs((vals[0] - vals[1]) - want) < 0.02 * abs(want), (at, vals, want)


def test_infinities_stay_in_their_row():
    T, H, I = 70, 136, 72
    x, f = _block(T, H, I, BF, 61)
    clean = f.forward(x)
    x[33, 5], x[40, 1], x[64, 0] = float("inf"), float("nan"), float("-inf")
    out = f.forward(x)
    rows = torch.ones(T, dtype=torch.bool)
    rows[[33, 40, 64]] = False
    assert torch.equal(out[rows], clean[rows])
    assert out[40].isnan().all() and not out[33].isfinite().any()


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("big", [100.0, 3e4, 1e12, 1e18])
def test_saturated_gates(act, big):
    """Far from zero the activation is g or 0 and its derivative 1 or 0, with nothing overflowing on the way."""
    T, H, I = 9, 16, 8
    x = torch.zeros(T, H, dtype=BF, device="cuda")
    x[:, 0], x[:, 1] = 1.0, 1.0
    w1, w2 = torch.zeros(2 * I, H, dtype=BF, device="cuda"), torch.zeros(H, I, dtype=BF, device="cuda")
    w1[:4, 0], w1[4:I, 0], w1[I:, 1] = big, -big, 2.0
    w2[:I] = torch.eye(I)
    f = mx.GatedFFN(w1, w2, act=act)
    out, gu = f.forward(x, save=True)
    g = float(w1[0, 0])
    assert (out[:, :4].float() == 2 * g).all() and not out[:, 4:].any()
    dx, dw1, dw2 = f.backward(torch.ones_like(x), x, gu)
    assert dx.isfinite().all() and dw1.isfinite().all() and dw2.isfinite().all()
    # d_gate = 2 act'(gate), d_up = act(gate): over T equal tokens
    assert (dw1[:4, 0].float() == 2 * T).all() and not dw1[4:I].any() and not dw1[I + 4:].any()
    assert torch.allclose(dw1[I: I + 4, 1].float(), torch.full((4,), T * g, device="cuda"), rtol=2 * du.u(BF))


@pytest.mark.parametrize("T", [1, 20, 150])
def test_side_stream_and_repeat(T):
    x, f = _block(T, 520, 264, BF, 71)
    dout = du.normal((T, 520), 1.0, BF, 72)
    ref, gu = f.forward(x, save=True)
    grads = f.backward(dout, x, gu)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, gu2 = f.forward(x, save=True, stream=s)
    got = f.backward(dout, x, gu2, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, ref) and torch.equal(gu2, gu)
    assert all(torch.equal(a, b) for a, b in zip(got, grads))


def test_two_graphs_replayed_in_turn():
    """Forward and backward captured at two sizes; replays interleave with eager calls and read current inputs."""
    runs = []
    for T in (3, 140):
        x, f = _block(T, 392, 136, HF, 80 + T, act="gelu")
        dout = du.normal((T, 392), 1.0, HF, 90 + T)
        step = lambda x=x, f=f, dout=dout: (lambda o: (o[0],) + tuple(f.backward(dout, x, o[1])))(
            f.forward(x, save=True))
        step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = step()
        runs.append((x, step, g, outs))
    for k in range(3):
        for x, step, g, outs in runs:
            x.copy_(du.normal(tuple(x.shape), 1.0, HF, 1000 * k + x.shape[0]))
            g.replay()
            eager = step()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, eager)), (k, x.shape)


def test_binding_refusals():
    x, f = _block(4, 64, 32, BF, 5)
    z = torch.zeros
    for bad, needle in ((dict(x=z(4, 72, dtype=BF, device="cuda")), "shape"), (dict(x=x.half()), "float16"),
                        (dict(x=x.cpu()), "cpu"), (dict(x=x.t().contiguous().t()), "contiguous"),
                        (dict(x=x, out=z(4, 64, dtype=HF, device="cuda")), "out is"),
                        (dict(x=x, add=z(3, 64, dtype=BF, device="cuda")), "add has"),
                        (dict(x=x, add=z(4, 64, device="cuda"), out_dtype=BF), "add is")):
        with pytest.raises(ValueError, match=needle):
            f.forward(**bad)
    with pytest.raises(ValueError, match="save"):
        f.forward(x, save="fp8")
    out, gu = f.forward(x, save=True)
    with pytest.raises(ValueError, match="gate_up"):
        f.backward(out, x, gu[:, :32])
    with pytest.raises(ValueError, match="accumulate"):
        f.backward(out, x, gu, accumulate=True)
    with pytest.raises(ValueError, match="dw1"):
        f.backward(out, x, gu, dw1=z(64, 64, dtype=HF, device="cuda"), dw_dtype=BF)
    with pytest.raises(mx.MoeError, match="overlaps x"):
        f.forward(x, out=x)
    with pytest.raises(mx.MoeError, match="multiple of 8"):
        f.forward(torch.zeros(4, 68, dtype=BF, device="cuda")[:, :64])
    with pytest.raises(mx.MoeError, match="16-byte"):
        f.forward(torch.zeros(4, 72, dtype=BF, device="cuda")[:, 4:68])
    with pytest.raises(mx.MoeError, match="x_stride"):
        f.forward(x[:1].expand(4, 64))
