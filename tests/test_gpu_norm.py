"""The norm before a layer, forward and backward, against the float64 oracle.

Bounds.  A row's sums pass at most 32 additions in a thread, 6 across the lanes
and 16 across the waves: 64 * 2^-24 of the sum of magnitudes covers them with
the products' roundings.  1 / rms takes half of that error (its argument's
square root) and five more roundings: 40 * 2^-24.  The result's own rounding is
u = finfo(type).eps / 2.  dweight adds up to T rows in fp32: T * 2^-24 of the sum
of magnitudes."""
import numpy as np
import pytest
import torch

from oracle import mx as omx
from oracle import train as ot
from tests import dense_util as du

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("mxfp4_weight_mixture_amd")
BF, HF, F = torch.bfloat16, torch.float16, torch.float32
SUM, INV = 64 * du.F32, 40 * du.F32

SIZES = [(1, 8), (3, 24), (2, 504), (5, 512), (64, 520), (257, 1096), (33, 2216), (17, 4096), (4, 7168), (2, 8192),
         (3, 8200), (2, 16384), (2, 16392), (1, 32768), (700, 64)]


def _weight(H, dtype, seed=5):
    return (1 + 0.25 * torch.randn(H, generator=torch.Generator().manual_seed(seed))).to(dtype).to("cuda")


def _kept(x, residual):
    return x if residual is None else (x.float() + residual.float()).to(residual.dtype)


def _out_bound(r, w, eps, dtype):
    out, _ = ot.rms_norm(du.f64(r), du.f64(w), eps)
    return out, du.rounded(out, (INV + 2 * du.F32) * np.abs(out), dtype)


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("xt,rt,wt,ot_", [(BF, None, BF, BF), (HF, HF, HF, HF), (F, BF, BF, BF), (BF, F, F, F),
                                          (HF, F, HF, HF), (F, None, F, BF), (F, F, BF, F), (BF, BF, F, BF)])
def test_forward(T, H, xt, rt, wt, ot_):
    x, w = du.normal((T, H), 1.5, xt, T + H), _weight(H, wt)
    residual = None if rt is None else du.normal((T, H), 3.0, rt, T + H + 1)
    f = mx.RMSNorm(w, eps=1e-5)
    n = f.forward(x, residual, out_dtype=ot_)
    r = _kept(x, residual)
    assert n.codes is None and n.scales is None and (n.residual is None) == (rt is None) and n.out.dtype == ot_
    if rt is not None:
        assert torch.equal(n.residual, r)
    du.assert_within(n.out, *_out_bound(r, w, f.eps, ot_), "out")


@pytest.mark.parametrize("T,H", [(1, 32), (3, 64), (9, 96), (2, 4096), (5, 7168), (2, 16384 + 32), (130, 544)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_mxfp8_codes_are_those_of_the_fp32_values(T, H, dtype):
    x, residual, w = du.normal((T, H), 1.0, F, 3), du.normal((T, H), 2.0, dtype, 4), _weight(H, dtype)
    x[0, :16] = 0.0
    residual[0, :32] = 0.0
    x[0, :32] = 0.0                       # a block of zeros
    f = mx.RMSNorm(w)
    n = f.forward(x, residual, out_dtype=F, mxfp8=True)
    codes, scales = omx.quantize_mxfp8(du.f64(n.out))
    assert np.array_equal(n.scales.cpu().numpy(), scales)
    assert np.array_equal(n.codes.cpu().numpy(), codes)
    assert scales[0, 0] == 0 and not codes[0, :32].any()
    # beside 16-bit values and alone they are the same codes
    both, alone = f.forward(x, residual, mxfp8=True), f.forward(x, residual, out=False, mxfp8=True)
    assert alone.out is None and both.out.dtype == dtype
    for m in (both, alone):
        assert torch.equal(m.codes, n.codes) and torch.equal(m.scales, n.scales) and torch.equal(m.residual, n.residual)
    assert torch.equal(both.out, n.out.to(dtype))


def test_mxfp8_boundaries_and_what_is_not_finite():
    """With weights of a power of two per column and rows of equal size the values are known exactly."""
    H = 128
    x = torch.ones((4, H), device="cuda")
    w = torch.ones(H, device="cuda")
    w[:32] = 448.0                               # stays at scale 1
    w[32:64] = 449.0                             # takes the next power of two
    w[64:96] = 2.0 ** -130                       # below the smallest scale's reach: scale byte 0
    x[1, 100], x[2, 101], x[3, 7] = float("inf"), float("nan"), 0.0
    n = mx.RMSNorm(w, eps=0.0).forward(x, out_dtype=F, mxfp8=True)
    s = n.scales.cpu().numpy()
    assert s[0].tolist() == [127, 128, 0, 119]
    codes, scales = omx.quantize_mxfp8(du.f64(n.out[:1]))
    assert np.array_equal(n.codes[:1].cpu().numpy(), codes) and np.array_equal(s[:1], scales)
    # an infinite row: 1 / rms is 0, so the infinity's own value is NaN and the others are 0
    assert s[1].tolist() == [0, 0, 0, 255] and (n.codes[1, 96:] & 0x7f == 0x7f).all() and not n.codes[1, :96].any()
    assert (s[2] == 255).all() and (n.codes[2] & 0x7f == 0x7f).all()
    assert n.out[3].isfinite().all() and n.codes[3, 7] == 0


def _grads(dout, r, w, eps, dres, dx_dtype, dw_dtype, base=0.0):
    d, x, wt = du.f64(dout), du.f64(r), du.f64(w)
    dr = 0.0 if dres is None else du.f64(dres)
    dx, dw = ot.rms_norm_grad(d, x, wt, eps, dr)
    _, inv = ot.rms_norm(x, wt, eps)
    u, g, H = x * inv, d * wt, x.shape[1]
    c = np.abs((g * u).mean(axis=1, keepdims=True))
    e_c = SUM * np.abs(g * u).mean(axis=1, keepdims=True) + 2 * INV * c
    err = inv * (np.abs(u) * (e_c + (INV + 3 * du.F32) * c) + 3 * du.F32 * np.abs(g)) \
        + INV * inv * (np.abs(g) + np.abs(u) * c) + 2 * du.F32 * np.abs(dx)
    ew = (d.shape[0] * du.F32 + INV + 2 * du.F32) * np.abs(d * u).sum(axis=0)
    dw = dw + base
    ew = ew + du.F32 * (np.abs(dw) + np.abs(base))
    return (dx, du.rounded(dx, err, dx_dtype)), (dw, du.rounded(dw, ew, dw_dtype))


@pytest.mark.parametrize("T,H", SIZES + [(1300, 520), (513, 8)])
@pytest.mark.parametrize("xt,dt,wt,rt", [(BF, BF, BF, BF), (HF, HF, HF, None), (F, BF, BF, F), (BF, F, F, BF),
                                         (F, F, F, None)])
def test_backward(T, H, xt, dt, wt, rt):
    x, dout, w = du.normal((T, H), 1.5, xt, T), du.normal((T, H), 1.0, dt, T + 1), _weight(H, wt)
    dres = None if rt is None else du.normal((T, H), 0.5, rt, T + 2)
    f = mx.RMSNorm(w, eps=1e-5)
    dx, dw = f.backward(dout, x, dresidual=dres)
    assert dw.dtype == wt and dx.dtype in (BF, HF)
    for got, (ref, bound), name in zip((dx, dw), _grads(dout, x, w, f.eps, dres, dx.dtype, wt), ("dx", "dweight")):
        du.assert_within(got, ref, bound, name)
    a, none = f.backward(dout, x, dresidual=dres, dweight=False)
    assert none is None and torch.equal(a, dx)
    none, b = f.backward(dout, x, dresidual=dres, dx=None)
    assert none is None and torch.equal(b, dw)


@pytest.mark.parametrize("T", [1, 70, 600])
def test_strides_accumulation_and_in_place(T):
    H = 520
    x, res, w = du.normal((T, H), 1.0, BF, 1), du.normal((T, H), 1.0, F, 2), _weight(H, BF)
    f = mx.RMSNorm(w)
    want = f.forward(x, res)
    wide = torch.full((T + 2, H + 24), 7.0, dtype=BF, device="cuda")
    keep = torch.full((T, H + 8), 7.0, device="cuda")
    n = f.forward(du.strided(x, 16), du.strided(res, 8), out=wide[1: T + 1, 8: H + 8], residual_out=keep[:, :H])
    assert torch.equal(n.out, want.out) and torch.equal(n.residual, want.residual)
    wide[1: T + 1, 8: H + 8] = 7.0
    assert (wide == 7.0).all() and (keep[:, H:] == 7.0).all()
    # in place: the sum over the residual, the norm over x
    x2, res2 = x.clone(), res.clone()
    n = f.forward(x2, res2, out=x2, residual_out=res2)
    assert n.out is x2 and torch.equal(x2, want.out) and torch.equal(res2, want.residual)
    xf = x.float()
    n = f.forward(xf, res, residual_out=xf)
    assert torch.equal(xf, want.residual) and torch.equal(n.out, want.out)
    # gradients: added to an earlier one; dx over dout, over dresidual
    dout, dres, base = du.normal((T, H), 1.0, BF, 3), du.normal((T, H), 1.0, BF, 4), du.normal((H,), 2.0, F, 5)
    ref = _grads(dout, want.residual, w, f.eps, dres, BF, F, du.f64(base))
    dw = base.clone()
    dx, got = f.backward(du.strided(dout, 8), du.strided(want.residual, 16), dresidual=du.strided(dres, 24), dweight=dw,
                         accumulate=True)
    assert got is dw
    du.assert_within(dx, *ref[0], "dx")
    du.assert_within(dw, *ref[1], "dweight")
    d2, r2 = dout.clone(), dres.clone()
    f.backward(d2, want.residual, dresidual=dres, dx=d2)
    f.backward(dout, want.residual, dresidual=r2, dx=r2)
    assert torch.equal(d2, dx) and torch.equal(r2, dx)


def test_no_rows():
    f = mx.RMSNorm(_weight(64, BF))
    x = torch.zeros((0, 64), dtype=BF, device="cuda")
    n = f.forward(x, x, mxfp8=True)
    assert n.out.shape == n.codes.shape == (0, 64) and n.scales.shape == (0, 2)
    dx, dw = f.backward(x, x)
    assert dx.shape == (0, 64) and not dw.any()
    dw.fill_(2.0)
    f.backward(x, x, dweight=dw, accumulate=True)
    assert (dw == 2.0).all()


def test_zero_rows_and_rows_that_are_not_finite_stay_alone():
    T, H = 40, 264
    x, w = du.normal((T, H), 1.0, BF, 9), _weight(H, BF)
    f = mx.RMSNorm(w)
    clean, dout = f.forward(x).out, du.normal((T, H), 1.0, BF, 10)
    dclean, _ = f.backward(dout, x)
    x[3], x[7, 1], x[11, 0] = 0.0, float("nan"), float("inf")
    out, (dx, _) = f.forward(x).out, f.backward(dout, x)
    rest = torch.ones(T, dtype=torch.bool)
    rest[[3, 7, 11]] = False
    assert torch.equal(out[rest], clean[rest]) and torch.equal(dx[rest], dclean[rest])
    assert not out[3].any() and out[7].isnan().all() and out[11, 0].isnan() and not out[11, 1:].any()
    # a zero row: u = 0, so dx = dout * weight / sqrt(eps)
    want = du.f64(dout[3]) * du.f64(w) / np.sqrt(f.eps)
    du.assert_within(dx[3], want, du.rounded(want, INV * np.abs(want), BF), "dx of a zero row")


def test_gradient_against_differences():
    """Central differences of sum(dout * out) + sum(dres * r) by the fp32 forward."""
    T, H = 6, 40
    x, dout, dres, w = (du.normal((T, H), 1.0, F, 21), du.normal((T, H), 1.0, F, 22), du.normal((T, H), 1.0, F, 23),
                        _weight(H, F))
    dx, dw = mx.RMSNorm(w, eps=1e-3).backward(dout, x, dresidual=dres, dx=torch.empty_like(x))
    def loss(xx, ww):
        o = mx.RMSNorm(ww, eps=1e-3).forward(xx, out_dtype=F).out
        return ((dout.double() * o.double()).sum() + (dres.double() * xx.double()).sum()).item()
    h = 2.0 ** -8
    sx, sw = torch.sign(dx), torch.sign(dw)
    for got, want in (((loss(x + h * sx, w) - loss(x - h * sx, w)), (dx.abs().sum() * 2 * h).item()),
                      ((loss(x, w + h * sw) - loss(x, w - h * sw)), (dw.abs().sum() * 2 * h).item())):
        # the third-order remainder is h^2 = 1.5e-5 of the slope, times its curvature of order 1 to 10; fp32's
        # roundings of the 240 outputs, 2^-24 each of about 1, against a difference of 2 h times about 200
        assert abs(got - want) < 1e-3 * want


def test_rows_behind_4_gib():
    T, H = 70000, 32768
    x = torch.zeros((T, H), dtype=BF, device="cuda")
    w = _weight(H, BF)
    at = [0, 1, 32767, 65537, T - 1]
    x[at] = du.normal((len(at), H), 1.0, BF, 31)
    f = mx.RMSNorm(w)
    few = f.forward(x[at])
    out = f.forward(x, out=x).out
    assert torch.equal(out[at], few.out) and not out[2].any() and not out[T - 2].any()


@pytest.mark.parametrize("T", [1, 300])
def test_side_stream_repeat_and_two_graphs(T):
    H = 1096
    runs = []
    for k, rows in enumerate((T, T + 5)):
        x, res, dout = (du.normal((rows, H), 1.0, BF, 40 + 3 * k + i) for i in range(3))
        f = mx.RMSNorm(_weight(H, BF, k))
        def step(x=x, res=res, dout=dout, f=f, stream=None):
            n = f.forward(x, res, stream=stream)
            return (n.out, n.residual) + f.backward(dout, n.residual, dresidual=dout, stream=stream)
        want = step()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        got = step(stream=s)
        torch.cuda.current_stream().wait_stream(s)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = step()
        runs.append((x, step, g, outs))
    for k in range(3):
        for x, step, g, outs in runs:
            x.copy_(du.normal(tuple(x.shape), 1.0, BF, 100 * k + x.shape[0]))
            g.replay()
            eager = step()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, eager))


def test_binding_refusals():
    f = mx.RMSNorm(_weight(64, BF))
    x = torch.zeros((4, 64), dtype=BF, device="cuda")
    for kw, needle in ((dict(x=x[:, :32]), "shape"), (dict(x=x.half()), "float16"), (dict(x=x.cpu()), "cpu"),
                       (dict(x=x, residual=x[:3]), "shape"), (dict(x=x, residual_out=x), "without a residual"),
                       (dict(x=x, out=False), "no output"),
                       (dict(x=x, residual=x.float(), residual_out=torch.empty_like(x)), "residual_out is")):
        with pytest.raises(ValueError, match=needle):
            f.forward(**kw)
    with pytest.raises(ValueError, match="accumulate"):
        f.backward(x, x, accumulate=True)
    with pytest.raises(ValueError, match="dweight"):
        f.backward(x, x, dweight=torch.zeros(32, device="cuda"))
    with pytest.raises(mx.MoeError, match="32"):
        mx.RMSNorm(_weight(40, BF)).forward(torch.zeros((2, 40), dtype=BF, device="cuda"), mxfp8=True)
    with pytest.raises(mx.MoeError, match="out_dtype"):
        f.forward(x, out_dtype=HF)
    with pytest.raises(mx.MoeError, match="dx overlaps x"):
        f.backward(x.clone(), x, dx=x)
    with pytest.raises(mx.MoeError, match="16-byte"):
        f.forward(torch.zeros((4, 72), dtype=BF, device="cuda")[:, 4:68])
    with pytest.raises(ValueError, match="weight"):
        mx.RMSNorm(torch.ones((2, 8), device="cuda"))
