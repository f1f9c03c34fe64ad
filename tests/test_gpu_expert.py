"""The routed experts with 16-bit weights, forward and backward, against the float64 oracle, expert by expert.

Row counts cover none, one, every class of row tile (up to 64, 128, 256 rows) with its edges, and several tiles;
widths that no tile divides.  Bounds are the dense block's (dense_util), for each expert's rows; a token's gradient
adds up its rows' bounds and one fp32 rounding for each addition."""
import numpy as np
import pytest
import torch

from oracle import train as ot
from tests import dense_util as du

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("mxfp4_weight_mixture_amd")
BF, HF, F = torch.bfloat16, torch.float16, torch.float32

COUNTS = {"one": [1], "few": [0, 1, 3, 0, 2], "edges": [64, 65, 128, 129, 1, 0], "tiles": [256, 0, 257, 63, 320, 513],
          "skewed": [700, 0, 0, 3, 20, 1, 0, 90]}


def _offsets(counts, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(counts)]), dtype=torch.int32, device="cuda")


def _experts(E, H, I, dtype, seed, layout="split", act="silu"):
    w1, w2 = du.normal((E, 2 * I, H), H ** -0.5, dtype, seed), du.normal((E, H, I), I ** -0.5, dtype, seed + 1)
    return mx.ExpertFFN(w1, w2, layout=layout, act=act)


def _forward_bounds(x, off, f, out_dtype):
    """(out, bound), (gate_up, fp32 error) of rows [rows][H]; rows of no expert are NaN."""
    rows = x.shape[0]
    out, b = np.full((rows, f.H), np.nan), np.full((rows, f.H), np.nan)
    gu, e = np.full((rows, 2 * f.I), np.nan), np.full((rows, 2 * f.I), np.nan)
    w1, w2 = du.f64(f.w1), du.f64(f.w2)
    for i in range(f.E):
        s = slice(int(off[i]), int(off[i + 1]))
        if s.start < s.stop:
            out[s], b[s], gu[s], e[s], _, _ = du.ffn_bounds(x[s], w1[i], w2[i], f.layout, f.act, f.dtype, out_dtype)
    return (out, b), (gu, e)


def _grad_bounds(dout, x, off, f, save, dx_dtype, dw_dtype, base1=0.0, base2=0.0):
    w1, w2 = du.f64(f.w1), du.f64(f.w2)
    dx, bx = np.full(x.shape, np.nan), np.full(x.shape, np.nan)
    g1, b1, g2, b2 = np.zeros(w1.shape), np.zeros(w1.shape), np.zeros(w2.shape), np.zeros(w2.shape)
    base1, base2 = np.broadcast_to(base1, w1.shape), np.broadcast_to(base2, w2.shape)
    for i in range(f.E):
        s = slice(int(off[i]), int(off[i + 1]))
        if s.start < s.stop:
            (dx[s], bx[s]), (g1[i], b1[i]), (g2[i], b2[i]) = du.ffn_grad_bounds(
                dout[s], x[s], w1[i], w2[i], f.layout, f.act, f.dtype, save, dx_dtype, dw_dtype, base1[i], base2[i])
        else:
            g1[i], g2[i] = base1[i], base2[i]    # bounds 0: as they were
    return (dx, bx), (g1, b1), (g2, b2)


FORMS = [(BF, "split", "silu"), (HF, "interleaved", "gelu"), (HF, "split", "gelu"), (BF, "interleaved", "silu")]


@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("H,I", [(8, 8), (264, 72), (520, 264), (128, 384)])
@pytest.mark.parametrize("dtype,layout,act", FORMS)
def test_forward(counts, H, I, dtype, layout, act):
    n = COUNTS[counts]
    f, off = _experts(len(n), H, I, dtype, 7, layout, act), _offsets(n)
    x = du.normal((sum(n), H), 1.0, dtype, 8)
    (ref, bound), (gu, e_gu) = _forward_bounds(du.f64(x), off.tolist(), f, dtype)
    out, kept = f.forward(x, off, save=True)
    du.assert_within(out, ref, bound, "out")
    du.assert_within(kept, gu, e_gu + 1e-37, "gate_up")
    assert torch.equal(f.forward(x, off), out)
    _, half = f.forward(x, off, save="half")
    assert half.dtype == dtype and torch.equal(half, kept.to(dtype))


@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("H,I", [(8, 8), (264, 72), (520, 264)])
@pytest.mark.parametrize("dtype,layout,act,save", [f + (s,) for f, s in zip(FORMS, (True, True, "half", "half"))])
def test_backward(counts, H, I, dtype, layout, act, save):
    n = COUNTS[counts]
    f, off = _experts(len(n), H, I, dtype, 17, layout, act), _offsets(n)
    x, dout = du.normal((sum(n), H), 1.0, dtype, 18), du.normal((sum(n), H), 1.0, dtype, 19)
    _, gu = f.forward(x, off, save=save)
    got = f.backward(dout, x, off, gu)
    refs = _grad_bounds(du.f64(dout), du.f64(x), off.tolist(), f, gu.dtype, dtype, dtype)
    for g, (ref, bound), name in zip(got, refs, ("dx", "dw1", "dw2")):
        du.assert_within(g, ref, bound, name)
    # each alone is the same
    assert torch.equal(f.backward(dout, x, off, gu, dw1=False, dw2=None)[0], got[0])
    assert torch.equal(f.backward(dout, x, off, gu, dx=False, dw2=False)[1], got[1])
    assert torch.equal(f.backward(dout, x, off, gu, dx=None, dw1=False)[2], got[2])


def _routed(T, E, k, seed):
    g = torch.Generator().manual_seed(seed)
    ids, w = mx.route(torch.randn((T, E), generator=g).to("cuda"), k)
    off, src, dest = mx.permute(ids, E)
    return off, src, dest, w


@pytest.mark.parametrize("T,E,k,H,I", [(1, 8, 2, 72, 40), (7, 16, 3, 264, 72), (150, 5, 2, 136, 264),
                                       (400, 12, 4, 264, 136), (33, 300, 6, 64, 32)])
@pytest.mark.parametrize("dtype,layout,act", FORMS[:2])
def test_gathered_tokens(T, E, k, H, I, dtype, layout, act):
    off, src, dest, _ = _routed(T, E, k, T)
    f = _experts(E, H, I, dtype, 27, layout, act)
    x, dout = du.normal((T, H), 1.0, dtype, 28), du.normal((T * k, H), 1.0, dtype, 29)
    rows = dict(gather=src, gather_div=k)
    out, gu = f.forward(du.strided(x, 16), off, save=True, **rows)
    plain = x[src.long() // k]
    want, gu2 = f.forward(plain, off, save=True)
    assert torch.equal(out, want) and torch.equal(gu, gu2)
    dx, dw1, dw2 = f.backward(dout, du.strided(x, 8), off, gu, dest_row=dest, **rows)
    dxr, v1, v2 = f.backward(dout, plain, off, gu, dx=torch.empty((T * k, H), device="cuda"))
    assert torch.equal(dw1, v1) and torch.equal(dw2, v2)
    (ref, bound), _, _ = _grad_bounds(du.f64(dout), du.f64(plain), off.tolist(), f, F, F, dtype)
    d = dest.view(T, k).cpu().numpy()
    total = ref[d].sum(axis=1)
    du.assert_within(dx, total, du.rounded(total, bound[d].sum(axis=1) + k * du.F32 * np.abs(ref[d]).sum(axis=1), dtype),
                     "dx")
    # the tokens' sum is in slot order, of the rows' fp32 gradients
    acc = torch.zeros((T, H), device="cuda")
    for j in range(k):
        acc += dxr[dest.view(T, k)[:, j].long()]
    assert torch.equal(dx, acc.to(dtype))


def test_rows_outside_the_experts_and_tokens_that_are_not_there():
    """A device's share of the experts (first offset above 0), padding behind the last, gathers outside the tokens."""
    n, H, I, T, k = [5, 0, 130, 2], 136, 72, 60, 3
    rows = T * k
    f, off = _experts(4, H, I, BF, 37), _offsets(n, first=9)
    lo, hi = 9, 9 + sum(n)
    g = torch.Generator().manual_seed(3)
    gather = torch.randint(0, T * k, (rows,), generator=g).to(torch.int32).to("cuda")
    gather[11], gather[20], gather[30] = -1, T * k, 2 ** 31 - 1
    gather[:lo], gather[hi:] = -(2 ** 31), 2 ** 31 - 1
    x, dout = du.normal((T, H), 1.0, BF, 38), du.normal((rows, H), 1.0, BF, 39)
    dout[:lo], dout[hi:] = float("nan"), float("nan")
    plain = torch.from_numpy(ot.gathered(du.f64(x), gather.cpu().numpy(), k)).to(BF).to("cuda")
    out = torch.full((rows, H), 5.0, dtype=BF, device="cuda")
    _, gu = f.forward(x, off, gather=gather, gather_div=k, out=out, save=True)
    assert (out[:lo] == 5.0).all() and (out[hi:] == 5.0).all()
    ref, bound = _forward_bounds(du.f64(plain), off.tolist(), f, BF)[0]
    du.assert_within(out[lo:hi], ref[lo:hi], bound[lo:hi], "out")
    gu[:lo], gu[hi:] = float("nan"), float("nan")
    # a dest_row that names rows in and outside the experts'
    dest = torch.randperm(rows, generator=g).to(torch.int32).to("cuda")
    dest[4], dest[9] = -5, rows + 7
    dx, dw1, dw2 = f.backward(dout, x, off, gu, gather=gather, gather_div=k, dest_row=dest)
    dxr = torch.full((rows, H), 4.0, device="cuda")
    _, v1, v2 = f.backward(dout, plain, off, gu, dx=dxr)
    assert torch.equal(dw1, v1) and torch.equal(dw2, v2) and dw1.isfinite().all() and not dw1[1].any()
    assert (dxr[:lo] == 4.0).all() and (dxr[hi:] == 4.0).all()
    acc = torch.zeros((T, H), device="cuda")
    for t in range(T):
        for j in range(k):
            d = int(dest[t * k + j])
            if lo <= d < hi:
                acc[t] += dxr[d]
    assert torch.equal(dx, acc.to(BF))


@pytest.mark.parametrize("counts", ["few", "skewed"])
def test_types_strides_and_accumulation(counts):
    n, H, I = COUNTS[counts], 264, 136
    rows = sum(n)
    f, off = _experts(len(n), H, I, BF, 47), _offsets(n)
    x, dout = du.normal((rows, H), 1.0, BF, 48), du.normal((rows, H), 1.0, BF, 49)
    wide = torch.full((rows + 2, H + 16), 3.0, device="cuda")
    out = wide[1: rows + 1, 8: H + 8]
    o, gu = f.forward(du.strided(x, 24), off, out=out, save=True)
    (ref, bound), _ = _forward_bounds(du.f64(x), off.tolist(), f, F)
    assert o is out
    du.assert_within(out, ref, bound, "out in fp32")
    wide[1: rows + 1, 8: H + 8] = 3.0
    assert (wide == 3.0).all()
    b1, b2 = du.normal(tuple(f.w1.shape), 3.0, F, 50), du.normal(tuple(f.w2.shape), 3.0, F, 51)
    g1, g2 = b1.clone(), b2.clone()
    dx = torch.full((rows, H + 8), 5.0, device="cuda")
    got = f.backward(du.strided(dout, 8), du.strided(x, 16), off, gu, dx=dx[:, :H], dw1=g1, dw2=g2, accumulate=True)
    refs = _grad_bounds(du.f64(dout), du.f64(x), off.tolist(), f, F, F, F, du.f64(b1), du.f64(b2))
    for v, (ref, bound), name in zip(got, refs, ("dx", "dw1", "dw2")):
        du.assert_within(v, ref, bound, name)
    assert (dx[:, H:] == 5.0).all()
    for e, c in enumerate(n):
        if c == 0:
            assert torch.equal(g1[e], b1[e]) and torch.equal(g2[e], b2[e])


def test_no_rows():
    f, off = _experts(3, 64, 32, BF, 3), _offsets([0, 0, 0])
    x = torch.zeros((0, 64), dtype=BF, device="cuda")
    out, gu = f.forward(x, off, save=True)
    assert out.shape == (0, 64) and gu.shape == (0, 64)
    dx, dw1, dw2 = f.backward(out, x, off, gu)
    assert dx.shape == (0, 64) and not dw1.any() and not dw2.any()
    dw1.fill_(2.0), dw2.fill_(3.0)
    f.backward(out, x, off, gu, dw1=dw1, dw2=dw2, accumulate=True)
    assert (dw1 == 2.0).all() and (dw2 == 3.0).all()
    # rows there are, none of them an expert's; tokens without rows
    x5 = torch.full((5, 64), float("nan"), dtype=BF, device="cuda")
    out = torch.full((5, 64), 7.0, dtype=BF, device="cuda")
    _, gu = f.forward(x5, off, out=out, save=True)
    assert (out == 7.0).all()
    _, dw1, dw2 = f.backward(x5, x5, off, gu)
    assert not dw1.any() and not dw2.any()
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    dest = torch.zeros(4, dtype=torch.int32, device="cuda")
    dx, _, _ = f.backward(x, x5[:4], off, gu[:0], gather=none, gather_div=1, dest_row=dest)
    assert dx.shape == (4, 64) and not dx.any()


def test_offsets_that_do_not_ascend_stay_in_bounds():
    """Nothing is promised of the results but that rows that are not there are not touched."""
    f = _experts(6, 64, 32, BF, 3)
    off = torch.tensor([-7, 300, 10, 2 ** 31 - 1, -(2 ** 31), 40, 1000], dtype=torch.int32, device="cuda")
    buf = torch.full((3 * 300, 64), 7.0, dtype=BF, device="cuda")
    x = torch.zeros((300, 64), dtype=BF, device="cuda")
    _, gu = f.forward(x, off, out=buf[300:600], save=True)
    dx = torch.full((3 * 300, 64), 7.0, dtype=BF, device="cuda")
    f.backward(x, x, off, gu, dx=dx[300:600])
    torch.cuda.synchronize()
    for b in (buf, dx):
        assert (b[:300] == 7.0).all() and (b[600:] == 7.0).all()


def test_infinities_stay_with_their_expert_and_row():
    n, H, I = [70, 1, 0, 40], 136, 72
    f, off = _experts(4, H, I, BF, 61), _offsets(n)
    x, dout = du.normal((111, H), 1.0, BF, 62), du.normal((111, H), 1.0, BF, 63)
    clean, gu = f.forward(x, off, save=True)
    dx0, d10, d20 = f.backward(dout, x, off, gu)
    x[3, 5], f.w1[1, 0, 0] = float("inf"), float("nan")
    out, gu = f.forward(x, off, save=True)
    dx, d1, d2 = f.backward(dout, x, off, gu)
    rest = torch.ones(111, dtype=torch.bool)
    rest[[3, 70]] = False
    assert torch.equal(out[rest], clean[rest]) and torch.equal(dx[rest], dx0[rest])
    assert torch.equal(d1[2:], d10[2:]) and torch.equal(d2[2:], d20[2:]) and not out[3].isfinite().any()


def test_one_expert_is_the_dense_block_and_the_order_of_experts_does_not_matter():
    H, I, T = 520, 264, 300
    f = _experts(3, H, I, BF, 71)
    x = du.normal((3 * T, H), 1.0, BF, 72)
    out = f.forward(x, _offsets([T, T, T]))
    for e in range(3):
        s = slice(e * T, (e + 1) * T)
        ref, bound, *_ = du.ffn_bounds(du.f64(x[s]), du.f64(f.w1[e]), du.f64(f.w2[e]), "split", "silu", BF, BF)
        du.assert_within(out[s], ref, bound, "an expert alone")
    turned = mx.ExpertFFN(f.w1.flip(0).contiguous(), f.w2.flip(0).contiguous())
    back = turned.forward(torch.cat([x[2 * T:], x[T: 2 * T], x[:T]]), _offsets([T, T, T]))
    assert torch.equal(torch.cat([back[2 * T:], back[T: 2 * T], back[:T]]), out)


def test_gradients_against_differences():
    """The directional derivatives of sum(dout * out), by central differences of the forward kernel in fp32 out."""
    T, E, k, H, I = 24, 4, 2, 64, 40
    off, src, dest, _ = _routed(T, E, k, 5)
    f = _experts(E, H, I, HF, 81, "interleaved", "gelu")
    x, dout = du.normal((T, H), 1.0, HF, 82), du.normal((T * k, H), 1.0, HF, 83)
    rows = dict(gather=src, gather_div=k)
    _, gu = f.forward(x, off, save=True, **rows)
    dx, dw1, dw2 = f.backward(dout, x, off, gu, dest_row=dest, **rows)
    d = 2.0 ** -4
    for grad, base, at in ((dx, x, "x"), (dw1, f.w1, "w1"), (dw2, f.w2, "w2")):
        step = torch.sign(grad.float()).to(HF) * d * base.float().std().to(HF)
        vals, args = [], {"x": x, "w1": f.w1, "w2": f.w2}
        for sgn in (1, -1):
            a = dict(args)
            a[at] = base + sgn * step
            out = mx.ExpertFFN(a["w1"], a["w2"], layout="interleaved", act="gelu").forward(a["x"], off, out_dtype=F, **rows)
            vals.append((out.double() * dout.double()).sum().item())
        want = (grad.double() * ((base + step).double() - (base - step).double())).sum().item()
        # second-order remainder: the step is 1/16 of the values' spread, so its cube is 2.4e-4 of them;
        # the slope along the gradient's signs is a sum of magnitudes, far above fp16's 2^-11 roundings
        assert abs((vals[0] - vals[1]) - want) < 0.02 * abs(want), (at, vals, want)


@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (40, 12, 3), (300, 6, 2)])
def test_side_stream_repeat_and_two_graphs(T, E, k):
    H, I = 264, 136
    runs = []
    for i, t in enumerate((T, T + 9)):
        off, src, dest, _ = _routed(t, E, k, t)
        f = _experts(E, H, I, BF, 90 + i)
        x, dout = du.normal((t, H), 1.0, BF, 91), du.normal((t * k, H), 1.0, BF, 92)
        def step(stream=None, f=f, x=x, off=off, src=src, dest=dest, dout=dout):
            rows = dict(gather=src, gather_div=k, stream=stream)
            out, gu = f.forward(x, off, save=True, **rows)
            return (out,) + tuple(f.backward(dout, x, off, gu, dest_row=dest, **rows))
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
        runs.append((x, step, g, outs, (off, src, dest)))
    for r in range(3):
        for x, step, g, outs, idx in runs:
            x.copy_(du.normal(tuple(x.shape), 1.0, BF, 1000 * r + x.shape[0]))
            if r == 2:     # another routing of the same sizes: the graph reads the current offsets
                off, src, dest, _ = _routed(x.shape[0], E, k, 77)
                for a, b in zip(idx, (off, src, dest)):
                    a.copy_(b)
            g.replay()
            eager = step()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, eager)), (r, x.shape)


def test_binding_refusals():
    f, off = _experts(3, 64, 32, BF, 5), _offsets([1, 2, 1])
    x = torch.zeros((4, 64), dtype=BF, device="cuda")
    idx = torch.zeros(6, dtype=torch.int32, device="cuda")
    for a, kw, needle in (((x[:, :32], off), {}, "shape"), ((x.half(), off), {}, "float16"), ((x.cpu(), off), {}, "cpu"),
                          ((x, off[:3]), {}, "expert_offsets"), ((x, off.long()), {}, "expert_offsets"),
                          ((x, off), dict(gather_div=2), "without gather"), ((x, off), dict(gather=idx.long()), "gather"),
                          ((x, off), dict(out=torch.empty((3, 64), dtype=BF, device="cuda")), "out has"),
                          ((x, off), dict(save="fp8"), "save")):
        with pytest.raises(ValueError, match=needle):
            f.forward(*a, **kw)
    out, gu = f.forward(x, off, save=True)
    with pytest.raises(ValueError, match="gate_up"):
        f.backward(out, x, off, gu[:3])
    with pytest.raises(ValueError, match="dest_row"):
        f.backward(torch.zeros((6, 64), dtype=BF, device="cuda"), x, off, torch.zeros((6, 64), device="cuda"), gather=idx)
    with pytest.raises(ValueError, match="accumulate"):
        f.backward(out, x, off, gu, accumulate=True)
    with pytest.raises(ValueError, match="dw1"):
        f.backward(out, x, off, gu, dw1=torch.zeros((3, 64, 64), dtype=HF, device="cuda"), dw_dtype=BF)
    with pytest.raises(ValueError, match="are not"):
        mx.ExpertFFN(f.w1, f.w2[:2])
    with pytest.raises(mx.MoeError, match="overlaps x"):
        f.forward(x, off, out=x)
    with pytest.raises(mx.MoeError, match="gather_div"):
        f.forward(x, off, gather=idx, gather_div=0)
