"""The experts with 16-bit weights in every kernel that a call may choose, at the sizes that choose it.

Each case names the tiles it is for: few rows with long sums; 64 x 64 tiles; narrow tiles (128 columns); wide ones (256)
with each kind of remainder, and weight gradients in tiles of 128 and of 256.  Whole results would take the float64
oracle long, so it computes parts that are exact by themselves: out and dx for some rows of every expert (its first and
last ones, the tiles' edges, others drawn), dw1 and dw2 for some inner indices i (their rows of w1 and columns of w2
alone: gate i and up i see no other).  Bounds: dense_util."""
import numpy as np
import pytest
import torch

from oracle import train as ot
from tests import dense_util as du

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("mxfp4_weight_mixture_amd")
BF, HF, F = torch.bfloat16, torch.float16, torch.float32

CASES = {
    "few, up to 16 rows": ([1, 0, 3, 16, 2], 1096, 1032),
    "few, several tiles of 32 rows": ([1, 0, 50, 3, 17, 1], 1096, 1032),
    "few, then narrow (short second sum)": ([5] * 40 + [0, 33], 1160, 520),
    "64 x 64": ([65, 0, 128, 1, 200], 1096, 520),
    "narrow": ([30, 0, 64, 65, 130, 1, 128, 129] * 3, 1096, 776),
    "narrow, streaming": ([2, 0, 40, 1] * 40, 520, 392),
    "wide, 256 x 256 gradients": ([1100, 1290, 0, 900, 1124], 4096, 1024),
    "wide, 128 x 128 gradients": ([4133, 3867], 1096, 776),
}


def _case(name, dtype, layout, act):
    counts, H, I = CASES[name]
    E, rows = len(counts), sum(counts)
    w1 = du.normal((E, 2 * I, H), H ** -0.5, dtype, 3)
    f = mx.ExpertFFN(w1, du.normal((E, H, I), I ** -0.5, dtype, 4), layout=layout, act=act)
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(5)
    tokens = 16 if name.endswith("up to 16 rows") else max(rows // 2, 1)
    gather = torch.randint(0, 2 * tokens, (rows,), generator=g).to(torch.int32).to("cuda")
    x = du.strided(du.normal((tokens, H), 1.0, dtype, 6), 24)
    return counts, f, off, x, gather


def _some(count, g):
    edges = {0, 15, 16, 31, 32, 63, 64, 127, 128, 255, 256, count - 1, count // 256 * 256, count // 64 * 64}
    return sorted({r for r in edges if 0 <= r < count} | set(torch.randint(0, count, (6,), generator=g).tolist()))


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("dtype,layout,act", [(BF, "split", "silu"), (HF, "interleaved", "gelu")])
def test_every_kernel(name, dtype, layout, act):
    counts, f, off, x, gather = _case(name, dtype, layout, act)
    rows, H, I, E = sum(counts), f.H, f.I, f.E
    how = dict(gather=gather, gather_div=2)
    out, gu = f.forward(x, off, save=True, **how)
    assert torch.equal(f.forward(x, off, **how), out)
    plain = x[gather.long() // 2]
    assert torch.equal(f.forward(plain, off), out) or name.startswith("few")   # (the rows' bound picks the tiles there)
    dout = du.normal((rows, H), 1.0, dtype, 7)
    _, dw1, dw2 = f.backward(dout, x, off, gu, dx=False, **how)
    dxr, v1, v2 = f.backward(dout, plain, off, gu, dx=torch.empty((rows, H), device="cuda"))
    assert torch.equal(dw1, v1) and torch.equal(dw2, v2)
    g = torch.Generator().manual_seed(11)
    for e in sorted(range(E), key=lambda i: -counts[i])[:4] + [E - 1]:
        if not counts[e]:
            assert not dw1[e].any() and not dw2[e].any()
            continue
        s = slice(int(off[e]), int(off[e + 1]))
        xe, de, w1, w2 = du.f64(plain[s]), du.f64(dout[s]), du.f64(f.w1[e]), du.f64(f.w2[e])
        at = _some(counts[e], g)
        ref, bound, kept, e_kept, _, _ = du.ffn_bounds(xe[at], w1, w2, layout, act, dtype, dtype)
        du.assert_within(out[s][at], ref, bound, f"out of expert {e}")
        du.assert_within(gu[s][at], kept, e_kept + 1e-37, f"gate_up of expert {e}")
        (ref, bound), _, _ = du.ffn_grad_bounds(de[at], xe[at], w1, w2, layout, act, dtype, F, F, dtype)
        du.assert_within(dxr[s][at], ref, bound, f"dx of expert {e}")
        i = sorted({0, 31, 32, 63, 64, 127, 128, I - 1} & set(range(I)))
        gate, up = (i, [I + k for k in i]) if layout == "split" else ([2 * k for k in i], [2 * k + 1 for k in i])
        both = gate + up if layout == "split" else [r for p in zip(gate, up) for r in p]
        _, (r1, b1), (r2, b2) = du.ffn_grad_bounds(de, xe, w1[both], w2[:, i], layout, act, dtype, F, F, dtype)
        du.assert_within(dw1[e][both], r1, b1, f"dw1 of expert {e}")
        du.assert_within(dw2[e][:, i], r2, b2, f"dw2 of expert {e}")


@pytest.mark.parametrize("name", ["few, several tiles of 32 rows", "narrow", "64 x 64"])
def test_values_behind_rows_and_in_foreign_tokens(name):
    """Rows beside the experts' hold NaN, tokens that do not exist count as zeros, in these kernels too."""
    counts, f, _, x, gather = _case(name, BF, "split", "silu")
    rows, lo = sum(counts), 7
    off = torch.tensor(lo + np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    gather = torch.cat([torch.full((lo,), 2 ** 31 - 1, dtype=torch.int32, device="cuda"), gather,
                        torch.full((9,), -(2 ** 31), dtype=torch.int32, device="cuda")])
    gather[lo], gather[lo + rows - 1], gather[lo + rows // 2] = -1, 2 * x.shape[0], 2 ** 31 - 1
    plain = torch.from_numpy(ot.gathered(du.f64(x), gather.cpu().numpy(), 2)).to(BF).to("cuda")
    out = torch.full((rows + lo + 9, f.H), 5.0, dtype=BF, device="cuda")
    f.forward(x, off, gather=gather, gather_div=2, out=out)
    plain[:lo], plain[lo + rows:] = float("nan"), float("nan")
    want = torch.full_like(out, 5.0)
    f.forward(plain, off, out=want)
    assert torch.equal(out, want) and (out[:lo] == 5.0).all() and (out[lo + rows:] == 5.0).all()
    assert out.isfinite().all()


@pytest.mark.parametrize("E", [1024, 1025, 2100, 8192])
def test_many_experts(E):
    """More experts than the lists' threads; rows of some in several tiles."""
    g = torch.Generator().manual_seed(E)
    counts = (torch.rand(E, generator=g) < 0.1).int() * torch.randint(1, 4, (E,), generator=g)
    counts[3], counts[E // 2], counts[E - 1] = 300, 70, 1
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[1:] = counts.cumsum(0)
    H, I, rows = 16, 8, int(off[-1])
    w1, w2 = du.normal((E, 2 * I, H), H ** -0.5, BF, 1), du.normal((E, H, I), I ** -0.5, BF, 2)
    f, offd = mx.ExpertFFN(w1, w2), off.to("cuda")
    x, dout = du.normal((rows, H), 1.0, BF, 3), du.normal((rows, H), 1.0, BF, 4)
    out, gu = f.forward(x, offd, save=True)
    dx, dw1, dw2 = f.backward(dout, x, offd, gu)
    x64, d64, w1, w2 = du.f64(x), du.f64(dout), du.f64(w1), du.f64(w2)
    for e in torch.nonzero(counts)[:, 0].tolist():
        s = slice(int(off[e]), int(off[e + 1]))
        ref, bound, *_ = du.ffn_bounds(x64[s], w1[e], w2[e], "split", "silu", BF, BF)
        du.assert_within(out[s], ref, bound, f"out of expert {e}")
        for got, (ref, bound) in zip((dx[s], dw1[e], dw2[e]), du.ffn_grad_bounds(d64[s], x64[s], w1[e], w2[e], "split",
                                                                                "silu", BF, F, BF, BF)):
            du.assert_within(got, ref, bound, f"gradients of expert {e}")
    empty = (counts == 0).to("cuda")
    assert not dw1[empty].any() and not dw2[empty].any()


@pytest.mark.parametrize("E,H,I", [(64, 64, 32), (64, 1096, 776), (6, 4096, 1024)])
def test_offsets_that_ask_for_more_tiles_than_there_are_rows(E, H, I):
    """Every second expert claims every row: nothing is promised but that other memory is not touched."""
    rows = 2000
    f = mx.ExpertFFN(torch.zeros((E, 2 * I, H), dtype=BF, device="cuda"), torch.zeros((E, H, I), dtype=BF, device="cuda"))
    off = torch.tensor([0, rows] * (E // 2) + [0], dtype=torch.int32, device="cuda")
    buf = torch.full((3 * rows, H), 7.0, dtype=BF, device="cuda")
    x = torch.zeros((rows, H), dtype=BF, device="cuda")
    _, gu = f.forward(x, off, out=buf[rows: 2 * rows], save=True)
    dx = torch.full((3 * rows, H), 7.0, dtype=BF, device="cuda")
    f.backward(x, x, off, torch.zeros_like(gu), dx=dx[rows: 2 * rows])
    torch.cuda.synchronize()
    for b in (buf, dx):
        assert (b[:rows] == 7.0).all() and (b[2 * rows:] == 7.0).all()


def test_weights_behind_4_gib():
    E, H, I, rows = 260, 4096, 2048, 200
    w1, w2 = torch.zeros((E, 2 * I, H), dtype=BF, device="cuda"), torch.zeros((E, H, I), dtype=BF, device="cuda")
    for e in (E - 1, 130):
        w1[e], w2[e] = du.normal((2 * I, H), H ** -0.5, BF, e), du.normal((H, I), I ** -0.5, BF, e + 1)
    f = mx.ExpertFFN(w1, w2)
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[131:], off[E] = 60, rows
    x, dout = du.normal((rows, H), 1.0, BF, 5), du.normal((rows, H), 1.0, BF, 6)
    out, gu = f.forward(x, off.to("cuda"), save=True)
    dx, dw1, dw2 = f.backward(dout, x, off.to("cuda"), gu)
    for e, s in ((130, slice(0, 60)), (E - 1, slice(60, rows))):
        x64, d64, a, b = du.f64(x[s]), du.f64(dout[s]), du.f64(w1[e]), du.f64(w2[e])
        at = [0, 31, x64.shape[0] - 1]
        ref, bound, *_ = du.ffn_bounds(x64[at], a, b, "split", "silu", BF, BF)
        du.assert_within(out[s][at], ref, bound, "out")
        du.assert_within(dx[s][at], *du.ffn_grad_bounds(d64[at], x64[at], a, b, "split", "silu", BF, F, BF, BF)[0], "dx")
        i = [0, 100, I - 1]
        both = i + [I + k for k in i]
        _, (r1, b1), (r2, b2) = du.ffn_grad_bounds(d64, x64, a[both], b[:, i], "split", "silu", BF, F, BF, BF)
        du.assert_within(dw1[e][both], r1, b1, "dw1")
        du.assert_within(dw2[e][:, i], r2, b2, "dw2")
    assert not dw1[:130].any() and not dw2[131: E - 1].any()
