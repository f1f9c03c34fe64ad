"""Experts spread over devices: each share's forward, combine and way back beside the whole's, rows of the other
share never written (NaN in their place) and never read; rows that are not there in the combine."""
import numpy as np
import pytest
import torch

from oracle import moe as omoe
from tests import dense_util as du

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("mxfp4_weight_mixture_amd")
BF, HF, F = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("dtype", [BF, HF, F])
@pytest.mark.parametrize("T,k,H", [(1, 1, 8), (40, 16, 136), (9, 20, 1096), (700, 2, 64)])
def test_combine_of_rows_that_are_not_there(T, k, H, dtype):
    g = np.random.default_rng(T + k)
    dest = g.permutation(T * k).astype(np.int32)
    y, w = du.normal((T * k, H), 1.0, dtype, 3), torch.from_numpy(g.random((T, k)).astype(np.float32)).to("cuda")
    lost = g.random(T * k) < 0.4
    lost[: k] = True                     # a token without any row
    y64, w64 = du.f64(y), np.where(lost.reshape(T, k), 0.0, du.f64(w))
    y[torch.from_numpy(dest[lost]).long().to("cuda")] = float("nan")
    d = dest.copy()
    d[lost] = g.choice([-1, T * k, 2 ** 31 - 1, -(2 ** 31)], lost.sum())
    out, xn = mx.combine(y, torch.from_numpy(d).to("cuda"), w, rms_next=True)
    ref = omoe.combine(y64, dest, w64)
    du.assert_within(out, ref, k * du.F32 * omoe.combine(np.abs(y64), dest, w64) + 1e-37)
    assert (out[0] == 0).all()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("T,E,k,H,I,cut", [(70, 9, 2, 136, 72, 4), (33, 16, 4, 264, 40, 15), (2, 8, 3, 64, 32, 1),
                                           (300, 6, 6, 1096, 264, 3)])
def test_two_shares_add_up(T, E, k, H, I, cut, dtype):
    w1, w2 = du.normal((E, 2 * I, H), H ** -0.5, dtype, 1), du.normal((E, H, I), I ** -0.5, dtype, 2)
    x, dout = du.normal((T, H), 1.0, dtype, 3), du.normal((T, H), 1.0, F, 4)
    ids, w = mx.route(du.normal((T, E), 1.0, F, 5), k)
    off, src, dest = mx.permute(ids, E)
    rows = dict(gather=src, gather_div=k)

    def step(a, b):
        f, o = mx.ExpertFFN(w1[a:b], w2[a:b]), off[a: b + 1].contiguous()
        d = torch.where((dest >= off[a]) & (dest < off[b]), dest, -1)
        y = torch.full((T * k, H), float("nan"), dtype=dtype, device="cuda")
        _, gu = f.forward(x, o, out=y, save=True, **rows)
        dy = torch.full_like(y, float("nan"))
        _, dw = mx.combine_backward(dout, y, d, w, dy=dy)
        dx, dw1, dw2 = f.backward(dy, x, o, gu, dest_row=d, dx=torch.empty((T, H), device="cuda"), **rows)
        lo, hi = int(off[a]), int(off[b])
        assert y[lo:hi].isfinite().all() and y[:lo].isnan().all() and y[hi:].isnan().all() and dy[:lo].isnan().all()
        return mx.combine(y, d, w), dw, dx, dw1, dw2

    whole, first, second = step(0, E), step(0, cut), step(cut, E)
    for a, p, q in zip(whole[:3], first, second):
        # the same products; the sums over the token's rows are split: k additions in fp32
        assert p.isfinite().all() and q.isfinite().all()
        # (terms bounded by 8 times the largest result: a sum of k of them, rounded k times)
        assert (a.double() - p.double() - q.double()).abs().max() <= 2 * k * du.F32 * 8 * k * a.abs().max()
    # one share alone holds each of the k weights' gradients and each expert's weights
    assert torch.equal(first[1] + second[1], whole[1])
    d1, d2 = torch.cat([first[3], second[3]]), torch.cat([first[4], second[4]])
    for e, (got, want) in enumerate(zip((d1, d2), whole[3:])):
        err = (got.double() - want.double()).norm() / want.double().norm()
        assert err <= 2 * du.u(dtype), (e, float(err))
