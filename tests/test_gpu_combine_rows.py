"""fp16 rows through the combine, alone and as the experts' default result on its way through a training step.

Bound: k products and additions in fp32, k * 2^-24 of the sum of magnitudes."""
import numpy as np
import pytest
import torch

from oracle import moe as omoe
from tests import dense_util as du
from tests import test_gpu_train_layer as tl

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("mxfp4_weight_mixture_amd")
BF, HF, F = torch.bfloat16, torch.float16, torch.float32


def _case(T, k, H, dtype, seed=1):
    g = np.random.default_rng(seed)
    dest = g.permutation(T * k).astype(np.int32)
    w = g.random((T, k)).astype(np.float32)
    return du.normal((T * k, H), 1.0, dtype, seed), torch.from_numpy(dest).to("cuda"), torch.from_numpy(w).to("cuda")


@pytest.mark.parametrize("T,k,H", [(1, 1, 8), (77, 5, 264), (40, 16, 7168), (3, 64, 8200), (2, 3, 16392)])
def test_combine_of_fp16_rows(T, k, H):
    y, dest, w = _case(T, k, H, HF)
    out, xn = mx.combine(y, dest, w, rms_next=True)
    y64, w64, d = du.f64(y), du.f64(w), dest.cpu().numpy()
    ref = omoe.combine(y64, d, w64)
    du.assert_within(out, ref, k * du.F32 * omoe.combine(np.abs(y64), d, w64) + 1e-37)
    # the same numbers in fp32 rows: the same products in the same order
    same, same_next = mx.combine(y.float(), dest, w, rms_next=True)
    assert torch.equal(out, same)
    assert (xn.float() - same_next.float()).abs().max() <= 2.0 ** -7 * same_next.float().abs().max()
    nxt = omoe.rms_rescale(ref)
    assert np.all(np.abs(du.f64(xn) - nxt) <= 2.0 ** -7 * np.abs(nxt) + 1e-30)


def test_infinities_and_subnormals_of_fp16_rows():
    y, dest, w = _case(6, 2, 64, HF)
    y[3], y[7] = float("inf"), 2.0 ** -24
    out = mx.combine(y, dest, w)
    assert torch.equal(out, mx.combine(y.float(), dest, w)) and out.isinf().any()


def _default_step(x, residual, dout, dres, w1, w2, wr, wn, k, layout, act):
    """test_gpu_train_layer's step with every call's default types."""
    E, norm, experts = w1.shape[0], mx.RMSNorm(wn, eps=1e-5), mx.ExpertFFN(w1, w2, layout=layout, act=act)
    n = norm.forward(x, residual)
    ids, w = mx.route((n.out.float() @ wr.float().t()).contiguous(), k)
    off, src, dest = mx.permute(ids, E)
    rows = dict(gather=src, gather_div=k)
    y, gu = experts.forward(n.out, off, save=True, **rows)
    assert y.dtype == w1.dtype
    out = mx.combine(y, dest, w)
    dy, dw = mx.combine_backward(dout, y, dest, w)
    dlogits = mx.route_backward(dw, ids, w, E)
    dn, dw1, dw2 = experts.backward(dy, n.out, off, gu, dest_row=dest, dx=torch.empty(x.shape, device="cuda"), **rows)
    dn += dlogits @ wr.float()
    dwr = dlogits.t().contiguous() @ n.out.float()
    dx, dwn = norm.backward(dn, n.residual, dresidual=dres, dw_dtype=F)
    return dict(out=out, dx=dx, dwn=dwn, dwr=dwr, dw1=dw1, dw2=dw2), (ids, n.residual)


@pytest.mark.parametrize("dtype", [HF, BF])
@pytest.mark.parametrize("T,E,k,H,I,layout,act", [(70, 9, 2, 136, 72, "split", "silu"),
                                                  (33, 16, 4, 264, 40, "interleaved", "gelu")])
def test_training_step_in_default_types(T, E, k, H, I, layout, act, dtype):
    w = tl._weights(E, H, I, dtype, 11)
    x, residual = du.normal((T, H), 1.0, F, 21), du.normal((T, H), 1.0, dtype, 22)
    dout, dres = du.normal((T, H), 1.0, F, 23), du.normal((T, H), 1.0, dtype, 24)
    got, (ids, r) = _default_step(x, residual, dout, dres, *w, k, layout, act)
    want = tl._autograd(r, ids, dout, dres, *w, layout, act)
    # 2-norms, as test_training_step_against_autograd: at most eight roundings to 16 bits, doubled
    for name, ref in want.items():
        err = (got[name].double().cpu() - ref).norm() / ref.norm()
        assert err <= 16 * du.u(dtype), (name, float(err))
