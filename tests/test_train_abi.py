"""Refusals of the norm, the router's gradients and the experts with 16-bit weights, on the CPU: every check runs
before any device call."""
import ctypes

import pytest

mx = pytest.importorskip("mxfp4_weight_mixture_amd", reason="libmxmoe.so is not built")

P = 1 << 20          # distinct 16-byte aligned addresses, far enough apart for the sizes below
S = mx.STATUS


def _refused(st, status, needle):
    msg = mx.lib.moe_last_error_message().decode()
    assert st == S[status] and needle in msg, (st, msg)


def _norm(**kw):
    d = dict(T=4, H=64, dtype=0, x_dtype=0, residual_dtype=0, weight_dtype=0, out_dtype=0, eps=1e-6, x=P, residual=2 * P,
             weight=3 * P, residual_out=4 * P, out=5 * P, codes=6 * P, scales=7 * P, x_stride=64, residual_stride=64,
             residual_out_stride=64, out_stride=64)
    d.update(kw)
    return mx.NormArgs(**d)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(T=-1), "MOE_ERR_SHAPE", "T = -1"),
    (dict(T=1 << 22), "MOE_ERR_SHAPE", "T ="),
    (dict(H=60), "MOE_ERR_SHAPE", "H = 60"),
    (dict(H=0), "MOE_ERR_SHAPE", "H = 0"),
    (dict(H=32776, x_stride=32776), "MOE_ERR_SHAPE", "H = 32776"),
    (dict(H=72, x_stride=72, residual_stride=72, residual_out_stride=72, out_stride=72), "MOE_ERR_SHAPE", "H % 32"),
    (dict(eps=-1e-6), "MOE_ERR_INVALID_ARG", "eps"),
    (dict(eps=float("nan")), "MOE_ERR_INVALID_ARG", "eps"),
    (dict(eps=float("inf")), "MOE_ERR_INVALID_ARG", "eps"),
    (dict(dtype=2), "MOE_ERR_INVALID_ARG", "dtype"),
    (dict(x_dtype=1), "MOE_ERR_INVALID_ARG", "x_dtype"),
    (dict(residual_dtype=1), "MOE_ERR_INVALID_ARG", "residual_dtype"),
    (dict(weight_dtype=1), "MOE_ERR_INVALID_ARG", "weight_dtype"),
    (dict(out_dtype=3), "MOE_ERR_INVALID_ARG", "out_dtype"),
    (dict(x_stride=60), "MOE_ERR_SHAPE", "x_stride"),
    (dict(residual_stride=68), "MOE_ERR_SHAPE", "residual_stride"),
    (dict(residual_out_stride=1 << 22), "MOE_ERR_SHAPE", "residual_out_stride"),
    (dict(out_stride=0), "MOE_ERR_SHAPE", "out_stride"),
    (dict(residual_out=None), "MOE_ERR_INVALID_ARG", "come together"),
    (dict(residual=None), "MOE_ERR_INVALID_ARG", "come together"),
    (dict(scales=None), "MOE_ERR_INVALID_ARG", "come together"),
    (dict(x=None), "MOE_ERR_INVALID_ARG", "null"),
    (dict(weight=None), "MOE_ERR_INVALID_ARG", "null"),
    (dict(out=None, codes=None, scales=None), "MOE_ERR_INVALID_ARG", "no output"),
    (dict(x=P + 8), "MOE_ERR_INVALID_ARG", "x is not 16-byte"),
    (dict(codes=6 * P + 8), "MOE_ERR_INVALID_ARG", "codes is not 16-byte"),
    (dict(out=2 * P), "MOE_ERR_INVALID_ARG", "out overlaps residual"),
    (dict(out=P + 16), "MOE_ERR_INVALID_ARG", "out overlaps x"),
    (dict(out=P, out_dtype=2), "MOE_ERR_INVALID_ARG", "out overlaps x"),
    (dict(residual_out=2 * P, residual_out_stride=72), "MOE_ERR_INVALID_ARG", "residual_out overlaps residual"),
    (dict(out=4 * P), "MOE_ERR_INVALID_ARG", "out and residual_out"),
    (dict(scales=6 * P + 255), "MOE_ERR_INVALID_ARG", "codes and scales"),
    (dict(scales=3 * P), "MOE_ERR_INVALID_ARG", "scales overlaps weight"),
])
def test_norm_refusals(kw, status, needle):
    _refused(mx.lib.moe_rms_norm_forward(ctypes.byref(_norm(**kw)), None), status, needle)


def _norm_grad(**kw):
    d = dict(T=4, H=64, dtype=0, dout_dtype=0, x_dtype=0, weight_dtype=0, dresidual_dtype=0, dx_dtype=0, dw_dtype=0,
             accumulate=0, eps=1e-6, dout=P, x=2 * P, weight=3 * P, dresidual=4 * P, dx=5 * P, dweight=6 * P,
             dout_stride=64, x_stride=64, dresidual_stride=64, dx_stride=64, workspace=7 * P, workspace_bytes=P)
    d.update(kw)
    return mx.NormGradArgs(**d)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(T=-1), "MOE_ERR_SHAPE", "T = -1"),
    (dict(H=12), "MOE_ERR_SHAPE", "H = 12"),
    (dict(eps=-1.0), "MOE_ERR_INVALID_ARG", "eps"),
    (dict(dout_dtype=1), "MOE_ERR_INVALID_ARG", "dout_dtype"),
    (dict(x_dtype=1), "MOE_ERR_INVALID_ARG", "x_dtype"),
    (dict(weight_dtype=4), "MOE_ERR_INVALID_ARG", "weight_dtype"),
    (dict(dresidual_dtype=1), "MOE_ERR_INVALID_ARG", "dresidual_dtype"),
    (dict(dx_dtype=1), "MOE_ERR_INVALID_ARG", "dx_dtype"),
    (dict(dw_dtype=1), "MOE_ERR_INVALID_ARG", "dw_dtype"),
    (dict(accumulate=2), "MOE_ERR_INVALID_ARG", "accumulate"),
    (dict(dout_stride=60), "MOE_ERR_SHAPE", "dout_stride"),
    (dict(x_stride=63), "MOE_ERR_SHAPE", "x_stride"),
    (dict(dresidual_stride=0), "MOE_ERR_SHAPE", "dresidual_stride"),
    (dict(dx_stride=1 << 30), "MOE_ERR_SHAPE", "dx_stride"),
    (dict(dout=None), "MOE_ERR_INVALID_ARG", "null"),
    (dict(workspace=None), "MOE_ERR_WORKSPACE", "need"),
    (dict(workspace_bytes=100), "MOE_ERR_WORKSPACE", "need"),
    (dict(dweight=6 * P + 4), "MOE_ERR_INVALID_ARG", "dweight is not 16-byte"),
    (dict(dx=2 * P), "MOE_ERR_INVALID_ARG", "dx overlaps x"),
    (dict(dx=P, dx_stride=72), "MOE_ERR_INVALID_ARG", "dx overlaps dout"),
    (dict(dx=4 * P, dx_dtype=2), "MOE_ERR_INVALID_ARG", "dx overlaps dresidual"),
    (dict(dweight=3 * P), "MOE_ERR_INVALID_ARG", "dweight overlaps weight"),
    (dict(workspace=5 * P), "MOE_ERR_INVALID_ARG", "dx and workspace"),
])
def test_norm_backward_refusals(kw, status, needle):
    _refused(mx.lib.moe_rms_norm_backward(ctypes.byref(_norm_grad(**kw)), None), status, needle)


def _combine(**kw):
    d = dict(dout=P, y=2 * P, y_dtype=0, dest_row=3 * P, topk_w=4 * P, T=4, k=2, H=64, dy=5 * P, dy_dtype=0,
             dtopk_w=6 * P, stream=None)
    d.update(kw)
    return mx.lib.moe_combine_backward(*d.values())


@pytest.mark.parametrize("kw,status,needle", [
    (dict(T=-1), "MOE_ERR_SHAPE", "T = -1"),
    (dict(T=1 << 22), "MOE_ERR_SHAPE", "T ="),
    (dict(k=0), "MOE_ERR_SHAPE", "k = 0"),
    (dict(k=65), "MOE_ERR_SHAPE", "k = 65"),
    (dict(H=36), "MOE_ERR_SHAPE", "H = 36"),
    (dict(y_dtype=3), "MOE_ERR_INVALID_ARG", "y_dtype"),
    (dict(dy_dtype=-1), "MOE_ERR_INVALID_ARG", "dy_dtype"),
    (dict(dout=None), "MOE_ERR_INVALID_ARG", "null"),
    (dict(y=None), "MOE_ERR_INVALID_ARG", "null"),
    (dict(topk_w=None), "MOE_ERR_INVALID_ARG", "null"),
    (dict(topk_w=4 * P + 2), "MOE_ERR_INVALID_ARG", "4-byte"),
    (dict(dy=5 * P + 8), "MOE_ERR_INVALID_ARG", "dy is not 16-byte"),
    (dict(dy=2 * P), "MOE_ERR_INVALID_ARG", "dy overlaps y"),
    (dict(dy=4 * P), "MOE_ERR_INVALID_ARG", "dy overlaps topk_w"),
    (dict(dtopk_w=4 * P + 4), "MOE_ERR_INVALID_ARG", "dtopk_w overlaps topk_w"),
    (dict(dtopk_w=5 * P + 4), "MOE_ERR_INVALID_ARG", "dtopk_w and dy"),
])
def test_combine_backward_refusals(kw, status, needle):
    _refused(_combine(**kw), status, needle)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(T=-1), "MOE_ERR_SHAPE", "T = -1"),
    (dict(T=1 << 26), "MOE_ERR_SHAPE", "T ="),
    (dict(E=0), "MOE_ERR_SHAPE", "E = 0"),
    (dict(E=1025), "MOE_ERR_SHAPE", "E = 1025"),
    (dict(k=9), "MOE_ERR_SHAPE", "k = 9"),
    (dict(dw=None), "MOE_ERR_INVALID_ARG", "null"),
    (dict(dl=None), "MOE_ERR_INVALID_ARG", "null"),
    (dict(dl=4 * P + 1), "MOE_ERR_INVALID_ARG", "4-byte"),
    (dict(ids=2 * P + 1), "MOE_ERR_INVALID_ARG", "4-byte"),
    (dict(dl=3 * P), "MOE_ERR_INVALID_ARG", "overlaps topk_w"),
])
def test_route_backward_refusals(kw, status, needle):
    d = dict(dw=P, ids=2 * P, w=3 * P, T=4, E=8, k=2, dl=4 * P, stream=None)
    d.update(kw)
    _refused(mx.lib.moe_route_backward(*d.values()), status, needle)


def test_norm_workspace_query():
    q = mx.lib.moe_rms_norm_grad_workspace_size
    assert q(4, 64) >= 4 * 64 * 4 and q(1 << 20, 7168) == q(1 << 21, 7168)
    assert q(-1, 64) == q(4, 0) == q(1 << 22, 64) == q(4, 40000) == 0
