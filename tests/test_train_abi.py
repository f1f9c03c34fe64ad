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
    assert q(4, 64) >= 64 * 4 and q(4, 7168) >= 4 * 7168 * 4 and q(1 << 20, 7168) == q(1 << 21, 7168)
    assert q(-1, 64) == q(4, 0) == q(1 << 22, 64) == q(4, 40000) == 0


def _expert(**kw):
    d = dict(rows=8, H=64, I=32, E=3, layout=1, gate_act=0, dtype=0, out_dtype=0, save_dtype=2, tokens=4, gather_div=2,
             x=P, gather=2 * P, expert_offsets=3 * P, w1=4 * P, w2=5 * P, out=6 * P, gate_up=7 * P, x_stride=64,
             out_stride=64, workspace=8 * P, workspace_bytes=P)
    d.update(kw)
    return mx.ExpertFfnArgs(**d)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(rows=-1), "MOE_ERR_SHAPE", "rows = -1"),
    (dict(rows=(1 << 28) + 1), "MOE_ERR_SHAPE", "rows ="),
    (dict(rows=1 << 20, I=1 << 16), "MOE_ERR_SHAPE", "too many"),
    (dict(E=8192, I=1 << 15, H=1 << 10, x_stride=1 << 10, out_stride=1 << 10), "MOE_ERR_SHAPE", "experts of"),
    (dict(H=60), "MOE_ERR_SHAPE", "H = 60"),
    (dict(I=4), "MOE_ERR_SHAPE", "I = 4"),
    (dict(E=0), "MOE_ERR_SHAPE", "E = 0"),
    (dict(E=8193), "MOE_ERR_SHAPE", "E = 8193"),
    (dict(layout=0), "MOE_ERR_INVALID_ARG", "layout"),
    (dict(gate_act=2), "MOE_ERR_INVALID_ARG", "gate_act"),
    (dict(dtype=2), "MOE_ERR_INVALID_ARG", "dtype"),
    (dict(out_dtype=1), "MOE_ERR_INVALID_ARG", "out_dtype"),
    (dict(save_dtype=1), "MOE_ERR_INVALID_ARG", "save_dtype"),
    (dict(x_stride=56), "MOE_ERR_SHAPE", "x_stride"),
    (dict(out_stride=68), "MOE_ERR_SHAPE", "out_stride"),
    (dict(tokens=-1), "MOE_ERR_SHAPE", "tokens = -1"),
    (dict(gather_div=0), "MOE_ERR_SHAPE", "gather_div = 0"),
    (dict(tokens=1 << 24), "MOE_ERR_SHAPE", "2^30"),
    (dict(x=None), "MOE_ERR_INVALID_ARG", "null"),
    (dict(expert_offsets=None), "MOE_ERR_INVALID_ARG", "null"),
    (dict(workspace=None), "MOE_ERR_WORKSPACE", "need"),
    (dict(workspace_bytes=64), "MOE_ERR_WORKSPACE", "need"),
    (dict(x=P + 8), "MOE_ERR_INVALID_ARG", "x is not 16-byte"),
    (dict(gather=2 * P + 2), "MOE_ERR_INVALID_ARG", "gather is not 4-byte"),
    (dict(out=P + 256), "MOE_ERR_INVALID_ARG", "out overlaps x"),
    (dict(out=3 * P), "MOE_ERR_INVALID_ARG", "out overlaps expert_offsets"),
    (dict(gate_up=6 * P + 512), "MOE_ERR_INVALID_ARG", "out and gate_up"),
    (dict(workspace=5 * P - 256), "MOE_ERR_INVALID_ARG", "workspace overlaps w2"),
])
def test_expert_refusals(kw, status, needle):
    _refused(mx.lib.moe_expert_ffn_forward(ctypes.byref(_expert(**kw)), None), status, needle)


def _expert_grad(**kw):
    d = dict(rows=8, H=64, I=32, E=3, layout=1, gate_act=0, dtype=0, save_dtype=2, dx_dtype=0, dw_dtype=0, accumulate=0,
             tokens=4, gather_div=2, dout=P, x=2 * P, gather=3 * P, dest_row=4 * P, expert_offsets=5 * P, w1=6 * P,
             w2=7 * P, gate_up=8 * P, dx=9 * P, dw1=10 * P, dw2=11 * P, dout_stride=64, x_stride=64, dx_stride=64,
             workspace=12 * P, workspace_bytes=P)
    d.update(kw)
    return mx.ExpertFfnGradArgs(**d)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(rows=-1), "MOE_ERR_SHAPE", "rows = -1"),
    (dict(H=0), "MOE_ERR_SHAPE", "H = 0"),
    (dict(E=-1), "MOE_ERR_SHAPE", "E = -1"),
    (dict(save_dtype=1), "MOE_ERR_INVALID_ARG", "save_dtype"),
    (dict(dx_dtype=1), "MOE_ERR_INVALID_ARG", "dx_dtype"),
    (dict(dw_dtype=1), "MOE_ERR_INVALID_ARG", "dw_dtype"),
    (dict(accumulate=2), "MOE_ERR_INVALID_ARG", "accumulate"),
    (dict(dout_stride=60), "MOE_ERR_SHAPE", "dout_stride"),
    (dict(x_stride=0), "MOE_ERR_SHAPE", "x_stride"),
    (dict(dx_stride=66), "MOE_ERR_SHAPE", "dx_stride"),
    (dict(gather_div=0), "MOE_ERR_SHAPE", "gather_div = 0"),
    (dict(tokens=1 << 20, gather_div=1 << 12), "MOE_ERR_SHAPE", "overflows"),
    (dict(dest_row=None), "MOE_ERR_INVALID_ARG", "dest_row"),
    (dict(dout=None), "MOE_ERR_INVALID_ARG", "null"),
    (dict(gate_up=None), "MOE_ERR_INVALID_ARG", "null"),
    (dict(rows=0, expert_offsets=None), "MOE_ERR_INVALID_ARG", "null"),
    (dict(workspace_bytes=64), "MOE_ERR_WORKSPACE", "need"),
    (dict(dw1=10 * P + 8), "MOE_ERR_INVALID_ARG", "dw1 is not 16-byte"),
    (dict(dx=P), "MOE_ERR_INVALID_ARG", "dx overlaps dout"),
    (dict(dx=4 * P), "MOE_ERR_INVALID_ARG", "dx overlaps dest_row"),
    (dict(dw2=7 * P), "MOE_ERR_INVALID_ARG", "dw2 overlaps w2"),
    (dict(dw2=10 * P), "MOE_ERR_INVALID_ARG", "dw1 and dw2"),
])
def test_expert_backward_refusals(kw, status, needle):
    _refused(mx.lib.moe_expert_ffn_backward(ctypes.byref(_expert_grad(**kw)), None), status, needle)


def test_expert_workspace_queries():
    f, b = mx.lib.moe_expert_ffn_workspace_size, mx.lib.moe_expert_ffn_grad_workspace_size
    assert f(8, 64, 32, 3) >= 8 * 32 * 2 and b(8, 64, 32, 3, 0) >= 8 * 96 * 2
    assert b(8, 64, 32, 3, 1) >= b(8, 64, 32, 3, 0) + 8 * 64 * 6
    for bad in ((-1, 64, 32, 3), (8, 0, 32, 3), (8, 64, 1 << 19, 3), (8, 64, 32, 8193)):
        assert f(*bad) == 0 and b(*bad, 1) == 0
