"""Refusals of the dense entry points, on the CPU: every check runs before any device call."""
import ctypes

import pytest
import torch

mx = pytest.importorskip("mxfp4_weight_mixture_amd", reason="libmxmoe.so is not built")

P = 1 << 20          # distinct 16-byte aligned addresses, far enough apart for the sizes below
BIG = 1 << 40


def _ffn(**kw):
    d = dict(T=4, H=64, I=32, layout=1, gate_act=0, dtype=0, out_dtype=0, save_dtype=0, x=P, w1=2 * P, w2=3 * P,
             out=4 * P, x_stride=64, out_stride=64, workspace=6 * P, workspace_bytes=P)
    d.update(kw)
    return mx.FfnArgs(**d)


def _grad(**kw):
    d = dict(T=4, H=64, I=32, layout=1, gate_act=0, dtype=0, save_dtype=2, dx_dtype=0, dw_dtype=0, dout=P, x=2 * P,
             w1=3 * P, w2=4 * P, gate_up=5 * P, dx=6 * P, dw1=7 * P, dw2=8 * P, dout_stride=64, x_stride=64,
             dx_stride=64, workspace=9 * P, workspace_bytes=P)
    d.update(kw)
    return mx.FfnGradArgs(**d)


def _adapter(**kw):
    d = dict(T=4, K=64, N=32, num_adapters=3, R=8, epilogue=0, gate_act=0, dtype=0, out_dtype=0, x=P, w=2 * P,
             ids=3 * P, a=4 * P, b=5 * P, out=6 * P, x_stride=64, out_stride=32, workspace=8 * P, workspace_bytes=P)
    d.update(kw)
    return mx.AdapterArgs(**d)


def _refused(fn, args, status, needle):
    st = fn(ctypes.byref(args) if args is not None else None, None)
    msg = mx.lib.moe_last_error_message().decode()
    assert st == mx.STATUS[status] and needle in msg, (st, msg)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(T=-1), "MOE_ERR_SHAPE", "T = -1"),
    (dict(T=(1 << 28) + 1), "MOE_ERR_SHAPE", "too many"),
    (dict(T=1 << 20, I=1 << 16, H=64), "MOE_ERR_SHAPE", "too many"),
    (dict(H=60), "MOE_ERR_SHAPE", "H = 60"),
    (dict(I=0), "MOE_ERR_SHAPE", "I = 0"),
    (dict(I=(1 << 18) + 8), "MOE_ERR_SHAPE", "I ="),
    (dict(layout=0), "MOE_ERR_INVALID_ARG", "layout"),
    (dict(gate_act=2), "MOE_ERR_INVALID_ARG", "gate_act"),
    (dict(dtype=2), "MOE_ERR_INVALID_ARG", "dtype"),
    (dict(out_dtype=1), "MOE_ERR_INVALID_ARG", "out_dtype"),
    (dict(save_dtype=1), "MOE_ERR_INVALID_ARG", "save_dtype"),
    (dict(x_stride=56), "MOE_ERR_SHAPE", "x_stride"),
    (dict(x_stride=68), "MOE_ERR_SHAPE", "x_stride"),
    (dict(out_stride=(1 << 22) + 8), "MOE_ERR_SHAPE", "out_stride"),
    (dict(add=5 * P, add_stride=0), "MOE_ERR_SHAPE", "add_stride"),
    (dict(x=None), "MOE_ERR_INVALID_ARG", "null"),
    (dict(w2=None), "MOE_ERR_INVALID_ARG", "null"),
    (dict(workspace=None), "MOE_ERR_WORKSPACE", "need"),
    (dict(workspace_bytes=16), "MOE_ERR_WORKSPACE", "need"),
    (dict(x=P + 8), "MOE_ERR_INVALID_ARG", "x is not 16-byte"),
    (dict(workspace=6 * P + 8), "MOE_ERR_INVALID_ARG", "workspace is not 16-byte"),
    (dict(out=P), "MOE_ERR_INVALID_ARG", "out overlaps x"),
    (dict(out=3 * P + 16), "MOE_ERR_INVALID_ARG", "out overlaps w2"),
    (dict(gate_up=4 * P + 16), "MOE_ERR_INVALID_ARG", "out and gate_up"),
    (dict(add=4 * P + 16, add_stride=64), "MOE_ERR_INVALID_ARG", "out overlaps add"),
    (dict(add=4 * P, add_stride=72), "MOE_ERR_INVALID_ARG", "out overlaps add"),
    (dict(workspace=2 * P), "MOE_ERR_INVALID_ARG", "workspace overlaps w1"),
])
def test_ffn_refusals(kw, status, needle):
    _refused(mx.lib.moe_gated_ffn_forward, _ffn(**kw), status, needle)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(T=-1), "MOE_ERR_SHAPE", "T = -1"),
    (dict(H=12), "MOE_ERR_SHAPE", "H = 12"),
    (dict(layout=3), "MOE_ERR_INVALID_ARG", "layout"),
    (dict(dtype=5), "MOE_ERR_INVALID_ARG", "dtype"),
    (dict(save_dtype=1), "MOE_ERR_INVALID_ARG", "save_dtype"),
    (dict(dx_dtype=1), "MOE_ERR_INVALID_ARG", "dx_dtype"),
    (dict(dw_dtype=-1), "MOE_ERR_INVALID_ARG", "dw_dtype"),
    (dict(accumulate=2), "MOE_ERR_INVALID_ARG", "accumulate"),
    (dict(dout_stride=8), "MOE_ERR_SHAPE", "dout_stride"),
    (dict(dx_stride=0), "MOE_ERR_SHAPE", "dx_stride"),
    (dict(gate_up=None), "MOE_ERR_INVALID_ARG", "null"),
    (dict(x=None), "MOE_ERR_INVALID_ARG", "null"),
    (dict(w1=None), "MOE_ERR_INVALID_ARG", "null"),
    (dict(workspace_bytes=0), "MOE_ERR_WORKSPACE", "need"),
    (dict(dw1=8 * P + 16), "MOE_ERR_INVALID_ARG", "dw1 and dw2"),
    (dict(dx=P), "MOE_ERR_INVALID_ARG", "dx overlaps dout"),
    (dict(dw2=4 * P), "MOE_ERR_INVALID_ARG", "dw2 overlaps w2"),
    (dict(dw2=8 * P + 4), "MOE_ERR_INVALID_ARG", "dw2 is not 16-byte"),
])
def test_ffn_gradient_refusals(kw, status, needle):
    _refused(mx.lib.moe_gated_ffn_backward, _grad(**kw), status, needle)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(T=-3), "MOE_ERR_SHAPE", "T = -3"),
    (dict(T=1 << 22, N=1 << 16, out_stride=1 << 16), "MOE_ERR_SHAPE", "too many"),
    (dict(K=4), "MOE_ERR_SHAPE", "K = 4"),
    (dict(N=33), "MOE_ERR_SHAPE", "N = 33"),
    (dict(N=24, epilogue=1, out_stride=14), "MOE_ERR_SHAPE", "multiple of 4"),
    (dict(num_adapters=-1), "MOE_ERR_SHAPE", "num_adapters"),
    (dict(num_adapters=65537), "MOE_ERR_SHAPE", "num_adapters"),
    (dict(R=0), "MOE_ERR_SHAPE", "R = 0"),
    (dict(R=12), "MOE_ERR_SHAPE", "R = 12"),
    (dict(R=264), "MOE_ERR_SHAPE", "R = 264"),
    (dict(epilogue=3), "MOE_ERR_INVALID_ARG", "epilogue"),
    (dict(epilogue=2, gate_act=9), "MOE_ERR_INVALID_ARG", "gate_act"),
    (dict(epilogue=1, w=None), "MOE_ERR_INVALID_ARG", "needs w"),
    (dict(dtype=2), "MOE_ERR_INVALID_ARG", "dtype"),
    (dict(out_dtype=1), "MOE_ERR_INVALID_ARG", "out_dtype"),
    (dict(x_stride=40), "MOE_ERR_SHAPE", "x_stride"),
    (dict(out_stride=24), "MOE_ERR_SHAPE", "out_stride"),
    (dict(add=7 * P, add_stride=16), "MOE_ERR_SHAPE", "add_stride"),
    (dict(ids=None), "MOE_ERR_INVALID_ARG", "null"),
    (dict(b=None), "MOE_ERR_INVALID_ARG", "null"),
    (dict(ids=3 * P + 2), "MOE_ERR_INVALID_ARG", "4-byte"),
    (dict(workspace_bytes=8), "MOE_ERR_WORKSPACE", "need"),
    (dict(a=4 * P + 8), "MOE_ERR_INVALID_ARG", "a is not 16-byte"),
    (dict(out=P), "MOE_ERR_INVALID_ARG", "out overlaps x"),
    (dict(out=3 * P), "MOE_ERR_INVALID_ARG", "out overlaps ids"),
    (dict(epilogue=1, out_stride=32, add=6 * P, add_stride=32), "MOE_ERR_INVALID_ARG", "out overlaps add"),
])
def test_adapter_refusals(kw, status, needle):
    _refused(mx.lib.moe_adapter_linear, _adapter(**kw), status, needle)


def test_null_args_and_size_queries():
    for fn in (mx.lib.moe_gated_ffn_forward, mx.lib.moe_gated_ffn_backward, mx.lib.moe_adapter_linear):
        _refused(fn, None, "MOE_ERR_INVALID_ARG", "null args")
    assert mx.lib.moe_gated_ffn_workspace_size(-1, 64, 32) == 0
    assert mx.lib.moe_gated_ffn_workspace_size(5, 64, 32) >= 5 * 32 * 2
    assert mx.lib.moe_gated_ffn_grad_workspace_size(5, 64, 32) >= 5 * 96 * 2
    assert mx.lib.moe_adapter_workspace_size(5, 64, 32, 3, 8) >= 5 * 8 * 2
    assert mx.lib.moe_adapter_workspace_size(5, 64, 32, -1, 8) == 0
    # sizes past 32 bits are not cut: a million tokens of a 28672-wide block
    assert mx.lib.moe_gated_ffn_workspace_size(1 << 20, 8192, 28672) >= (1 << 20) * 28672 * 2


@pytest.mark.parametrize("make,needle", [
    (lambda z: mx.GatedFFN(z(64, 16, dtype=torch.float32), z(16, 32)), "float32"),
    (lambda z: mx.GatedFFN(z(64, 16), z(16, 32)), "device tensor"),
    (lambda z: mx.AdapterLinear(None, z(2, 8, 16, dtype=torch.float64), z(2, 16, 8)), "float64"),
])
def test_binding_refuses_host_tensors_and_other_types(make, needle):
    with pytest.raises(ValueError, match=needle):
        make(lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype))
