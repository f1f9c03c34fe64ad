"""Sizes past what one launch can count (2^32 threads) are refused, on the CPU: such a launch would not run, without an
error.  (The calls that are to pass the size check are refused for a later argument.)"""
import ctypes

import pytest

mx = pytest.importorskip("mxfp4_weight_mixture_amd", reason="libmxmoe.so is not built")

P = ctypes.c_void_p(1 << 20)


def _refusal(st):
    assert st != 0
    return mx.lib.moe_last_error_message().decode()


@pytest.mark.parametrize("call", [lambda T, E: mx.lib.moe_route(P, T, E, 2, P, P, None),
                                  lambda T, E: mx.lib.moe_route_backward(P, P, P, T, E, 2, P, None)])
def test_routing(call):
    """four tokens a block of 256 threads"""
    for T in ((1 << 26) - 3, (1 << 26) - 1, 1 << 26, 2 ** 31 - 1):
        assert f"T = {T}" in _refusal(call(T, 8))
    assert "E = 1025" in _refusal(call((1 << 26) - 4, 1025))


@pytest.mark.parametrize("y_dtype,H,most", [(1, 8192, (1 << 22) - 1), (3, 8192, (1 << 22) - 1), (0, 4096, (1 << 23) - 1),
                                            (1, 512, (1 << 26) - 1), (0, 8, (1 << 26) - 1)])
def test_combine(y_dtype, H, most):
    """a block of up to 1024 threads a token, 512 for fp32 rows"""
    call = lambda T, y: mx.lib.moe_combine(y, y_dtype, P, P, T, 2, H, P, None, None)
    for T in (most + 1, 2 ** 31 - 1):
        assert f"T = {T}" in _refusal(call(T, P))
    assert "null" in _refusal(call(most, None))


def _expert_grad(**kw):
    p = 1 << 20
    d = dict(rows=8, H=64, I=32, E=3, layout=1, gate_act=0, dtype=0, save_dtype=2, dx_dtype=0, dw_dtype=0, accumulate=0,
             tokens=1 << 22, gather_div=2, dout=p, x=2 * p, gather=3 * p, dest_row=4 * p, expert_offsets=5 * p, w1=6 * p,
             w2=7 * p, gate_up=8 * p, dx=9 * p, dw1=10 * p, dw2=11 * p, dout_stride=64, x_stride=64, dx_stride=64,
             workspace=12 * p, workspace_bytes=64)
    d.update(kw)
    return _refusal(mx.lib.moe_expert_ffn_backward(ctypes.byref(mx.ExpertFfnGradArgs(**d)), None))


@pytest.mark.parametrize("kw,needle", [
    # what forward takes, backward takes: as many tokens as x may have, and any number without dx
    (dict(), "workspace 64 bytes"), (dict(tokens=(1 << 24) - 1), "workspace 64 bytes"),
    (dict(tokens=1 << 27, x_stride=8, H=8, dx_stride=8, dout_stride=8, dw1=None), "workspace 64 bytes"),
    (dict(dx=None, dest_row=None), "workspace 64 bytes"),
    (dict(tokens=1 << 22, gather_div=1 << 10, dx=None, dest_row=None), "workspace 64 bytes"),
    (dict(tokens=1 << 22, gather_div=1 << 9), "overflows"), (dict(tokens=1 << 24), "2^30"),
])
def test_tokens_of_the_experts_backward(kw, needle):
    assert needle in _expert_grad(**kw)
