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
