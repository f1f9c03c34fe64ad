"""What the combine takes for its rows, on the CPU: each type under its own number, everything else refused."""
import ctypes

import pytest
import torch

from tests.test_stream_buffers import mx, world, z  # noqa: F401  (world is a fixture)

F, BF, HF, I32 = torch.float32, torch.bfloat16, torch.float16, torch.int32


def _args(T=5, k=2, H=32, y=BF):
    return z(T * k, H, dtype=y), z(T * k, dtype=I32), z(T, k, dtype=F)


@pytest.mark.parametrize("dtype,name", [(F, "MOE_OUT_FP32"), (BF, "MOE_OUT_BF16"), (HF, "MOE_OUT_FP16")])
def test_each_type_of_rows_goes_by_its_own_number(world, monkeypatch, dtype, name):  # noqa: F811
    seen = []
    monkeypatch.setattr(world.lib, "moe_combine", lambda *a: seen.append(a[1]) or 0, raising=False)
    mx.combine(*_args(y=dtype))
    assert seen == [mx.OUT[name]]


@pytest.mark.parametrize("change,needle", [
    (lambda y, d, w: (y.double(), d, w), "y must"), (lambda y, d, w: (y.view(torch.int16), d, w), "y must"),
    (lambda y, d, w: (y[:9], d, w), "y must"), (lambda y, d, w: (z(32, 10).t(), d, w), "y must"),
    (lambda y, d, w: (y.view(-1), d, w), "y must"), (lambda y, d, w: (y, d.long(), w), "dest_row"),
    (lambda y, d, w: (y, d[:9], w), "dest_row"),
    (lambda y, d, w: (y, d, w.double()), "topk_w"), (lambda y, d, w: (y, d, z(2, 5, dtype=F).t()), "topk_w"),
])
def test_other_rows_are_refused(world, change, needle):  # noqa: F811
    with pytest.raises(ValueError, match=needle):
        mx.combine(*change(*_args()))
    assert not world.lib.calls


def test_the_entry_point_takes_three_types():
    """(refused for the next argument: the type passed)"""
    p = ctypes.c_void_p(16)
    for t, needle in ((0, "H = 12"), (1, "H = 12"), (3, "H = 12"), (2, "y_dtype 2"), (4, "y_dtype 4"), (-1, "y_dtype -1")):
        assert mx.lib.moe_combine(p, t, p, p, 4, 2, 12, p, None, None) != 0
        assert needle in mx.lib.moe_last_error_message().decode()
