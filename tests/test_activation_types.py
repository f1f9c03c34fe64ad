"""Activations of the MXFP4 products, on the CPU: bf16, or codes with their scales; the norm's fp16 or fp32 output (what
it gives beside fp16 weights, or when asked) is refused, not read as bf16."""
import pytest
import torch

from tests.test_stream_buffers import Stream, _layer, mx, world, z  # noqa: F401  (world is a fixture)

F, HF, BF, U8 = torch.float32, torch.float16, torch.bfloat16, torch.uint8


def _gemm(x, scales):
    mx.grouped_gemm(x, z(4, 64, 16, dtype=U8), z(4, 64, 1, dtype=U8), z(5, dtype=torch.int32), a_scales=scales)


def _forward(x, scales):
    _layer().forward(z(5, 4, dtype=F), x, scales)


def _capture(x, scales):
    _layer().capture(z(5, 4, dtype=F), x, scales)


def _streamed(x, scales):
    mx.prefill_streamed([z(64, dtype=U8)], [z(64, dtype=U8)], z(1, 5, 4, dtype=F), x, z(5, 32, dtype=F), T=5, H=32, I=32,
                        E=4, k=2, num_layers=1, depth=1, copy_stream=Stream("copy"))


CALLS = [_gemm, _forward, _capture, _streamed]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("dtype", [HF, F, torch.float64, U8])
def test_other_types_are_refused(world, call, dtype):  # noqa: F811
    with pytest.raises(ValueError, match="bfloat16"):
        call(z(5, 32, dtype=dtype), None)
    assert not world.lib.calls


@pytest.mark.parametrize("call", CALLS[:3])
@pytest.mark.parametrize("dtype", [BF, HF, F])
def test_values_with_scales_are_refused(world, call, dtype):  # noqa: F811
    with pytest.raises(ValueError, match="codes"):
        call(z(5, 32, dtype=dtype), z(5, 1, dtype=U8))
    assert not world.lib.calls


@pytest.mark.parametrize("call", CALLS)
def test_bf16_and_its_bits_are_taken(world, call):  # noqa: F811
    for dtype in (BF, torch.int16):
        call(z(5, 32, dtype=dtype), None)
    if call is not _streamed:
        for dtype in (U8, torch.float8_e4m3fn):
            call(z(5, 32, dtype=U8).view(dtype), z(5, 1, dtype=U8))
    assert world.lib.calls
