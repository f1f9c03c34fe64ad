"""Logits and expert ids on the CPU: contiguous fp32 and int32, or refused (logits in 16 bits, a product of 16-bit
activations, would be read past their end)."""
import pytest
import torch

from tests.test_stream_buffers import Stream, _layer, mx, world, z  # noqa: F401  (world is a fixture)

F, HF, BF, U8, I32 = torch.float32, torch.float16, torch.bfloat16, torch.uint8, torch.int32


def _streamed(logits):
    mx.prefill_streamed([z(64, dtype=U8)], [z(64, dtype=U8)], logits, z(5, 32), z(5, 32, dtype=F), T=5, H=32, I=32, E=4,
                        k=2, num_layers=1, depth=1, copy_stream=Stream("copy"))


CALLS = {"route": lambda t: mx.route(t, 2), "layer": lambda t: _layer().forward(t, z(5, 32)),
         "captured layer": lambda t: _layer().capture(t, z(5, 32)), "streamed prefill": _streamed}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("logits", [z(5, 4), z(5, 4, dtype=HF), z(5, 4, dtype=torch.float64), z(4, 5, dtype=F).t(),
                                    z(5, 8, dtype=F)[:, :4]], ids=["bf16", "fp16", "fp64", "turned", "columns"])
def test_other_logits_are_refused(world, name, logits):  # noqa: F811
    with pytest.raises(ValueError, match="logits"):
        CALLS[name](logits)
    assert not world.lib.calls


@pytest.mark.parametrize("name", CALLS)
def test_fp32_logits_are_taken(world, name):  # noqa: F811
    CALLS[name](z(5, 4, dtype=F))
    assert world.lib.calls


@pytest.mark.parametrize("ids", [z(5, 2, dtype=torch.int64), z(2, 5, dtype=I32).t(), z(5, 2, dtype=F)])
def test_other_ids_are_refused(world, ids):  # noqa: F811
    with pytest.raises(ValueError, match="topk_ids"):
        mx.permute(ids, 4)
    assert not world.lib.calls
