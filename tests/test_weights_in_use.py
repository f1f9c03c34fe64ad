"""Weights whose memory is another one than when their object was made (an optimizer or a move gave the tensor new
storage, or the attribute a new tensor), on the CPU: a call reads them where they are now."""
import pytest
import torch

from tests.test_stream_buffers import mx, world, z  # noqa: F401  (world is a fixture)
from tests.test_train_stream_buffers import dev

F, I32 = torch.float32, torch.int32


def _experts():
    f = mx.ExpertFFN(z(3, 64, 32), z(3, 32, 32))
    off, how = z(4, dtype=I32), dict(gather=z(10, dtype=I32), gather_div=2)
    return f, ("w1", "w2"), {
        "moe_expert_ffn_forward": lambda: f.forward(z(5, 32), off, **how),
        "moe_expert_ffn_backward": lambda: f.backward(z(10, 32), z(5, 32), off, z(10, 64), dest_row=z(10, dtype=I32), **how)}


def _ffn():
    f = mx.GatedFFN(z(64, 32), z(32, 32))
    return f, ("w1", "w2"), {"moe_gated_ffn_forward": lambda: f.forward(z(5, 32)),
                             "moe_gated_ffn_backward": lambda: f.backward(z(5, 32), z(5, 32), z(5, 64))}


def _norm():
    f = mx.RMSNorm(dev(z(32)))
    return f, ("weight",), {"moe_rms_norm_forward": lambda: f.forward(z(5, 32), z(5, 32)),
                            "moe_rms_norm_backward": lambda: f.backward(z(5, 32), z(5, 32))}


@pytest.mark.parametrize("make", [_experts, _ffn, _norm])
@pytest.mark.parametrize("replace", ["storage", "attribute"])
def test_calls_read_the_weights_where_they_are(world, monkeypatch, make, replace):  # noqa: F811
    f, names, calls = make()
    kept = [getattr(f, n) for n in names]     # (so that the old memory is not given out again)
    old = [t.data_ptr() for t in kept]
    for n in names:
        t = getattr(f, n)
        new = t.clone()
        if replace == "attribute":
            setattr(f, n, new)
        else:
            before = t.data
            kept.append(before)
            t.data = new
    for entry, call in calls.items():
        seen = []
        monkeypatch.setattr(world.lib, entry, lambda ref, s: seen.extend(getattr(ref._obj, n) for n in names) or 0,
                            raising=False)
        call()
        assert seen == [getattr(f, n).data_ptr() for n in names], entry
        assert not set(seen) & set(old), entry
