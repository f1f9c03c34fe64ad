"""A call with a shared expert that is refused has enqueued nothing: `out` keeps its values, and a captured layer
with one allocates nothing when it is replayed."""
import pytest
import torch

from tests import dense_util as du
from tests.gpu_util import device_weights
from workloads import gen

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("mxfp4_weight_mixture_amd")
BF, F = torch.bfloat16, torch.float32


def _layer(T=24, H=256):
    s = gen.LayerShape(T=T, H=H, I=128, E=8, k=2, act="bf16", layout="split", cfg_id=420)
    li = gen.layer_inputs(s)
    ffn = mx.GatedFFN(du.normal((384, H), H ** -0.5, BF, 1), du.normal((H, 192), 192 ** -0.5, BF, 2))
    return mx.Layer(*device_weights(s), k=2, layout="split", shared=ffn), torch.from_numpy(li.logits).to("cuda"), \
        li.x_bf16.to("cuda")


def test_refused_calls_leave_out_alone():
    layer, logits, x = _layer()
    T, H = x.shape
    flat = torch.zeros(2 * T * (H + 8), dtype=BF, device="cuda")
    out = torch.full((T, H), 7.0, device="cuda")
    rows = lambda start, stride: flat[start: start + (T - 1) * stride + H].as_strided((T, H), (stride, 1),
                                                                                       start)
    for bad, needle in ((rows(0, H + 4), "multiple of 8"), (rows(4, H), "16-byte"), (rows(0, 0), "x_stride"),
                        (out.view(BF)[:, :H], "overlaps")):
        for call in (layer.forward, layer.capture):
            with pytest.raises(mx.MoeError, match=needle):
                call(logits, x, out=out, x_shared=bad)
    for bad, needle in ((torch.zeros(T + 1, H, device="cuda"), "out has shape"), (out.half(), "float16")):
        for call in (layer.forward, layer.capture):
            with pytest.raises(ValueError, match=needle):
                call(logits, x, out=bad)
    torch.cuda.synchronize()
    assert (out == 7.0).all()
    want = layer.forward(logits, x)
    assert torch.equal(layer.forward(logits, x, out=out), want) and (out != 7.0).any()


def test_replays_allocate_nothing_and_equal_calls():
    layer, logits, x = _layer(T=90)
    g = layer.capture(logits, x)
    count = lambda: torch.cuda.memory_stats()["allocation.all.allocated"]
    before = count()
    got = g.replay()
    assert count() == before
    side = torch.cuda.Stream()
    for k in range(3):
        x.copy_(du.normal(tuple(x.shape), 1.0, BF, 30 + k))
        want = layer.forward(logits, x)
        side.wait_stream(torch.cuda.current_stream())
        g.replay(stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, want), k
    g.close()
