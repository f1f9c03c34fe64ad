"""Calls on the current stream and on a side stream in flight at the same time, without a wait between them: each
gives what it gives alone, bitwise.  (Inputs are ready beforehand; scratch of equal size is freed and taken again
all the time.)"""
import pytest
import torch

from tests import dense_util as du
from tests.gpu_util import device_weights, device_x
from workloads import gen

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("mxfp4_weight_mixture_amd")
BF = torch.bfloat16


def _calls():
    """name -> call(input number, stream) of each kind, with two inputs of equal sizes."""
    T, H, I, n = 3000, 2048, 1024, 5
    f = mx.GatedFFN(du.normal((2 * I, H), H ** -0.5, BF, 1), du.normal((H, I), I ** -0.5, BF, 2))
    lin = mx.AdapterLinear(f.w1, du.normal((n, 64, H), H ** -0.5, BF, 3), du.normal((n, 2 * I, 64), 0.125, BF, 4))
    xs = [du.normal((T, H), 1.0, BF, 10 + i) for i in range(2)]
    douts = [du.normal((T, H), 1.0, BF, 20 + i) for i in range(2)]
    kept = [f.forward(x, save=True)[1] for x in xs]
    ids = [(torch.arange(T, device="cuda") * n // T).int(), (torch.arange(T, device="cuda") // 700).int()]
    s = gen.LayerShape(T=900, H=512, I=256, E=8, k=2, act="bf16", cfg_id=410, layout="split")
    li = gen.layer_inputs(s)
    w, x0 = device_weights(s), device_x(li)[0]
    shared = mx.GatedFFN(du.normal((512, 512), 512 ** -0.5, BF, 5), du.normal((512, 256), 256 ** -0.5, BF, 6))
    layer = mx.Layer(*w, k=2, layout="split", shared=shared)
    logits = [torch.from_numpy(li.logits).to("cuda"), torch.from_numpy(li.logits[::-1].copy()).to("cuda")]
    graphs = [layer.capture(lg, x0) for lg in logits]
    return {
        "ffn": lambda i, st: [f.forward(xs[i], stream=st)],
        "ffn backward": lambda i, st: list(f.backward(douts[i], xs[i], kept[i], stream=st)),
        "adapters": lambda i, st: [lin.forward(xs[i], ids[i], stream=st)],
        "route": lambda i, st: list(mx.route(logits[i], 2, stream=st)),
        "layer": lambda i, st: [layer.forward(logits[i], x0, stream=st)],
        "captured layer": lambda i, st: [graphs[i].replay(stream=st)],
    }


def _same(got, want, what):
    assert len(got) == len(want)
    assert all(torch.equal(a, b) for a, b in zip(got, want)), what


@pytest.fixture(scope="module")
def calls():
    return _calls()


@pytest.mark.parametrize("name", ["ffn", "ffn backward", "adapters", "route", "layer", "captured layer"])
def test_current_and_side_stream_in_flight(calls, name):
    call = calls[name]
    want = []
    for i in range(2):
        want.append([t.clone() for t in call(i, None)])
        torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        got = []
        for r in range(4):
            got.append((0, call(0, None)))
            got.append((1, call(1, side)))
        torch.cuda.synchronize()
        for i, g in got:
            _same(g, want[i], (name, i))


@pytest.mark.parametrize("name", ["ffn", "ffn backward", "adapters", "layer"])
def test_results_read_late_on_the_current_stream(calls, name):
    """A side stream's result is read on the current stream behind a long queue and dropped at once: the side
    stream's next call must not get its memory before it has been read."""
    call = calls[name]
    want = [[t.clone() for t in call(i, None)] for i in range(2)]
    torch.cuda.synchronize()
    a = torch.randn(4096, 4096, device="cuda")
    side, main = torch.cuda.Stream(), torch.cuda.current_stream()
    for r in range(4):
        got = call(r % 2, side)
        main.wait_stream(side)
        for _ in range(3):
            a @ a
        copies = [t.clone() for t in got]
        del got
        call(1 - r % 2, side)
        torch.cuda.synchronize()
        _same(copies, want[r % 2], (name, r))


def test_layers_in_two_captured_graphs():
    """One layer captured into two graphs, with eager calls of other sizes between: replays of both at once, and
    after a larger call has replaced the layer's workspace, give the eager results."""
    s = gen.LayerShape(T=300, H=512, I=256, E=8, k=2, act="bf16", cfg_id=411, layout="split")
    li = gen.layer_inputs(s)
    shared = mx.GatedFFN(du.normal((512, 512), 512 ** -0.5, BF, 5), du.normal((512, 256), 256 ** -0.5, BF, 6))
    layer = mx.Layer(*device_weights(s), k=2, layout="split", shared=shared)
    logits = torch.from_numpy(li.logits).to("cuda")
    x = device_x(li)[0]
    layer.forward(logits, x)
    torch.cuda.synchronize()
    runs = []
    for T in (300, 200):
        lg, xx = logits[:T].clone(), x[:T].clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = layer.forward(lg, xx)
        runs.append((g, lg, xx, out))
    side = torch.cuda.Stream()
    for k in range(4):
        for _, _, xx, _ in runs:
            xx.copy_(du.normal(tuple(xx.shape), 1.0, BF, 50 + k))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            runs[1][0].replay()
        runs[0][0].replay()
        torch.cuda.synchronize()
        for _, lg, xx, out in runs:
            assert torch.equal(layer.forward(lg, xx), out), k
        layer.forward(torch.cat([logits] * (k + 2)), torch.cat([x] * (k + 2)))
        torch.cuda.synchronize()


def test_inputs_dropped_at_once():
    """Inputs and weights made for one call on a side stream, dropped when it returns, while the current stream
    allocates and fills memory of their sizes and the side stream is far behind."""
    T, H, I = 3000, 2048, 1024
    make = lambda: (du.normal((2 * I, H), H ** -0.5, BF, 1), du.normal((H, I), I ** -0.5, BF, 2),
                    du.normal((T, H), 1.0, BF, 3), du.normal((T, H), 1.0, BF, 4))
    w1, w2, x, add = make()
    want = mx.GatedFFN(w1, w2).forward(x, add=add)
    a = torch.randn(4096, 4096, device="cuda")
    side = torch.cuda.Stream()
    for _ in range(3):
        w1, w2, x, add = make()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(5):
                a @ a
        got = mx.GatedFFN(w1, w2).forward(x, add=add, stream=side)
        sizes = [t.numel() for t in (w1, w2, x, add)]
        del w1, w2, x, add
        junk = [torch.full((n,), float("nan"), dtype=BF, device="cuda") for n in sizes]
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        del junk
