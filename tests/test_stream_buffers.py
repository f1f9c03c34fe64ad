"""Where the binding's calls allocate, on the CPU: a call that enqueues on a given stream takes its scratch and
results from that stream's memory (a block of the current stream may still be in use there), and its results are
kept for both streams.  Streams, allocations and the library are stand-ins: nothing runs."""
import contextlib
import ctypes

import pytest
import torch

mx = pytest.importorskip("mxfp4_weight_mixture_amd", reason="libmxmoe.so is not built")

BF = torch.bfloat16


class Stream:
    def __init__(self, name, device=None):
        self.name, self.cuda_stream, self.device, self.synced = name, id(self) % 2 ** 31, torch.device("cpu"), 0

    def synchronize(self):
        self.synced += 1


class Library:
    """Size queries answer 64 bytes, everything else succeeds; which stream each call got is kept."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            if name.endswith(("_workspace_size", "_bytes")):
                return 64
            if name.endswith(("_offset", "_check")):   # (nothing enqueued)
                return 0
            self.calls.append((name, [a.value for a in args if isinstance(a, ctypes.c_void_p)]))
            return 0
        return call


class World:
    def __init__(self, patch):
        self.main, self.side = Stream("main"), Stream("side")
        self.current, self.made, self.kept = self.main, [], {}
        empty, empty_like = torch.empty, torch.empty_like

        def made(t):
            self.made.append((t, self.current))
            return t

        @contextlib.contextmanager
        def on(stream):
            before, self.current = self.current, stream
            yield
            self.current = before

        patch.setattr(torch, "empty", lambda *a, **k: made(empty(*a, **k)))
        patch.setattr(torch, "empty_like", lambda *a, **k: made(empty_like(*a, **k)))
        patch.setattr(torch.cuda, "current_stream", lambda device=None: self.current)
        patch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
        patch.setattr(torch.cuda, "synchronize", lambda device=None: None)
        patch.setattr(torch.cuda, "stream", on)
        patch.setattr(torch.cuda, "Stream", lambda device=None: Stream("new"))
        patch.setattr(torch.Tensor, "record_stream", lambda t, s: self.kept.setdefault(id(t), set()).add(s.name),
                      raising=False)
        patch.setattr(mx, "_weight", lambda name, w: None)
        patch.setattr(mx, "_on_current_device", lambda device, stream: None)
        self.lib = Library()
        patch.setattr(mx, "lib", self.lib)


@pytest.fixture
def world(monkeypatch):
    with monkeypatch.context() as m:
        yield World(m)


def z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


def _ffn():
    return mx.GatedFFN(z(64, 32), z(32, 32))


def _layer(**kw):
    u = torch.uint8
    return mx.Layer(z(4, 64, 16, dtype=u), z(4, 64, 1, dtype=u), z(4, 32, 16, dtype=u), z(4, 32, 1, dtype=u), k=2, **kw)


CALLS = {
    "route": lambda s: mx.route(z(5, 4, dtype=torch.float32), 2, stream=s),
    "permute": lambda s: mx.permute(z(5, 2, dtype=torch.int32), 4, stream=s),
    "grouped_gemm": lambda s: mx.grouped_gemm(z(5, 32), z(4, 64, 16, dtype=torch.uint8),
                                              z(4, 64, 1, dtype=torch.uint8), z(5, dtype=torch.int32), stream=s),
    "grouped_gemm to mxfp8": lambda s: mx.grouped_gemm(
        z(5, 32), z(4, 64, 16, dtype=torch.uint8), z(4, 64, 1, dtype=torch.uint8), z(5, dtype=torch.int32),
        epilogue="split", out_dtype="mxfp8", stream=s),
    "tile_weights": lambda s: mx.tile_weights(z(4, 64, 16, dtype=torch.uint8), z(4, 64, 1, dtype=torch.uint8),
                                              stream=s),
    "untile_weights": lambda s: mx.untile_weights(z(4, 64, 16, dtype=torch.uint8), z(4, 64, 1, dtype=torch.uint8),
                                                  stream=s),
    "combine": lambda s: mx.combine(z(10, 32), z(10, dtype=torch.int32), z(5, 2, dtype=torch.float32),
                                    rms_next=True, stream=s),
    "ffn": lambda s: _ffn().forward(z(5, 32), save=True, stream=s),
    "ffn backward": lambda s: _ffn().backward(z(5, 32), z(5, 32), z(5, 64), stream=s),
    "adapters": lambda s: mx.AdapterLinear(z(16, 32), z(2, 8, 32), z(2, 16, 8)).forward(
        z(5, 32), z(5, dtype=torch.int32), stream=s),
    "layer": lambda s: _layer().forward(z(5, 4, dtype=torch.float32), z(5, 32), stream=s),
    "layer with a shared expert": lambda s: _layer(shared=_ffn()).forward(z(5, 4, dtype=torch.float32), z(5, 32),
                                                                         stream=s),
    "streamed prefill": lambda s: mx.prefill_streamed(
        [z(64, dtype=torch.uint8)], [z(64, dtype=torch.uint8)], z(1, 5, 4, dtype=torch.float32), z(5, 32),
        z(5, 32, dtype=torch.float32), T=5, H=32, I=32, E=4, k=2, num_layers=1, depth=1, compute_stream=s,
        copy_stream=Stream("copy")),
}


@pytest.mark.parametrize("name", CALLS)
def test_buffers_belong_to_the_stream_that_uses_them(world, name):
    res = CALLS[name](world.side)
    res = res if isinstance(res, tuple) else (res,)
    assert world.lib.calls and all(world.side.cuda_stream in streams for _, streams in world.lib.calls)
    assert world.made and {s.name for _, s in world.made} == {"side"}
    # the caller goes on with the results on the current stream and frees them there
    assert all(world.kept.get(id(t), set()) >= {"main", "side"} for t in res)


@pytest.mark.parametrize("name", CALLS)
def test_buffers_of_calls_on_the_current_stream(world, name):
    CALLS[name](None)
    assert {s.name for _, s in world.made} == {"main"}


def test_a_layer_on_two_streams(world):
    """The kept workspace is not taken to another stream, where it may still be in use; on one stream it stays."""
    layer, logits, x = _layer(), z(5, 4, dtype=torch.float32), z(5, 32)
    seen = []
    for stream in (None, None, world.side, world.side, None):
        layer.forward(logits, x, stream=stream)
        seen.append(layer._ws)
    assert seen[0] is seen[1] and seen[2] is seen[3]
    assert len({t.data_ptr() for t in (seen[0], seen[2], seen[4])}) == 3


def test_a_captured_layer_owns_its_memory_before_it_is_replayed(world):
    """Replays may go to any stream: nothing earlier may still use the graph's buffers."""
    _layer().capture(z(5, 4, dtype=torch.float32), z(5, 32))
    assert world.main.synced


def test_a_refused_shared_expert_comes_before_any_launch(world):
    """What the library refuses of the shared expert's tensors is refused before the routed experts are enqueued,
    in a call and in a captured layer."""
    order = []

    class Refusing(Library):
        def __getattr__(self, name):
            if name == "moe_last_error_message":
                return lambda: b"refused"
            call = super().__getattr__(name)
            if name not in ("moe_gated_ffn_check", "moe_gated_ffn_forward"):
                return lambda *a: (order.append(name), call(*a))[1]
            return lambda *a: (order.append(name), mx.STATUS["MOE_ERR_SHAPE"])[1]

    mx.lib = Refusing()
    layer, logits, x = _layer(shared=_ffn()), z(5, 4, dtype=torch.float32), z(5, 32)
    with pytest.raises(mx.MoeError, match="refused"):
        layer.forward(logits, x)
    with pytest.raises(mx.MoeError, match="refused"):
        layer.capture(logits, x)
    assert "moe_layer_forward" not in order and "moe_layer_graph_create" not in order
    # nothing of the call's tensors fits: the binding's own checks come first, too
    with pytest.raises(ValueError, match="out"):
        layer.forward(logits, x, out=z(6, 32, dtype=torch.float32))
    assert "moe_layer_forward" not in order


def test_captured_calls_of_a_layer_share_no_workspace(world, monkeypatch):
    """Graphs that a caller captures keep the memory they were captured on: no two calls in captures, and none
    outside, use one workspace, whatever stream they are captured on."""
    layer, logits, x = _layer(), z(5, 4, dtype=torch.float32), z(5, 32)
    held = []
    for capturing, stream in ((False, None), (True, None), (True, None), (False, None), (True, world.side),
                              (False, world.side), (False, world.side)):
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing)
        layer.forward(logits, x, stream=stream)
        held.append(layer._ws)
    assert held[5] is held[6]
    assert len({id(t) for t in held[:6]}) == 6


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("bad", [lambda: z(5, 32), lambda: z(4, 32, dtype=torch.float32),
                                 lambda: z(5, 40, dtype=torch.float32)[:, :32],
                                 lambda: z(32, 5, dtype=torch.float32).t()])
def test_a_layer_refuses_results_it_would_not_fill(world, bad, shared):
    """The routed experts' sum is fp32, [T][H], row behind row: another type, fewer rows or rows further apart are
    refused before anything is enqueued."""
    layer, logits, x = _layer(**(dict(shared=_ffn()) if shared else {})), z(5, 4, dtype=torch.float32), z(5, 32)
    for call in (layer.forward, layer.capture):
        with pytest.raises(ValueError, match="out"):
            call(logits, x, out=bad())
    assert not world.lib.calls
    layer.forward(logits, x, out=z(5, 32, dtype=torch.float32))
    assert world.lib.calls


def _codes(*shape):
    return z(*shape, dtype=torch.uint8)


def _fp32(*shape):
    return z(*shape, dtype=torch.float32)


def _int32(*shape):
    return z(*shape, dtype=torch.int32)


# name -> (call of a stream and its inputs, the inputs)
TAKES = {
    "route": (lambda s, lg: mx.route(lg, 2, stream=s), lambda: [_fp32(5, 4)]),
    "permute": (lambda s, ids: mx.permute(ids, 4, stream=s), lambda: [_int32(5, 2)]),
    "grouped_gemm": (lambda s, a, w, ws, off, sc, ga: mx.grouped_gemm(a, w, ws, off, a_scales=sc, a_gather=ga, stream=s),
                     lambda: [_codes(5, 32), _codes(4, 64, 16), _codes(4, 64, 1), _int32(5), _codes(5, 1), _int32(5)]),
    "tile_weights": (lambda s, w, ws: mx.tile_weights(w, ws, stream=s), lambda: [_codes(4, 64, 16), _codes(4, 64, 1)]),
    "untile_weights": (lambda s, w, ws: mx.untile_weights(w, ws, stream=s),
                       lambda: [_codes(4, 64, 16), _codes(4, 64, 1)]),
    "combine": (lambda s, y, d, w: mx.combine(y, d, w, stream=s), lambda: [z(10, 32), _int32(10), _fp32(5, 2)]),
    "ffn": (lambda s, x, add: _ffn().forward(x, add=add, stream=s), lambda: [z(5, 32), z(5, 32)]),
    "ffn backward": (lambda s, d, x, gu: _ffn().backward(d, x, gu, stream=s), lambda: [z(5, 32), z(5, 32), z(5, 64)]),
    "adapters": (lambda s, x, ids, add: mx.AdapterLinear(z(16, 32), z(2, 8, 32), z(2, 16, 8)).forward(
        x, ids, add=add, stream=s), lambda: [z(5, 32), _int32(5), z(5, 16)]),
    "layer": (lambda s, lg, x, xs: _layer().forward(lg, x, xs, stream=s), lambda: [_fp32(5, 4), _codes(5, 32),
                                                                                   _codes(5, 1)]),
    "layer to x_next": (lambda s, lg, x, xn: _layer().forward(lg, x, x_next=xn, stream=s),
                        lambda: [_fp32(5, 4), z(5, 32), z(5, 32)]),
    "layer with a shared expert": (lambda s, lg, x, xs, sh: _layer(shared=_ffn()).forward(lg, x, xs, x_shared=sh, stream=s),
                                   lambda: [_fp32(5, 4), _codes(5, 32), _codes(5, 1), z(5, 32)]),
    "streamed prefill": (lambda s, slot, lg, x, out, li: mx.prefill_streamed(
        [_codes(64)], [slot], lg, x, out, T=5, H=32, I=32, E=4, k=2, num_layers=1, depth=1, layer_inputs=li,
        compute_stream=s, copy_stream=Stream("copy")),
        lambda: [_codes(64), _fp32(1, 5, 4), z(5, 32), _fp32(5, 32), z(1, 5, 32)]),
}


@pytest.mark.parametrize("name", ["ffn", "ffn backward", "adapters", "layer", "layer with a shared expert"])
def test_weights_live_as_long_as_the_streams_work(world, name, monkeypatch):
    """So may the weights, with the object that holds them."""
    made = []
    monkeypatch.setitem(globals(), "z", lambda *a, _z=z, **k: made.append(_z(*a, **k)) or made[-1])
    call, make = TAKES[name]
    call(world.side, *make())
    assert len(made) >= 4 and all("side" in world.kept.get(id(t), ()) for t in made)


@pytest.mark.parametrize("name", TAKES)
def test_inputs_live_as_long_as_the_streams_work(world, name):
    """A caller may drop its inputs at once: the allocator keeps their memory until the stream is done with them."""
    call, make = TAKES[name]
    inputs = make()
    call(world.side, *inputs)
    assert all("side" in world.kept.get(id(t), ()) for t in inputs)
    if name == "streamed prefill":   # the slots are filled, the logits read on the copy stream
        assert all("copy" in world.kept.get(id(t), ()) for t in inputs[:2])
