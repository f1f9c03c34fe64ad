"""Where the calls of the norm, the router's gradients and the experts with 16-bit weights allocate, on the CPU, with
the stand-ins of test_stream_buffers: scratch and results on the stream of the call, inputs, weights and results kept
for both streams, however soon the caller drops them."""
import pytest
import torch

from tests.test_stream_buffers import BF, mx, world, z  # noqa: F401  (world is a fixture)

F, I32 = torch.float32, torch.int32


class _Tensor(torch.Tensor):
    is_cuda = True
    __torch_function__ = torch._C._disabled_torch_function_impl


def dev(t):
    """A tensor that the binding takes for a device tensor."""
    return t.as_subclass(_Tensor)


def _experts():
    return mx.ExpertFFN(z(3, 64, 32), z(3, 32, 32))


CALLS = {
    "norm": (lambda s, w, x, r: tuple(mx.RMSNorm(w).forward(x, r, mxfp8=True, stream=s)), lambda: [dev(z(32)), z(5, 32), z(5, 32)]),
    "norm backward": (lambda s, w, d, x, r: mx.RMSNorm(w).backward(d, x, dresidual=r, stream=s),
                      lambda: [dev(z(32)), z(5, 32), z(5, 32), z(5, 32)]),
    "combine backward": (lambda s, d, y, dest, w: mx.combine_backward(d, y, dest, w, stream=s),
                         lambda: [z(5, 32, dtype=F), z(10, 32), z(10, dtype=I32), z(5, 2, dtype=F)]),
    "route backward": (lambda s, d, ids, w: mx.route_backward(d, ids, w, 4, stream=s),
                       lambda: [z(5, 2, dtype=F), z(5, 2, dtype=I32), z(5, 2, dtype=F)]),
    "experts": (lambda s, x, off, src: _experts().forward(x, off, gather=src, gather_div=2, save=True, stream=s),
                lambda: [z(5, 32), z(4, dtype=I32), z(10, dtype=I32)]),
    "experts backward": (lambda s, d, x, off, gu, src, dest: _experts().backward(
        d, x, off, gu, gather=src, gather_div=2, dest_row=dest, stream=s),
        lambda: [z(10, 32), z(5, 32), z(4, dtype=I32), z(10, 64), z(10, dtype=I32), z(10, dtype=I32)]),
}


@pytest.mark.parametrize("name", CALLS)
def test_buffers_belong_to_the_stream_that_uses_them(world, name):  # noqa: F811
    call, make = CALLS[name]
    inputs = make()
    res = call(world.side, *inputs)
    res = res if isinstance(res, tuple) else (res,)
    assert world.lib.calls and all(world.side.cuda_stream in streams for _, streams in world.lib.calls)
    assert world.made and {s.name for _, s in world.made} == {"side"}
    assert all(world.kept.get(id(t), set()) >= {"main", "side"} for t in res if t is not None)


@pytest.mark.parametrize("name", CALLS)
def test_buffers_of_calls_on_the_current_stream(world, name):  # noqa: F811
    call, make = CALLS[name]
    call(None, *make())
    assert {s.name for _, s in world.made} == {"main"}


@pytest.mark.parametrize("name", CALLS)
def test_inputs_live_as_long_as_the_streams_work(world, name):  # noqa: F811
    call, make = CALLS[name]
    inputs = make()
    call(world.side, *inputs)
    assert all("side" in world.kept.get(id(t), ()) for t in inputs)


@pytest.mark.parametrize("name", ["experts", "experts backward"])
def test_weights_live_as_long_as_the_streams_work(world, name, monkeypatch):  # noqa: F811
    made = []
    monkeypatch.setitem(globals(), "z", lambda *a, _z=z, **k: made.append(_z(*a, **k)) or made[-1])
    call, make = CALLS[name]
    call(world.side, *make())
    assert len(made) >= 5 and all("side" in world.kept.get(id(t), ()) for t in made)
