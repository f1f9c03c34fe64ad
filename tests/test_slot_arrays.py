"""dest_row as [T*k] or [T][k], on the CPU: taken as it lies in memory, or copied on the stream of the call (which does
not wait for the current one)."""
import pytest
import torch

from tests.test_stream_buffers import mx, world, z  # noqa: F401  (world is a fixture)

F, I32 = torch.float32, torch.int32


def _combine_backward(s, dest):
    mx.combine_backward(z(5, 32, dtype=F), z(10, 32), dest, z(5, 2, dtype=F), stream=s)


def _combine(s, dest):
    mx.combine(z(10, 32), dest, z(5, 2, dtype=F), stream=s)


def _experts_backward(s, dest):
    f = mx.ExpertFFN(z(3, 64, 32), z(3, 32, 32))
    f.backward(z(10, 32), z(5, 32), z(4, dtype=I32), z(10, 64), gather=z(10, dtype=I32), gather_div=2, dest_row=dest,
               stream=s)


CALLS = [_combine, _combine_backward, _experts_backward]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("side", [True, False])
def test_contiguous_rows_are_taken_as_they_lie(world, monkeypatch, call, side):  # noqa: F811
    seen = []

    def entry(*args):
        seen.append([a.value for a in args if hasattr(a, "value")] + [getattr(getattr(a, "_obj", None), "dest_row", None)
                                                                      for a in args])
        return 0

    for name in ("moe_combine", "moe_combine_backward", "moe_expert_ffn_backward"):
        monkeypatch.setattr(world.lib, name, entry, raising=False)
    for dest in (z(10, dtype=I32), z(5, 2, dtype=I32)):
        call(world.side if side else None, dest)
        assert dest.data_ptr() in seen[-1]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("side", [True, False])
@pytest.mark.parametrize("dest", [torch.arange(10, dtype=I32).view(2, 5).t(), torch.arange(20, dtype=I32).view(5, 4)[:, ::2],
                                  torch.arange(20, dtype=I32)[::2]], ids=["t", "columns", "steps"])
def test_rows_that_are_not_contiguous_are_copied_on_the_calls_stream(world, monkeypatch, call, side, dest):  # noqa: F811
    copies, contiguous, reshape = [], torch.Tensor.contiguous, torch.Tensor.reshape

    def seen(f):
        def copy(t, *a):
            r = f(t, *a)
            if r.data_ptr() != t.data_ptr():
                copies.append((world.current.name, r.flatten().tolist()))
            return r
        return copy

    monkeypatch.setattr(torch.Tensor, "contiguous", seen(contiguous))
    monkeypatch.setattr(torch.Tensor, "reshape", seen(reshape))
    call(world.side if side else None, dest)
    assert copies == [("side" if side else "main", [x for r in dest.tolist() for x in (r if isinstance(r, list) else [r])])]
    assert world.lib.calls
    if side:
        assert "side" in world.kept[id(dest)]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("dest", [z(9, dtype=I32), z(5, 2, dtype=torch.int64), z(5, 2, 1, dtype=I32)])
def test_other_rows_are_refused(world, call, dest):  # noqa: F811
    with pytest.raises(ValueError, match="dest_row must"):
        call(None, dest)
    assert not world.lib.calls
