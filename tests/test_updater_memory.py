"""What the updater's Python objects hold on to, with stand-ins for the GPU's streams and allocator (no GPU needed)."""
import contextlib
import types
import weakref

import pytest
import torch

from gaussian_splatting_rasterizer_amd import updater


class Stream:
    def __init__(self, number):
        self.cuda_stream = number


def scratch_object():
    """An _Op whose workspaces are CPU tensors, and the set whose content says whether its stream is being captured."""
    op, capture = updater._Op.__new__(updater._Op), set()
    op.torch = types.SimpleNamespace(empty=torch.empty, uint8=torch.uint8,
                                     cuda=types.SimpleNamespace(is_current_stream_capturing=lambda: bool(capture)))
    op.device, op.workspace, op._home = torch.device("cpu"), None, None
    return op, capture


@pytest.mark.parametrize("before", [False, True], ids=["allocated in the capture", "allocated before"])
def test_captured_scratch_memory_is_kept(before):
    """A graph replays into the workspace of its capture, so a larger call afterwards must not give that memory back."""
    (op, capture), stream = scratch_object(), Stream(1)
    if before:
        op._scratch(1000, stream)
    capture.add("graph")
    captured = weakref.ref(op._scratch(1000, stream))
    capture.clear()
    op._scratch(5000, stream)
    op._scratch(9000, stream)
    assert captured() is not None and op.workspace.numel() >= 9000
    del op
    assert captured() is None


def test_other_scratch_memory_is_given_back():
    (op, capture), stream = scratch_object(), Stream(1)
    first = weakref.ref(op._scratch(1000, stream))
    op._scratch(5000, stream)
    assert first() is None and op._scratch(400, stream).numel() >= 5000
    capture.add("graph")
    captured = weakref.ref(op._scratch(400, stream))
    capture.clear()
    second = weakref.ref(op._scratch(9000, stream))
    op._scratch(20000, stream)
    assert second() is None and captured() is not None


class Recorded:
    """A tensor that notes the streams it was recorded on."""

    def __init__(self):
        self.streams = []

    def record_stream(self, stream):
        self.streams.append(stream)


def stream_object(current):
    op = updater._Op.__new__(updater._Op)
    op.device = types.SimpleNamespace(index=0)
    op.torch = types.SimpleNamespace(
        Tensor=Recorded,
        cuda=types.SimpleNamespace(current_stream=lambda device: current, current_device=lambda: 0,
                                   stream=lambda s: contextlib.nullcontext(),
                                   device=lambda d: contextlib.nullcontext()))
    return op


def test_tensors_of_another_stream_are_recorded():
    """Given a stream, the arguments' and the weights' memory must not be reused before its work is done, nor the
    results' before the current stream's."""
    here, side = Stream(1), Stream(2)
    op = stream_object(here)
    x, grad, weight, y, dx = (Recorded() for _ in range(5))
    op._held = (weight,)
    out = op._on(side, lambda stream, *a: (y, {"x": dx}), x, {"x": grad, "w": None}, True, None)
    assert out == (y, {"x": dx})
    assert all(t.streams == [side] for t in (x, grad, weight))
    assert y.streams == [here] and dx.streams == [here]


@pytest.mark.parametrize("given", [False, True])
def test_nothing_is_recorded_on_the_current_stream(given):
    here = Stream(1)
    op = stream_object(here)
    x, y = Recorded(), Recorded()
    assert op._on(here if given else None, lambda stream, *a: y, x) is y
    assert x.streams == [] and y.streams == []
