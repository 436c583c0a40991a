"""What the updater's Python objects hold on to, with stand-ins for the GPU's streams and allocator (no GPU needed)."""
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
