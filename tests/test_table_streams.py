"""The streams of the tables that kernels read in device memory: the plans'
and the pointer sets'.  Host side only (tests/fake_gpu.py): no kernel runs.

The allocator hands memory out again in the order of the stream it was taken
on.  So a table has to be filled in that order, and every other stream that
reads it has to be recorded, or the memory may be written to while it is read."""
import pytest
import torch

import fsdp_sharded_state_amd as fs
from fake_gpu import FakeGpu, Stream

SHAPES = [(8, 64), (33,)]


@pytest.fixture
def gpu(monkeypatch):
    return FakeGpu(monkeypatch)


def _plan():
    return fs.fs_plan(SHAPES, "bf16", 2, False, "fsdp2")


PLANS = {"plan": _plan, "mx4": lambda: fs.fs_mx4_plan(_plan()), "reshard": lambda: fs.fs_reshard_plan(_plan(), _plan())}


@pytest.mark.parametrize("kind", list(PLANS))
@pytest.mark.parametrize("stream,current", [(Stream(70), 0), (None, 50), (None, 0), (70, 0), (Stream(0), 50), (0, 50)])
def test_tables_are_copied_on_the_stream_whose_memory_they_take(gpu, kind, stream, current):
    """Memory of another stream may still be written to by what that stream has under way."""
    p = PLANS[kind]()
    with gpu.on(Stream(current)):
        p.upload(stream=stream)
    (name, args), = gpu.calls
    want = current if stream is None else getattr(stream, "cuda_stream", stream)
    assert name.endswith("upload") and args[1] == p.workspace.data_ptr()
    assert (args[3] or 0) == want and p.workspace.pool == want


@pytest.mark.parametrize("kind", list(PLANS))
@pytest.mark.parametrize("stream,current", [(2, 0), (None, 2)])
def test_tables_are_not_copied_on_the_per_thread_stream(gpu, kind, stream, current):
    """It is another stream in every host thread, but one to the allocator; the copy is waited for anyway."""
    p = PLANS[kind]()
    with gpu.on(Stream(current)):
        p.upload(stream=stream)
    (_, args), = gpu.calls
    assert (args[3] or 0) == 0 and p.workspace.pool == 0
