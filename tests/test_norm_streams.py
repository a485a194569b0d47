"""A stream that the calls with a workspace refuse (no GPU call is made)."""
import pytest
import torch

import fsdp_sharded_state_amd as fs


@pytest.mark.parametrize("scratch", [0, 64])
def test_the_per_thread_stream_is_refused(monkeypatch, scratch):
    """hipStreamPerThread (handle 2) is another stream in every host thread,
    but one to the allocator: two threads would get the same workspace."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 2, raising=False)

    def launched(*args):
        raise AssertionError("the call was launched")

    for stream in (2, None):      # given by its handle, and as the current stream
        with pytest.raises(ValueError, match="per-thread"):
            fs._launch(0, stream, launched, scratch=scratch)
