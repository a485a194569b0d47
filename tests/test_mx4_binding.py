"""What the binding of the 4-bit calls says and hands on.  Host side only (tests/fake_gpu.py)."""
import pytest
import torch

import fsdp_sharded_state_amd as fs
from fake_gpu import FakeGpu


@pytest.fixture
def gpu(monkeypatch):
    return FakeGpu(monkeypatch)


def test_a_seed_on_another_gpu_is_named_by_what_it_is(gpu):
    """A quantisation has no gradients."""
    with pytest.raises(ValueError, match="^seed is on cuda:0, the other arguments on cuda:1$"):
        fs._scalar_ptr(torch.empty(1, dtype=torch.int64, device="cuda"), torch.int64, 1, "seed")
