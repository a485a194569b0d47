"""Where the tables of pointer sets lie, and how long.  Host side only (tests/fake_gpu.py)."""
import pytest
import torch

import fsdp_sharded_state_amd as fs
from fake_gpu import FakeGpu


@pytest.fixture
def gpu(monkeypatch):
    return FakeGpu(monkeypatch)


@pytest.mark.parametrize("shapes", [[(0,), (8, 64)], [(0, 3), (0,), (5,), (0,)]])
def test_a_parameter_without_elements_may_lie_anywhere(gpu, shapes):
    """Nothing is read of it, and the table of the others goes to their GPU all the same."""
    plan = fs.fs_plan(shapes, "bf16", 2, False, "fsdp2").upload()
    params = [gpu.empty(*s) if 0 not in s else torch.zeros(s, dtype=torch.bfloat16) for s in shapes]
    fs.fs_pack(plan, params, gpu.empty(plan.gathered_numel))
    tab = plan.ptr_table(params, "params")
    assert tab.is_cuda and tab.tolist() == [p.data_ptr() if p.numel() else 0 for p in params]
    assert gpu.calls[-1][0] == "fs_pack" and gpu.calls[-1][1][1] == tab.data_ptr()
