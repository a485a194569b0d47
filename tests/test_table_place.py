"""Where the tables of pointer sets lie, and how long.  Host side only (tests/fake_gpu.py)."""
import gc
import threading
import weakref

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


@pytest.mark.parametrize("name", ["fs_pack", "fs_unpack", "fs_pack_cast", "fs_pack_mx4", "fs_unpack_mx4"])
def test_a_call_holds_its_table_until_it_has_launched(gpu, monkeypatch, name):
    """Another thread's calls on the plan may release the set between its being made and the launch."""
    plan = fs.fs_plan([(8, 64)], "bf16", 2, False, "fsdp2").upload()
    mp = fs.fs_mx4_plan(plan).upload()
    dtype = torch.float32 if name == "fs_pack_cast" else torch.bfloat16
    params, whole, whole4 = [gpu.empty(8, 64, dtype=dtype)], gpu.empty(plan.gathered_numel), gpu.empty(mp.gathered_bytes, dtype=torch.uint8)
    others = [[gpu.empty(8, 64)] for _ in range(9)]
    alive = []
    real = plan.ptr_table

    def made(*args, **kw):
        tab = real(*args, **kw)
        alive.append(weakref.ref(tab))
        for o in others:
            real(o, "others")
        return tab

    def launched(*args):
        gc.collect()
        assert alive[0]() is not None and alive[0]().data_ptr() in args

    monkeypatch.setattr(plan, "ptr_table", made)
    gpu.during[name] = launched
    {"fs_pack": lambda: fs.fs_pack(plan, params, whole), "fs_unpack": lambda: fs.fs_unpack(plan, whole, params),
     "fs_pack_cast": lambda: fs.fs_pack_cast(plan, params, whole), "fs_pack_mx4": lambda: fs.fs_pack_mx4(mp, params, whole4),
     "fs_unpack_mx4": lambda: fs.fs_unpack_mx4(mp, whole4, params)}[name]()
    assert gpu.calls[-1][0] == name


@pytest.mark.parametrize("change", ["releases", "adds"])
def test_two_threads_may_release_sets_of_one_plan(gpu, change):
    """Between one thread's look at the sets and its release of one, another may release the same or add its own."""
    plan = fs.fs_plan([(8, 64)], "bf16", 2, False, "fsdp2").upload()
    sets = [[gpu.empty(8, 64)] for _ in range(9)]
    for s in sets[:8]:
        plan.ptr_table(s, "params")

    class Pinned(set):
        def __contains__(self, key):        # the other thread's turn
            if change == "releases":
                plan._ptr_cache.pop(key, None)
                return False
            if len(plan._ptr_cache) < 12:
                plan._ptr_cache[len(plan._ptr_cache)] = None
            return key == next(iter(plan._ptr_cache))

    plan._pinned = Pinned()
    assert plan.ptr_table(sets[8], "params").tolist() == [sets[8][0].data_ptr()]


def test_a_pinned_set_stays(gpu):
    """Also where another thread released it between its lookup and its being pinned."""
    plan = fs.fs_plan([(8, 64)], "bf16", 2, False, "fsdp2").upload()
    params = [gpu.empty(8, 64)]
    plan.ptr_table(params, "params")

    class Pinned(set):
        def add(self, key):
            plan._ptr_cache.pop(key)        # the other thread's turn, before the pin is there
            super().add(key)

    plan._pinned = Pinned()
    gpu.capturing = True
    tab = plan.ptr_table(params, "params")
    gpu.capturing = False
    (key, held), = plan._ptr_cache.items()
    assert held.memory is tab and key in plan._pinned


@pytest.mark.parametrize("kind", ["plan", "mx4", "reshard"])
def test_tables_stay_where_they_are(gpu, kind):
    """They do not change; a captured graph reads them at every replay, and a second upload may come in between."""
    plans = [fs.fs_plan([(8, 64)], "bf16", n, False, "fsdp2") for n in (2, 4)]
    p = {"plan": lambda: plans[0], "mx4": lambda: fs.fs_mx4_plan(plans[0]), "reshard": lambda: fs.fs_reshard_plan(*plans)}[kind]()
    ws = weakref.ref(p.upload().workspace)
    assert p.upload() is p and p.upload("cuda:0") is p
    gc.collect()
    assert ws() is p.workspace and len(gpu.calls) == 1


@pytest.mark.parametrize("kind", ["plan", "mx4", "reshard"])
def test_two_threads_may_upload_one_plan(gpu, kind):
    """The second one waits and finds the tables there; two copies at once could leave the library with the one that is dropped."""
    plans = [fs.fs_plan([(8, 64)], "bf16", n, False, "fsdp2") for n in (2, 4)]
    p = {"plan": lambda: plans[0], "mx4": lambda: fs.fs_mx4_plan(plans[0]), "reshard": lambda: fs.fs_reshard_plan(*plans)}[kind]()
    other = threading.Thread(target=p.upload)

    def copying(*args):
        if not gpu.calls[1:]:
            other.start()
            other.join(0.3)

    gpu.during[{"plan": "fs_plan_upload", "mx4": "fs_mx4_plan_upload", "reshard": "fs_reshard_upload"}[kind]] = copying
    p.upload()
    other.join()
    assert len(gpu.calls) == 1 and p.workspace.data_ptr() == gpu.calls[0][1][1]
