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


def _calls():
    """Every call that reads a plan's tables: name, and a function that makes the plan and gives (owner of the tables, call(stream))."""
    def pack(gpu, f, dtype=torch.bfloat16, out=True, **kw):
        p = _plan().upload()
        params, whole = [gpu.empty(*s, dtype=dtype) for s in SHAPES], gpu.empty(p.gathered_numel)
        return p, lambda stream: f(p, params, whole, stream=stream) if out else f(p, whole, params, stream=stream)

    def mx4(gpu, call):
        mp = fs.fs_mx4_plan(_plan()).upload()
        params, whole = [gpu.empty(*s) for s in SHAPES], gpu.empty(mp.gathered_bytes, dtype=torch.uint8)
        return mp, lambda stream: call(mp, params, whole, stream)

    def local(gpu):
        p = _plan().upload()
        pieces, shard = [gpu.empty(n) for n in p.local_numels(1)], gpu.empty(p.shard_numel)
        return p, lambda stream: p.load_local(shard, 1, pieces, stream=stream)

    def reshard(gpu):
        r = fs.fs_reshard_plan(_plan(), _plan()).upload()
        a, b = gpu.empty(r.src_info.gathered_numel), gpu.empty(r.dst_info.gathered_numel)
        return r, lambda stream: fs.fs_reshard(r, a, b, stream=stream)

    def reduce(mp, params, whole, stream):
        rows = whole.view(2, -1)
        fs.fs_reduce_shard_mx4(mp, [rows[0], rows[1]], torch.empty(mp.plan.shard_numel, device="cuda"), rank=0, stream=stream)

    return {"fs_pack": lambda g: pack(g, fs.fs_pack), "fs_pack_cast": lambda g: pack(g, fs.fs_pack_cast, torch.float32),
            "fs_unpack": lambda g: pack(g, fs.fs_unpack, out=False), "fs_load_local": local, "fs_reshard": reshard,
            "fs_pack_mx4": lambda g: mx4(g, lambda mp, ps, w, s: fs.fs_pack_mx4(mp, ps, w, stream=s)),
            "fs_unpack_mx4": lambda g: mx4(g, lambda mp, ps, w, s: fs.fs_unpack_mx4(mp, w, ps, stream=s)),
            "fs_reduce_shard_mx4": lambda g: mx4(g, reduce)}


CALLS = _calls()


@pytest.mark.parametrize("name", list(CALLS))
def test_streams_that_read_a_plans_tables_are_recorded(gpu, name):
    """Once each; a plan that goes out of scope then gives its tables back behind their work."""
    owner, call = CALLS[name](gpu)
    ws = owner.workspace

    def launched(stream, handle):
        call(stream)
        assert gpu.calls[-1][0] == name and (gpu.calls[-1][1][-1] or 0) == handle

    launched(None, 0)
    launched(Stream(0), 0)
    assert ws.recorded == []                        # the stream that they were taken on
    for _ in range(2):
        launched(Stream(70), 70)
        with gpu.on(Stream(50)):
            launched(None, 50)
    assert ws.recorded == [70, 50]
    with gpu.on(Stream(50)):
        launched(Stream(0), 0)
        launched(90, 90)                            # a bare handle may be destroyed before the plan is: the plan is to be kept
    assert ws.recorded == [70, 50]


@pytest.mark.parametrize("name", [n for n in CALLS if n not in ("fs_reshard", "fs_reduce_shard_mx4")])
def test_streams_that_read_a_pointer_table_are_recorded(gpu, name):
    """Also a table that another current stream's call has made."""
    owner, call = CALLS[name](gpu)
    plan = getattr(owner, "plan", owner)
    call(None)
    (key, held), = plan._ptr_cache.items()
    tab = held.memory
    assert tab.pool == 0 and tab.recorded == []
    for _ in range(2):
        with gpu.on(Stream(50)):
            call(None)
        call(Stream(70))
    with gpu.on(Stream(70)):
        call(Stream(0))
    assert tab.recorded == [50, 70] and not plan._pinned
    call(90)
    assert tab.recorded == [50, 70] and plan._pinned == {key}


def test_a_table_made_for_another_stream_than_the_current_one(gpu):
    """It is filled in the current stream's order, before the call goes on, and read on the call's."""
    plan = _plan().upload()
    params, whole = [gpu.empty(*s) for s in SHAPES], gpu.empty(plan.gathered_numel)
    with gpu.on(Stream(50)):
        fs.fs_pack(plan, params, whole, stream=Stream(70))
    (held,) = plan._ptr_cache.values()
    assert held.memory.pool == 50 and held.memory.recorded == [70]
    assert not plan._pinned
    gpu.capturing = True
    fs.fs_pack(plan, params, whole, stream=Stream(70))
    assert len(plan._pinned) == 1


def test_the_per_thread_stream_pins_a_table(gpu):
    """The allocator cannot tell it from another thread's."""
    plan = _plan().upload()
    params, whole = [gpu.empty(*s) for s in SHAPES], gpu.empty(plan.gathered_numel)
    with gpu.on(Stream(2)):
        fs.fs_pack(plan, params, whole)
    assert len(plan._pinned) == 1
