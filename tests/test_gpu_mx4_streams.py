"""The 4-bit calls' plans on several streams, and uploads between captures."""
import threading

import pytest
import torch

import fsdp_sharded_state_amd as fs
from gpu_util import say

pytestmark = pytest.mark.gpu

SHAPES, WORLD = [(64,), (96, 64), (64, 96), (96,)], 4


def _group(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    params = [torch.randn(s, generator=g, device="cuda").bfloat16() for s in SHAPES]
    plan = fs.fs_plan(SHAPES, "bf16", WORLD, False, "fsdp2", 2)
    return params, plan, fs.fs_mx4_plan(plan).upload()


def _step(mp, params, gathered, outs, g32, stream=None):
    fs.fs_pack_mx4(mp, params, gathered, stream=stream)
    fs.fs_unpack_mx4(mp, gathered, outs, stream=stream)
    fs.fs_reduce_shard_mx4(mp, [gathered[:mp.shard_bytes]] * (2 * WORLD), g32, rank=1, grad_acc=2, stream=stream)


def _buffers(mp, params):
    return torch.empty(mp.gathered_bytes, dtype=torch.uint8, device="cuda"), [torch.empty_like(p) for p in params], torch.empty(mp.plan.shard_numel, device="cuda")


@pytest.mark.parametrize("kind", ["given", "current", "handle"])
def test_a_plan_on_another_stream_than_its_upload(kind):
    """The results are the ones of the stream that it was uploaded on; the tables are recorded on the other, where a torch
    stream is given or current."""
    params, plan, mp = _group(1)
    here, there = _buffers(mp, params), _buffers(mp, params)
    s = torch.cuda.Stream()
    for stream, b in ((torch.cuda.current_stream(), here), (s, there)):
        torch.cuda.synchronize()
        say("stream", kind, stream)
        if kind == "current":
            with torch.cuda.stream(stream):
                _step(mp, params, *b)
        else:
            _step(mp, params, *b, stream=stream if kind == "given" else stream.cuda_stream)
        torch.cuda.synchronize()
    assert torch.equal(here[0], there[0]) and torch.equal(here[2], there[2]) and all(map(torch.equal, here[1], there[1]))
    if kind != "handle":
        assert s.cuda_stream in mp._table.known
        # the parameters' table and that of the outputs there; the outputs here have one of their own
        assert sum(s.cuda_stream in t.known for t in plan._ptr_cache.values()) == 2 and not plan._pinned
    else:
        assert s.cuda_stream not in mp._table.known and len(plan._pinned) == len(plan._ptr_cache) == 3


def test_tables_uploaded_and_read_on_a_side_stream():
    params, plan, mp = _group(2)
    want = _buffers(mp, params)
    _step(mp, params, *want, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    say("upload on a side stream")
    side = fs.fs_mx4_plan(fs.fs_plan(SHAPES, "bf16", WORLD, False, "fsdp2", 2)).upload(stream=s)
    got = _buffers(mp, params)
    _step(side, params, *got, stream=s)
    del side
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2]) and all(map(torch.equal, got[1], want[1]))


def test_a_captured_graph_reads_the_tables_it_was_captured_with():
    """A later upload takes another workspace: what was captured before it goes on reading the earlier one, what comes
    after reads the later.  Both graphs, replayed in turn and side by side, give the eager results."""
    params, plan, mp = _group(3)
    sets = [_buffers(mp, params) for _ in range(2)]

    def step(b):
        _step(mp, params, *b)

    def state(b):
        return [t.clone() for t in (b[0], *b[1], b[2])]

    for b in sets:
        step(b)
    torch.cuda.synchronize()
    want, graphs, later = [state(b) for b in sets], [], []
    for k, b in enumerate(sets):
        say("capture", k)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(b)
        graphs.append(graph)
        later.append(torch.zeros(mp.workspace_bytes, dtype=torch.uint8, device="cuda"))
        rc = fs.lib().fs_mx4_plan_upload(mp._h, later[-1].data_ptr(), later[-1].numel(), torch.cuda.current_stream().cuda_stream)
        assert rc == 0
    streams = [torch.cuda.Stream() for _ in graphs]
    for turn in range(4):
        for b in sets:
            for t in (b[0], *b[1], b[2]):
                t.zero_()
        torch.cuda.synchronize()
        say("replay", turn)
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for k, b in enumerate(sets):
            assert all(map(torch.equal, state(b), want[k])), f"turn {turn}, graph {k}"
        step(sets[0])                       # eager, from the last upload's tables
        torch.cuda.synchronize()
        assert all(map(torch.equal, state(sets[0]), want[0]))


def test_a_captured_dequantisation_replays_with_new_values():
    """Of a matrix and of a gathered weight in chunks, into bf16 and fp32."""
    params, plan, mp = _group(4)
    gathered = torch.empty(mp.gathered_bytes, dtype=torch.uint8, device="cuda")
    fs.fs_pack_mx4(mp, params, gathered)
    q, w = fs.fs_mx4_empty(77, 130), mp.matrix(gathered, 1)
    x = torch.randn(77, 130, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda")
    fs.fs_mx4_quantize(x, q)
    outs = [torch.empty(s, dtype=t, device="cuda") for t in (torch.bfloat16, torch.float32) for s in (q.shape, w.shape)]

    def step():
        for k, o in enumerate(outs):
            fs.fs_mx4_dequantize(w if k % 2 else q, o)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for turn in range(4):
        fs.fs_mx4_quantize(x * (turn + 2), q)
        fs.fs_pack_mx4(mp, [p * (turn + 2) for p in params], gathered)
        for o in outs:
            o.zero_()
        say("replay", turn)
        graph.replay()
        got = [o.clone() for o in outs]
        torch.cuda.synchronize()
        step()
        assert all(map(torch.equal, got, outs)) and all((o != 0).any() for o in outs), f"turn {turn}"


def test_threads_on_one_plan():
    """Each on a stream of its own and with more sets of parameters than the plan keeps tables of, some shared with the
    other threads: every result is the single-threaded one."""
    _, plan, mp = _group(6)
    sets = [[torch.randn(s, generator=torch.Generator(device="cuda").manual_seed(10 * k + i), device="cuda").bfloat16()
             for i, s in enumerate(SHAPES)] for k in range(14)]
    want = []
    for params in sets:
        b = _buffers(mp, params)
        fs.fs_pack_mx4(mp, params, b[0])
        fs.fs_unpack_mx4(mp, b[0], b[1])
        want.append((b[0], b[1]))
    torch.cuda.synchronize()
    errors = []

    def run(k):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for turn in range(6):
                    got = []
                    for j in [*range(3 * k, 3 * k + 3), 12, 13]:        # 12 and 13 are everyone's
                        b = _buffers(mp, sets[j])
                        fs.fs_pack_mx4(mp, sets[j], b[0], stream=stream if turn % 2 else None)
                        fs.fs_unpack_mx4(mp, b[0], b[1], stream=stream if turn % 2 else None)
                        got.append((j, b))
                    stream.synchronize()
                    for j, b in got:
                        assert torch.equal(b[0], want[j][0]) and all(map(torch.equal, b[1], want[j][1])), f"thread {k}, turn {turn}, set {j}"
        except Exception as e:     # noqa: BLE001
            errors.append(e)

    say("four threads on one plan")
    threads = [threading.Thread(target=run, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
