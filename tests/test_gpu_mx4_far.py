"""The 4-bit calls on more than 2^31 elements and past 2^32 bytes, and with
random bits whose counter passes 2^32: windows at the start, where an
index passes a power of two, and at the end, bit for bit against the 64-bit definitions
(tests/mx4_ref.py)."""
import numpy as np
import pytest
import torch

import fsdp_sharded_state_amd as fs
import mx4_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _room(gigabytes):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gigabytes << 30:
        pytest.skip(f"needs {gigabytes} GiB of free GPU memory")


@pytest.fixture(autouse=True)
def _give_back():
    yield
    torch.cuda.empty_cache()


def _filled(shape, dtype, seed):
    """Normals, the same 64M again and again (an odd count, so that no two rows begin alike)."""
    base = torch.randn((1 << 26) + 37, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)
    x = torch.empty(shape, dtype=dtype, device="cuda")
    flat, n = x.view(-1), base.numel()
    whole = flat.numel() // n
    flat[:whole * n].view(whole, n).copy_(base.expand(whole, n))
    flat[whole * n:].copy_(base[:flat.numel() - whole * n])
    return x


def _f64(t):
    return t.float().cpu().double().numpy()


def _seed(v):
    return None if v is None else torch.tensor([v], dtype=torch.int64, device="cuda")


def _check_row(q, x_row, r, seed, orientation):
    """Row r of a quantised matrix against its elements, as float64."""
    nb = ref.blocks(x_row.size)
    full = np.zeros(nb * 32)
    full[:x_row.size] = x_row
    c, s = ref.encode(full.reshape(nb, 32), seed, r * nb + np.arange(nb), orientation)
    assert np.array_equal(q.codes[r].cpu().numpy(), c.reshape(-1)) and np.array_equal(q.scales[r].cpu().numpy(), s), f"row {r}"
    return ref.decode(c, s[:, None]).reshape(-1)[:x_row.size]


@pytest.mark.parametrize("dtype,seed", [("bf16", None), ("bf16", -3), ("fp32", 8)])
def test_quantize_rows_and_back(dtype, seed):
    rows, cols = 70000, 33000                   # 2.3e9 elements: 31 bits of them end in row 65075
    _room(24)
    x, q = _filled((rows, cols), DT[dtype], 1), fs.fs_mx4_empty(rows, cols)
    say("rows", dtype, seed)
    fs.fs_mx4_quantize(x, q, seed=_seed(seed))
    checked = {r: _check_row(q, _f64(x[r]), r, None if seed is None else seed % 2 ** 64, 0) for r in (0, 32538, 65075, 65076, rows - 1)}
    say("back", dtype, seed)
    fs.fs_mx4_dequantize(q, x)
    for r, want in checked.items():
        assert np.array_equal(_f64(x[r]), want), f"row {r}"


def test_quantize_both_ways_past_32_bits_of_the_counter():
    rows, cols = 32771, (1 << 20) + 33          # 1.07e9 blocks either way: four groups of random bits each
    _room(120)
    x, by_row, by_col = _filled((rows, cols), torch.bfloat16, 2), fs.fs_mx4_empty(rows, cols), fs.fs_mx4_empty(cols, rows)
    assert 4 * rows * ref.blocks(cols) > 2 ** 32 and 4 * cols * ref.blocks(rows) > 2 ** 32
    say("both ways")
    fs.fs_mx4_quantize(x, by_row, by_col, seed=_seed(77))
    for r in (0, rows // 2, rows - 1):
        _check_row(by_row, _f64(x[r]), r, 77, 0)
    for c in (0, 1, cols // 2, 1047553, cols - 2, cols - 1):        # the counter passes 2^32 in column 1047553
        _check_row(by_col, _f64(x[:, c]), c, 77, 1)


def test_copy_in_and_out():
    shapes, world = [((1 << 35) + (1 << 20) + 77,), (1001,)], 4
    _room(170)
    plan = fs.fs_plan(shapes, "bf16", world, True, "fsdp1")
    mp = fs.fs_mx4_plan(plan).upload()
    params = [_filled(s, torch.bfloat16, 3 + i) for i, s in enumerate(shapes)]
    gathered = torch.empty(mp.gathered_bytes, dtype=torch.uint8, device="cuda")
    assert 4 * mp.shard_blocks * world > 2 ** 32 and mp.shard_bytes > 2 ** 32
    say("copy-in")
    fs.fs_pack_mx4(mp, params, gathered, seed=_seed(9))
    shards = gathered.view(world, -1)
    outs = [torch.empty_like(p) for p in params]
    say("copy-out")
    fs.fs_unpack_mx4(mp, gathered, outs)
    windows = 0
    for _, src, n, p, r in plan.segments():
        b = mp.piece(p, r)[0]
        nb, some = ref.blocks(n), 300
        starts = {0, nb // 2, max(0, nb - some)} | {max(0, min(nb - some, (edge - src) // 32 - some // 2)) for edge in (1 << 31, 1 << 32, 1 << 35) if src < edge < src + n}
        starts |= {max(0, min(nb - some, edge - b - some // 2)) for edge in (1 << 27, 1 << 28)}      # 2^31 and 2^32 bytes of codes
        for at in starts:
            hi = min(nb, at + some)
            x = np.zeros((hi - at) * 32)
            part = slice(src + at * 32, min(src + n, src + hi * 32))
            x[:part.stop - part.start] = _f64(params[p][part])
            c, s = ref.encode(x.reshape(-1, 32), 9, r * mp.shard_blocks + b + at + np.arange(hi - at))
            shard = shards[r]
            assert np.array_equal(shard[(b + at) * 16:(b + hi) * 16].cpu().numpy(), c.reshape(-1)), f"codes of {p} on {r} from block {at} on"
            assert np.array_equal(shard[mp.shard_blocks * 16 + b + at:mp.shard_blocks * 16 + b + hi].cpu().numpy(), s)
            assert np.array_equal(_f64(outs[p][part]), ref.decode(c, s[:, None]).reshape(-1)[:part.stop - part.start])
            windows += 1
    assert windows >= 4 * 4
    for r in (0, 3):                            # a rank's own copy-in gives the same bytes
        one = torch.empty(mp.shard_bytes, dtype=torch.uint8, device="cuda")
        say("copy-in of rank", r)
        fs.fs_pack_mx4(mp, params, one, rank=r, seed=_seed(9))
        assert torch.equal(one, shards[r])


def test_reduce():
    shapes, world, rank = [((1 << 32) + 12345,), (77,)], 2, 1
    _room(40)
    plan = fs.fs_plan(shapes, "bf16", world, False, "fsdp2")
    mp = fs.fs_mx4_plan(plan).upload()
    assert plan.shard_numel > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(4)
    slices = torch.randint(0, 256, (3 * world, mp.shard_bytes), generator=g, device="cuda", dtype=torch.uint8)
    slices[:, 16 * mp.shard_blocks:17 * mp.shard_blocks].random_(120, 131, generator=g)
    out = torch.full((plan.shard_numel,), float("nan"), device="cuda")
    say("reduce")
    fs.fs_reduce_shard_mx4(mp, slices, out, rank=rank, grad_acc=3)
    covered = 0
    for dst, _, n, p, r in plan.segments():
        if r != rank:
            continue
        b, elem, nb, some = mp.piece(p, r)[0], dst - r * plan.shard_numel, ref.blocks(n), 300
        for at in {0, nb // 2, max(0, nb - some), max(0, min(nb - some, (1 << 26) - some // 2)), max(0, min(nb - some, (1 << 25) - some // 2))}:
            hi = min(nb, at + some)
            m = min(n - at * 32, (hi - at) * 32)
            total = None
            for s in slices:
                v = ref.decode(s[(b + at) * 16:(b + hi) * 16].cpu().numpy(),
                               s[16 * mp.shard_blocks + b + at:16 * mp.shard_blocks + b + hi].cpu().numpy()).astype(np.float32)[:m]
                total = v if total is None else total + v
            assert np.array_equal(out[elem + at * 32:elem + at * 32 + m].cpu().numpy(), total / np.float32(world)), f"piece {p} from block {at} on"
            covered += m
    assert covered > 10000 and not out.isnan().any()
