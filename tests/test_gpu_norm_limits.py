"""The gradient norm at the limit of its one-launch form, and the reduce with
norm over several passes and launch spans together and with NaN and infinities
in its slices."""
import math

import numpy as np
import pytest
import torch

import norm_ref as ref
import synth
from gpu_util import Guarded, bits, say
from test_norm_limits import MOST, TILES

pytestmark = pytest.mark.gpu

fs = pytest.importorskip("fsdp_sharded_state_amd")

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
CODE = {BF: fs.FS_BF16, F32: fs.FS_FP32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fs.lib()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def scalars():
    """total and norm, holding something else."""
    return torch.full((1,), -7.0, dtype=F64, device="cuda"), torch.full((1,), -7.0, device="cuda")


def views_of(sizes, dtype, start):
    """Tensors of their own buffers, `start` elements into a 512-byte aligned
    one, NaN around each."""
    out = []
    for i, n in enumerate(sizes):
        flat = torch.full((n + start + 8,), math.nan, dtype=dtype, device="cuda")
        v = flat[start:start + n]
        v.copy_(synth.normal_f32(5 + i, synth.STREAM_PARAMS, n, 1.0, device="cuda"))
        out.append(v)
    return out


@pytest.mark.parametrize("norm_type", [2, math.inf])
@pytest.mark.parametrize("start", ["line", "last element of a line"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_at_the_one_launch_limit(dtype, start, norm_type):
    most, off = MOST[CODE[dtype]], 0 if start == "line" else 128 // torch.finfo(dtype).bits * 8 - 1
    lists = [[most(TILES)], [most(TILES) + 1], [most(1)] * TILES, [most(1)] * (TILES + 1), [1] * TILES, [1] * (TILES + 1),
             [most(64), most(64)], [most(64), most(64) + 1]]
    for sizes in lists:
        say("one-launch limit", dtype, start, norm_type, len(sizes), sizes[-1])
        views = views_of(sizes, dtype, off)
        total, norm = scalars()
        fs.fs_grad_norm(views, total, norm, norm_type=norm_type)
        ref.check_total(total, views, norm_type)
        ref.check_norm(norm, float(total), norm_type)


SPAN = {"fp32": 32 << 20, "bf16": 16 << 20}   # elements of one launch


@pytest.mark.parametrize("rd,N,A,n,aligned", [
    ("fp32", 4, 9, (32 << 20) + 4099, True),       # passes of 32 and 4 terms: two chunk shapes in one call
    ("fp32", 8, 5, (32 << 20) + 4099, True),       # 32 and 8
    ("fp32", 7, 7, (128 << 20) + 4099, True),      # 32 and 17 in the longest calls' shape, five spans
    ("fp32", 8, 5, (32 << 20) + 4099, False),
    ("fp32", 4, 16, (64 << 20) + 5, True),         # two whole passes of 32
    ("bf16", 8, 5, (32 << 20) + 4099, True),       # four micro-steps, then one; three spans
    ("bf16", 16, 3, (16 << 20) + 8200, True),      # two, then one
    ("bf16", 8, 5, (16 << 20) + 4099, False),
])
def test_reduce_norm_over_passes_and_spans(rd, N, A, n, aligned):
    """More than 32 terms and more than one launch span: each span's launches
    leave partial totals in its last pass only.  One slice holds the few
    nonzero elements: one at a time for the maximum, and all of one size for
    the sum of squares, so that a lost or overwritten partial total shows."""
    say("reduce norm passes x spans", rd, N, A, n, aligned)
    terms, step, first = N * A, 8 if aligned else 3, 0 if aligned else 1
    buf = torch.zeros(first + n + step * terms, dtype=BF, device="cuda")
    windows = [buf[first + step * k:first + step * k + n] for k in range(terms)]
    own = torch.zeros(first + n, dtype=BF, device="cuda")[first:]
    sl = windows[:-1] + [own]
    edges = list(range(SPAN[rd], n, SPAN[rd]))
    at = sorted({0, 1, 2047, 2048, n // 2, n - 1} | {e + d for e in edges for d in (-1, 0)})
    out, plain = torch.full((n,), 9.0, device="cuda"), torch.empty(n, device="cuda")
    total, norm = scalars()

    # each place in turn: the maximum is that one element's
    for k in at:
        own[k] = 3.0
        fs.fs_reduce_shard_ex(sl, plain, N, A, rd)
        fs.fs_reduce_shard_norm(sl, out, total, norm, world=N, grad_acc=A, reduce_dtype=rd, norm_type=math.inf)
        assert torch.equal(out, plain), k
        assert float(plain[k]) > 0 and float(total) == float(plain.abs().max()) == float(norm), k
        own[k] = 0.0
    # and all of them
    for i, k in enumerate(at):
        own[k] = 1.0 + i / 32
    fs.fs_reduce_shard_ex(sl, plain, N, A, rd)
    fs.fs_reduce_shard_norm(sl, out, total, norm, world=N, grad_acc=A, reduce_dtype=rd)
    assert torch.equal(out, plain)
    x = plain[plain != 0].cpu().numpy().astype(np.float64)
    want = math.fsum(x * x)
    # the zeros add nothing, so only the nonzero elements' sums round
    assert len(x) == len(at) and abs(float(total) - want) <= ref.total_tol(len(x)) * want
    ref.check_norm(norm, float(total), 2)
    # random gradients: the averages bit for bit
    buf.copy_(synth.normal_bf16(17, synth.STREAM_PARAMS, buf.numel(), 1e-3, device="cuda"))
    fs.fs_reduce_shard_ex(windows, plain, N, A, rd)
    fs.fs_reduce_shard_norm(windows, out, total, norm, world=N, grad_acc=A, reduce_dtype=rd)
    assert torch.equal(out, plain)
    want = sum(float(torch.dot(p, p)) for p in (q.double() for q in plain.split(1 << 24)))
    assert abs(float(total) - want) <= 2 * ref.total_tol(n) * want


@pytest.mark.parametrize("norm_type", [2, math.inf])
@pytest.mark.parametrize("rd", ["fp32", "bf16"])
@pytest.mark.parametrize("n,N,A,shift", [
    (1001, 4, 1, 0), (1001, 4, 2, 1), (100_003, 8, 1, 0), (100_003, 8, 5, 0), (100_003, 4, 2, 3), (2_500_001, 8, 2, 0),
])
def test_reduce_norm_of_nan_and_infinities(n, N, A, shift, rd, norm_type):
    """They reach the averages, and show in the total and the norm."""
    say("reduce norm special", n, N, A, shift, rd, norm_type)
    base = [synth.normal_bf16(23, synth.stream_grad(j, k, N), n, 1e-3, device="cuda") for j in range(A) for k in range(N)]
    last = N * A - 1
    cases = [   # (slice, element, value) of each
        [(0, n - 1, math.nan)],
        [(last, 0, math.inf)],
        [(last // 2, n // 2, -math.inf)],
        [(0, n // 3, math.inf), (1, n // 3, -math.inf)],      # their sum is NaN
        [(0, 5, math.inf), (last, n - 2, math.nan)],
        [(0, n - 1, 3.0e38), (1, n - 1, 3.0e38)],             # beyond fp32 in the running sum
    ]
    for puts in cases:
        sl = [Guarded(n, BF, shift=shift, fill=b) for b in base]
        for k, e, x in puts:
            sl[k].t[e] = x
        plain, got = Guarded(n, F32, shift=shift), Guarded(n, F32, shift=shift)
        total, norm = scalars()
        fs.fs_reduce_shard_ex([s.t for s in sl], plain.t, N, A, rd)
        fs.fs_reduce_shard_norm([s.t for s in sl], got.t, total, norm, world=N, grad_acc=A, reduce_dtype=rd,
                                norm_type=norm_type)
        torch.cuda.synchronize()
        for g in sl + [plain, got]:
            g.check()
        np.testing.assert_array_equal(bits(got.t), bits(plain.t))
        assert not math.isfinite(float(total))
        ref.check_total(total, [got.t], norm_type)
        ref.check_norm(norm, float(total), norm_type)
