"""The gradient norm over many tensors, clipping, the reduce that yields the
norm and the AdamW step that clips, against 64-bit numpy (tests/norm_ref.py),
the library's own unfused calls (bit for bit) and the oracle."""
import math

import numpy as np
import pytest
import torch

import norm_ref as ref
import oracle
import synth
from gpu_util import Guarded, bits, say

pytestmark = pytest.mark.gpu

fs = pytest.importorskip("fsdp_sharded_state_amd")

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
NORMS = [2, math.inf]


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


def grads(n, dtype, seed, sd=1e-3):
    make = synth.normal_bf16 if dtype == BF else synth.normal_f32
    return make(seed, synth.STREAM_PARAMS, n, sd, device="cuda")


def packed(sizes, dtypes, seed, fill=math.nan, gap=1, shift=0):
    """Tensors cut out of one buffer per type, `gap` elements of `fill` before
    and between them (so most start off any alignment, next to NaN), and the
    buffers."""
    flats, at, views = {}, {}, []
    for dt in (BF, F32):
        n = shift + gap + sum(s + gap for s, d in zip(sizes, dtypes) if d == dt)
        flats[dt], at[dt] = torch.full((n,), fill, dtype=dt, device="cuda"), shift + gap
    for i, (s, d) in enumerate(zip(sizes, dtypes)):
        v = flats[d][at[d]:at[d] + s]
        v.copy_(grads(s, d, seed + i))
        at[d] += s + gap
        views.append(v)
    return views, flats


SIZE_LISTS = {
    "none": [],
    "empty_tensors": [0, 0],
    "one_element": [1],
    "tiny": [1, 2, 0, 3, 5, 7, 8, 9, 15, 16, 17],
    "one_tile_edges": [2047 * 4, 2048 * 4, 2048 * 4 + 1, 2048 * 8, 2048 * 8 + 3],
    "mid": [100_003, 1, 65_536, 0, 31],
    "spread": [1 << k for k in range(0, 20)] + [(1 << k) + 1 for k in range(0, 20)],
    "many": [3 + 37 * (i % 11) for i in range(500)],
    "large": [9_000_001, 5, 4_100_000],
    "16_tensors": [33] * 16,
    "17_tensors": [33] * 17,
    "192_tensors": [5] * 192,
    "193_tensors": [5] * 193,
    "mostly_empty": [0 if i % 30 else 70 + i for i in range(300)],
    "around_one_launch": [127 * 256, 200],           # 127 KB in fp32: one launch
    "past_one_launch": [128 * 256, 130 * 256],
}


@pytest.mark.parametrize("norm_type", NORMS)
@pytest.mark.parametrize("kind", ["bf16", "fp32", "mixed"])
@pytest.mark.parametrize("name", list(SIZE_LISTS))
def test_norm_over_lists(name, kind, norm_type):
    say("norm", name, kind, norm_type)
    sizes = SIZE_LISTS[name]
    dts = [BF if kind == "bf16" or (kind == "mixed" and i % 3) else F32 for i in range(len(sizes))]
    views, _ = packed(sizes, dts, seed=3)
    total, norm = scalars()
    fs.fs_grad_norm(views, total, norm, norm_type=norm_type)
    ref.check_total(total, views, norm_type)
    ref.check_norm(norm, float(total), norm_type)
    again, _ = scalars()
    fs.fs_grad_norm(fs.fs_grad_list(views), again, norm_type=norm_type)   # the same bits on every run
    assert float(again) == float(total)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_and_clip_at_every_start_and_length(dtype):
    """Starts 0..9 elements off a 16-byte boundary, lengths 0..20, NaN on both
    sides: neither read into the norm nor written by the clip."""
    say("edges", dtype)
    for start in range(10):
        for n in range(21):
            flat = torch.full((64,), math.nan, dtype=dtype, device="cuda")
            v = flat[start:start + n]
            v.copy_(grads(n, dtype, 100 + n, sd=1.0))
            before = bits(flat)
            g = ref.as64(v)
            total, norm = scalars()
            fs.fs_grad_norm([v], total, norm)
            ref.check_total(total, [v], 2)
            if n == 0:
                continue
            coef = ref.coef64(float(total), 2, 0.5 * float(norm), 1e-6)
            fs.fs_clip_grads([v], total, 0.5 * float(norm))
            tol = ref.CLIP_BF16 if dtype == BF else ref.CLIP_F32
            assert (np.abs(ref.as64(v) - g * coef) <= tol * np.abs(g * coef) + 1e-45).all(), (start, n)
            after = bits(flat)
            after[start:start + n] = before[start:start + n]
            np.testing.assert_array_equal(after, before)


@pytest.mark.parametrize("norm_type", NORMS)
def test_norm_accumulates(norm_type):
    say("accumulate", norm_type)
    views, _ = packed([1000, 77, 300_001], [BF, F32, BF], seed=9)
    total, norm = scalars()
    for i, v in enumerate(views):
        fs.fs_grad_norm([v], total, norm, norm_type=norm_type, accumulate=i > 0)
    ref.check_total(total, views, norm_type, extra_n=len(views))
    ref.check_norm(norm, float(total), norm_type)
    fs.fs_grad_norm([], total, norm, norm_type=norm_type, accumulate=True)     # an empty list adds nothing
    ref.check_total(total, views, norm_type, extra_n=len(views) + 1)
    fs.fs_grad_norm([], total, norm, norm_type=norm_type)
    assert float(total) == 0.0 and float(norm) == 0.0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("norm_type", NORMS)
@pytest.mark.parametrize("n", [5, 4096, 700_001])
def test_norm_of_special_values(n, norm_type, dtype):
    say("special", n, norm_type, dtype)
    total, norm = scalars()
    base = grads(n, dtype, 5)

    def measure(*puts):
        g = base.clone()
        for at, x in puts:
            g[at] = x
        fs.fs_grad_norm([g], total, norm, norm_type=norm_type)
        ref.check_total(total, [g], norm_type)
        ref.check_norm(norm, float(total), norm_type)

    measure((n - 1, math.nan))
    measure((0, -math.inf))
    measure((n // 2, math.inf), (1, math.nan))
    measure((n // 2, 3.0e38), (0, -3.0e38))         # squares beyond fp32, not beyond a double
    measure((n // 2, -0.0))
    base = torch.full((n,), 1e-39, dtype=dtype, device="cuda")   # subnormal, squares far below fp32
    measure()
    base = torch.zeros(n, dtype=dtype, device="cuda")
    measure()
    # NaN stays when a list is joined to it, and joins what stands
    total.fill_(math.nan)
    fs.fs_grad_norm([base], total, norm, norm_type=norm_type, accumulate=True)
    assert math.isnan(float(total)) and math.isnan(float(norm))
    total.fill_(1.0)
    base[0] = math.nan
    fs.fs_grad_norm([base], total, norm, norm_type=norm_type, accumulate=True)
    assert math.isnan(float(total))


@pytest.mark.parametrize("norm_type", NORMS)
@pytest.mark.parametrize("kind", ["bf16", "fp32", "mixed"])
@pytest.mark.parametrize("name", list(SIZE_LISTS))
def test_clip_over_lists(name, kind, norm_type):
    say("clip", name, kind, norm_type)
    sizes = SIZE_LISTS[name]
    dts = [BF if kind == "bf16" or (kind == "mixed" and i % 3) else F32 for i in range(len(sizes))]
    views, flats = packed(sizes, dts, seed=21, fill=7.0)
    total, norm = scalars()
    t = 2.25 if norm_type == 2 else 1.5              # a total of all ranks: the norm is 1.5
    total.fill_(t)
    old = [ref.as64(v) for v in views]
    flat_old = {d: bits(f) for d, f in flats.items()}
    fs.fs_clip_grads(views, total, 0.7, norm, norm_type=norm_type)
    assert float(norm) == 1.5 and float(total) == t
    coef = ref.coef64(t, norm_type, 0.7, 1e-6)
    for v, g in zip(views, old):
        tol = ref.CLIP_BF16 if v.dtype == BF else ref.CLIP_F32
        got, want = ref.as64(v), g * coef
        assert (np.abs(got - want) <= tol * np.abs(want) + (1e-38 if v.dtype == BF else 1e-45)).all()
    for v in views:
        v.fill_(0)
    for d, f in flats.items():                       # what lies between the tensors is as it was
        now = f.clone()
        assert int((now != 0).sum()) == sum(1 for d2 in dts if d2 == d) + 1
        np.testing.assert_array_equal(bits(now)[bits(now) != 0], flat_old[d][bits(now) != 0])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_clip_special_totals(dtype):
    say("clip special", dtype)
    n = 30_011
    g = grads(n, dtype, 77)
    g[5], g[6], g[7], g[8], g[9] = math.nan, math.inf, -math.inf, -0.0, 2.0 ** -130      # the last is subnormal
    total, norm = scalars()
    cases = [   # total, norm type, max_norm, eps, coefficient
        (0.25, 2, 1.0, 1e-6, 1.0),
        (0.0, 2, 0.0, 0.0, 1.0),                      # nothing to clip: no 0 / 0
        (1.0, 2, 1.0, 0.0, 1.0),                      # exactly at the limit
        (math.inf, 2, math.inf, 1e-6, 1.0),           # no limit
        (math.inf, math.inf, 1.0, 1e-6, 0.0),
        (4.0, math.inf, 0.0, 1e-6, 0.0),
        (math.nan, 2, 1.0, 1e-6, math.nan),
        (math.nan, math.inf, math.inf, 1e-6, math.nan),
        (16.0, 2, 1.0, 0.0, 0.25),
    ]
    for t, nt, mx, eps, coef in cases:
        x = g.clone()
        total.fill_(t)
        fs.fs_clip_grads([x], total, mx, norm, norm_type=nt, norm_eps=eps)
        if coef == 1.0:
            np.testing.assert_array_equal(bits(x), bits(g))          # NaN payloads included
        else:
            want = (g.float() * coef).to(dtype)                      # a power of two, zero or NaN: exact
            assert torch.equal(torch.isnan(x), torch.isnan(want))
            keep = ~torch.isnan(want)
            np.testing.assert_array_equal(bits(x[keep]), bits(want[keep]))


REDUCE_CASES = [  # n, world, grad_acc, shift
    (0, 2, 1, 0), (1, 1, 1, 0), (7, 2, 1, 0), (1023, 4, 1, 0), (1024, 3, 2, 0), (4095, 8, 1, 0), (4096, 8, 2, 0),
    (4097, 16, 1, 0), (16383, 8, 4, 0), (16385, 8, 3, 0), (40_007, 8, 5, 0), (33_001, 5, 7, 0), (250_001, 8, 4, 0),
    (3, 2, 1, 1), (2049, 2, 2, 1), (30_011, 5, 7, 3), (70_000, 8, 1, 5), (1 << 20, 8, 1, 0), (3_000_001, 2, 1, 0),
]


@pytest.mark.parametrize("norm_type", NORMS)
@pytest.mark.parametrize("rd", ["fp32", "bf16"])
@pytest.mark.parametrize("n,N,A,shift", REDUCE_CASES)
def test_reduce_norm(n, N, A, shift, rd, norm_type):
    say("reduce norm", n, N, A, shift, rd, norm_type)
    sl = [Guarded(n, BF, shift=shift, fill=synth.normal_bf16(4, synth.stream_grad(j, k, N), n, 1e-3, device="cuda"))
          for j in range(A) for k in range(N)]
    plain, got = Guarded(n, F32, shift=shift), Guarded(n, F32, shift=shift)
    fs.fs_reduce_shard_ex([s.t for s in sl], plain.t, N, A, rd)
    total, norm = scalars()
    fs.fs_reduce_shard_norm([s.t for s in sl], got.t, total, norm, world=N, grad_acc=A, reduce_dtype=rd,
                            norm_type=norm_type)
    torch.cuda.synchronize()
    for g in sl + [plain, got]:
        g.check()
    np.testing.assert_array_equal(bits(got.t), bits(plain.t))
    ref.check_total(total, [got.t], norm_type)
    ref.check_norm(norm, float(total), norm_type)
    before = float(total)
    fs.fs_reduce_shard_norm(fs.fs_grad_list([s.t for s in sl]), got.t, total, norm, world=N, grad_acc=A,
                            reduce_dtype=rd, norm_type=norm_type, accumulate=True)
    # the same total once more, joined to itself: exactly twice it, or it
    assert float(total) == (2 * before if norm_type == 2 else before)


@pytest.mark.parametrize("n,terms", [((1 << 23) + 5, 4), (2_100_003, 32), (2_100_003, 40), ((1 << 21) - 1, 24), (5_000_011, 17), ((1 << 27) + 4099, 17)])
def test_reduce_norm_in_every_chunk_shape(n, terms):
    """The shapes that go by length and term count; the slices are
    windows of one buffer, 8 elements apart."""
    say("reduce norm shapes", n, terms)
    g = torch.Generator(device="cuda").manual_seed(n)
    buf = torch.empty(n + 8 * terms, dtype=BF, device="cuda")
    for piece in buf.split(1 << 24):
        piece.copy_(torch.randn(piece.numel(), generator=g, device="cuda").mul_(1e-3))
    sl = [buf[8 * k:8 * k + n] for k in range(terms)]
    out, plain = torch.full((n,), 9.0, device="cuda"), torch.empty(n, device="cuda")
    total, norm = scalars()
    fs.fs_reduce_shard_norm(sl, out, total, norm, world=terms)
    fs.fs_reduce_shard(sl, plain, terms)
    assert torch.equal(out, plain)
    want = sum(float(torch.dot(p, p)) for p in (q.double() for q in plain.split(1 << 24)))
    assert abs(float(total) - want) <= 2 * ref.total_tol(n) * want
    ref.check_norm(norm, float(total), 2)
    fs.fs_reduce_shard_norm(sl, out, total, norm, world=terms, norm_type=math.inf)
    assert float(total) == float(plain.abs().max())


@pytest.mark.parametrize("rd", ["fp32", "bf16"])
def test_reduce_norm_over_launch_spans(rd):
    """Longer than two launch spans, 33 terms in two passes for fp32, a ragged end."""
    n, N = (2 << 25) + 4099, 2
    say("reduce norm spans", n, rd)
    sl = [grads(n, BF, 60 + k) for k in range(N)]
    out, plain = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    total, norm = scalars()
    fs.fs_reduce_shard_norm(sl, out, total, norm, world=N, reduce_dtype=rd)
    fs.fs_reduce_shard_ex(sl, plain, N, 1, rd)
    assert torch.equal(out, plain)
    want = sum(float(torch.dot(p, p)) for p in plain.double().split(1 << 22))
    assert abs(float(total) - want) <= 2 * ref.total_tol(n) * want
    ref.check_norm(norm, float(total), 2)
    peak = plain.abs().max()
    plain[n - 1] = -3.0                             # the last element, by way of the slices
    for s in sl:
        s[n - 1] = -3.0
    fs.fs_reduce_shard_norm(sl, out, total, norm, world=N, reduce_dtype=rd, norm_type=math.inf)
    assert float(peak) < 3.0 and float(total) == 3.0 and float(norm) == 3.0


def _adam_state(n, seed, shift=0):
    th = synth.normal_f32(seed, synth.STREAM_MASTER, n, 0.02, device="cuda")
    m = synth.normal_f32(seed, synth.STREAM_EXP_AVG, n, 1e-3, device="cuda")
    v = synth.normal_f32(seed, synth.STREAM_EXP_AVG_SQ, n, 1e-3, device="cuda") ** 2
    return [Guarded(n, F32, shift=shift, fill=x) for x in (th, m, v)]


@pytest.mark.parametrize("gdt", [BF, F32])
@pytest.mark.parametrize("n,shift", [(0, 0), (1, 0), (3, 1), (255, 0), (256, 0), (1021, 0), (5003, 3), (250_001, 0)])
def test_adamw_clip(n, shift, gdt):
    """Bit for bit the plain step on the scaled gradient, and the oracle's step within its tolerance."""
    hp = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=7)
    for t, nt, mx in [(2.25, 2, 0.7), (1.5, math.inf, 0.7), (0.25, 2, 1.0), (math.inf, 2, 1.0)]:
        say("adamw clip", n, shift, gdt, t, nt)
        g = Guarded(n, gdt, shift=shift, fill=grads(n, gdt, 31))
        total, _ = scalars()
        total.fill_(t)
        coef = np.float32(ref.coef64(t, nt, mx, 1e-6))
        scaled = g.t.float() * float(coef)
        a, b = _adam_state(n, 8, shift), _adam_state(n, 8, shift)
        th0, m0, v0 = (x.t.cpu().numpy().copy() for x in a)
        pa, pb = Guarded(n, BF, shift=shift), Guarded(n, BF, shift=shift)
        fs.fs_adamw_step_clip(*(x.t for x in a), g.t, pa.t, total=total, max_norm=mx, norm_type=nt, **hp)
        fs.fs_adamw_step(*(x.t for x in b), scaled, pb.t, **hp)
        torch.cuda.synchronize()
        for x in a + b + [pa, pb, g]:
            x.check()
        for x, y in zip(a + [pa], b + [pb]):
            np.testing.assert_array_equal(bits(x.t), bits(y.t))
        if n and math.isfinite(t):
            rt, rm, rv, _ = oracle.adamw_step(th0, m0, v0, scaled.cpu().numpy(),
                                              oracle.AdamWHparams(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8,
                                                                  weight_decay=0.1, step=7))
            assert np.all(np.abs(a[0].t.cpu().numpy() - rt) <= 1e-6 * np.maximum(np.abs(rt), np.abs(th0)))
            assert np.all(np.abs(a[1].t.cpu().numpy() - rm) <= 1e-6 * np.abs(rm) + 1e-45)
            assert np.all(np.abs(a[2].t.cpu().numpy() - rv) <= 1e-6 * np.abs(rv) + 1e-45)
        # without the bf16 copy: the same state
        c = _adam_state(n, 8, shift)
        fs.fs_adamw_step_clip(*(x.t for x in c), g.t, total=total, max_norm=mx, norm_type=nt, **hp)
        for x, y in zip(c, b):
            np.testing.assert_array_equal(bits(x.t), bits(y.t))


def test_adamw_clip_nan_total_and_launch_spans():
    n = (64 << 20) + 4101
    say("adamw clip spans", n)
    total, _ = scalars()
    total.fill_(4.0)
    g = grads(n, BF, 2)
    a, b = [[torch.full((n,), x, device="cuda") for x in (0.02, 1e-3, 1e-6)] for _ in range(2)]
    fs.fs_adamw_step_clip(*a, g, total=total, max_norm=1.0, norm_eps=0.0, step=3)
    fs.fs_adamw_step(*b, g.float().mul_(0.5), step=3)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    total.fill_(math.nan)
    fs.fs_adamw_step_clip(*a, g, total=total, max_norm=1.0, step=3)
    assert all(bool(torch.isnan(x).all()) for x in a)


def test_clipped_step_of_all_ranks():
    """The calls together, as a step uses them: N logical ranks reduce their
    shards, each adding its total to one; every rank's AdamW clips by it.  The
    norm is that of the unsharded averaged gradient, and the parameters are
    those of a 64-bit AdamW on the unsharded, clipped gradient."""
    shapes, N, A = synth.mlp_tiny_shapes(), 4, 2
    for mode, uo in (("fsdp2", False), ("fsdp1", True)):
        say("clipped step", mode)
        plan = fs.fs_plan(shapes, "bf16", N, uo, mode, A).upload()
        S = plan.shard_numel
        full = []
        for k in range(N * A):
            g, off = [], 0
            for s in shapes:
                n = int(np.prod(s))
                g.append(synth.normal_bf16(1, synth.stream_grad(0, k, N), n, 1e-2, device="cuda", start=off))
                off += n
            buf = torch.empty(plan.gathered_numel, dtype=BF, device="cuda")
            fs.fs_pack(plan, g, buf)
            full.append((buf, g))
        total, norm = scalars()
        g32 = [torch.empty(S, device="cuda") for _ in range(N)]
        for r in range(N):
            fs.fs_reduce_shard_norm([b[r * S:(r + 1) * S] for b, _ in full], g32[r], total, norm, world=N, grad_acc=A,
                                    accumulate=r > 0)
        # unsharded: the average of every parameter's gradients
        avg = [sum(ref.as64(g[i]) for _, g in full) / N for i in range(len(shapes))]
        want = math.sqrt(sum(float(np.square(x).sum()) for x in avg))
        # each average was rounded A*N times to fp32 on its way, N*A - 1 adds of like terms and a division
        assert abs(float(norm) - want) <= (N * A + 2) * ref.U24 * want
        # the same norm from the local views, parameter by parameter, over all ranks
        twin = plan.twin("fp32").upload()
        total2, norm2 = scalars()
        for r in range(N):
            fs.fs_grad_norm(twin.local_views(g32[r], r), total2, norm2, accumulate=r > 0)
        assert abs(float(total2) - float(total)) <= ref.total_tol(N * S) * float(total)
        max_norm = 0.3 * want
        th, masters = [], []
        for r in range(N):
            p16 = torch.empty(S, dtype=BF, device="cuda")
            state = _adam_state(S, 40 + r)
            th0, m0, v0 = (ref.as64(x.t) for x in state)
            fs.fs_adamw_step_clip(*(x.t for x in state), g32[r], p16, total=total, max_norm=max_norm, step=5)
            g = ref.as64(g32[r]) * (max_norm / (want + 1e-6))
            lr, b1, b2, eps, wd = (float(np.float32(x)) for x in (1e-3, 0.9, 0.999, 1e-8, 0.01))
            m = b1 * m0 + (1 - b1) * g
            v = b2 * v0 + (1 - b2) * g * g
            step = lr * (m / (1 - b1 ** 5)) / (np.sqrt(v / (1 - b2 ** 5)) + eps)
            t64 = th0 * (1 - lr * wd) - step
            # theta: one rounding of its own; g is off by (N*A + 6) * 2^-24 (norm, coefficient, product), which
            # moves the step by no more than twice that
            tol = ref.U24 * np.maximum(np.abs(t64), np.abs(th0)) + 2 * (N * A + 6) * ref.U24 * lr * (
                b1 * np.abs(m0) + np.abs((1 - b1) * g)) / (1 - b1 ** 5) / (np.sqrt(v / (1 - b2 ** 5)) + eps)
            assert (np.abs(ref.as64(state[0].t) - t64) <= 1.01 * tol).all()
            assert (np.abs(ref.as64(p16) - ref.as64(state[0].t)) <= ref.U8 * np.abs(ref.as64(state[0].t))).all()
            th.append(p16)
            masters.append(state[0].t)
        # clipping the shards in place and stepping without a clip ends in the same bits
        for r in range(N):
            state = _adam_state(S, 40 + r)
            g = g32[r].clone()
            fs.fs_clip_grads(twin.local_views(g, r), total, max_norm)
            p16 = torch.empty(S, dtype=BF, device="cuda")
            fs.fs_adamw_step(*(x.t for x in state), g, p16, step=5)
            np.testing.assert_array_equal(bits(state[0].t), bits(masters[r]))
            np.testing.assert_array_equal(bits(p16), bits(th[r]))


def test_long_tensor_past_32_bit_offsets():
    """A tensor of more than 2^32 bytes and 2^31 elements: what its end holds
    counts, and the clip reaches it."""
    n = (1 << 31) + 4099
    say("long", n)
    g = torch.zeros(n, dtype=BF, device="cuda")
    at = [0, (1 << 30) + 5, (1 << 31) - 1, 1 << 31, n - 1]
    for i, k in enumerate(at):
        g[k] = float(1 << i)
    total, norm = scalars()
    fs.fs_grad_norm([g[1:]], total, norm)
    assert float(total) == 4.0 + 16.0 + 64.0 + 256.0
    fs.fs_grad_norm([g], total, norm, norm_type=math.inf)
    assert float(total) == 16.0
    fs.fs_clip_grads([g], total, 4.0, norm, norm_type=math.inf, norm_eps=0.0)
    assert [float(g[k]) for k in at] == [0.25, 0.5, 1.0, 2.0, 4.0]
    assert int(torch.count_nonzero(g)) == len(at)


def test_captured_and_replayed():
    """The four calls in one graph, twice, in a shared pool; replays between
    eager work on the same stream, each against the eager result."""
    n, N = 50_021, 4
    say("graph")
    sl = [[grads(n, BF, 10 * q + k) for k in range(N)] for q in range(2)]
    lists = [fs.fs_grad_list(s) for s in sl]

    def buffers():
        return dict(out=torch.zeros(n, device="cuda"), total=scalars()[0], norm=scalars()[1], t2=scalars()[0],
                    clip=torch.zeros(n, device="cuda"), st=[x.t for x in _adam_state(n, 3)],
                    p=torch.zeros(n, dtype=BF, device="cuda"))

    def step(q, b):
        fs.fs_reduce_shard_norm(lists[q], b["out"], b["total"], b["norm"], world=N)
        b["clip"].copy_(b["out"])
        fs.fs_clip_grads([b["clip"]], b["total"], 0.01)
        fs.fs_grad_norm([b["clip"][:7], b["clip"][7:]], b["t2"])
        fs.fs_adamw_step_clip(*b["st"], b["out"], b["p"], total=b["total"], max_norm=0.01, step=2)

    eager, captured, graphs = [buffers() for _ in range(2)], [buffers() for _ in range(2)], []
    pool = torch.cuda.graph_pool_handle()
    for q in range(2):
        b = captured[q]
        keep = [x.clone() for x in b["st"]]
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step(q, b)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            step(q, b)
        for x, k in zip(b["st"], keep):
            x.copy_(k)
        graphs.append(g)
    for rep in range(4):
        for q in (0, 1):
            for k in range(N):                      # new gradients in the same places
                sl[q][k].copy_(grads(n, BF, 1000 * rep + 10 * q + k, sd=1e-3 * (rep + 1)))
            step(q, eager[q])
            graphs[q].replay()
            torch.cuda.synchronize()
            e, c = eager[q], captured[q]
            assert float(e["total"]) == float(c["total"]) and float(e["t2"]) == float(c["t2"]) > 0
            assert float(e["norm"]) == float(c["norm"])
            for x, y in zip([e["out"], e["clip"], e["p"], *e["st"]], [c["out"], c["clip"], c["p"], *c["st"]]):
                np.testing.assert_array_equal(bits(x), bits(y))


@pytest.mark.parametrize("seed", range(24))
def test_random_lists(seed):
    """Random counts, sizes, types, gaps and starts: total, norm and clip."""
    rng = np.random.default_rng(seed)
    n = int(np.exp(rng.uniform(0, np.log(400))))
    most = np.exp(rng.uniform(0, np.log(300_000 if n > 40 else 3_000_000)))
    sizes = [int(x) for x in np.exp(rng.uniform(0, np.log(most + 1), n)) - (rng.random(n) < 0.1)]
    dts = [BF if rng.random() < 0.5 else F32 for _ in sizes]
    say("random list", seed, n, int(most))
    views, flats = packed(sizes, dts, seed=1000 * seed, gap=int(rng.integers(0, 6)), shift=int(rng.integers(0, 9)))
    norm_type = NORMS[seed % 2]
    gl = fs.fs_grad_list(views)
    total, norm = scalars()
    fs.fs_grad_norm(gl, total, norm, norm_type=norm_type)
    ref.check_total(total, views, norm_type)
    ref.check_norm(norm, float(total), norm_type)
    nans = {d: int(torch.isnan(f).sum()) for d, f in flats.items()}
    old, mx = [ref.as64(v) for v in views], 0.6 * float(norm)
    fs.fs_clip_grads(gl, total, mx, norm_type=norm_type, norm_eps=0.0)
    coef = ref.coef64(float(total), norm_type, mx, 0.0)
    for v, g in zip(views, old):
        tol = ref.CLIP_BF16 if v.dtype == BF else ref.CLIP_F32
        assert (np.abs(ref.as64(v) - g * coef) <= tol * np.abs(g * coef) + (1e-38 if v.dtype == BF else 1e-45)).all()
    assert nans == {d: int(torch.isnan(f).sum()) for d, f in flats.items()}


def test_threads_share_a_list():
    """Four host threads, each with its stream and total, one list and one set of slices."""
    import threading
    say("threads")
    sizes = [70_001, 5, 400_000]
    views, _ = packed(sizes, [F32, BF, BF], seed=4)
    gl, sl = fs.fs_grad_list(views), fs.fs_grad_list([grads(50_000, BF, k) for k in range(8)])
    want, want_r = scalars()[0], scalars()[0]
    out0 = torch.empty(50_000, device="cuda")
    fs.fs_grad_norm(gl, want)
    fs.fs_reduce_shard_norm(sl, out0, want_r, world=8)
    torch.cuda.synchronize()
    bad = []

    def work(k):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                t, r = torch.zeros(1, dtype=F64, device="cuda"), torch.zeros(1, dtype=F64, device="cuda")
                out = torch.empty(50_000, device="cuda")
                for _ in range(25):
                    fs.fs_grad_norm(gl, t)
                    fs.fs_reduce_shard_norm(sl, out, r, world=8)
                    if float(t) != float(want) or float(r) != float(want_r) or not torch.equal(out, out0):
                        bad.append(k)
        except Exception as e:  # noqa: BLE001 -- reported below
            bad.append((k, repr(e)))

    ts = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not bad, bad


def test_streams_of_their_own():
    """Two streams at once, each given as an object or a raw handle, one list
    between them; and the allocator's reuse of a finished call's workspace."""
    say("streams")
    big = [grads(6_000_011, F32, 1), grads(3_000_003, BF, 2)]
    gl = fs.fs_grad_list(big)
    want, _ = scalars()
    fs.fs_grad_norm(gl, want)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[torch.zeros(1, dtype=F64, device="cuda") for _ in range(20)] for _ in streams]
    torch.cuda.synchronize()
    for i in range(20):
        for k, s in enumerate(streams):
            fs.fs_grad_norm(gl, outs[k][i], stream=s if i % 2 else s.cuda_stream)
        torch.full((1 << 14,), 1e30, dtype=F64, device="cuda")     # takes what the current stream's pool has free
    fs.fs_grad_norm(gl, want, stream=0)                             # the null stream
    torch.cuda.synchronize()
    assert all(float(t) == float(want) for row in outs for t in row)


def test_a_lists_memory_that_moved_is_refused():
    t = torch.ones(1000, device="cuda")
    gl = fs.fs_grad_list([t[:500], t[500:]])
    total, _ = scalars()
    fs.fs_grad_norm(gl, total)
    assert float(total) == 1000.0
    t.untyped_storage().resize_(0)
    with pytest.raises(ValueError, match="memory"):
        fs.fs_grad_norm(gl, total)
    with pytest.raises(ValueError, match="memory"):
        fs.fs_clip_grads(gl, total, 1.0)
    # an alias is held: a replaced gradient leaves the list's memory alone
    p = torch.nn.Parameter(torch.ones(64, device="cuda"))
    p.grad = torch.full((64,), 2.0, device="cuda")
    gl = fs.fs_grad_list([p.grad])
    p.grad = None
    torch.zeros(64, device="cuda")
    fs.fs_grad_norm(gl, total)
    assert float(total) == 256.0


def test_refused_on_the_gpu():
    a = torch.ones(64, 64, device="cuda")
    total, norm = scalars()
    with pytest.raises(ValueError, match="contiguous"):
        fs.fs_grad_norm([a.t()], total)
    with pytest.raises(ValueError, match="dtype"):
        fs.fs_grad_norm([a.half()], total)
    with pytest.raises(ValueError, match="is on"):
        fs.fs_grad_norm([a], total.cpu())
    with pytest.raises(ValueError, match="tensor 1"):
        fs.fs_grad_list([a, a.cpu()])
    with pytest.raises(fs.FsError, match="share memory"):
        fs.fs_clip_grads([a, a[3]], total, 1.0)
    with pytest.raises(fs.FsError, match="overlaps tensor 0"):
        fs.fs_grad_norm([a.view(-1)], total, a.view(-1)[5:6])
    with pytest.raises(fs.FsError, match="max_norm"):
        fs.fs_clip_grads([a], total, -1.0)
    with pytest.raises(ValueError, match="slice"):
        fs.fs_reduce_shard_norm([a.view(-1)], a.view(-1), total, world=1)
    assert bool((a == 1).all()) and float(total) == -7.0
