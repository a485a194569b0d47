"""Microscaled 4-bit operators on the GPU against their 64-bit definitions
(tests/mx4_ref.py): codes, scales and decoded values bit for bit, the reduce
bit for bit, products within the tolerance that mx4_ref.py derives."""
import ctypes
import math
import threading

import numpy as np
import pytest
import torch

import fsdp_sharded_state_amd as fs
import mx4_ref as ref
import synth
from gpu_util import say

pytestmark = pytest.mark.gpu

CANARY = 0xA5
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _values(shape, dtype, seed, spread=3.0):
    """Normals times powers of two of wide spread, some exact midpoints and zeros of both signs."""
    g = _gen(seed)
    x = torch.randn(shape, generator=g, device="cuda") * torch.exp2(torch.randn(shape, generator=g, device="cuda") * spread)
    grid = torch.randint(-24, 25, shape, generator=g, device="cuda") * 0.25
    pick = torch.rand(shape, generator=g, device="cuda")
    return torch.where(pick < 0.1, grid, torch.where(pick > 0.97, -torch.zeros_like(x), x)).to(DT[dtype])


def _f64(t):
    return t.detach().float().cpu().double().numpy()


def _seed(v):
    return torch.tensor([v], dtype=torch.int64, device="cuda")


class Guard:
    """A matrix of 4-bit blocks between canaries, with row strides beyond the rows' bytes."""

    def __init__(self, rows, cols, more=0):
        nb = ref.blocks(cols)
        self.rows, self.nb, self.cs, self.ss = rows, nb, 16 * nb + 16 * more, nb + more
        self.codes = torch.full((128 + rows * self.cs,), CANARY, dtype=torch.uint8, device="cuda")
        self.scales = torch.full((128 + rows * self.ss,), CANARY, dtype=torch.uint8, device="cuda")
        self.c = self.codes[64:].as_strided((rows, 16 * nb), (self.cs, 1))
        self.s = self.scales[64 - more:].as_strided((rows, nb), (self.ss, 1))     # any byte address
        self.m = fs.Mx4Matrix(self.c, self.s, cols)

    def check(self, codes, scales):
        assert np.array_equal(self.s.cpu().numpy(), scales), "scales differ"
        got = self.c.cpu().numpy()
        assert np.array_equal(got, codes), f"{(got != codes).sum()} code bytes differ"
        self.c.fill_(CANARY)
        self.s.fill_(CANARY)
        assert (self.codes == CANARY).all() and (self.scales == CANARY).all(), "bytes between the rows were written"


# ------------------------------------------------------------------ matrices --

SHAPES = [(1, 1), (1, 31), (1, 32), (1, 33), (1, 4096), (2, 64), (31, 33), (33, 31), (64, 256), (128, 128), (127, 129),
          (129, 127), (257, 100), (300, 8), (5, 1000), (1000, 5), (96, 416), (513, 640)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_quantize(rows, cols, dtype):
    for case, (which, seed, pad, shift, more) in enumerate([("both", None, 0, 0, 0), ("both", -7, 3, 1, 2), ("row", 1 << 62, 8, 8, 0),
                                                           ("col", None, 5, 0, 1), ("col", 12345, 0, 3, 0), ("row", None, 24, 0, 3)]):
        say("quantize", rows, cols, dtype, which, seed)
        base = _values((rows * (cols + pad) + shift + 1,), dtype, 100 * rows + cols + case)
        x = base[shift:].as_strided((rows, cols), (cols + pad, 1))
        r = Guard(rows, cols, more) if which != "col" else None
        c = Guard(cols, rows, more) if which != "row" else None
        fs.fs_mx4_quantize(x, r and r.m, c and c.m, seed=None if seed is None else _seed(seed))
        v, bits = _f64(x), None if seed is None else seed & (2 ** 64 - 1)
        if r:
            r.check(*ref.encode_matrix(v, bits, 0))
        if c:
            c.check(*ref.encode_matrix(v.T, bits, 1))


@pytest.mark.parametrize("rows,cols,pad", [(8200, 1100, 0), (300, 33000, 5), (70000, 33, 8)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("seed", [None, 7])
def test_quantize_and_back_of_many_tiles(rows, cols, pad, dtype, seed):
    """Rows alone, and both ways: every block of some rows and columns, and all of them against each other."""
    say(f"many tiles {rows} {cols} {pad} {dtype} {seed}")
    x = _values((rows, cols + pad), dtype, rows)[:, :cols]
    alone, both, col = Guard(rows, cols), Guard(rows, cols), Guard(cols, rows)
    sd = None if seed is None else _seed(seed)
    fs.fs_mx4_quantize(x, alone.m, seed=sd)
    fs.fs_mx4_quantize(x, both.m, col.m, seed=sd)
    out = torch.full((rows, cols + pad), 7.0, device="cuda")
    fs.fs_mx4_dequantize(alone.m, out[:, :cols])
    assert torch.equal(alone.c, both.c) and torch.equal(alone.s, both.s)
    assert (out[:, cols:] == 7).all()
    for q, v, n, o in ((alone, x, cols, 0), (col, x.T, rows, 1)):
        take = sorted({0, 1, 17, q.rows // 2, q.rows - 16, q.rows - 1})
        c, s = q.c[take].cpu().numpy(), q.s[take].cpu().numpy()
        nb, host = ref.blocks(n), _f64(v[take])
        full = np.zeros((len(take), nb * ref.BLOCK))
        full[:, :n] = host
        index = (np.array(take)[:, None] * nb + np.arange(nb)).reshape(-1)
        wc, ws = ref.encode(full.reshape(-1, ref.BLOCK), seed, index, o)
        assert np.array_equal(c, wc.reshape(len(take), -1)) and np.array_equal(s, ws.reshape(len(take), -1))
        if o == 0:
            assert np.array_equal(_f64(out[take][:, :cols]), _decoded(q.c[take], q.s[take], cols))
    for q in (alone, both, col):
        q.check(q.c.cpu().numpy().copy(), q.s.cpu().numpy().copy())    # the canaries between


@pytest.mark.parametrize("seed", [None, 99])
def test_quantize_every_bf16_value(seed):
    """Each value beside a maximum of its own binade, of 1 to 7 binades more, and alone."""
    u = np.arange(65536, dtype=np.uint32)
    rows = []
    for more in (0, 1, 2, 3, 7):
        e = np.minimum(((u >> 7) & 255) + more, 254)
        rows.append(np.where((u & 0x7F80) == 0x7F80, 0, (e << 7) | 0x15))     # a partner; none beside inf and NaN
    m = np.stack([u, *rows], 1).astype(np.uint16)
    blocks = np.zeros((5 * 65536, 32), np.uint16)
    for k in range(5):
        blocks[k * 65536:(k + 1) * 65536, 2 * k] = m[:, 0]
        if k:
            blocks[k * 65536:(k + 1) * 65536, 31 - k] = m[:, k]
    for dtype in ("bf16", "fp32"):
        x = torch.from_numpy(blocks.view(np.int16).copy()).view(torch.bfloat16).cuda().to(DT[dtype])
        q = fs.fs_mx4_empty(x.shape[0], 32)
        say("every bf16 value", dtype, seed)
        fs.fs_mx4_quantize(x, q, seed=None if seed is None else _seed(seed))
        v = (blocks.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
        c, s = ref.encode_matrix(v, seed, 0)
        assert np.array_equal(q.scales.cpu().numpy(), s) and np.array_equal(q.codes.cpu().numpy(), c)


@pytest.mark.parametrize("seed", [None, 3])
def test_quantize_fp32_beside_midpoints_and_at_the_ends(seed):
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.5, 1, 1.5, 2, 3, 4, 6, 7, 7.999], np.float32)
    near = np.concatenate([mids, np.nextafter(mids, np.float32(0)), np.nextafter(mids, np.float32(8))])
    near = np.concatenate([near, -near]).astype(np.float64)
    rows = []
    for e in (-149, -140, -128, -127, -126, -125, -60, -1, 0, 1, 60, 124, 125):
        for top in (4.0, 4.5, 6.0, 6.0000005, 7.99):
            with np.errstate(over="ignore"):
                v = np.ldexp(near, e).astype(np.float32)
                b = np.zeros((4, 32), np.float32)
                b[:, 0] = np.float32(np.ldexp(top, e))
            for k in range(4):
                part = v[k * 24:(k + 1) * 24]
                b[k, 4:4 + len(part)] = np.where(np.abs(part) <= b[k, 0], part, 0)
            rows.append(b)
    x = np.concatenate(rows + [np.zeros((1, 32), np.float32), np.full((1, 32), np.nan, np.float32),
                               np.full((1, 32), -np.inf, np.float32), np.full((1, 32), 3.4e38, np.float32)])
    x[-3, 1:] = 1.0
    q = fs.fs_mx4_empty(x.shape[0], 32)
    fs.fs_mx4_quantize(torch.from_numpy(x).cuda(), q, seed=None if seed is None else _seed(seed))
    c, s = ref.encode_matrix(x.astype(np.float64), seed, 0)
    assert np.array_equal(q.scales.cpu().numpy(), s) and np.array_equal(q.codes.cpu().numpy(), c)


def test_stochastic_rounding_is_unbiased():
    """The mean over T seeds of an element between two codes a step apart is
    off by at most 2^-17 of a step (the random bits' grain) and its sampling
    error: each draw has variance at most step^2 / 4, so 6 sigma is
    3 * step / sqrt(T)."""
    T, scale = 4096, 2.0 ** -3
    x = torch.rand(1, 32, generator=_gen(1), device="cuda") * 0.75          # amax under 6/8: one scale
    x[0, 0] = 0.75
    total = torch.zeros(32, device="cuda", dtype=torch.float64)
    q, out = fs.fs_mx4_empty(1, 32), torch.empty(1, 32, device="cuda")
    for t in range(T):
        fs.fs_mx4_quantize(x, q, seed=_seed(t))
        fs.fs_mx4_dequantize(q, out)
        total += out[0].double()
    y = x[0].double() / scale
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0)) * scale
    assert ((total / T - x[0].double()).abs() <= step * (3 / math.sqrt(T) + 2.0 ** -17)).all()


def _random_matrix(rows, cols, seed, lo=120, hi=134):
    g = _gen(seed)
    nb = ref.blocks(cols)
    codes = torch.randint(0, 256, (rows, 16 * nb), generator=g, device="cuda", dtype=torch.uint8)
    if cols % 32:                                   # zeros after the last element
        flat = torch.zeros(rows, 32 * nb, dtype=torch.uint8, device="cuda")
        flat[:, 0::2], flat[:, 1::2] = codes & 15, codes >> 4
        flat[:, cols:] = 0
        codes = flat[:, 0::2] | (flat[:, 1::2] << 4)
    return codes.contiguous(), torch.randint(lo, hi, (rows, nb), generator=g, device="cuda", dtype=torch.uint8)


def _decoded(codes, scales, cols):
    return ref.decode(codes.cpu().numpy(), scales.cpu().numpy())[:, :cols]


def test_dequantize_every_code_at_every_scale():
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").view(16, 16).repeat(256, 1)
    scales = torch.arange(256, dtype=torch.uint8, device="cuda").repeat_interleave(16).view(-1, 1)
    want = _decoded(codes, scales, 32)
    for dt in (torch.float32, torch.bfloat16):
        out = torch.empty(4096, 32, dtype=dt, device="cuda")
        fs.fs_mx4_dequantize(fs.Mx4Matrix(codes, scales, 32), out)
        with np.errstate(over="ignore"):
            exact = torch.from_numpy(want.astype(np.float32)).to(dt).float()     # in fp32 exact up to overflow
        nan = torch.isnan(exact)
        got = out.float().cpu()
        assert torch.equal(torch.isnan(got), nan)
        assert torch.equal(torch.where(nan, 0, got).view(torch.int32), torch.where(nan, 0, exact).view(torch.int32))


@pytest.mark.parametrize("rows,cols", SHAPES)
def test_dequantize(rows, cols):
    codes, scales = _random_matrix(rows, cols, rows * 7 + cols)
    want = torch.from_numpy(_decoded(codes, scales, cols).astype(np.float32))
    for dt, pad, shift in ((torch.float32, 0, 0), (torch.float32, 3, 1), (torch.bfloat16, 0, 0), (torch.bfloat16, 7, 3)):
        raw = torch.full((64 + shift + rows * (cols + pad),), -77.0, dtype=dt, device="cuda")
        out = raw[32 + shift:].as_strided((rows, cols), (cols + pad, 1))
        say("dequantize", rows, cols, dt, pad)
        fs.fs_mx4_dequantize(fs.Mx4Matrix(codes, scales, cols), out)
        assert torch.equal(out.cpu(), want.to(dt))
        out.fill_(-77.0)
        assert (raw == -77.0).all()


# -------------------------------------------------------------------- shards --

GROUPS = {
    "mlp": synth.mlp_tiny_shapes(),
    "odd": [(5, 7), (1,), (), (0, 4), (33,), (3, 32), (100, 64), (2, 5, 9), (257,), (8191,), (3, 8193)],
    "tiny": [(1,)] * 20,
    "one": [(70000,)],
}


def _group(name, world, mode, orig, dtype):
    shapes = GROUPS[name]
    plan = fs.fs_plan(shapes, dtype, world, orig, mode)
    mp = fs.fs_mx4_plan(plan).upload()
    rows = [(plan.param(i).chunk_rows, plan.param(i).row) for i in range(len(shapes))]
    pieces, blocks, nbytes = ref.layout(plan.segments(), rows, mode, world, len(shapes))
    return shapes, plan, mp, pieces, blocks, nbytes


MODES = [("fsdp1", False), ("fsdp1", True), ("fsdp2", False)]


@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("world", [1, 3, 8])
@pytest.mark.parametrize("mode,orig", MODES)
def test_pack_and_unpack(name, world, mode, orig):
    for dtype, seed, shift in (("bf16", None, 0), ("fp32", None, 1), ("bf16", 17, 3), ("fp32", -1, 0)):
        say("pack", name, world, mode, orig, dtype, seed)
        shapes, plan, mp, pieces, blocks, nbytes = _group(name, world, mode, orig, dtype)
        numels = [math.prod(s) for s in shapes]
        params = [_values((n + shift,), dtype, 31 * i + world)[shift:].view(s) for i, (s, n) in enumerate(zip(shapes, numels))]
        want = ref.pack(pieces, blocks, nbytes, world, [_f64(p).reshape(-1) for p in params],
                        None if seed is None else seed & (2 ** 64 - 1))
        raw = torch.full((32 + mp.gathered_bytes,), CANARY, dtype=torch.uint8, device="cuda")
        out = raw[16:16 + mp.gathered_bytes]
        s = None if seed is None else _seed(seed)
        fs.fs_pack_mx4(mp, params, out, seed=s)
        assert np.array_equal(out.cpu().numpy().reshape(world, nbytes), want)
        assert (raw[:16] == CANARY).all() and (raw[16 + mp.gathered_bytes:] == CANARY).all()
        for r in range(world):
            shard = torch.full((nbytes,), CANARY, dtype=torch.uint8, device="cuda")
            fs.fs_pack_mx4(mp, params, shard, rank=r, seed=s)
            assert np.array_equal(shard.cpu().numpy(), want[r]), f"rank {r}"
        flats = [torch.full((n + 8 + shift,), -77.0, dtype=DT[dtype], device="cuda") for n in numels]
        outs = [f[4 + shift:4 + shift + n].view(sh) for f, n, sh in zip(flats, numels, shapes)]
        fs.fs_unpack_mx4(mp, out, outs)
        for i, (o, f, n) in enumerate(zip(outs, flats, numels)):
            v = np.zeros(n)
            for (p, r), (b, src, ln) in pieces.items():
                if p == i:
                    v[src:src + ln] = ref.piece_values(want[r], blocks, b, ln)
            assert torch.equal(o.reshape(-1).cpu(), torch.from_numpy(v.astype(np.float32)).to(DT[dtype])), f"parameter {i}"
            o.fill_(-77.0)
            assert (f == -77.0).all()


@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("world,acc", [(1, 1), (3, 1), (8, 1), (3, 5), (8, 9), (64, 2), (65, 2)])
@pytest.mark.parametrize("mode,orig", MODES)
def test_reduce_bit_exact(name, world, acc, mode, orig):
    shapes, plan, mp, pieces, blocks, nbytes = _group(name, world, mode, orig, "bf16")
    terms = world * acc
    for rank in {0, world // 2, world - 1}:
        say("reduce", name, world, acc, mode, orig, rank)
        g = _gen(rank + terms)
        slices = torch.randint(0, 256, (terms, nbytes), generator=g, device="cuda", dtype=torch.uint8)   # pads hold anything
        if blocks:
            slices[:, blocks * 16:blocks * 17] = torch.randint(110, 125, (terms, blocks), generator=g, device="cuda", dtype=torch.uint8)
        n = plan.shard_numel
        raw = torch.full((n + 9,), -77.0, device="cuda")
        out = raw[5:5 + n]
        rows = list(slices) if terms % 2 else slices
        fs.fs_reduce_shard_mx4(mp, rows, out, rank=rank, grad_acc=acc)
        want = np.zeros(n, np.float32)
        pos = {(p, r): dst - r * n for dst, _, _, p, r in plan.segments()}
        host = slices.cpu().numpy()
        for (p, r), (b, _, ln) in pieces.items():
            if r != rank:
                continue
            s = None
            for t in range(terms):
                v = ref.piece_values(host[t], blocks, b, ln).astype(np.float32)
                s = v if s is None else s + v
            want[pos[p, r]:pos[p, r] + ln] = s / np.float32(world)
        assert np.array_equal(out.cpu().numpy().view(np.uint32), want.view(np.uint32))
        assert (raw[:5] == -77.0).all() and (raw[5 + n:] == -77.0).all()


def test_reduce_carries_nan_and_infinity():
    mp = fs.fs_mx4_plan(fs.fs_plan([(2, 64)], "bf16", 2, False, "fsdp2")).upload()
    s = torch.zeros(2, mp.shard_bytes, dtype=torch.uint8, device="cuda")
    s[0, mp.shard_blocks * 16] = 255                     # block 0 of slice 0: NaN
    s[:, 16] = 0x77                                      # block 1 starts with 6, 6
    s[:, mp.shard_blocks * 16 + 1] = 254                 # times 2^127: over fp32
    out = torch.empty(64, device="cuda")
    fs.fs_reduce_shard_mx4(mp, s, out, rank=0)
    assert torch.isnan(out[:32]).all() and torch.isinf(out[32:34]).all() and (out[34:] == 0).all()


# ------------------------------------------------------------------ products --

def _check_product(a, b, out, m, n, k):
    A, B = _decoded(*a, k), _decoded(*b, k)
    want = A @ B.T if k else np.zeros((m, n))
    tol, half = ref.product_tolerance(A, B, out.dtype == torch.bfloat16)
    got = _f64(out)
    err = np.abs(got - want) - tol - half * (np.abs(want) + tol)
    assert err.max() <= 0, f"off by {np.abs(got - want).max()}"


MNK = [(1, 1, 1), (1, 1, 32), (1, 17, 33), (2, 16, 64), (16, 16, 128), (17, 15, 127), (15, 33, 129), (1, 300, 1000), (33, 64, 160),
       (64, 64, 256), (65, 63, 257), (100, 1, 4000), (128, 128, 512), (127, 129, 480), (130, 260, 1376), (256, 256, 256),
       (257, 300, 1024), (8, 2048, 2048), (3, 1000, 5000), (300, 520, 2080), (512, 256, 130), (31, 96, 7000),
       (900, 1000, 1), (1000, 900, 33), (700, 1100, 480), (1300, 700, 481), (600, 2000, 545), (2500, 3000, 100), (2700, 3100, 700)]


@pytest.mark.parametrize("m,n,k", MNK)
def test_matmul(m, n, k):
    a, b = _random_matrix(m, k, m + 3 * n + 5 * k), _random_matrix(n, k, 7 * m + n + k)
    for dt, pad, shift in ((torch.float32, 0, 0), (torch.bfloat16, 0, 0), (torch.bfloat16, 3, 1), (torch.float32, 5, 3)):
        raw = torch.full((64 + shift + m * (n + pad),), -77.0, dtype=dt, device="cuda")
        out = raw[32 + shift:].as_strided((m, n), (n + pad, 1))
        say("matmul", m, n, k, dt, pad)
        fs.fs_mx4_matmul(fs.Mx4Matrix(*a, k), fs.Mx4Matrix(*b, k), out)
        _check_product(a, b, out, m, n, k)
        out.fill_(-77.0)
        assert (raw == -77.0).all()


@pytest.mark.parametrize("m,n,k", [(1, 70, 96), (40, 33, 224), (200, 260, 544), (260, 300, 1056)])
def test_matmul_with_strides_and_chunks(m, n, k):
    """Rows further apart than their bytes, scales at any byte address, b's rows in chunks."""
    a, b = _random_matrix(m, k, 1), _random_matrix(n, k, 2)
    ga, gb = Guard(m, k, 3), Guard(n, k, 5)
    for g, (c, s) in ((ga, a), (gb, b)):
        g.c.copy_(c)
        g.s.copy_(s)
    out = torch.empty(m, n, device="cuda")
    fs.fs_mx4_matmul(ga.m, gb.m, out)
    _check_product(a, b, out, m, n, k)
    nb = ref.blocks(k)
    for chunk in (1, 16, 33, n - 1):
        count = -(-n // chunk)
        stride = -(-(chunk * 17 * nb + 8) // 16) * 16
        buf = torch.full((count, stride), CANARY, dtype=torch.uint8, device="cuda")
        for c in range(count):
            part = slice(c * chunk, min(n, (c + 1) * chunk))
            cc, ss = b[0][part], b[1][part]
            buf[c, :cc.numel()] = cc.reshape(-1)
            buf[c, chunk * 16 * nb + 5:chunk * 16 * nb + 5 + ss.numel()] = ss.reshape(-1)
        st = fs.Mx4MatrixStruct(buf.data_ptr(), buf.data_ptr() + chunk * 16 * nb + 5, n, k, 16 * nb, nb, chunk, stride)
        say("chunks of", chunk)
        out.fill_(-1)
        fs.fs_mx4_matmul(fs.Mx4Matrix(*a, k), fs.Mx4Matrix._gathered(st, buf), out)
        _check_product(a, b, out, m, n, k)
        outt = torch.empty(n, m, device="cuda")
        fs.fs_mx4_matmul(fs.Mx4Matrix._gathered(st, buf), fs.Mx4Matrix(*a, k), outt)
        _check_product(b, a, outt, n, m, k)


@pytest.mark.parametrize("m,n,k,chunk,stride", [(200, 600, 512, 300, 600 << 20), (2048, 2100, 256, 700, 3 << 30), (3, 600, 512, 300, 3 << 30)])
def test_matmul_with_chunks_far_apart(m, n, k, chunk, stride):
    """Offsets past 31 and 32 bits."""
    a, b = _random_matrix(m, k, 1), _random_matrix(n, k, 2)
    nb, count = k // 32, -(-n // chunk)
    buf = torch.empty((count - 1) * stride + chunk * 17 * nb, dtype=torch.uint8, device="cuda")
    for c in range(count):
        cc, ss = b[0][c * chunk:(c + 1) * chunk], b[1][c * chunk:(c + 1) * chunk]
        at = c * stride
        buf[at:at + cc.numel()] = cc.reshape(-1)
        buf[at + chunk * 16 * nb:at + chunk * 16 * nb + ss.numel()] = ss.reshape(-1)
    st = fs.Mx4MatrixStruct(buf.data_ptr(), buf.data_ptr() + chunk * 16 * nb, n, k, 16 * nb, nb, chunk, stride)
    out, outt = torch.empty(m, n, device="cuda"), torch.empty(n, m, device="cuda")
    say("far chunks", m, n, k)
    fs.fs_mx4_matmul(fs.Mx4Matrix(*a, k), fs.Mx4Matrix._gathered(st, buf), out)
    _check_product(a, b, out, m, n, k)
    fs.fs_mx4_matmul(fs.Mx4Matrix._gathered(st, buf), fs.Mx4Matrix(*a, k), outt)
    _check_product(b, a, outt, n, m, k)
    w = torch.empty(n, k, dtype=torch.bfloat16, device="cuda")
    fs.fs_mx4_dequantize(fs.Mx4Matrix._gathered(st, buf), w)
    assert torch.equal(w.cpu().double(), torch.from_numpy(_decoded(*b, k)))


@pytest.mark.parametrize("m,n,k", [(1, 64, 128), (20, 40, 96), (256, 512, 512), (300, 300, 300), (2100, 2300, 400), (600, 700, 97)])
def test_matmul_special_scales(m, n, k):
    a, b = _random_matrix(m, k, 3), _random_matrix(n, k, 4)
    a[1][m - 1, -1] = 255                                # NaN in a's last row
    b[1][n // 2, 0] = 255                                # and in one of b's
    out = torch.empty(m, n, device="cuda")
    fs.fs_mx4_matmul(fs.Mx4Matrix(*a, k), fs.Mx4Matrix(*b, k), out)
    nan = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    nan[m - 1] = True
    nan[:, n // 2] = True
    assert torch.equal(torch.isnan(out), nan)
    lo, hi = (_random_matrix(m, k, 5, 0, 60), _random_matrix(n, k, 6, 180, 250))      # the products' range, not the factors'
    fs.fs_mx4_matmul(fs.Mx4Matrix(*lo, k), fs.Mx4Matrix(*hi, k), out)
    _check_product(lo, hi, out, m, n, k)
    big = _random_matrix(m, k, 7, 250, 254), _random_matrix(n, k, 8, 250, 254)          # over fp32: infinities or NaN, no fault
    fs.fs_mx4_matmul(fs.Mx4Matrix(*big[0], k), fs.Mx4Matrix(*big[1], k), out)
    assert not torch.isfinite(out[_f64_zero_free(big, k)]).any()


def _f64_zero_free(big, k):
    """Outputs with a term over fp32's range: 2^128 or more after every cancellation is impossible to tell here, so
    only those whose largest single term is over it."""
    A, B = (np.abs(_decoded(*x, k)) for x in big)
    hit = np.array([[(A[i] * B[j]).max() > 2.0 ** 130 for j in range(B.shape[0])] for i in range(min(A.shape[0], 4))])
    full = np.zeros((A.shape[0], B.shape[0]), bool)
    full[:hit.shape[0]] = hit
    return torch.from_numpy(full).cuda()


def test_matmul_of_nothing():
    out = torch.full((5, 7), 3.0, device="cuda")
    fs.fs_mx4_matmul(fs.fs_mx4_empty(5, 0), fs.fs_mx4_empty(7, 0), out)
    assert (out == 0).all()
    fs.fs_mx4_matmul(fs.fs_mx4_empty(0, 64), fs.fs_mx4_empty(7, 64), torch.empty(0, 7, device="cuda"))
    fs.fs_mx4_matmul(fs.fs_mx4_empty(5, 64), fs.fs_mx4_empty(0, 64), torch.empty(5, 0, device="cuda"))


@pytest.mark.parametrize("m,n", [(300, 700), (1100, 1300), (2100, 2300), (5000, 4700)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_matmul_without_columns_at_every_size(m, n, dtype):
    """No term at all: zeros, also where a workgroup takes one tile after the other."""
    say(f"no columns {m} {n} {dtype}")
    out = torch.full((m, n + 3), 3.0, dtype=DT[dtype], device="cuda")
    fs.fs_mx4_matmul(fs.fs_mx4_empty(m, 0), fs.fs_mx4_empty(n, 0), out[:, :n])
    assert (out[:, :n] == 0).all() and (out[:, n:] == 3).all()


@pytest.mark.parametrize("m,n,k", [(2048, 4096, 4096), (1000, 5000, 2304), (4096, 512, 8192), (7, 11008, 4096), (64, 4096, 11008)])
def test_matmul_large_exact_sums(m, n, k):
    """Small integers at one scale: every partial sum is an integer (in units
    of 1/4) below 2^24, so fp32 sums in any order are exact, bit for bit."""
    g = _gen(m + n + k)
    small = torch.tensor([0, 1, 2, 9, 10], device="cuda", dtype=torch.uint8)       # 0, 0.5, 1, -0.5, -1

    def matrix(rows):
        c = small[torch.randint(0, 5, (rows, k), generator=g, device="cuda")]
        return (c[:, 0::2] | (c[:, 1::2] << 4)).contiguous(), torch.full((rows, k // 32), 127, dtype=torch.uint8, device="cuda"), c

    def values(c):
        return torch.tensor([0, .5, 1, 0, 0, 0, 0, 0, 0, -.5, -1], device="cuda")[c.long()]

    (ac, as_, av), (bc, bs, bv) = matrix(m), matrix(n)
    out = torch.empty(m, n, device="cuda")
    fs.fs_mx4_matmul(fs.Mx4Matrix(ac, as_, k), fs.Mx4Matrix(bc, bs, k), out)
    assert torch.equal(out, values(av) @ values(bv).t())


@pytest.mark.parametrize("world,rows,row,other", [(1, 40, 64, 96), (3, 100, 96, 33), (8, 64, 256, 64), (8, 37, 32, 1), (2, 300, 1024, 512)])
def test_gathered_parameters_as_matrices(world, rows, row, other):
    """A weight read where the all-gather left it gives what it gives unpacked and quantised again."""
    shapes = [(other,), (rows, row), (row,), (2, rows, row)]
    mp = fs.fs_mx4_plan(fs.fs_plan(shapes, "bf16", world, False, "fsdp2")).upload()
    params = [_values(s, "bf16", i) for i, s in enumerate(shapes)]
    gathered = torch.empty(mp.gathered_bytes, dtype=torch.uint8, device="cuda")
    fs.fs_pack_mx4(mp, params, gathered)
    outs = [torch.empty_like(p) for p in params]
    fs.fs_unpack_mx4(mp, gathered, outs)
    for i, cols in ((1, row), (3, rows * row)):
        if cols % 32:
            with pytest.raises(fs.FsError, match="whole blocks"):
                mp.matrix(gathered, i)
            continue
        w = mp.matrix(gathered, i)
        d0 = shapes[i][0]
        assert w.shape == (d0, cols)
        plain = torch.empty(d0, cols, dtype=torch.bfloat16, device="cuda")
        fs.fs_mx4_dequantize(w, plain)
        assert torch.equal(plain, outs[i].view(d0, cols))
        x = fs.fs_mx4_empty(5, cols)
        fs.fs_mx4_quantize(_values((5, cols), "bf16", 77, 0.5), x)
        again = fs.fs_mx4_empty(d0, cols)
        again.codes.copy_(_codes_of(params[i].view(d0, cols))[0])
        again.scales.copy_(_codes_of(params[i].view(d0, cols))[1])
        got, want = (torch.empty(5, d0, device="cuda") for _ in range(2))
        fs.fs_mx4_matmul(x, w, got)
        fs.fs_mx4_matmul(x, again, want)
        assert torch.equal(got, want)


def _codes_of(x):
    c, s = ref.encode_matrix(_f64(x))
    return torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda()


def _lossless(shape, seed):
    """Integers of at most 3 in magnitude with a 4 in every block of rows and columns, which quantise without loss."""
    x = torch.randint(-3, 4, shape, generator=_gen(seed), device="cuda").float()
    i, j = torch.meshgrid(torch.arange(shape[0]), torch.arange(shape[1]), indexing="ij")
    x[(i % 32 == j % 32).cuda()] = 4.0
    return x


def test_gradients_of_a_linear_layer():
    """y = x W^T with loss sum(g * y): the three products give the formula's
    gradients, and the differences of the loss (which is linear in each
    factor, and here exact in fp32)."""
    M, N, K = 64, 96, 128
    x, w, g = _lossless((M, K), 1), _lossless((N, K), 2), _lossless((M, N), 3)

    def q(t):
        r, c = fs.fs_mx4_empty(*t.shape), fs.fs_mx4_empty(t.shape[1], t.shape[0])
        fs.fs_mx4_quantize(t, r, c)
        return r, c

    def product(a, b):
        out = torch.empty(a.shape[0], b.shape[0], device="cuda")
        fs.fs_mx4_matmul(a, b, out)
        return out

    (xr, xc), (wr, wc), (gr, gc) = q(x), q(w), q(g)
    y, dx, dw = product(xr, wr), product(gr, wc), product(gc, xc)
    X, W, G = (t.double() for t in (x, w, g))
    assert torch.equal(y.double(), X @ W.t()) and torch.equal(dx.double(), G @ W) and torch.equal(dw.double(), G.t() @ X)

    def loss(xx, ww):
        return (G * product(q(xx)[0], q(ww)[0]).double()).sum().item()

    base = loss(x, w)
    for i, j in ((0, 1), (5, 40), (63, 126)):
        x2 = x.clone()
        x2[i, j] = 4.0 if x[i, j] < 4 else 3.0        # stays lossless: a 4 is left in every other block position
        if i % 32 != j % 32:
            assert loss(x2, w) - base == (x2[i, j] - x[i, j]).item() * dx[i, j].item()
    for i, j in ((1, 0), (33, 70), (95, 2)):
        w2 = w.clone()
        w2[i, j] = 4.0
        assert loss(x, w2) - base == (4.0 - w[i, j]).item() * dw[i, j].item()


# ------------------------------------------------------- graphs, streams, use --

def _step_buffers():
    shapes = [(64,), (96, 64), (64, 96), (96,)]
    world, acc = 4, 2
    plan = fs.fs_plan(shapes, "bf16", world, False, "fsdp2", acc)
    mp = fs.fs_mx4_plan(plan).upload()
    return shapes, world, acc, plan, mp


def test_training_step_in_four_bits():
    """Copy-in, products on the gathered weights, their gradients, the copy-in
    of every rank's gradients with random rounding, the reduce and AdamW,
    against the same chain in 64 bits (quantisation and reduce bit for bit)."""
    shapes, world, acc, plan, mp = _step_buffers()
    pieces, blocks, nbytes = ref.layout(plan.segments(), [(plan.param(i).chunk_rows, plan.param(i).row) for i in range(4)],
                                        "fsdp2", world, 4)
    params = [_values(s, "bf16", i, 0.5) for i, s in enumerate(shapes)]
    gathered = torch.empty(mp.gathered_bytes, dtype=torch.uint8, device="cuda")
    fs.fs_pack_mx4(mp, params, gathered)
    w_up, w_down = mp.matrix(gathered, 1), mp.matrix(gathered, 2)
    slices, hosts, rank, tokens = [], [], 2, 40
    for t in range(world * acc):
        x = _values((tokens, 64), "bf16", 50 + t, 0.5)
        xr, xc = fs.fs_mx4_empty(tokens, 64), fs.fs_mx4_empty(64, tokens)
        fs.fs_mx4_quantize(x, xr, xc)
        h = torch.empty(tokens, 96, dtype=torch.bfloat16, device="cuda")
        fs.fs_mx4_matmul(xr, w_up, h)
        hr, hc = fs.fs_mx4_empty(tokens, 96), fs.fs_mx4_empty(96, tokens)
        fs.fs_mx4_quantize(h, hr, hc)
        y = torch.empty(tokens, 64, device="cuda")
        fs.fs_mx4_matmul(hr, w_down, y)
        # loss = sum(y^2) / 2: dy = y; the weights' gradients contract over tokens
        dr, dc = fs.fs_mx4_empty(tokens, 64), fs.fs_mx4_empty(64, tokens)
        fs.fs_mx4_quantize(y, dr, dc, seed=_seed(t))
        dw_down = torch.empty(64, 96, device="cuda")
        fs.fs_mx4_matmul(dc, hc, dw_down)
        H, X = _decoded(hr.codes, hr.scales, 96), _decoded(xr.codes, xr.scales, 64)
        W2 = np.concatenate([ref.piece_values(gathered.cpu().numpy().reshape(world, -1)[r], blocks, pieces[2, r][0], pieces[2, r][2])
                             for r in range(world)]).reshape(64, 96)
        want = H @ W2.T
        tol, _ = ref.product_tolerance(H, W2, False)
        assert (np.abs(_f64(y) - want) <= tol).all()
        D, Hc = _decoded(dc.codes, dc.scales, tokens), _decoded(hc.codes, hc.scales, tokens)
        tol, _ = ref.product_tolerance(D, Hc, False)
        assert (np.abs(_f64(dw_down) - D @ Hc.T) <= tol).all()
        grads = [torch.randn(64, device="cuda"), torch.randn(96, 64, device="cuda"), dw_down, torch.randn(96, device="cuda")]
        s = torch.empty(mp.shard_bytes, dtype=torch.uint8, device="cuda")
        fs.fs_pack_mx4(mp, grads, s, rank=rank, seed=_seed(1000 + t))
        host = ref.pack(pieces, blocks, nbytes, world, [_f64(v).reshape(-1) for v in grads], 1000 + t)[rank]
        assert np.array_equal(s.cpu().numpy(), host)
        slices.append(s)
        hosts.append(host)
    n = plan.shard_numel
    g32 = torch.empty(n, device="cuda")
    fs.fs_reduce_shard_mx4(mp, slices, g32, rank=rank, grad_acc=acc)
    want = np.zeros(n, np.float32)
    for dst, _, ln, p, r in plan.segments():
        if r == rank:
            total = None
            for host in hosts:
                v = ref.piece_values(host, blocks, pieces[p, r][0], ln).astype(np.float32)
                total = v if total is None else total + v
            want[dst - r * n:dst - r * n + ln] = total / np.float32(world)
    assert np.array_equal(g32.cpu().numpy(), want)
    master, m, v = (torch.zeros(n, device="cuda") for _ in range(3))
    fs.fs_adamw_step(master, m, v, g32, None, lr=1e-2, weight_decay=0.0, step=1)
    g = want.astype(np.float64)     # step 1 from zero state: theta = -lr * g / (|g| + eps')
    expect = -np.float64(np.float32(1e-2)) * g / (np.abs(g) + 1e-8)
    assert np.allclose(master.cpu().numpy(), expect, rtol=1e-5, atol=1e-9)


def test_captured_step_replays_with_new_values():
    shapes, world, acc, plan, mp = _step_buffers()
    params = [_values(s, "bf16", i) for i, s in enumerate(shapes)]
    outs = [torch.empty_like(p) for p in params]
    gathered = torch.empty(mp.gathered_bytes, dtype=torch.uint8, device="cuda")
    slices = torch.empty(world * acc, mp.shard_bytes, dtype=torch.uint8, device="cuda")
    g32 = torch.empty(plan.shard_numel, device="cuda")
    seed = _seed(5)
    x, xq, xc = _values((33, 64), "bf16", 9), fs.fs_mx4_empty(33, 64), fs.fs_mx4_empty(64, 33)
    y = torch.empty(33, 96, device="cuda")
    w = mp.matrix(gathered, 1)
    wide, tall = fs.fs_mx4_empty(300, 4096), fs.fs_mx4_empty(260, 4096)
    for q, s in ((wide, 1), (tall, 2)):
        c, sc = _random_matrix(*q.shape, s)
        q.codes.copy_(c)
        q.scales.copy_(sc)
    big = torch.empty(300, 260, device="cuda")

    def step():
        fs.fs_pack_mx4(mp, params, gathered, seed=seed)
        fs.fs_unpack_mx4(mp, gathered, outs)
        fs.fs_mx4_quantize(x, xq, xc, seed=seed)
        fs.fs_mx4_matmul(xq, w, y)
        fs.fs_mx4_matmul(wide, tall, big)
        for k in range(world * acc):
            fs.fs_pack_mx4(mp, params, slices[k], rank=1, seed=seed)
        fs.fs_reduce_shard_mx4(mp, slices, g32, rank=1, grad_acc=acc)

    def state():
        return [t.clone() for t in (gathered, *outs, xq.codes, xc.codes, y, big, g32)]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    seen = []
    for k in range(4):
        seed.fill_(100 + k)
        x.copy_(_values((33, 64), "bf16", 20 + k))
        wide.scales.fill_(120 + k)
        graph.replay()
        got = state()
        step()
        torch.cuda.synchronize()
        want = state()
        assert all(torch.equal(p, q) for p, q in zip(got, want)), f"replay {k}"
        seen.append(got[0])
    assert not torch.equal(seen[0], seen[1])


def test_two_captured_graphs_at_once():
    """Two graphs of the same calls on the same plan, each into buffers of its own, replayed side by side on
    two streams; a second upload comes between their captures."""
    shapes, world, acc, plan, _ = _step_buffers()
    mp = fs.fs_mx4_plan(plan).upload()
    params = [_values(s, "bf16", i) for i, s in enumerate(shapes)]
    quantised = _random_matrix(300, 2048, 1), _random_matrix(200, 2048, 2)
    a, b = (fs.Mx4Matrix(*q, 2048) for q in quantised)
    sets = [(torch.empty(mp.gathered_bytes, dtype=torch.uint8, device="cuda"), torch.empty(plan.shard_numel, device="cuda"),
             torch.empty(300, 200, device="cuda"), fs.fs_mx4_empty(300, 200), fs.fs_mx4_empty(200, 300), _seed(k))
            for k in range(2)]

    def step(gathered, g32, out, row, col, seed):
        fs.fs_pack_mx4(mp, params, gathered, seed=seed)
        fs.fs_reduce_shard_mx4(mp, [gathered[:mp.shard_bytes]] * (world * acc), g32, rank=0, grad_acc=acc)
        fs.fs_mx4_matmul(a, b, out)
        fs.fs_mx4_quantize(out, row, col, seed=seed)

    def state(s):
        return [t.clone() for t in (s[0], s[1], s[2], s[3].codes, s[3].scales, s[4].codes, s[4].scales)]

    want = []
    for s in sets:
        step(*s)
        want.append(state(s))
    torch.cuda.synchronize()
    graphs, streams = [torch.cuda.CUDAGraph() for _ in sets], [torch.cuda.Stream() for _ in sets]
    for g, s in zip(graphs, sets):
        with torch.cuda.graph(g):
            step(*s)
        mp.upload()
    for turn in range(4):
        for s in sets:
            for t in (s[0], s[1], s[2], s[3].codes, s[4].codes):
                t.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            for g, st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    g.replay()
        torch.cuda.synchronize()
        for k, s in enumerate(sets):
            assert all(torch.equal(p, q) for p, q in zip(state(s), want[k])), f"turn {turn}, graph {k}"


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("cols", [33, 4096])
def test_one_row_has_no_stride(dtype, cols):
    """The strides of matrices of one row are not looked at: here ones that no larger matrix could have."""
    nb = ref.blocks(cols)
    x = _values((1, cols), dtype, 3)
    codes = torch.empty(16 * nb, dtype=torch.uint8, device="cuda").as_strided((1, 16 * nb), (5, 1))
    scales = torch.empty(nb, dtype=torch.uint8, device="cuda").as_strided((1, nb), (0, 1))
    q, out = fs.Mx4Matrix(codes, scales, cols), torch.empty(cols, device="cuda").as_strided((1, cols), (1, 1))
    fs.fs_mx4_quantize(x.as_strided((1, cols), (7, 1)), q)
    c, s = ref.encode_matrix(_f64(x))
    assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scales.cpu().numpy(), s)
    fs.fs_mx4_dequantize(q, out)
    assert np.array_equal(_f64(out), _decoded(codes, scales, cols))
    y = torch.empty(1, dtype=torch.float32, device="cuda").as_strided((1, 1), (0, 1))
    fs.fs_mx4_matmul(q, q, y)
    _check_product((codes, scales), (codes, scales), y, 1, 1, cols)


def test_other_streams_and_threads():
    """Each thread on its own stream, each with its own buffers, gives the single-threaded results."""
    shapes, world, acc, plan, _ = _step_buffers()
    a, b = _random_matrix(300, 2048, 1), _random_matrix(200, 2048, 2)

    def work(k, stream):
        mp = fs.fs_mx4_plan(plan2[k]).upload()
        params = [_values(s, "bf16", 10 * k + i) for i, s in enumerate(shapes)]
        gathered = torch.empty(mp.gathered_bytes, dtype=torch.uint8, device="cuda")
        out = torch.empty(300, 200, device="cuda")
        A, B = fs.Mx4Matrix(*a, 2048), fs.Mx4Matrix(*b, 2048)
        for _ in range(20):
            fs.fs_pack_mx4(mp, params, gathered, seed=seeds[k], stream=stream)
            fs.fs_mx4_matmul(A, B, out, stream=stream)
        torch.cuda.synchronize()
        return gathered, out

    plan2 = [fs.fs_plan(shapes, "bf16", world, False, "fsdp2", acc) for _ in range(8)]
    seeds = [_seed(k) for k in range(4)]
    torch.cuda.synchronize()
    want = [work(k, None) for k in range(4)]
    plan2 = [fs.fs_plan(shapes, "bf16", world, False, "fsdp2", acc) for _ in range(8)]
    got, errors = [None] * 4, []

    def run(k):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                got[k] = work(k, s if k % 2 else None)
        except Exception as e:     # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for g, w in zip(got, want):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


def test_refusals_on_the_gpu():
    """What needs an uploaded plan to be reached; nothing is launched."""
    plan = fs.fs_plan([(8, 64)], "bf16", 2, False, "fsdp2")
    mp = fs.fs_mx4_plan(plan).upload()
    L, P, O = fs.lib(), 1 << 20, 1 << 30
    for args, code in (((P, 0, O, 2, None, None), fs.FS_E_INVAL), ((P, 0, O, -2, None, None), fs.FS_E_INVAL),
                       ((P, 2, O, -1, None, None), fs.FS_E_DTYPE), ((P, 0, O + 8, -1, None, None), fs.FS_E_ALIGN),
                       ((P, 0, None, -1, None, None), fs.FS_E_INVAL), ((None, 0, O, -1, None, None), fs.FS_E_INVAL),
                       ((P, 0, O, -1, O + 16, None), fs.FS_E_INVAL), ((P, 0, O, -1, P + 4, None), fs.FS_E_ALIGN)):
        assert L.fs_pack_mx4(mp._h, *args) == code
    for args, code in (((None, P, 0, None), fs.FS_E_INVAL), ((O, None, 0, None), fs.FS_E_INVAL),
                       ((O + 4, P, 0, None), fs.FS_E_ALIGN), ((O, P, 7, None), fs.FS_E_DTYPE)):
        assert L.fs_unpack_mx4(mp._h, *args) == code

    def reduce(rank=0, acc=1, ptrs=(O, O + 4096), out=P):
        return L.fs_reduce_shard_mx4(mp._h, rank, acc, (ctypes.c_void_p * len(ptrs))(*ptrs), out, None)

    for kw, code in ((dict(rank=2), fs.FS_E_INVAL), (dict(rank=-1), fs.FS_E_INVAL), (dict(acc=0), fs.FS_E_INVAL),
                     (dict(ptrs=(O, None)), fs.FS_E_INVAL), (dict(ptrs=(O, O + 8)), fs.FS_E_ALIGN), (dict(out=None), fs.FS_E_INVAL),
                     (dict(out=P + 2), fs.FS_E_ALIGN), (dict(out=O + 64), fs.FS_E_INVAL)):
        assert reduce(**kw) == code
    ws = mp.workspace
    assert mp.upload().workspace is ws and mp.upload(device=ws.device).workspace is ws      # there already
    host = torch.empty(1 << 12, dtype=torch.uint8)
    assert L.fs_mx4_plan_upload(mp._h, (host.data_ptr() + 15) & ~15, 3000, None) == fs.FS_E_INVAL
    with pytest.raises(ValueError, match="no longer"):
        m = fs.fs_mx4_empty(4, 64)
        m.codes.set_(torch.zeros(4, 32, dtype=torch.uint8, device="cuda"))
        fs.fs_mx4_dequantize(m, torch.empty(4, 64, device="cuda"))
