"""Large products of 4-bit matrices on data: a workgroup that takes tile after
tile, and operands with strides, chunks and scales at any address.  Small
values at a few scales, so that every partial sum is exact in fp32 whatever its
order: the results have to be equal, not close.

Sizes by the dispatch rule for 256 CUs: 1100 by 1300 takes tiles of 128 by 128;
4200 by 4400, 4500 by 4700 and 2400 by 3900 take 256 by 256 (306, 342 and 160 tiles, of
which the first two are more than there are workgroups)."""
import pytest
import torch

import fsdp_sharded_state_amd as fs
import mx4_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu

CANARY = 0xA5
SMALL = [0, 1, 2, 9, 10]                # 0, 0.5, 1, -0.5, -1
VALUES = {0: 0.0, 1: 0.5, 2: 1.0, 9: -0.5, 10: -1.0}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _matrix(rows, k, seed):
    """Codes (rows, 16 a block), scales of 2^-1 to 2^1, and the values (rows, k).  A product's terms are multiples of
    1/16 of at most 4: sums of up to 2^18 of them are exact in fp32."""
    g, nb = _gen(seed), ref.blocks(k)
    c = torch.tensor(SMALL, dtype=torch.uint8, device="cuda")[torch.randint(0, 5, (rows, nb * 32), generator=g, device="cuda")]
    c[:, k:] = 0
    s = torch.randint(126, 129, (rows, nb), generator=g, device="cuda").to(torch.uint8)
    table = torch.zeros(16, device="cuda")
    for code, v in VALUES.items():
        table[code] = v
    v = table[c.long()] * torch.exp2(s.float() - 127).repeat_interleave(32, 1)
    return (c[:, 0::2] | (c[:, 1::2] << 4)).contiguous(), s, v[:, :k].contiguous()


def _plain(m, k):
    return fs.Mx4Matrix(m[0], m[1], k)


def _out(m, n, dtype, pad, shift):
    raw = torch.full((64 + shift + m * (n + pad),), -77.0, dtype=dtype, device="cuda")
    return raw, raw[32 + shift:].as_strided((m, n), (n + pad, 1))


def _equal(raw, out, want, label):
    want = want.to(out.dtype)
    bad = out != want
    assert not bad.any(), f"{label}: {int(bad.sum())} differ, first at {bad.nonzero()[0].tolist()}"
    out.fill_(-77.0)
    assert (raw == -77.0).all(), f"{label}: written outside the output"


def test_sums_are_exact_as_said():
    assert 2 ** 18 * 4 * 16 <= 2 ** 24


# k of one group of 16 blocks (fewer and all of them, a last one partly filled), of two, three and seven.
@pytest.mark.parametrize("m,n", [(4500, 4700), (4200, 4400), (2400, 3900)])
@pytest.mark.parametrize("k", [32, 40, 480, 500, 512, 513, 1000, 1500, 3500])
def test_tile_after_tile(m, n, k):
    a, b = _matrix(m, k, m + k), _matrix(n, k, n + 2 * k)
    want = a[2] @ b[2].t()
    for dtype, pad, shift in ((torch.float32, 0, 0), (torch.bfloat16, 0, 0), (torch.bfloat16, 4, 0), (torch.bfloat16, 3, 1), (torch.float32, 5, 3)):
        say("tile after tile", m, n, k, dtype, pad, shift)
        raw, out = _out(m, n, dtype, pad, shift)
        fs.fs_mx4_matmul(_plain(a, k), _plain(b, k), out)
        _equal(raw, out, want, f"{dtype} pad {pad} shift {shift}")


@pytest.mark.parametrize("k", [500, 1500])
def test_nan_of_one_row_stays_in_its_row(k):
    """Also in tiles that a workgroup takes second, whose scales are loaded while the first are in use."""
    m, n = 4500, 4700
    a, b = _matrix(m, k, 1), _matrix(n, k, 2)
    want = a[2] @ b[2].t()
    for row, col in ((0, n - 1), (m - 1, 0), (2305, 4444), (4300, 2500)):
        a2, b2 = a[1].clone(), b[1].clone()
        a2[row, -1] = 255
        b2[col, 0] = 255
        say("nan", k, row, col)
        out = torch.empty(m, n, device="cuda")
        fs.fs_mx4_matmul(fs.Mx4Matrix(a[0], a2, k), fs.Mx4Matrix(b[0], b2, k), out)
        w = want.clone()
        w[row] = float("nan")
        w[:, col] = float("nan")
        assert torch.equal(out.isnan(), w.isnan()) and torch.equal(out.nan_to_num(7.0), w.nan_to_num(7.0))


def _laid_out(m, k, chunk, code_stride=None, scale_more=0, shift=0, chunk_stride=None):
    """The matrix with its rows in chunks (0: one run), code rows code_stride apart, scale rows scale_more bytes further
    apart than their blocks, and the scales `shift` bytes after the codes' end: (Mx4Matrix, the buffer)."""
    codes, scales, _ = m
    rows, nb = scales.shape
    cs, ss = code_stride or 16 * nb, nb + scale_more
    run = min(chunk, rows) if chunk else rows
    count = -(-rows // run)
    bytes_ = run * cs + shift + run * ss
    stride = chunk_stride or -(-bytes_ // 16) * 16
    assert stride >= bytes_ and stride % 16 == 0
    buf = torch.empty((count - 1) * stride + bytes_, dtype=torch.uint8, device="cuda")
    if buf.numel() < 1 << 30:
        buf.fill_(CANARY)
    for c in range(count):
        part = slice(c * run, min(rows, (c + 1) * run))
        here = min(rows, (c + 1) * run) - c * run
        at = c * stride
        buf[at:].as_strided((here, 16 * nb), (cs, 1)).copy_(codes[part])
        buf[at + run * cs + shift:].as_strided((here, nb), (ss, 1)).copy_(scales[part])
    st = fs.Mx4MatrixStruct(buf.data_ptr(), buf.data_ptr() + run * cs + shift, rows, k, cs, ss, chunk, stride if chunk else 0)
    return fs.Mx4Matrix._gathered(st, buf)


@pytest.mark.parametrize("m,n", [(1100, 1300), (4200, 4400)])
@pytest.mark.parametrize("k", [96, 1000, 1504])
def test_strides_and_chunks(m, n, k):
    """Chunks of one row, of ones that divide neither 128 nor 256, with a last one partly filled, of all rows and more."""
    a, b, nb = _matrix(m, k, 3), _matrix(n, k, 4), ref.blocks(k)
    want = a[2] @ b[2].t()
    raw, out = _out(m, n, torch.float32, 0, 0)
    for chunk, more, scale_more, shift in ((0, 3, 5, 7), (1, 0, 0, 3), (33, 1, 0, 0), (300, 0, 2, 9), (256, 0, 0, 0), (n - 1, 2, 1, 13), (n + 5, 0, 0, 1)):
        say("b in chunks of", chunk, m, n, k)
        lb = _laid_out(b, k, chunk, 16 * (nb + more), scale_more, shift)
        fs.fs_mx4_matmul(_plain(a, k), lb, out)
        _equal(raw, out, want, f"b in chunks of {chunk}")
        say("a in chunks of", chunk, m, n, k)
        la = _laid_out(a, k, chunk, 16 * (nb + more), scale_more, shift)
        fs.fs_mx4_matmul(la, lb, out)
        _equal(raw, out, want, f"a and b in chunks of {chunk}")


@pytest.mark.parametrize("m,n", [(1100, 1300), (4200, 4400)])
@pytest.mark.parametrize("chunk,code_stride,chunk_stride", [
    (0, (4 << 20) - 16, None), (0, 4 << 20, None),                  # rows as far apart as 32-bit offsets hold, and further
    (300, None, (512 << 20) - 16), (300, None, 512 << 20),          # chunks, of which 256 rows lie in two
    (33, 1 << 20, (64 << 20) - 128), (33, 1 << 20, 64 << 20),       # in nine
])
def test_rows_at_the_reach_of_offsets(m, n, chunk, code_stride, chunk_stride):
    """On either side of the rule that the large shapes' 32-bit offsets set."""
    if chunk == 33 and m > 2000:
        m, n = 2400, 3900                                           # (119 chunks of 64 MB)
    k = 480
    a, b = _matrix(m, k, 5), _matrix(n, k, 6)
    want = a[2] @ b[2].t()
    raw, out = _out(m, n, torch.float32, 0, 0)
    far = _laid_out(b, k, chunk, code_stride, 1, 5, chunk_stride)
    say("far rows", m, n, chunk, code_stride, chunk_stride)
    fs.fs_mx4_matmul(_plain(a, k), far, out)
    _equal(raw, out, want, "b")
    raw, out = _out(n, m, torch.float32, 0, 0)
    fs.fs_mx4_matmul(far, _plain(a, k), out)
    _equal(raw, out, want.t(), "a")
    del far
    torch.cuda.empty_cache()


@pytest.mark.parametrize("world", [1, 3, 8])
@pytest.mark.parametrize("m,n", [(1100, 1300), (4200, 4400)])
def test_a_gathered_weight_in_a_large_product(world, m, n):
    k = 1024
    shapes = [(k,), (n, k), (33,)]
    w = torch.tensor([0, .5, 1, -.5, -1], device="cuda")[torch.randint(0, 5, (n, k), generator=_gen(7), device="cuda")]
    params = [torch.ones(k, device="cuda"), w, torch.ones(33, device="cuda")]
    mp = fs.fs_mx4_plan(fs.fs_plan(shapes, "bf16", world, False, "fsdp2")).upload()
    gathered = torch.empty(mp.gathered_bytes, dtype=torch.uint8, device="cuda")
    fs.fs_pack_mx4(mp, params, gathered)        # multiples of a half up to 1 lose nothing
    a = _matrix(m, k, 8)
    raw, out = _out(m, n, torch.bfloat16, 0, 0)
    say("gathered weight", world, m, n)
    fs.fs_mx4_matmul(_plain(a, k), mp.matrix(gathered, 1), out)
    _equal(raw, out, a[2] @ w.t(), "x W^T")
    raw, out = _out(n, m, torch.float32, 0, 0)
    fs.fs_mx4_matmul(mp.matrix(gathered, 1), _plain(a, k), out)
    _equal(raw, out, w @ a[2].t(), "W x^T")
