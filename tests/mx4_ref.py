"""Plain 64-bit definitions of the microscaled 4-bit format for the tests:
blocks of 32 e2m1 elements with an e8m0 scale, written from the format's
definition with numpy, without the library."""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK, PIECE, LINE = 32, 8, 128


def blocks(n):
    return -(-n // BLOCK)


def philox(seed, groups, orientation):
    """Philox4x32 with 7 rounds: the output words of each group, as (n, 4) uint64 of 32 bits."""
    m32 = np.uint64(0xFFFFFFFF)
    g = np.asarray(groups, dtype=np.uint64)
    c = [g & m32, g >> np.uint64(32), np.full_like(g, orientation), np.zeros_like(g)]
    k = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for _ in range(7):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), p1 & m32,
             (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), p0 & m32]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, -1)


def random16(seed, block_index, orientation):
    """(n, 32) random 16-bit numbers of the blocks with these indices."""
    idx = np.asarray(block_index, dtype=np.uint64)
    w = philox(seed, idx[:, None] * np.uint64(4) + np.arange(4, dtype=np.uint64), orientation)   # (n, 4 groups, 4 words)
    return np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], -1).reshape(len(idx), BLOCK).astype(np.int64)


def encode(x, seed=None, block_index=None, orientation=0):
    """(n, 32) float64 (values of fp32 or bf16) -> codes (n, 16) uint8, scales (n,) uint8."""
    x = np.asarray(x, dtype=np.float64)
    amax = np.abs(x).max(1)
    finite = np.isfinite(amax)
    safe = np.where(finite, amax, 0)
    frac, ex = np.frexp(safe)                    # safe = frac * 2^ex, frac in [0.5, 1)
    e = np.where(safe > 0, np.maximum(ex - 3, -127), -127)
    if seed is not None:
        e = e + ((frac > 0.75) & (ex - 3 >= -127) & (safe > 0))
    y = np.ldexp(np.where(finite[:, None], np.abs(x), 0), -e[:, None])
    if seed is None:
        code = np.zeros(x.shape, np.int64)
        for i in range(7):                       # past the midpoint; on it where the upper index is even
            mid = (GRID[i] + GRID[i + 1]) / 2
            code += (y >= mid) if i % 2 else (y > mid)
    else:
        assert y.max(initial=0) <= 6
        low = np.minimum(np.searchsorted(GRID, y, side="right") - 1, 6)
        f = (y - GRID[low]) / (GRID[low + 1] - GRID[low])
        code = low + (f > (random16(seed, block_index, orientation) + 0.5) / 65536)
    code = code + 8 * np.signbit(x)
    code[~finite] = 0
    code = code.astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), np.where(finite, e + 127, 255).astype(np.uint8)


def decode(codes, scales):
    """codes (..., 16 a block), scales (..., blocks) -> float64 values (..., 32 a block)."""
    codes, scales = np.asarray(codes), np.asarray(scales)
    c = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[:-1] + (-1,))
    v = np.where(c & 8, -1.0, 1.0) * GRID[c & 7]
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return v * np.repeat(s, BLOCK, axis=-1)


def encode_matrix(x, seed=None, orientation=0):
    """Row blocks of a matrix: codes (rows, 16*nb), scales (rows, nb)."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    nb = blocks(cols)
    full = np.zeros((rows, nb * BLOCK))
    full[:, :cols] = x
    c, s = encode(full.reshape(-1, BLOCK), seed, np.arange(rows * nb), orientation)
    return c.reshape(rows, nb * 16), s.reshape(rows, nb)


def layout(segments, params, mode, world, n_params):
    """The quantised shards of a plan, from its segments (dst, src, len, param, rank): pieces {(param, rank):
    (first block, source element, count)} and the shard's blocks and bytes.  params: (chunk_rows, row)."""
    up = lambda n: -(-n // PIECE) * PIECE    # noqa: E731
    pieces, total = {}, 0
    if mode == "fsdp2":
        first = []
        for chunk, row in params:
            first.append(total)
            total += up(blocks(chunk * row))
        for _, src, ln, p, r in segments:
            pieces[p, r] = (first[p], src, ln)
    else:
        used = [0] * world
        for _, src, ln, p, r in sorted(segments):
            pieces[p, r] = (used[r], src, ln)
            used[r] += up(blocks(ln))
        total = max(used, default=0)
    return pieces, total, -(-17 * total // LINE) * LINE


def pack(pieces, shard_blocks, shard_bytes, world, params, seed=None):
    """The gathered buffer (world, shard_bytes) of flat float64 parameters."""
    out = np.zeros((world, shard_bytes), np.uint8)
    for (p, r), (b, src, n) in pieces.items():
        nb = blocks(n)
        x = np.zeros(nb * BLOCK)
        x[:n] = params[p][src:src + n]
        c, s = encode(x.reshape(-1, BLOCK), seed, r * shard_blocks + b + np.arange(nb))
        out[r, b * 16:(b + nb) * 16] = c.reshape(-1)
        out[r, shard_blocks * 16 + b:shard_blocks * 16 + b + nb] = s
    return out


def piece_values(shard, shard_blocks, b, n):
    """Float64 values of a piece of n elements in one rank's shard bytes."""
    nb = blocks(n)
    return decode(shard[b * 16:(b + nb) * 16], shard[shard_blocks * 16 + b:shard_blocks * 16 + b + nb])[:n]


def product_tolerance(a, b, bf16):
    """How far a product may be off, elementwise.  Every product of two
    elements is exact (two significant bits each); a sum of K of them in fp32,
    in any order, with each of its K - 1 additions off by at most a whole
    step (2^-23 of the partial sum, itself at most the sum of magnitudes),
    is off by (K - 1) * 2^-23 * sum |a||b| to first order; 2^-22 covers the
    rest.  A bf16 result is rounded once more by half a step, 2^-8."""
    mag = np.abs(a) @ np.abs(b).T
    tol = max(a.shape[1] - 1, 0) * 2.0 ** -22 * mag
    return tol, (2.0 ** -8 if bf16 else 0.0)
