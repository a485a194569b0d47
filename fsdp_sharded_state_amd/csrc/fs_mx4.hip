// fs_mx4.hip -- quantising and dequantising in blocks of 32 4-bit elements:
// matrices, and the shards of a group (copy-in, copy-out and the reduce of
// quantised slices).
#include <string.h>

#include "fs_mx4.h"

using namespace fsi;

namespace {

constexpr int kQuads = kThreads / 4;                       // blocks a workgroup handles at a time
constexpr int kTileSteps = kMx4TileBlocks / kQuads;        // a lane's quarters of a tile
static_assert(kTileSteps * kQuads == kMx4TileBlocks, "a tile is whole steps");
static_assert(kThreads >= kMx4TileBlocks, "a thread for every block of a tile or pad");

// The waves of a workgroup that exchange units through LDS: those of fp32 elements, the others need none.
template <class T>
constexpr int kWavesExchanging = kUnits<T> > 1 ? kThreads / 64 : 1;

// ------------------------------------------------------------------ shards --

// Copy-in: a tile a workgroup, all its loads on their way before the first block is made.  Its codes and scales
// go through LDS: 16 bytes a lane are stored for the four that a lane makes at a time, and four scales
// for one.  HBM bounds it: one 7B block in bf16 78 to 81 us, 6.3 to 6.6 TB/s, with its buffers again and again, 94 with
// buffers in turn that are in no cache.  At random 97 and 98: there the vector instructions do.
template <class T, bool STOCHASTIC>
__global__ __launch_bounds__(kThreads) void pack_mx4_kernel(const Mx4Tile *__restrict__ tiles, uint32_t ntiles,
                                                            const Mx4Run *__restrict__ pads,
                                                            const void *const *__restrict__ params,
                                                            uint8_t *__restrict__ out, int32_t first_rank,
                                                            int64_t shard_blocks, int64_t shard_bytes,
                                                            const uint64_t *__restrict__ seed_at) {
    __shared__ u32x4 lds_units[kWavesExchanging<T>][128];
    __shared__ __attribute__((aligned(16))) uint32_t lds_codes[kMx4TileBlocks * 4];
    __shared__ __attribute__((aligned(4))) uint8_t lds_scales[kMx4TileBlocks];
    const int tid = threadIdx.x;
    if (blockIdx.x >= ntiles) {   // blocks of no piece, or the bytes after the last scale
        const Mx4Run run = pads[blockIdx.x - ntiles];
        uint8_t *shard = out + (run.rank - first_rank) * shard_bytes;
        if (run.n == 0) {
            const int64_t end = shard_blocks * (kMx4BlockBytes + 1);
            for (int64_t k = end + tid; k < shard_bytes; k += kThreads) shard[k] = 0;
        } else if (tid < run.n) {
            *reinterpret_cast<u32x4 *>(shard + (run.at + tid) * kMx4BlockBytes) = u32x4{0, 0, 0, 0};
            shard[shard_blocks * kMx4BlockBytes + run.at + tid] = 0;
        }
        return;
    }
    const Mx4Tile t = tiles[blockIdx.x];
    const T *src = static_cast<const T *>(params[t.param]) + t.src;
    const uint64_t seed = STOCHASTIC ? *seed_at : 0;
    const uint64_t group = 4 * (uint64_t)(t.rank * shard_blocks + t.blk);
    constexpr int U = kUnits<T>, E = kUnit<T>;
    const int first = (tid & ~63) * U + (tid & 63);
    u32x4 v[kTileSteps][U];
    with_past(on16(src), [&](auto past) {
#pragma unroll
        for (int i = 0; i < kTileSteps; ++i)
#pragma unroll
            for (int h = 0; h < U; ++h) {
                const int at = E * (i * kThreads * U + first + 64 * h);
                v[i][h] = load_unit<past>(src + at, t.n - at);
            }
    });
#pragma unroll
    for (int i = 0; i < kTileSteps; ++i) {
        const int q = i * kThreads + tid;
        const Raw8<T> r = own_units(v[i], lds_units[U > 1 ? tid >> 6 : 0]);
        uint32_t s;
        lds_codes[q] = encode8<STOCHASTIC>(r, seed, group + q, 0, &s);
        if ((tid & 3) == 0) lds_scales[q >> 2] = (uint8_t)s;
    }
    __syncthreads();
    uint8_t *shard = out + (t.rank - first_rank) * shard_bytes;
    if (tid < t.nblk)
        *reinterpret_cast<u32x4 *>(shard + (t.blk + tid) * kMx4BlockBytes) = *reinterpret_cast<const u32x4 *>(lds_codes + 4 * tid);
    if (4 * tid < t.nblk)   // whole words: blocks come in eights
        *reinterpret_cast<uint32_t *>(shard + shard_blocks * kMx4BlockBytes + t.blk + 4 * tid) =
            *reinterpret_cast<const uint32_t *>(lds_scales + 4 * tid);
}

// Copy-out: a lane makes 16 bytes of values at a time, whole cache lines a wave.  HBM bounds it: one 7B block in bf16
// 73 to 75 us, 6.8 to 7.0 TB/s, again and again or right after its copy-in; 99, 5.2 TB/s, with buffers in turn.
template <class T>
__global__ __launch_bounds__(kThreads) void unpack_mx4_kernel(const Mx4Tile *__restrict__ tiles,
                                                              const uint8_t *__restrict__ gathered,
                                                              void *const *__restrict__ params, int64_t shard_blocks,
                                                              int64_t shard_bytes) {
    const int tid = threadIdx.x;
    const Mx4Tile t = tiles[blockIdx.x];
    T *dst = static_cast<T *>(params[t.param]) + t.src;
    const uint8_t *shard = gathered + t.rank * shard_bytes;
    const uint8_t *codes = shard + t.blk * kMx4BlockBytes;
    const uint8_t *scales = shard + shard_blocks * kMx4BlockBytes + t.blk;
    constexpr int E = kUnit<T>, kSteps = kMx4Tile / E / kThreads;
    uint32_t c[kSteps], s[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int q = i * kThreads + tid;
        if (E * q < t.n) {
            c[i] = unit_codes<T>(codes, q);
            s[i] = ld(scales + q / (kMx4Block / E));
        }
    }
    with_past(on16(dst), [&](auto past) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int q = i * kThreads + tid;
            if (E * q < t.n) store_unit<past>(dst + E * q, decode_unit(T{}, c[i], scale_value(s[i])), t.n - E * q);
        }
    });
}

// In the reduce a workgroup takes one of kParts parts of a tile, so that a wave lives for
// one round of loads and many are on a CU.  The parts share cache lines
// of scales, and go to one XCD: eight tiles at a time, the last ones in turn.
constexpr uint32_t kParts = kTileSteps, kXcds = 8;

struct TilePart {
    uint32_t tile, part;
};
__device__ __forceinline__ TilePart part_of(uint32_t id, uint32_t ntiles) {
    if (id < ntiles / kXcds * kXcds * kParts) return {id / (kXcds * kParts) * kXcds + id % kXcds, id / kXcds % kParts};
    return {id / kParts, id % kParts};
}

constexpr int kMx4Terms = 64;   // slices of one launch; the sums of more are carried through `out`
struct Mx4Slices {
    const uint8_t *p[kMx4Terms];
};

// A lane's 8 elements of `COUNT` slices from `first` on, all their loads on their way at once.
template <int COUNT>
__device__ __forceinline__ void add_slices(float (&acc)[8], const Mx4Slices &slices, int first, int64_t code0, int64_t scale0,
                                           int q) {
    uint32_t c[COUNT], s[COUNT];
#pragma unroll
    for (int j = 0; j < COUNT; ++j) {
        c[j] = reinterpret_cast<const uint32_t *>(slices.p[first + j] + code0)[q];
        s[j] = slices.p[first + j][scale0 + (q >> 2)];
    }
#pragma unroll
    for (int j = 0; j < COUNT; ++j) {
        float v[8];
        decode8(v, c[j], scale_value(s[j]));
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] += v[k];
    }
}

// The sums are in fp32, slice by slice.  HBM's mix of many read streams and a write bounds it: one 7B block's
// shard of 8 slices 35.3 us, 5.9 TB/s, three of 32 slices 276, 5.8 TB/s.  In parts of tiles the two took 41.6 and 296
// where whole tiles took 44.3 and 350, two steps of them at a time 48 and 295, four 53 and 302; with the parts of a
// tile on one XCD and stores past the caches 40.6 and 282.
__global__ __launch_bounds__(kThreads) void reduce_mx4_kernel(const Mx4Tile *__restrict__ tiles, uint32_t ntiles,
                                                              const Mx4Run *__restrict__ gaps, Mx4Slices slices,
                                                              int nterms, int first_pass, float divide, float scale,
                                                              float *__restrict__ out, int64_t shard_blocks) {
    __shared__ u32x4 lds_units[kThreads / 64][128];
    const int tid = threadIdx.x;
    const uint32_t id = blockIdx.x;
    if (id >= ntiles * kParts) {   // elements of no piece
        const Mx4Run run = gaps[id - ntiles * kParts];
        for (int k = tid; k < run.n; k += kThreads) out[run.at + k] = 0.f;
        return;
    }
    const TilePart at = part_of(id, ntiles);
    const Mx4Tile t = tiles[at.tile];
    if (at.part == 0 && tid < t.fill) out[t.elem + t.n + tid] = 0.f;
    const int q = at.part * kThreads + tid, valid = t.n - 8 * q;
    if (t.n - 8 * (q & ~63) <= 0) return;   // whole waves
    const int64_t code0 = t.blk * kMx4BlockBytes, scale0 = shard_blocks * kMx4BlockBytes + t.blk;
    float *dst = out + t.elem + 8 * q;
    float acc[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        acc[k] = -0.f;   // adds nothing to any value, zeros of either sign among them
        if (!first_pass && k < valid) acc[k] = dst[k];
    }
    if (valid > 0) {
        int j = 0;
        for (; j + 8 <= nterms; j += 8) add_slices<8>(acc, slices, j, code0, scale0, q);
        if (j + 4 <= nterms) {
            add_slices<4>(acc, slices, j, code0, scale0, q);
            j += 4;
        }
        for (; j < nterms; ++j) add_slices<1>(acc, slices, j, code0, scale0, q);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] = divide != 0.f ? acc[k] / divide : acc[k] * scale;
    u32x4 v[2];
    units_in_turn(v, acc, lds_units[tid >> 6]);
    const int first = 8 * (q & ~63) + 4 * (tid & 63);
    with_past(on16(out + t.elem), [&](auto past) {
#pragma unroll
        for (int h = 0; h < 2; ++h) store_unit<past>(out + t.elem + first + 256 * h, v[h], t.n - first - 256 * h);
    });
}

// ---------------------------------------------------------------- matrices --

struct Mx4Out {
    uint8_t *codes, *scales;
    int64_t code_stride, scale_stride;
};

// Neighbours share the cache lines of codes and scales: a run of tiles to each XCD.
__device__ __forceinline__ uint32_t tile_run(uint32_t id, uint32_t tiles) {
    const uint32_t each = tiles / kXcds, rest = tiles % kXcds, xcd = id % kXcds;
    return xcd * each + min(xcd, rest) + id / kXcds;
}

// Along rows alone, and back: a tile is 16 rows by 128 elements, a lane's eight of them or a unit.
constexpr int kRowLanes = 16, kRowTileCols = 8 * kRowLanes, kRowTileRows = kThreads / kRowLanes;

// STEPS tiles of the row-major order, one after the other, where there are many: their codes and scales then go through
// LDS, to be stored 16 bytes and one a lane.  Past 4096 tiles 8192 by 11008 bf16 takes 44 us for 50 a tile at a time, random
// 59 to 64 for 67, 1.25M by 32 46 for 65, 4096 by 4096 8.6 for 9.7; 2048 by 4096 takes 5.2 either way, 1024 by 4096 3.8
// for 3.3 and 16 by 4096 2.4 for 1.8.
constexpr int kManySteps = 4;
constexpr int64_t kManyTiles = 4096;
template <class T, bool STOCHASTIC, int STEPS>
__global__ __launch_bounds__(kThreads) void quantize_rows_mx4_kernel(int64_t rows, int64_t cols, const T *__restrict__ x,
                                                                     int64_t ldx, uint32_t tiles_x, Mx4Out by_row,
                                                                     const uint64_t *__restrict__ seed_at) {
    constexpr int U = kUnits<T>, E = kUnit<T>, kRowUnits = kRowTileCols / E, kTileBlocks = kRowTileCols / kMx4Block;
    __shared__ u32x4 lds_units[kWavesExchanging<T>][128];
    __shared__ __attribute__((aligned(16))) uint32_t lds_codes[kRowTileRows][STEPS * kRowLanes];
    __shared__ uint8_t lds_scales[kRowTileRows][STEPS * kTileBlocks];
    const uint32_t first = tile_run(blockIdx.x, gridDim.x) * STEPS;
    const int tid = threadIdx.x, lr = tid / kRowLanes, lq = tid % kRowLanes;
    const int64_t nb = (cols + kMx4Block - 1) / kMx4Block;
    uint32_t ty[STEPS], tx[STEPS];   // tiles beyond the last one lie below the matrix
    ty[0] = first / tiles_x, tx[0] = first % tiles_x;
#pragma unroll
    for (int i = 1; i < STEPS; ++i) {
        const bool wrap = tx[i - 1] + 1 == tiles_x;
        ty[i] = ty[i - 1] + wrap, tx[i] = wrap ? 0 : tx[i - 1] + 1;
    }
    u32x4 v[STEPS][U];
    with_past(on16(x) && ldx * sizeof(T) % 16 == 0, [&](auto past) {
#pragma unroll
        for (int i = 0; i < STEPS; ++i)
#pragma unroll
            for (int h = 0; h < U; ++h) {
                const int u = (tid & ~63) * U + 64 * h + (tid & 63);
                const int64_t r = (int64_t)ty[i] * kRowTileRows + u / kRowUnits, c = (int64_t)tx[i] * kRowTileCols + E * (u % kRowUnits);
                v[i][h] = load_unit<past>(x + r * ldx + c, r < rows ? (int)imax(0, imin(E, cols - c)) : 0);
            }
    });
    const uint64_t seed = STOCHASTIC ? *seed_at : 0;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const Raw8<T> e = own_units(v[i], lds_units[U > 1 ? tid >> 6 : 0]);
        const int64_t r = (int64_t)ty[i] * kRowTileRows + lr, b = (int64_t)tx[i] * kTileBlocks + lq / 4;
        uint32_t s;
        const uint32_t code = encode8<STOCHASTIC>(e, seed, 4 * (uint64_t)(r * nb + b) + (lq & 3), 0, &s);
        if (STEPS > 1) {
            lds_codes[lr][i * kRowLanes + lq] = code;
            if ((lq & 3) == 0) lds_scales[lr][i * kTileBlocks + lq / 4] = (uint8_t)s;
        } else if (r < rows && b < nb) {
            *reinterpret_cast<uint32_t *>(by_row.codes + r * by_row.code_stride + b * kMx4BlockBytes + 4 * (lq & 3)) = code;
            if ((lq & 3) == 0) by_row.scales[r * by_row.scale_stride + b] = (uint8_t)s;
        }
    }
    if (STEPS == 1) return;
    __syncthreads();
    static_assert(STEPS == 1 || STEPS * kTileBlocks * kRowTileRows == kThreads, "a thread for every block");
    const int row = tid / (STEPS * kTileBlocks), at = tid % (STEPS * kTileBlocks);
    const uint32_t tile = first + at / kTileBlocks;
    const int64_t r = (int64_t)(tile / tiles_x) * kRowTileRows + row, b = (int64_t)(tile % tiles_x) * kTileBlocks + at % kTileBlocks;
    if (r < rows && b < nb) {
        *reinterpret_cast<u32x4 *>(by_row.codes + r * by_row.code_stride + b * kMx4BlockBytes) =
            *reinterpret_cast<const u32x4 *>(&lds_codes[row][4 * at]);
        by_row.scales[r * by_row.scale_stride + b] = lds_scales[row][at];
    }
}

// Back: a lane takes a unit of U rows of the tile.  8192 by 11008 to bf16 takes 31 to 37 us, 6.2 to 7.3 TB/s, where the codes
// are in the caches still (right after their making, or the same buffers again and again), to fp32 57 to 62; with buffers
// in turn that are in no cache 51 and 99, 4.5 and 4.1 TB/s, two thirds of a copy's rate.
template <class T>
__global__ __launch_bounds__(kThreads) void dequantize_mx4_kernel(Mx4Mat m, int64_t rows, int64_t cols, T *__restrict__ out,
                                                                  int64_t ldo, uint32_t tiles_x) {
    constexpr int U = kUnits<T>, E = kUnit<T>, kRowUnits = kRowTileCols / E;
    const uint32_t id = tile_run(blockIdx.x, gridDim.x);
    const int64_t r0 = (int64_t)(id / tiles_x) * kRowTileRows + threadIdx.x / kRowUnits;
    const int64_t c = (int64_t)(id % tiles_x) * kRowTileCols + E * (threadIdx.x % kRowUnits);
    if (c >= cols) return;
    uint32_t w[U], s[U];
#pragma unroll
    for (int h = 0; h < U; ++h) {
        const int64_t r = r0 + h * (kRowTileRows / U);
        if (r < rows) {
            int64_t code, scale;
            m.row((uint32_t)r, &code, &scale);
            w[h] = unit_codes<T>(m.codes + code, c / E);
            s[h] = ld(m.scales + scale + c / kMx4Block);
        }
    }
    with_past(on16(out) && ldo * sizeof(T) % 16 == 0, [&](auto past) {
#pragma unroll
        for (int h = 0; h < U; ++h) {
            const int64_t r = r0 + h * (kRowTileRows / U);
            if (r < rows) store_unit<past>(out + r * ldo + c, decode_unit(T{}, w[h], scale_value(s[h])), (int)imin(E, cols - c));
        }
    });
}

// Along columns, with or without rows: a workgroup takes 128 rows by 256 bytes, and the columns' blocks come from a
// copy in LDS.  There a lane takes 32 rows of a word, one or two blocks of its own, so no
// lanes join; the lanes of a quad take the column's four blocks, which they store side by side.
// 8192 by 11008 bf16 both ways: 62 to 66 us to nearest, 4.2 to 4.5 TB/s, which HBM and the LDS copy bound; 86 to 94 random,
// bound by the vector instructions, of which the random bits' multiplications (28 for 16 elements) take several times an
// addition's cycles.
// Columns alone 51 to 55 and 53 to 58.  From fp32 99 to 105 and 119 to 123.  With buffers in turn that are in no cache 76 and 88,
// columns alone 57 and 60, from fp32 117 and 122.
constexpr int kColTileRows = 128;
template <class T>
constexpr int kColTileCols = 256 / sizeof(T);

// The blocks in column `at` of a wave's 32 rows of LDS words: one for fp32, two for bf16.
__device__ __forceinline__ void column_raws(Raw8<float> (&v)[1][4], const uint32_t *w) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[0][k >> 1].v[k & 1] = u32x4{w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]};
}
__device__ __forceinline__ void column_raws(Raw8<uint16_t> (&v)[2][4], const uint32_t *w) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // the low halves of two rows, and the high ones
            lo[i] = __builtin_amdgcn_perm(w[8 * k + 2 * i + 1], w[8 * k + 2 * i], 0x05040100);
            hi[i] = __builtin_amdgcn_perm(w[8 * k + 2 * i + 1], w[8 * k + 2 * i], 0x07060302);
        }
        v[0][k].v = u32x4{lo[0], lo[1], lo[2], lo[3]};
        v[1][k].v = u32x4{hi[0], hi[1], hi[2], hi[3]};
    }
}

template <class T, bool ROWS, bool STOCHASTIC>
__global__ __launch_bounds__(kThreads) void quantize_cols_mx4_kernel(int64_t rows, int64_t cols, const T *__restrict__ x,
                                                                     int64_t ldx, uint32_t tiles_x, Mx4Out by_row,
                                                                     Mx4Out by_col, const uint64_t *__restrict__ seed_at) {
    constexpr int kCols = kColTileCols<T>, kColLanes = kCols / 8, kColSteps = kColTileRows * kColLanes / kThreads;
    constexpr int U = kUnits<T>, E = kUnit<T>, kRowUnits = kCols / E;
    constexpr int kColBlocks = kColTileRows / kMx4Block;   // of a column
    // Bytes of a row in LDS, and more between blocks of them: neither the writes of rows nor the reads of four blocks'
    // words by the lanes of a quad meet in a bank.
    constexpr int kPitch = 256 + 16, kBetween = 64;
    __shared__ __attribute__((aligned(16))) uint8_t lds[kColTileRows * kPitch + kColBlocks * kBetween];
    auto lds_row = [&](int r) { return lds + r * kPitch + r / kMx4Block * kBetween; };
    const uint32_t id = tile_run(blockIdx.x, gridDim.x);
    const int64_t r0 = (int64_t)(id / tiles_x) * kColTileRows, c0 = (int64_t)(id % tiles_x) * kCols;
    const uint64_t seed = STOCHASTIC ? *seed_at : 0;
    const int64_t nbr = (cols + kMx4Block - 1) / kMx4Block, nbc = (rows + kMx4Block - 1) / kMx4Block;
    u32x4 v[kColSteps * U];
    with_past(on16(x) && ldx * sizeof(T) % 16 == 0, [&](auto past) {
#pragma unroll
        for (int i = 0; i < kColSteps * U; ++i) {
            const int q = i * kThreads + threadIdx.x;
            const int64_t r = r0 + q / kRowUnits, c = c0 + E * (q % kRowUnits);
            v[i] = load_unit<past>(x + r * ldx + c, r < rows ? (int)imax(0, imin(E, cols - c)) : 0);
        }
    });
#pragma unroll
    for (int i = 0; i < kColSteps * U; ++i) {
        const int q = i * kThreads + threadIdx.x;
        *reinterpret_cast<u32x4 *>(lds_row(q / kRowUnits) + q % kRowUnits * 16) = v[i];
    }
    if (U > 1) __syncthreads();   // a lane's eights come from LDS
    if (ROWS) {
        constexpr int kStep = kThreads / kColLanes;   // rows between a lane's loads
        const int lq = threadIdx.x % kColLanes;
        const int64_t r1 = r0 + threadIdx.x / kColLanes, b = c0 / kMx4Block + lq / 4;
        uint8_t *codes = by_row.codes + r1 * by_row.code_stride + b * kMx4BlockBytes + 4 * (lq & 3);
        uint8_t *scales = by_row.scales + r1 * by_row.scale_stride + b;
        uint64_t group = 4 * (uint64_t)(r1 * nbr + b) + (lq & 3);
#pragma unroll
        for (int i = 0; i < kColSteps; ++i) {
            Raw8<T> e;
            if (U == 1) __builtin_memcpy(&e, &v[i], 16);
            else __builtin_memcpy(&e, __builtin_assume_aligned(lds_row(i * kStep + threadIdx.x / kColLanes) + lq * sizeof e, 16), sizeof e);
            uint32_t s;
            const uint32_t code = encode8<STOCHASTIC>(e, seed, group, 0, &s);
            if (r1 + i * kStep < rows && b < nbr) {
                *reinterpret_cast<uint32_t *>(codes) = code;
                if ((lq & 3) == 0) *scales = (uint8_t)s;
            }
            codes += kStep * by_row.code_stride;
            scales += kStep * by_row.scale_stride;
            group += 4 * kStep * (uint64_t)nbr;
        }
    }
    if (U == 1) __syncthreads();
    constexpr int kWide = 4 / sizeof(T);   // columns a lane
    static_assert(kCols / kWide * kColBlocks == kThreads, "a lane takes the blocks of one word's columns");
    const int lb = threadIdx.x % kColBlocks, lc = threadIdx.x / kColBlocks;   // a quad's codes follow each other
    const int64_t b = r0 / kMx4Block + lb;
    if (b >= nbc) return;
    uint32_t w[kMx4Block];
#pragma unroll
    for (int k = 0; k < kMx4Block; ++k) w[k] = *reinterpret_cast<const uint32_t *>(lds_row(lb * kMx4Block) + k * kPitch + lc * 4);
    Raw8<T> e[kWide][4];
    column_raws(e, w);
#pragma unroll
    for (int j = 0; j < kWide; ++j) {
        const int64_t c = c0 + lc * kWide + j;
        const uint32_t s = scale_byte<STOCHASTIC>(max(max(amax8(e[j][0]), amax8(e[j][1])), max(amax8(e[j][2]), amax8(e[j][3]))));
        uint32_t code[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) code[k] = encode8_at<STOCHASTIC>(e[j][k], s, seed, 4 * (uint64_t)(c * nbc + b) + k, 1);
        if (c < cols) {
            *reinterpret_cast<u32x4 *>(by_col.codes + c * by_col.code_stride + b * kMx4BlockBytes) = u32x4{code[0], code[1], code[2], code[3]};
            by_col.scales[c * by_col.scale_stride + b] = (uint8_t)s;
        }
    }
}

// ---------------------------------------------------------------- launching --

int current_device(const char *what, int *dev) {
    if (hipGetDevice(dev) != hipSuccess) return fail(FS_E_HIP, "%s: no current device", what);
    return FS_OK;
}

// The tables live on the device they were uploaded to.
int check_plan(const char *what, fs_mx4_plan_t p) {
    if (!p) return fail(FS_E_INVAL, "%s: plan is NULL", what);
    if (!p->dev_ws) return fail(FS_E_INVAL, "%s: plan has no uploaded workspace (call fs_mx4_plan_upload)", what);
    int dev = -1;
    if (int rc = current_device(what, &dev)) return rc;
    if (dev != p->dev_id)
        return fail(FS_E_INVAL, "%s: the plan was uploaded on device %d, current device is %d", what, p->dev_id, dev);
    return FS_OK;
}

int check_dtype(const char *what, fs_dtype dtype) {
    if (dtype != FS_BF16 && dtype != FS_FP32) return fail(FS_E_DTYPE, "%s: unknown dtype %d", what, (int)dtype);
    return FS_OK;
}
int64_t width(fs_dtype dtype) { return dtype == FS_BF16 ? 2 : 4; }

// A grid's threads are counted in 32 bits.
constexpr int64_t kMaxGrid = UINT32_MAX / kThreads;

const Mx4Tile *tiles_at(fs_mx4_plan_t p, int32_t rank) {
    return reinterpret_cast<const Mx4Tile *>(static_cast<const char *>(p->dev_ws) + p->ws_tiles) + p->tile_off[rank];
}
const Mx4Run *pads_at(fs_mx4_plan_t p, int32_t rank) {
    return reinterpret_cast<const Mx4Run *>(static_cast<const char *>(p->dev_ws) + p->ws_pads) + p->pad_off[rank];
}
const Mx4Run *gaps_at(fs_mx4_plan_t p, int32_t rank) {
    return reinterpret_cast<const Mx4Run *>(static_cast<const char *>(p->dev_ws) + p->ws_gaps) + p->gap_off[rank];
}

// f(T value, std::bool_constant) by the element type and whether there is a seed.
template <class F>
void by_type(fs_dtype dtype, bool stochastic, F &&f) {
    if (dtype == FS_BF16) {
        if (stochastic) f(uint16_t{}, std::true_type{});
        else f(uint16_t{}, std::false_type{});
    } else {
        if (stochastic) f(float{}, std::true_type{});
        else f(float{}, std::false_type{});
    }
}

int check_seed(const char *what, const uint64_t *seed) {
    if (misaligned(seed, 8)) return fail(FS_E_ALIGN, "%s: seed not 8-byte aligned", what);
    return FS_OK;
}

}  // namespace

extern "C" int fs_mx4_plan_upload(fs_mx4_plan_t p, void *workspace, size_t bytes, hipStream_t stream) {
    clear_error();
    const char *what = "fs_mx4_plan_upload";
    if (!p || !workspace) return fail(FS_E_INVAL, "%s: NULL argument", what);
    if (misaligned(workspace, 16)) return fail(FS_E_ALIGN, "%s: workspace must be 16-byte aligned", what);
    if ((int64_t)bytes < p->info.workspace_bytes)
        return fail(FS_E_INVAL, "%s: workspace too small (%zu < %lld bytes)", what, bytes, (long long)p->info.workspace_bytes);
    int dev = -1;
    if (int rc = current_device(what, &dev)) return rc;
    hipPointerAttribute_t a;
    memset(&a, 0, sizeof a);
    const hipError_t known = hipPointerGetAttributes(&a, workspace);
    if (known != hipSuccess) (void)hipGetLastError();   // the query's error is not a launch error
    if (known != hipSuccess || a.type != hipMemoryTypeDevice || a.device != dev)
        return fail(FS_E_INVAL, "%s: workspace must be device memory of the current device (%d)", what, dev);
    char *ws = static_cast<char *>(workspace);
    struct Part { int64_t off; const void *src; size_t bytes; };
    const Part parts[] = {{p->ws_tiles, p->tiles.data(), p->tiles.size() * sizeof(Mx4Tile)},
                          {p->ws_pads, p->pads.data(), p->pads.size() * sizeof(Mx4Run)},
                          {p->ws_gaps, p->gaps.data(), p->gaps.size() * sizeof(Mx4Run)}};
    for (const Part &part : parts) {
        if (part.bytes == 0) continue;
        const hipError_t e = hipMemcpyAsync(ws + part.off, part.src, part.bytes, hipMemcpyHostToDevice, stream);
        if (e != hipSuccess) return fail(FS_E_HIP, "%s: copy failed: %s", what, hipGetErrorString(e));
    }
    const hipError_t e = hipStreamSynchronize(stream);
    if (e != hipSuccess) return fail(FS_E_HIP, "%s: sync failed: %s", what, hipGetErrorString(e));
    p->dev_ws = workspace;
    p->dev_id = dev;
    return FS_OK;
}

extern "C" int fs_pack_mx4(fs_mx4_plan_t p, const void *const *params, fs_dtype param_dtype, void *out, int32_t rank,
                           const uint64_t *seed, hipStream_t stream) {
    clear_error();
    const char *what = "fs_pack_mx4";
    if (int rc = check_plan(what, p)) return rc;
    if (int rc = check_dtype(what, param_dtype)) return rc;
    if (rank < -1 || rank >= p->world) return fail(FS_E_INVAL, "%s: rank %d out of range [-1, %d)", what, rank, p->world);
    if (int rc = check_seed(what, seed)) return rc;
    const int32_t lo = rank < 0 ? 0 : rank, hi = rank < 0 ? p->world : rank + 1;
    const int64_t ntiles = p->tile_off[hi] - p->tile_off[lo], npads = p->pad_off[hi] - p->pad_off[lo];
    if (ntiles + npads == 0) return FS_OK;
    if (!out) return fail(FS_E_INVAL, "%s: out is NULL", what);
    if (!params) return fail(FS_E_INVAL, "%s: params is NULL", what);
    if (misaligned(out, 16)) return fail(FS_E_ALIGN, "%s: out not 16-byte aligned", what);
    if (seed && ranges_overlap(seed, 8, out, (hi - lo) * p->info.shard_bytes))
        return fail(FS_E_INVAL, "%s: seed inside out", what);
    if (ntiles + npads > kMaxGrid) return fail(FS_E_OVERFLOW, "%s: too many tiles for one launch", what);
    (void)hipGetLastError();
    by_type(param_dtype, seed != nullptr, [&](auto t, auto stochastic) {
        hipLaunchKernelGGL((pack_mx4_kernel<decltype(t), decltype(stochastic)::value>), dim3((uint32_t)(ntiles + npads)),
                           dim3(kThreads), 0, stream, tiles_at(p, lo), (uint32_t)ntiles, pads_at(p, lo), params,
                           static_cast<uint8_t *>(out), lo, p->info.shard_blocks, p->info.shard_bytes, seed);
    });
    return check_launch(what);
}

extern "C" int fs_unpack_mx4(fs_mx4_plan_t p, const void *gathered, void *const *params, fs_dtype param_dtype,
                             hipStream_t stream) {
    clear_error();
    const char *what = "fs_unpack_mx4";
    if (int rc = check_plan(what, p)) return rc;
    if (int rc = check_dtype(what, param_dtype)) return rc;
    const int64_t ntiles = (int64_t)p->tiles.size();
    if (ntiles == 0) return FS_OK;
    if (!gathered) return fail(FS_E_INVAL, "%s: gathered is NULL", what);
    if (!params) return fail(FS_E_INVAL, "%s: params is NULL", what);
    if (misaligned(gathered, 16)) return fail(FS_E_ALIGN, "%s: gathered not 16-byte aligned", what);
    if (ntiles > kMaxGrid) return fail(FS_E_OVERFLOW, "%s: too many tiles for one launch", what);
    (void)hipGetLastError();
    by_type(param_dtype, false, [&](auto t, auto) {
        hipLaunchKernelGGL((unpack_mx4_kernel<decltype(t)>), dim3((uint32_t)ntiles), dim3(kThreads), 0, stream,
                           tiles_at(p, 0), static_cast<const uint8_t *>(gathered), params, p->info.shard_blocks,
                           p->info.shard_bytes);
    });
    return check_launch(what);
}

extern "C" int fs_reduce_shard_mx4(fs_mx4_plan_t p, int32_t rank, int32_t grad_acc, const void *const *slices, float *out,
                                   hipStream_t stream) {
    clear_error();
    const char *what = "fs_reduce_shard_mx4";
    if (int rc = check_plan(what, p)) return rc;
    if (rank < 0 || rank >= p->world) return fail(FS_E_INVAL, "%s: rank %d out of range [0, %d)", what, rank, p->world);
    if (grad_acc < 1) return fail(FS_E_INVAL, "%s: grad_acc must be >= 1", what);
    if (p->shard_numel == 0) return FS_OK;
    if (!out || !slices) return fail(FS_E_INVAL, "%s: NULL argument", what);
    if (misaligned(out, 4)) return fail(FS_E_ALIGN, "%s: out not aligned to 4 bytes", what);
    const int64_t terms = (int64_t)p->world * grad_acc;
    if (terms > INT32_MAX) return fail(FS_E_OVERFLOW, "%s: too many slices", what);
    for (int64_t k = 0; k < terms; ++k) {
        if (!slices[k]) return fail(FS_E_INVAL, "%s: slice %lld is NULL", what, (long long)k);
        if (misaligned(slices[k], 16)) return fail(FS_E_ALIGN, "%s: slice %lld not 16-byte aligned", what, (long long)k);
        if (ranges_overlap(slices[k], p->info.shard_bytes, out, p->shard_numel * 4))
            return fail(FS_E_INVAL, "%s: out overlaps slice %lld", what, (long long)k);
    }
    const int64_t ntiles = p->tile_off[rank + 1] - p->tile_off[rank], ngaps = p->gap_off[rank + 1] - p->gap_off[rank];
    if (ntiles * kParts + ngaps > kMaxGrid) return fail(FS_E_OVERFLOW, "%s: too many tiles for one launch", what);
    (void)hipGetLastError();
    // dividing by a power of two is multiplying by its reciprocal, bit for bit
    const bool exact = (p->world & (p->world - 1)) == 0;
    for (int64_t k = 0; k < terms; k += kMx4Terms) {
        Mx4Slices s;
        memset(&s, 0, sizeof s);
        const int count = (int)imin(kMx4Terms, terms - k);
        for (int j = 0; j < count; ++j) s.p[j] = static_cast<const uint8_t *>(slices[k + j]);
        hipLaunchKernelGGL(reduce_mx4_kernel, dim3((uint32_t)(ntiles * kParts + ngaps)), dim3(kThreads), 0, stream,
                           tiles_at(p, rank), (uint32_t)ntiles, gaps_at(p, rank), s, count, k == 0,
                           k + count == terms && !exact ? (float)p->world : 0.f,
                           k + count == terms ? 1.f / (float)p->world : 1.f, out, p->info.shard_blocks);
    }
    return check_launch(what);
}

namespace fsi {

int check_matrix(const char *what, const char *name, const fs_mx4_matrix_t *m, Mx4Mat *out, Footprint (&covers)[2]) {
    constexpr int64_t kMost = (int64_t)1 << 56;   // sums of these stay within int64
    covers[0] = covers[1] = Footprint{nullptr, 0, 0, 0, name};
    memset(out, 0, sizeof *out);
    if (m->rows < 0 || m->cols < 0) return fail(FS_E_INVAL, "%s: %s has a negative size", what, name);
    if (m->rows > INT32_MAX || m->cols > INT32_MAX)
        return fail(FS_E_OVERFLOW, "%s: %s has more than 2^31 - 1 rows or columns", what, name);
    if (m->rows == 0 || m->cols == 0) return FS_OK;
    const int64_t nb = mx4_blocks(m->cols);
    if (!m->codes || !m->scales) return fail(FS_E_INVAL, "%s: %s is NULL", what, name);
    if (m->chunk_rows < 0) return fail(FS_E_INVAL, "%s: %s has negative chunk_rows", what, name);
    const int64_t run = m->chunk_rows ? imin(m->chunk_rows, m->rows) : m->rows;   // rows of a chunk
    if ((run > 1 && (m->code_stride < nb * kMx4BlockBytes || m->scale_stride < nb)))
        return fail(FS_E_INVAL, "%s: the rows of %s overlap", what, name);
    const int64_t chunks = m->chunk_rows ? (m->rows - 1) / m->chunk_rows + 1 : 1;   // chunk_rows may be any length
    if (misaligned(m->codes, 16) || (run > 1 && (m->code_stride & 15)) || (chunks > 1 && (m->chunk_stride & 15)))
        return fail(FS_E_ALIGN, "%s: the codes of %s are not on 16 bytes", what, name);
    if ((run > 1 && (m->code_stride > kMost / run || m->scale_stride > kMost / run)) ||
        (chunks > 1 && m->chunk_stride > kMost / chunks))
        return fail(FS_E_OVERFLOW, "%s: the strides of %s are too large", what, name);
    const int64_t codes = (run > 1 ? (run - 1) * m->code_stride : 0) + nb * kMx4BlockBytes;
    const int64_t scales = (run > 1 ? (run - 1) * m->scale_stride : 0) + nb;
    // the chunks' codes (or scales) follow each other; the two may lie between each other, as in a gathered buffer
    if (chunks > 1 && (m->chunk_stride < codes || m->chunk_stride < scales))
        return fail(FS_E_INVAL, "%s: the chunks of %s overlap", what, name);
    const int64_t far = chunks > 1 ? (chunks - 1) * m->chunk_stride : 0;
    out->codes = static_cast<const uint8_t *>(m->codes);
    out->scales = static_cast<const uint8_t *>(m->scales);
    out->code_stride = run > 1 ? m->code_stride : 0;
    out->scale_stride = run > 1 ? m->scale_stride : 0;
    covers[0] = {m->codes, far + codes, chunks > 1 ? 0 : out->code_stride, chunks > 1 ? far + codes : nb * kMx4BlockBytes, name};
    covers[1] = {m->scales, far + scales, chunks > 1 ? 0 : out->scale_stride, chunks > 1 ? far + scales : nb, name};
    if (chunks > 1) {
        uint32_t l = 0;
        while (((int64_t)1 << l) < m->chunk_rows) ++l;   // chunk_rows < rows < 2^31
        out->chunk_rows = (uint32_t)m->chunk_rows;
        out->chunk_shift = 31 + l;
        out->chunk_mul = (uint32_t)(((uint64_t)1 << (31 + l)) / (uint64_t)m->chunk_rows + 1);
        out->chunk_stride = m->chunk_stride;
    }
    return FS_OK;
}

}  // namespace fsi

namespace {

// Output matrix `m` of `rows` by `cols`; its codes and scales are appended to `all`, which must be disjoint of them.
int check_out(const char *what, const char *name, const fs_mx4_matrix_t *m, int64_t rows, int64_t cols, Mx4Out *out,
              Footprint *all, int *count) {
    Mx4Mat k;
    Footprint mine[2];
    if (m->rows != rows || m->cols != cols)
        return fail(FS_E_INVAL, "%s: %s must be %lld by %lld", what, name, (long long)rows, (long long)cols);
    if (m->chunk_rows != 0) return fail(FS_E_INVAL, "%s: %s is chunked", what, name);
    if (int rc = check_matrix(what, name, m, &k, mine)) return rc;
    for (const Footprint &f : mine) {
        for (int i = 0; i < *count; ++i)
            if (meet(f, all[i])) return fail(FS_E_INVAL, "%s: %s overlaps %s", what, name, all[i].name);
        all[(*count)++] = f;
    }
    *out = Mx4Out{const_cast<uint8_t *>(k.codes), const_cast<uint8_t *>(k.scales), k.code_stride, k.scale_stride};
    return FS_OK;
}

// Checks a plain matrix of `width` bytes an element and gives what it covers.
int check_plain(const char *what, const char *name, const void *p, int64_t rows, int64_t cols, int64_t ld, int64_t width,
                Footprint *covers) {
    *covers = Footprint{nullptr, 0, 0, 0, name};
    if (rows < 0 || cols < 0) return fail(FS_E_INVAL, "%s: negative size", what);
    if (rows > INT32_MAX || cols > INT32_MAX) return fail(FS_E_OVERFLOW, "%s: more than 2^31 - 1 rows or columns", what);
    if (rows == 0 || cols == 0) return FS_OK;
    if (!p) return fail(FS_E_INVAL, "%s: %s is NULL", what, name);
    if (misaligned(p, width)) return fail(FS_E_ALIGN, "%s: %s not aligned to its element size", what, name);
    if (rows > 1 && ld < cols) return fail(FS_E_INVAL, "%s: the rows of %s overlap", what, name);
    if (rows > 1 && ld > ((int64_t)1 << 56) / rows) return fail(FS_E_OVERFLOW, "%s: %s is too large", what, name);
    const int64_t stride = rows > 1 ? ld * width : 0;
    *covers = Footprint{p, (rows - 1) * stride + cols * width, stride, cols * width, name};
    return FS_OK;
}

int mat_tiles(const char *what, int64_t rows, int64_t cols, int64_t tile_rows, int64_t tile_cols, uint32_t *across, uint32_t *tiles) {
    const int64_t x = (cols + tile_cols - 1) / tile_cols, y = (rows + tile_rows - 1) / tile_rows;
    if (x * y > kMaxGrid) return fail(FS_E_OVERFLOW, "%s: too large for one launch", what);
    *across = (uint32_t)x;
    *tiles = (uint32_t)(x * y);
    return FS_OK;
}

}  // namespace

extern "C" int fs_mx4_quantize(int64_t rows, int64_t cols, const void *x, fs_dtype dtype, int64_t ldx,
                               const fs_mx4_matrix_t *by_row, const fs_mx4_matrix_t *by_col, const uint64_t *seed,
                               hipStream_t stream) {
    clear_error();
    const char *what = "fs_mx4_quantize";
    if (int rc = check_dtype(what, dtype)) return rc;
    if (!by_row && !by_col) return fail(FS_E_INVAL, "%s: no output", what);
    if (int rc = check_seed(what, seed)) return rc;
    Footprint all[6];
    int count = 0;
    if (int rc = check_plain(what, "x", x, rows, cols, ldx, width(dtype), &all[count++])) return rc;
    all[count++] = Footprint{seed, seed ? 8 : 0, 0, 8, "seed"};
    Mx4Out row{}, col{};
    if (by_row)
        if (int rc = check_out(what, "by_row", by_row, rows, cols, &row, all, &count)) return rc;
    if (by_col)
        if (int rc = check_out(what, "by_col", by_col, cols, rows, &col, all, &count)) return rc;
    uint32_t across, tiles;
    if (int rc = by_col ? mat_tiles(what, rows, cols, kColTileRows, dtype == FS_BF16 ? kColTileCols<uint16_t> : kColTileCols<float>, &across, &tiles)
                        : mat_tiles(what, rows, cols, kRowTileRows, kRowTileCols, &across, &tiles))
        return rc;
    const bool many = !by_col && tiles > kManyTiles;
    if (many) tiles = (tiles + kManySteps - 1) / kManySteps;
    if (tiles == 0) return FS_OK;
    (void)hipGetLastError();
    by_type(dtype, seed != nullptr, [&](auto t, auto stochastic) {
        using T = decltype(t);
        constexpr bool S = decltype(stochastic)::value;
        const T *src = static_cast<const T *>(x);
        const int64_t ld = rows > 1 ? ldx : 0;
        if (many)
            hipLaunchKernelGGL((quantize_rows_mx4_kernel<T, S, kManySteps>), dim3(tiles), dim3(kThreads), 0, stream, rows, cols,
                               src, ld, across, row, seed);
        else if (!by_col)
            hipLaunchKernelGGL((quantize_rows_mx4_kernel<T, S, 1>), dim3(tiles), dim3(kThreads), 0, stream, rows, cols, src, ld,
                               across, row, seed);
        else if (by_row)
            hipLaunchKernelGGL((quantize_cols_mx4_kernel<T, true, S>), dim3(tiles), dim3(kThreads), 0, stream, rows, cols,
                               src, ld, across, row, col, seed);
        else
            hipLaunchKernelGGL((quantize_cols_mx4_kernel<T, false, S>), dim3(tiles), dim3(kThreads), 0, stream, rows, cols,
                               src, ld, across, row, col, seed);
    });
    return check_launch(what);
}

extern "C" int fs_mx4_dequantize(const fs_mx4_matrix_t *m, void *out, fs_dtype dtype, int64_t ldo, hipStream_t stream) {
    clear_error();
    const char *what = "fs_mx4_dequantize";
    if (!m) return fail(FS_E_INVAL, "%s: the matrix is NULL", what);
    if (int rc = check_dtype(what, dtype)) return rc;
    Mx4Mat k;
    Footprint read[2], written;
    if (int rc = check_matrix(what, "the matrix", m, &k, read)) return rc;
    if (int rc = check_plain(what, "out", out, m->rows, m->cols, ldo, width(dtype), &written)) return rc;
    if (meet(written, read[0]) || meet(written, read[1])) return fail(FS_E_INVAL, "%s: out overlaps the matrix", what);
    uint32_t across, tiles;
    if (int rc = mat_tiles(what, m->rows, m->cols, kRowTileRows, kRowTileCols, &across, &tiles)) return rc;
    if (tiles == 0) return FS_OK;
    (void)hipGetLastError();
    by_type(dtype, false, [&](auto t, auto) {
        using T = decltype(t);
        hipLaunchKernelGGL(dequantize_mx4_kernel<T>, dim3(tiles), dim3(kThreads), 0, stream, k, m->rows, m->cols,
                           static_cast<T *>(out), m->rows > 1 ? ldo : 0, across);
    });
    return check_launch(what);
}
