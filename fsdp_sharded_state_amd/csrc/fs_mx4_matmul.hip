// fs_mx4_matmul.hip -- the product of two matrices of 4-bit blocks.
#include <string.h>

#include "fs_mx4.h"

using namespace fsi;

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

// The scaled matrix instruction on 16 by 16 outputs and 128 elements of k:
// lane l holds row l%16 and block l/16 of the four, its scale in byte 0 of
// the scale register; output element i of lane l is (row 4*(l/16) + i of the
// first operand, row l%16 of the second).  The second operand is taken from
// `a`, so that a lane's four outputs are consecutive in a row of `out`.
__device__ __forceinline__ f32x4 mfma16(u32x4 x, uint32_t sx, u32x4 y, uint32_t sy, f32x4 acc) {
    const i32x8 p = {(int)x.x, (int)x.y, (int)x.z, (int)x.w, 0, 0, 0, 0};
    const i32x8 q = {(int)y.x, (int)y.y, (int)y.z, (int)y.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(p, q, acc, 4, 4, 0, (int)sx, 0, (int)sy);
}

// The same on 32 by 32 outputs and 64 elements of k: lane l holds row l%32 and
// block l/32 of two, its scale in byte BX (BY); its output 4*g + e is row 8*g + 4*(l/32) + e of the first operand, row l%32 of the second.
template <int BX, int BY>
__device__ __forceinline__ f32x16 mfma32(u32x4 x, uint32_t sx, u32x4 y, uint32_t sy, f32x16 acc) {
    const i32x8 p = {(int)x.x, (int)x.y, (int)x.z, (int)x.w, 0, 0, 0, 0};
    const i32x8 q = {(int)y.x, (int)y.y, (int)y.z, (int)y.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(p, q, acc, 4, 4, BX, (int)sx, BY, (int)sy);
}

__device__ __forceinline__ void store4(float *p, f32x4 v, int64_t valid) {
    if (valid >= 4) {
        __builtin_memcpy(p, &v, 16);
    } else {
        for (int k = 0; k < 4; ++k)
            if (k < valid) p[k] = v[k];
    }
}
__device__ __forceinline__ void store4(uint16_t *p, f32x4 v, int64_t valid) {
    const bf16x4 h = __builtin_convertvector(v, bf16x4);   // rounded to nearest even, two values an instruction
    if (valid >= 4) {
        __builtin_memcpy(p, &h, 8);
    } else {
        uint16_t e[4];
        __builtin_memcpy(e, &h, 8);
        for (int k = 0; k < 4; ++k)
            if (k < valid) p[k] = e[k];
    }
}

// Workgroups go to the 8 XCDs in turn, each with an L2 of its own, and the grid is a
// multiple of 8 or there is a workgroup for every tile: tile `id` is on XCD id % 8.  An XCD
// takes a run of the tile order, in which kGroup tiles down are taken before the
// next column, so the tiles that it works on at a time share rows of both.
constexpr uint32_t kXcds = 8, kGroup = 4;
__device__ __forceinline__ void tile_of(uint32_t id, uint32_t tiles_m, uint32_t tiles_n, uint32_t *tm, uint32_t *tn) {
    const uint32_t total = tiles_m * tiles_n, each = total / kXcds, rest = total % kXcds;
    const uint32_t xcd = id % kXcds, k = id / kXcds;
    const uint32_t at = xcd * each + (xcd < rest ? xcd : rest) + k;   // the first `rest` XCDs have one more
    const uint32_t band = at / (kGroup * tiles_n), in = at % (kGroup * tiles_n);
    const uint32_t high = tiles_m - band * kGroup < kGroup ? tiles_m - band * kGroup : kGroup;
    *tm = band * kGroup + in % high;
    *tn = in / high;
}

// ------------------------------------------------------------ small products --
//
// A workgroup takes 16*FM by 16*FN outputs, and its KW waves share k: wave w
// takes the groups w, w + KW, ... of 16 blocks (four matrix instructions
// deep), fragments straight from memory, all of a group's loads on their way
// at once.  So small products fill the chip, and a single token's reads every
// weight once and no more.  The scales of a row's group come in one load, from
// which each quarter of the wave takes its byte.  The waves' sums are joined
// through LDS, in an order that the sizes alone give.  Rows beyond the matrices read the
// last one, and are not stored.  A launch and the latency of a few loads bound it: 1 by 11008 by 4096 takes 6.9 us, in
// which the weight is read at 3.5 TB/s, 333 by 1000 by 1377 5.1.
template <int FM_, int FN_, int KW_>
struct SmallShape {
    static constexpr int FM = FM_, FN = FN_, KW = KW_, kThreads = 64 * KW;
};

template <class T, class S>
__global__ __launch_bounds__(S::kThreads) void matmul_mx4_small_kernel(Mx4Mat a, Mx4Mat b, int64_t m, int64_t n, int32_t nb,
                                                                       T *__restrict__ out, int64_t ldo, uint32_t tiles_m,
                                                                       uint32_t tiles_n) {
    constexpr int FM = S::FM, FN = S::FN, F = FM + FN, KW = S::KW, kEntries = FM * FN * 64;
    __shared__ f32x4 sums[KW / 2][kEntries];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, kb = lane >> 4;
    uint32_t tm, tn;
    tile_of(blockIdx.x, tiles_m, tiles_n, &tm, &tn);
    const int64_t m0 = (int64_t)tm * 16 * FM, n0 = (int64_t)tn * 16 * FN;
    const uint8_t *code[F], *scale[F];   // of a's rows, then b's
#pragma unroll
    for (int i = 0; i < F; ++i) {
        int64_t c, q;
        if (i < FM) a.row((uint32_t)imin(m0 + 16 * i + r, m - 1), &c, &q);
        else b.row((uint32_t)imin(n0 + 16 * (i - FM) + r, n - 1), &c, &q);
        code[i] = (i < FM ? a.codes : b.codes) + c + kb * kMx4BlockBytes;
        scale[i] = (i < FM ? a.scales : b.scales) + q;
    }
    f32x4 acc[FN][FM] = {};
    auto multiply = [&](const u32x4 (&v)[4][F], const uint32_t (&s)[4][F]) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int j = 0; j < FM; ++j) acc[i][j] = mfma16(v[t][FM + i], s[t][FM + i], v[t][j], s[t][j], acc[i][j]);
    };
    const int32_t whole = nb & ~15;
    for (int32_t k0 = 16 * wave; k0 < whole; k0 += 16 * KW) {
        u32x4 v[4][F], q[F];
        uint32_t s[4][F];
#pragma unroll
        for (int i = 0; i < F; ++i) {
            q[i] = ld16_any(scale[i] + k0);
#pragma unroll
            for (int t = 0; t < 4; ++t) v[t][i] = *reinterpret_cast<const u32x4 *>(code[i] + (int64_t)(k0 + 4 * t) * kMx4BlockBytes);
        }
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
            for (int t = 0; t < 4; ++t) s[t][i] = word(q[i], t) >> (8 * kb);
        multiply(v, s);
    }
    if (whole < nb && (whole >> 4) % KW == wave) {   // the last group, block by block
        u32x4 v[4][F];
        uint32_t s[4][F];
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                v[t][i] = u32x4{0, 0, 0, 0};
                s[t][i] = 127;
                if (whole + 4 * t + kb < nb) {
                    v[t][i] = *reinterpret_cast<const u32x4 *>(code[i] + (int64_t)(whole + 4 * t) * kMx4BlockBytes);
                    s[t][i] = scale[i][whole + 4 * t + kb];
                }
            }
        multiply(v, s);
    }
    // the upper waves' sums to the lower ones, then theirs to all
    auto entry = [&](int i, int j) { return (i * FM + j) * 64 + lane; };
    if (wave >= KW / 2) {
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < FM; ++j) sums[wave - KW / 2][entry(i, j)] = acc[i][j];
    }
    __syncthreads();
    if (wave < KW / 2) {
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < FM; ++j) sums[wave][entry(i, j)] += acc[i][j];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < kEntries; e += S::kThreads) {
        f32x4 v = sums[0][e];
#pragma unroll
        for (int w = 1; w < KW / 2; ++w) v += sums[w][e];
        const int frag = e >> 6, l = e & 63;
        const int64_t row = m0 + 16 * (frag % FM) + (l & 15), col = n0 + 16 * (frag / FM) + 4 * (l >> 4);
        if (row < m && col < n) store4(out + row * ldo + col, v, n - col);
    }
}

// ------------------------------------------------------------ large products --
//
// A workgroup of eight waves takes 256 by 256 outputs, a wave 64 by 128.  k goes
// in steps of 4 blocks (64 bytes of a row), each one round of matrix
// instructions; the codes of four steps lie in LDS, filled by asynchronous
// loads that bypass the registers.  During a round the fragments of the next
// one are read.  Where a round starts, its own step's place in LDS is free
// again and takes the step four further on, so a load has three rounds to arrive.
//
// The 32 by 32 instruction is used as it keeps its rate with one scale register for each operand
// (33 cycles of the 32 that its size stands for; the 16 by 16 one took 23 to 30 for 16).
//
// A row's 16 scales for four steps are loaded at once and stored with
// those of either half of the wave side by side: one 64-bit read gives a lane
// its scales for four rounds, and the instruction selects the byte.
//
// A row's four 16-byte chunks are stored at places exchanged by two bits of
// the row, so that the 16 lanes of a read phase hit all banks; the loads write
// LDS in lane order, so each lane fetches the chunk that belongs at its place.
// The loads check their bounds: what lies beyond a row's blocks is fetched
// from an offset outside, which gives zeros.
//
// There is a workgroup for each CU (its LDS holds one), which takes tile after tile:
// the last rounds of a tile load the first steps of the next, so neither
// the start of a tile nor the writing of its outputs leaves the loads idle.
// Outputs go through LDS, a part of a wave's tile at a time, so that stores cover whole cache lines.
//
// 8192 by 11008 by 4096 to bf16 takes 194 to 206 us, 3.6 to 3.8 PFLOP/s, 11008 by 4096 by 8192 to fp32 187 to 200, 3.7 to 3.9,
// from one MI355X to another.  The matrix instructions alone, on data, run at 6.8 PFLOP/s here, as power holds the clock
// under 1.9 GHz: 109 us.  With the rounds' waits and LDS reads and without loads they take 135 to 140, the loads add about 23, the scales 9 of them, and
// the outputs the rest; 1376 and 688 tiles are 5.4 of 6 turns of 256 workgroups and 2.7 of 3.

constexpr int kStepBlocks = 4;       // blocks of k in a step
constexpr int kStepBytes = kStepBlocks * kMx4BlockBytes;
constexpr int kStages = 4;           // steps in LDS
// A tile's rows are addressed by 32-bit offsets from its first one.
constexpr int64_t kBigMaxOffset = (int64_t)1 << 31;

typedef __attribute__((address_space(3))) void *LdsPtr;

#ifdef __HIP_DEVICE_COMPILE__   // the host pass does not know the buffer builtins
// A buffer of kBigMaxOffset - 1 bytes from p on, which is the same in every lane.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_from(const uint8_t *p) {
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint64_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)v), hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32));
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void *>(hi << 32 | lo), 0, (int)(kBigMaxOffset - 1), 0x00020000);
}

// x, in a register that the compiler computes nothing from ahead of this place.
__device__ __forceinline__ int hidden(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

// Waits until no more than N of this wave's loads are on their way and its LDS
// accesses are done, then for every wave.  One piece of assembly, as the fence of __syncthreads
// would wait for every load into LDS, the steps still to come among them.
template <int N>
__device__ __forceinline__ void loads_and_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}
#endif

constexpr int kPartBytes = 2048;   // of LDS a wave's outputs go through

// A tile of BM rows of a by BN of b, in GM by GN waves.
template <int BM_, int BN_, int GM, int GN>
struct BigShape {
    static constexpr int BM = BM_, BN = BN_, kWaves = GM * GN, kThreads = 64 * kWaves;
    static constexpr int kGridN = GN;
    static constexpr int FM = BM / GM / 32, FN = BN / GN / 32;         // a wave's fragments
    static constexpr int kLoadRows = 64 * kMx4BlockBytes / kStepBytes;                // rows of one load
    static constexpr int LM = BM / kWaves / kLoadRows, LN = BN / kWaves / kLoadRows;  // a wave's loads of a step
    static constexpr int kRows = BM + BN, kScaleLoads = (kRows + kThreads - 1) / kThreads;
    static constexpr int kBuf = kRows * kStepBytes, kScales = kRows * 16;
    static constexpr int kPerCu = 163840 / (kStages * kBuf + 2 * kScales + kWaves * kPartBytes);   // workgroups of a CU, by their LDS
    static_assert(LM * kWaves * kLoadRows == BM && LN * kWaves * kLoadRows == BN && FM * GM * 32 == BM && FN * GN * 32 == BN, "whole fragments and loads");
    static_assert(FN % 2 == 0, "fragments of b come in pairs");
};

template <class T, class S>
__global__ __launch_bounds__(S::kThreads, S::kWaves * S::kPerCu / 4) void matmul_mx4_big_kernel(Mx4Mat a, Mx4Mat b, int64_t m, int64_t n,
                                                                                    int32_t nb, T *__restrict__ out,
                                                                                    int64_t ldo, uint32_t tiles_m,
                                                                                    uint32_t tiles_n) {
#ifdef __HIP_DEVICE_COMPILE__
    constexpr int BM = S::BM, BN = S::BN, FM = S::FM, FN = S::FN;
    // one array a stage, so that the compiler can tell the loads into one from the reads of another
    __shared__ __attribute__((aligned(128))) uint8_t buf0[S::kBuf], buf1[S::kBuf], buf2[S::kBuf], buf3[S::kBuf];   // a's rows, then b's
    __shared__ __attribute__((aligned(128))) uint8_t scl[2][S::kScales];
    __shared__ __attribute__((aligned(128))) uint8_t part[S::kWaves][kPartBytes];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t tiles = tiles_m * tiles_n;

    // The tile to load: this thread's rows, chunk `chunk` of each step.
    const int chunk = (lane & 3) ^ (lane >> 4);
    __amdgpu_buffer_rsrc_t ra, rb;
    uint32_t oa[S::LM], ob[S::LN];
    const uint8_t *sp[S::kScaleLoads];   // and of the scales
    auto aim = [&](int64_t m0, int64_t n0) {
        int64_t a0, b0, c, sc;
        const int l = hidden(lane), load_row = l >> 2;
        a.row((uint32_t)m0, &a0, &sc);
        b.row((uint32_t)n0, &b0, &sc);
        ra = buffer_from(a.codes + a0);
        rb = buffer_from(b.codes + b0);
#pragma unroll
        for (int j = 0; j < S::LM; ++j) {
            a.row((uint32_t)imin(m0 + (wave * S::LM + j) * S::kLoadRows + load_row, m - 1), &c, &sc);
            oa[j] = (uint32_t)(c - a0) + chunk * kMx4BlockBytes;
        }
#pragma unroll
        for (int j = 0; j < S::LN; ++j) {
            b.row((uint32_t)imin(n0 + (wave * S::LN + j) * S::kLoadRows + load_row, n - 1), &c, &sc);
            ob[j] = (uint32_t)(c - b0) + chunk * kMx4BlockBytes;
        }
#pragma unroll
        for (int j = 0; j < S::kScaleLoads; ++j) {
            const int q = j * S::kThreads + wave * 64 + l;   // rows beyond the tile (q >= kRows) are loaded, not stored
            if (q < BM) a.row((uint32_t)imin(m0 + q, m - 1), &c, &sc);
            else b.row((uint32_t)imin(n0 + q - BM, n - 1), &c, &sc);
            sp[j] = (q < BM ? a.scales : b.scales) + sc;
        }
    };

    constexpr int kLoads = S::LM + S::LN;   // of a step
    auto load_codes = [&](uint8_t *buf, int32_t step, int k) {   // one of them
        const uint32_t beyond = step * kStepBlocks + chunk < nb ? 0u : 0x80000000u;
        const int at = step * kStepBytes;
        if (k < S::LM)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (LdsPtr)(buf + (wave * S::LM + k) * 1024), 16, oa[k] | beyond, at, 0, 0);
        else
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (LdsPtr)(buf + BM * kStepBytes + (wave * S::LN + k - S::LM) * 1024), 16,
                                                     ob[k - S::LM] | beyond, at, 0, 0);
    };
    // 16 scales of a row; a last group is loaded so that it ends with the row, and shifted down.  A row of fewer comes
    // byte by byte, and needs the same shift.
    u32x4 sv[S::kScaleLoads];
    auto load_scales = [&](int32_t k0) {
        const int32_t first = k0 + 16 <= nb ? k0 : nb - 16;
#pragma unroll
        for (int j = 0; j < S::kScaleLoads; ++j) {
            if (nb >= 16) {
                sv[j] = ld16_any(sp[j] + first);
            } else {
                uint32_t w[4] = {};
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    if (first + k >= 0) w[k >> 2] |= (uint32_t)sp[j][first + k] << (8 * (k & 3));
                sv[j] = u32x4{w[0], w[1], w[2], w[3]};
            }
        }
    };
    auto store_scales = [&](uint8_t *s, int32_t k0) {
        const int over = (int)imax(0, imin(16, k0 + 16 - nb));   // bytes that belong to earlier groups
#pragma unroll
        for (int j = 0; j < S::kScaleLoads; ++j) {
            const int q = j * S::kThreads + tid;
            uint64_t lo = (uint64_t)sv[j].y << 32 | sv[j].x, hi = (uint64_t)sv[j].w << 32 | sv[j].z;
            if (over >= 8) lo = hi, hi = 0;
            const int bits = 8 * (over & 7);
            lo = over == 16 ? 0 : lo >> bits | (hi << 1) << (63 - bits);
            hi >>= bits;
            // the halves' bytes, even and odd ones, side by side
            const uint32_t w0 = (uint32_t)lo, w1 = (uint32_t)(lo >> 32), w2 = (uint32_t)hi, w3 = (uint32_t)(hi >> 32);
            if (S::kRows % S::kThreads == 0 || q < S::kRows)
                *reinterpret_cast<u32x4 *>(s + q * 16) =
                    u32x4{__builtin_amdgcn_perm(w1, w0, 0x06040200), __builtin_amdgcn_perm(w3, w2, 0x06040200),
                          __builtin_amdgcn_perm(w1, w0, 0x07050301), __builtin_amdgcn_perm(w3, w2, 0x07050301)};
        }
    };

    const int wm = wave / S::kGridN * (FM * 32), wn = wave % S::kGridN * (FN * 32);
    // Lane l reads row l%32 of a fragment and, of the step's four blocks, l/32 and l/32 + 2 in the round's two halves.
    const int r = lane & 31, q = lane >> 5;
    const int place = (q ^ ((r >> 2) & 3)) * kMx4BlockBytes;   // of the first half; the second's has bit 1 of the place flipped
    const int at_a = (wm + r) * kStepBytes + place, at_b = (BM + wn + r) * kStepBytes + place;
    const int at_sx = (BM + wn + r) * 16 + q * 8, at_sy = (wm + r) * 16 + q * 8;
    // An LDS instruction holds an offset of 16 bits, so the upper stages have bases
    // of their own, hidden from the compiler, which would otherwise make one for every read.
    const int base_a[2][2] = {{at_a, at_a ^ 32}, {hidden(at_a + 65536), hidden((at_a ^ 32) + 65536)}};
    const int base_b[2][2] = {{at_b, at_b ^ 32}, {hidden(at_b + 65536), hidden((at_b ^ 32) + 65536)}};
    // Fragments of the two halves.  Each is read anew as soon as its products are issued.  What the round needs to its end,
    // a's second half and the last of b's, is doubled, so that the last reads have products after them to arrive behind.
    u32x4 x[2][FN], xl[2], y0[FM], y1[2][FM];
    u32x2 sx[FN], sy[FM], nsy[FM];      // scales for four rounds
    auto read_x = [&](u32x4 &x, const uint8_t *buf, int up, int h, int i) {
        x = *reinterpret_cast<const u32x4 *>(&buf[base_b[up][h] - up * 65536 + i * 32 * kStepBytes]);
    };
    auto read_y = [&](u32x4 &y, const uint8_t *buf, int up, int h, int j) {
        y = *reinterpret_cast<const u32x4 *>(&buf[base_a[up][h] - up * 65536 + j * 32 * kStepBytes]);
    };
    auto read_sx = [&](const uint8_t *s, int i) { sx[i] = *reinterpret_cast<const u32x2 *>(s + at_sx + i * 512); };
    auto read_sy = [&](const uint8_t *s) {
#pragma unroll
        for (int j = 0; j < FM; ++j) nsy[j] = *reinterpret_cast<const u32x2 *>(s + at_sy + j * 512);
    };
    f32x16 acc[FN][FM];
    // Round `st` of four with the fragments at hand, which reads the next round's from `buf` and, in the last of four, the
    // next scales from `s`.  It loads step `step` into `to`, spread over the products: a wave's loads in a row would
    // wait for each other, and its products for them.
    auto round = [&](auto st_, const uint8_t *buf, const uint8_t *s, uint8_t *to, int32_t step) {
        constexpr int st = decltype(st_)::value, byte = 2 * (st & 1);
        constexpr int up = st == 1 || st == 2;
        auto load = [&](int i) {
#pragma unroll
            for (int k = i * kLoads / (2 * FN); k < (i + 1) * kLoads / (2 * FN); ++k) load_codes(to, step, k);
        };
#pragma unroll
        for (int i = 0; i < FN; ++i) {
#pragma unroll
            for (int j = 0; j < FM; ++j)
                acc[i][j] = mfma32<byte, byte>(x[0][i], st < 2 ? sx[i].x : sx[i].y, y0[j], st < 2 ? sy[j].x : sy[j].y, acc[i][j]);
            load(i);
            read_x(x[0][i], buf, up, 0, i);
            if (i < FM) read_y(y1[(st & 1) ^ 1][i], buf, up, 1, i);
            if (i == FN - 1) {
                read_x(xl[(st & 1) ^ 1], buf, up, 1, FN - 1);
#pragma unroll
                for (int j = 0; j < FM; ++j) read_y(y0[j], buf, up, 0, j);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < FN; ++i) {
#pragma unroll
            for (int j = 0; j < FM; ++j)
                acc[i][j] = mfma32<byte + 1, byte + 1>(i == FN - 1 ? xl[st & 1] : x[1][i], st < 2 ? sx[i].x : sx[i].y, y1[st & 1][j],
                                                       st < 2 ? sy[j].x : sy[j].y, acc[i][j]);
            load(FN + i);
            if (i < FN - 1) read_x(x[1][i], buf, up, 1, i);
            if (st == 3) read_sx(s, i);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // A wave's outputs: 16 rows by 128 bytes at a time through its part of LDS.  A row's 16-byte pieces are exchanged by
    // its low bits, so that neither side meets in a bank.
    uint8_t *mine = part[wave];
    auto store_tile = [&](int64_t m0, int64_t n0) {
        constexpr int kWide = 128 / sizeof(T), kFrags = kWide / 32;   // columns and fragments of a part
        constexpr int kPiece = 16 / sizeof(T);                        // elements of 16 bytes
        const int l = hidden(lane), r = l & 15, q = l >> 5;
        const int64_t row = m0 + wm + (l >> 3), col = n0 + wn + (l & 7) * kPiece;
        const bool past = on16(out) && ldo * sizeof(T) % 16 == 0;   // past the caches: 194 us for 209 (11008 by 4096 by 8192)
#pragma unroll
        for (int j = 0; j < 2 * FM; ++j)
#pragma unroll
            for (int h = 0; h < FN / kFrags; ++h) {
                if (((l >> 4) & 1) == (j & 1)) {
#pragma unroll
                    for (int i = 0; i < kFrags; ++i)
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            const int at = 32 * i + 8 * g + 4 * q, piece = at / kPiece, low = at % kPiece;
                            const f32x16 &v = acc[h * kFrags + i][j >> 1];
                            store4(reinterpret_cast<T *>(mine + r * 128 + ((piece ^ (r & 7)) * 16)) + low,
                                   f32x4{v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]}, 4);
                        }
                }
                wave_meets();
                u32x4 v[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int lr = (l >> 3) + 8 * k;
                    v[k] = *reinterpret_cast<const u32x4 *>(mine + lr * 128 + (((l & 7) ^ (lr & 7)) * 16));
                }
                wave_meets();
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int64_t to = row + 16 * j + 8 * k, from = col + h * kWide;
                    if (to < m) {
                        T *p = out + to * ldo + from;
                        if (from + kPiece <= n) {
                            if (past) st16(reinterpret_cast<char *>(p), v[k]);
                            else st16_any(p, v[k]);
                        } else {
                            T e[kPiece];
                            __builtin_memcpy(e, &v[k], 16);
                            for (int c = 0; c < kPiece; ++c)
                                if (from + c < n) p[c] = e[c];
                        }
                    }
                }
            }
    };
    constexpr int kBehind = 2 * kLoads;   // loads of the two latest steps

    // Groups of four steps.  Without a block there is one all the same, which multiplies zeros: the way to the next tile
    // leads through it.
    const int32_t groups = nb > 0 ? (nb + 15) / 16 : 1;
    uint32_t tile = blockIdx.x, tm, tn;
    tile_of(tile, tiles_m, tiles_n, &tm, &tn);
    aim((int64_t)tm * BM, (int64_t)tn * BN);
    load_scales(0);
#pragma unroll
    for (int k = 0; k < kLoads; ++k) load_codes(buf0, 0, k);
#pragma unroll
    for (int k = 0; k < kLoads; ++k) load_codes(buf1, 1, k);
#pragma unroll
    for (int k = 0; k < kLoads; ++k) load_codes(buf2, 2, k);
#pragma unroll
    for (int k = 0; k < kLoads; ++k) load_codes(buf3, 3, k);
    store_scales(scl[0], 0);
    loads_and_barrier<kBehind + kLoads>();
    read_sy(scl[0]);
#pragma unroll
    for (int i = 0; i < FN; ++i) {
        read_x(x[0][i], buf0, 0, 0, i);
        if (i < FN - 1) read_x(x[1][i], buf0, 0, 1, i);
        else read_x(xl[0], buf0, 0, 1, i);
        read_sx(scl[0], i);
    }
#pragma unroll
    for (int j = 0; j < FM; ++j) {
        read_y(y0[j], buf0, 0, 0, j);
        read_y(y1[0][j], buf0, 0, 1, j);
    }
    int odd = 0;
    for (;;) {
        const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
        const bool more = tile + gridDim.x < tiles;
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < FM; ++j) acc[i][j] = f32x16{};
        for (int32_t g = 0; g < groups; ++g) {
            int32_t load = g + 1;   // the group to load
            if (load == groups && more) {
                tile += gridDim.x;
                tile_of(tile, tiles_m, tiles_n, &tm, &tn);
                aim((int64_t)tm * BM, (int64_t)tn * BN);
                load = 0;
            }
            uint8_t *next = scl[odd ^= 1];
#pragma unroll
            for (int i = 0; i < FM; ++i) sy[i] = nsy[i];
            loads_and_barrier<kBehind>();
            load_scales(16 * load);
            round(std::integral_constant<int, 0>{}, buf1, next, buf0, 4 * load);
            loads_and_barrier<kBehind>();
            round(std::integral_constant<int, 1>{}, buf2, next, buf1, 4 * load + 1);
            loads_and_barrier<kBehind>();
            round(std::integral_constant<int, 2>{}, buf3, next, buf2, 4 * load + 2);
            store_scales(next, 16 * load);
            loads_and_barrier<kBehind>();
            read_sy(next);
            round(std::integral_constant<int, 3>{}, buf0, next, buf3, 4 * load + 3);
        }
        store_tile(m0, n0);
        if (!more) break;
    }
    loads_and_barrier<0>();             // nothing may be on its way into LDS when the workgroup ends
#endif
}

constexpr int kBig = 256;   // the longest side of a tile

// Workgroups that run at a time.
template <class S>
int64_t big_grid() {
    const CuLimits L = cu_limits();
    return (L.cus > 0 ? L.cus : 256) * S::kPerCu;
}

template <class T, class S>
int launch_big(const char *what, const Mx4Mat &a, const Mx4Mat &b, int64_t m, int64_t n, int64_t nb, void *out, int64_t ldo,
               hipStream_t stream) {
    const int64_t tm = (m + S::BM - 1) / S::BM, tn = (n + S::BN - 1) / S::BN;
    if (tm * tn > INT32_MAX) return fail(FS_E_OVERFLOW, "%s: too many outputs for one launch", what);
    hipLaunchKernelGGL((matmul_mx4_big_kernel<T, S>), dim3((uint32_t)imin(tm * tn, big_grid<S>())), dim3(S::kThreads), 0,
                       stream, a, b, m, n, (int32_t)nb, static_cast<T *>(out), ldo, (uint32_t)tm, (uint32_t)tn);
    return check_launch(what);
}

template <class T, class S>
int launch_small(const char *what, const Mx4Mat &a, const Mx4Mat &b, int64_t m, int64_t n, int64_t nb, void *out, int64_t ldo,
                 hipStream_t stream) {
    const int64_t tm = (m + 16 * S::FM - 1) / (16 * S::FM), tn = (n + 16 * S::FN - 1) / (16 * S::FN);
    if (tm * tn > UINT32_MAX / S::kThreads) return fail(FS_E_OVERFLOW, "%s: too many outputs for one launch", what);
    hipLaunchKernelGGL((matmul_mx4_small_kernel<T, S>), dim3((uint32_t)(tm * tn)), dim3(S::kThreads), 0, stream, a, b, m, n,
                       (int32_t)nb, static_cast<T *>(out), ldo, (uint32_t)tm, (uint32_t)tn);
    return check_launch(what);
}

// Whether the offsets of a tile's rows fit (those of any 256 consecutive ones).
bool big_offsets(const Mx4Mat &k, int64_t nb) {
    const int64_t jumps = k.chunk_rows ? kBig / k.chunk_rows + 1 : 0;
    return k.code_stride < kBigMaxOffset / kBig / 2 && nb * kMx4BlockBytes < kBigMaxOffset / 8 &&
           (jumps == 0 || k.chunk_stride < kBigMaxOffset / 4 / jumps);
}

}  // namespace

extern "C" int fs_mx4_matmul(const fs_mx4_matrix_t *a, const fs_mx4_matrix_t *b, void *out, fs_dtype dtype, int64_t ldo,
                             hipStream_t stream) {
    clear_error();
    const char *what = "fs_mx4_matmul";
    if (!a || !b) return fail(FS_E_INVAL, "%s: a matrix is NULL", what);
    if (dtype != FS_BF16 && dtype != FS_FP32) return fail(FS_E_DTYPE, "%s: unknown dtype %d", what, (int)dtype);
    Mx4Mat ka, kb;
    Footprint ra[2], rb[2];
    if (int rc = check_matrix(what, "a", a, &ka, ra)) return rc;
    if (int rc = check_matrix(what, "b", b, &kb, rb)) return rc;
    if (a->cols != b->cols)
        return fail(FS_E_INVAL, "%s: a has %lld columns, b %lld", what, (long long)a->cols, (long long)b->cols);
    const int64_t m = a->rows, n = b->rows, k = a->cols, w = dtype == FS_BF16 ? 2 : 4;
    if (m == 0 || n == 0) return FS_OK;
    if (!out) return fail(FS_E_INVAL, "%s: out is NULL", what);
    if (misaligned(out, w)) return fail(FS_E_ALIGN, "%s: out not aligned to its element size", what);
    if (m > 1 && ldo < n) return fail(FS_E_INVAL, "%s: the rows of out overlap", what);
    if (m > 1 && ldo > ((int64_t)1 << 56) / m) return fail(FS_E_OVERFLOW, "%s: out is too large", what);
    const int64_t nb = mx4_blocks(k), ld = m > 1 ? ldo : 0;
    const Footprint written{out, ((m - 1) * ld + n) * w, ld * w, n * w, "out"};
    for (const Footprint &f : {ra[0], ra[1], rb[0], rb[1]})
        if (meet(written, f)) return fail(FS_E_INVAL, "%s: out overlaps a matrix", what);
    (void)hipGetLastError();
    // By the tiles that there are for 256 CUs, measured over m from 1 to 4096, n and k from 512 to 11008 (us, in a graph).
    // 16 by 16 up to 512 tiles, or where 16 rows are all: 4.4 for 5.9 of the next (1 by 4096 by 4096), 7.1 for 8.9 (1 by
    //   11008 by 4096), 7.4 for 7.8 (128 by 1024 by 4096); past it 12.0 for 7.9 (256 by 1024 by 4096).
    // 32 by 32 up to 512: 7.9 for 12.0 (64 by 4096 by 4096), 5.4 for 6.9 (128 by 4096 by 1024); past it 17.0 for 12.4 (64 by
    //   11008 by 4096), 45 for 31 (1024 by 1024 by 11008).
    // 128 by 128 while 256 by 256 would give no more than 128: 16.5 for 27.7 (1024 by 4096 by 4096), 29.3 for 31.2 (2048 by 4096
    //   by 4096); past it 38.9 for 33.9 (1024 by 11008 by 4096), 141 for 109 (4096 by 11008 by 4096).
    auto tiles = [&](int64_t side) { return ((m + side - 1) / side) * ((n + side - 1) / side); };
    const bool offsets = big_offsets(ka, nb) && big_offsets(kb, nb);
    auto go = [&](auto t) {
        using T = decltype(t);
        if (m <= 16 || tiles(16) <= 512) return launch_small<T, SmallShape<1, 1, 8>>(what, ka, kb, m, n, nb, out, ld, stream);
        if (tiles(32) <= 512 || !offsets) return launch_small<T, SmallShape<2, 2, 8>>(what, ka, kb, m, n, nb, out, ld, stream);
        if (tiles(256) <= 128) return launch_big<T, BigShape<128, 128, 2, 2>>(what, ka, kb, m, n, nb, out, ld, stream);
        return launch_big<T, BigShape<256, 256, 4, 2>>(what, ka, kb, m, n, nb, out, ld, stream);
    };
    return dtype == FS_BF16 ? go(uint16_t{}) : go(float{});
}
