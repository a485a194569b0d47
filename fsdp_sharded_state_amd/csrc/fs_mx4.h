// fs_mx4.h -- the microscaled 4-bit block format as the kernels of both MX4
// sources make and read it.  Not part of the public ABI.
//
// A lane that quantises works on 8 consecutive elements: 4 bytes of codes, a quarter of a
// block.  The four lanes of a quad hold one block, so its largest magnitude
// is joined by two quad permutes and no LDS.  CDNA4 converts a pair of values
// to codes and back, scale and rounding included, in one instruction each
// (checked bit for bit against the definition over every bf16 value at every
// scale, fp32 values on and beside every midpoint, and every code at every
// scale): 4 instructions a lane, so the conversions stay under the HBM time.
#pragma once
#include <type_traits>

#include "fs_device.h"
#include "fs_mx4_plan.h"

namespace fsi {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// Accesses to global memory through any pointer.  Where the pointer was itself
// read from memory the compiler would take the generic ones, which are slower: the copy-out
// of 45M fp32 elements to odd addresses took 46 us with those, 34 with these.
template <class T>
using Global = __attribute__((address_space(1))) T;
template <class T>
__device__ __forceinline__ T ld(const T *p) {
    return *(const Global<T> *)reinterpret_cast<uintptr_t>(p);
}
template <class T>
__device__ __forceinline__ void st(T *p, T v) {
    *(Global<T> *)reinterpret_cast<uintptr_t>(p) = v;
}
// 16 bytes at any element-aligned address: the target allows unaligned vector accesses.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
__device__ __forceinline__ u32x4 ld16_any(const void *p) { return *(const Global<u32x4_any> *)reinterpret_cast<uintptr_t>(p); }
__device__ __forceinline__ void st16_any(void *p, u32x4 v) { *(Global<u32x4_any> *)reinterpret_cast<uintptr_t>(p) = v; }
// Past the caches, on 16 bytes.  Elements pass through once, and what a call
// leaves in the caches to be written back costs the next one: copy-in and copy-out of one 7B block
// in bf16 take 206 us without, 156 with.  Off 16 bytes lanes share sectors, which the caches have to join
// (45M fp32 elements to odd addresses: 34 us through the caches, 84 past them).
// The two kinds of access are chosen by a template argument: the compiler makes one of a choice beside them.
template <bool PAST>
__device__ __forceinline__ u32x4 ld16_el(const void *p) {
    if (PAST) return __builtin_nontemporal_load((const Global<u32x4> *)reinterpret_cast<uintptr_t>(p));
    return ld16_any(p);
}
template <bool PAST>
__device__ __forceinline__ void st16_el(void *p, u32x4 v) {
    if (PAST) __builtin_nontemporal_store(v, (Global<u32x4> *)reinterpret_cast<uintptr_t>(p));
    else st16_any(p, v);
}
// f(std::bool_constant<past>())
template <class F>
__device__ __forceinline__ void with_past(bool past, F &&f) {
    if (past) f(std::true_type{});
    else f(std::false_type{});
}

// Eight elements of either type as they lie in memory.
template <class T>
struct Raw8;
template <>
struct Raw8<uint16_t> {
    u32x4 v;
};
template <>
struct Raw8<float> {
    u32x4 v[2];
};

__device__ __forceinline__ bool on16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

__device__ __forceinline__ uint32_t word(const u32x4 &v, int k) { return k == 0 ? v.x : k == 1 ? v.y : k == 2 ? v.z : v.w; }
// Elements of 16 bytes, and units of that size in a lane's eight.
template <class T>
constexpr int kUnit = 16 / sizeof(T);
template <class T>
constexpr int kUnits = 8 / kUnit<T>;

// `valid` (any value) elements of a unit at p, zeros after them.
template <bool PAST>
__device__ __forceinline__ u32x4 load_unit(const uint16_t *p, int valid) {
    if (valid >= 8) return ld16_el<PAST>(p);
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t lo = 2 * k < valid ? ld(p + 2 * k) : 0, hi = 2 * k + 1 < valid ? ld(p + 2 * k + 1) : 0;
        w[k] = lo | (hi << 16);
    }
    return u32x4{w[0], w[1], w[2], w[3]};
}
template <bool PAST>
__device__ __forceinline__ u32x4 load_unit(const float *p, int valid) {
    if (valid >= 4) return ld16_el<PAST>(p);
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = k < valid ? __float_as_uint(ld(p + k)) : 0u;
    return u32x4{w[0], w[1], w[2], w[3]};
}
template <bool PAST>
__device__ __forceinline__ void store_unit(uint16_t *p, const u32x4 &v, int valid) {
    if (valid >= 8) {
        st16_el<PAST>(p, v);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < valid) st(p + k, (uint16_t)(word(v, k >> 1) >> (16 * (k & 1))));
    }
}
template <bool PAST>
__device__ __forceinline__ void store_unit(float *p, const u32x4 &v, int valid) {
    if (valid >= 4) {
        st16_el<PAST>(p, v);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < valid) st(p + k, __uint_as_float(word(v, k)));
    }
}

// The lanes of a wave meet, their LDS accesses before this place before those
// after it.  (The hardware keeps a wave's LDS accesses in order; this keeps the compiler to it.)
__device__ __forceinline__ void wave_meets() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// A lane's eight fp32 values are two units.  With each lane at its own two, an access of the wave would hold half of
// each cache line.  So units go to the lanes in turn, lane l taking
// units l and 64 + l of the wave's 128, and are exchanged through 2 KB of LDS for 2l and 2l + 1, its own: one 7B block
// in fp32 both ways 397 us -> 308, its shard's reduce 39.3 -> 34.9, 8192 by 11008 from fp32 92 -> 78 and back 99 -> 62.
__device__ __forceinline__ Raw8<uint16_t> own_units(const u32x4 (&v)[1], u32x4 *) { return Raw8<uint16_t>{v[0]}; }
__device__ __forceinline__ Raw8<float> own_units(const u32x4 (&v)[2], u32x4 *of_wave) {
    const int lane = threadIdx.x & 63;
    of_wave[lane] = v[0];
    of_wave[64 + lane] = v[1];
    wave_meets();
    const Raw8<float> r{{of_wave[2 * lane], of_wave[2 * lane + 1]}};
    wave_meets();
    return r;
}
// And back.
__device__ __forceinline__ void units_in_turn(u32x4 (&v)[2], const float (&own)[8], u32x4 *of_wave) {
    const int lane = threadIdx.x & 63;
    __builtin_memcpy(&of_wave[2 * lane], own, 32);
    wave_meets();
    v[0] = of_wave[lane];
    v[1] = of_wave[64 + lane];
    wave_meets();
}

// Element k as fp32.
__device__ __forceinline__ float elem(const Raw8<uint16_t> &r, int k) {
    const uint32_t w = word(r.v, k >> 1);
    return __uint_as_float(k & 1 ? w & 0xFFFF0000u : w << 16);
}
__device__ __forceinline__ float elem(const Raw8<float> &r, int k) { return __uint_as_float(word(r.v[k >> 2], k & 3)); }

// Bits of the largest magnitude as fp32: as integers they are ordered like
// the magnitudes, with the infinity above every number and NaN above it.
__device__ __forceinline__ uint32_t amax8(const Raw8<uint16_t> &r) {
    u16x2 m = __builtin_bit_cast(u16x2, r.v.x & 0x7FFF7FFFu);
#pragma unroll
    for (int k = 1; k < 4; ++k)
        m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, word(r.v, k) & 0x7FFF7FFFu));
    return (uint32_t)max(m.x, m.y) << 16;
}
__device__ __forceinline__ uint32_t amax8(const Raw8<float> &r) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max(m, word(r.v[k >> 2], k & 3) & 0x7FFFFFFFu);
    return m;
}

// The largest of the quad's four values, in each of its lanes.
__device__ __forceinline__ uint32_t quad_max(uint32_t x) {
    x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0xB1, 0xF, 0xF, true));   // lanes 1 0 3 2
    return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x4E, 0xF, 0xF, true));   // lanes 2 3 0 1
}

// The scale byte of a block whose largest magnitude has these bits.
template <bool STOCHASTIC>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
    const uint32_t e = amax >> 23;
    if (e == 255) return 255;
    uint32_t s = max(e, 2u) - 2;
    if (STOCHASTIC && e >= 2 && (amax & 0x7FFFFFu) > 0x400000u) ++s;
    return s;
}
// 2^(s - 127).  For 255 the infinity's bits: the conversions go by the
// exponent alone, and give NaN for every code.
__device__ __forceinline__ float scale_value(uint32_t s) { return __uint_as_float(max(s << 23, 0x00400000u)); }

// (a copy first: a bit cast of a vector's element takes the vector's first)
__device__ __forceinline__ bf16x2 bf16_pair(const u32x4 &v, int k) {
    const uint32_t w = word(v, k);
    return __builtin_bit_cast(bf16x2, w);
}

__device__ __forceinline__ uint32_t encode_nearest(const Raw8<uint16_t> &r, float scale) {
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, bf16_pair(r.v, 0), scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, bf16_pair(r.v, 1), scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, bf16_pair(r.v, 2), scale, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, bf16_pair(r.v, 3), scale, 3);
    return c;
}
__device__ __forceinline__ uint32_t encode_nearest(const Raw8<float> &r, float scale) {
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, elem(r, 0), elem(r, 1), scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, elem(r, 2), elem(r, 3), scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, elem(r, 4), elem(r, 5), scale, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, elem(r, 6), elem(r, 7), scale, 3);
    return c;
}

__device__ __forceinline__ uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) {
    return (uint32_t)__builtin_amdgcn_bitop3_b32((int)a, (int)b, (int)c, 0x96);   // the truth table of a ^ b ^ c
}

struct Random8 {
    uint32_t w[4];
};

// Philox4x32 with 7 rounds.  Seven are the fewest that pass its authors'
// statistical tests; with 16 bits an element a call serves 8 of them.
__device__ __forceinline__ Random8 philox8(uint64_t seed, uint64_t group, uint32_t orientation) {
    uint32_t c0 = (uint32_t)group, c1 = (uint32_t)(group >> 32), c2 = orientation, c3 = 0;
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
    for (int i = 0; i < 7; ++i) {
        const uint64_t p0 = (uint64_t)c0 * 0xD2511F53u, p1 = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = xor3((uint32_t)(p1 >> 32), c1, k0);
        c1 = (uint32_t)p1;
        c2 = xor3((uint32_t)(p0 >> 32), c3, k1);
        c3 = (uint32_t)p0;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return Random8{{c0, c1, c2, c3}};
}

// Stochastic codes of 8 elements: with y = |x| / 2^(s-127) <= 6, P the power
// of two at or below y but at least 1, and P/2 the step of y's codes, y goes
// up from the code at or below it where the fraction f of the step exceeds
// t = (r + 0.5) / 65536.  The instruction that rounds to nearest then makes the code.
//
// bf16: it is given y + (0.5 - t) * P/2, which it rounds up where f > t.  y
// has 8 significant bits and (0.5 - t) * P/2 is a multiple of P * 2^-18, so the
// sum is exact from y = 2^-18 on, and below that f < 2^-17 <= t: the sum, at
// most 0.25, goes down.  A tie, f = t, needs as many fraction bits as t has, which y has only below
// 0.5: there the even code, zero, is the lower one.  The sum may lie under the power of two
// at or below y, where the codes are denser: then that power is given, which is no more
// than the code at or below y, or rounds down to it.
__device__ __forceinline__ float power_below(float y) { return __uint_as_float(__float_as_uint(y) & 0x7F800000u); }
// The larger of two values, of which b is not negative: as integers, which need no care for NaN.
__device__ __forceinline__ float larger(float a, float b) {
    return __uint_as_float((uint32_t)max((int)__float_as_uint(a), (int)__float_as_uint(b)));
}
__device__ __forceinline__ float with_sign(float y, float x) { return __builtin_copysignf(y, x); }

__device__ __forceinline__ uint32_t encode_stochastic(const Raw8<uint16_t> &r, uint32_t s, const Random8 &rnd) {
    const float inv = __uint_as_float((254 - s) << 23);   // s <= 253
    float z[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float x = elem(r, k), y = fabsf(x) * inv;
        const float u = (float)(k & 1 ? rnd.w[k >> 1] >> 16 : rnd.w[k >> 1] & 0xFFFFu);
        const float q = power_below(y);
        z[k] = with_sign(larger(fmaf(larger(q, 1.f), fmaf(u, -0x1p-17f, 0.25f - 0x1p-18f), y), q), x);
    }
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, z[0], z[1], 1.f, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, z[2], z[3], 1.f, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, z[4], z[5], 1.f, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, z[6], z[7], 1.f, 3);
}
// fp32: y / (P/2) is exact, so are its whole part and its fraction; the whole
// part, one more where f > t, times P is twice the code's value.
__device__ __forceinline__ uint32_t encode_stochastic(const Raw8<float> &r, uint32_t s, const Random8 &rnd) {
    const float inv = __uint_as_float((254 - s) << 23);
    float z[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float x = elem(r, k), y = fabsf(x) * inv, p = larger(power_below(y), 1.f);
        const float steps = y * __uint_as_float(0x7F800000u - __float_as_uint(p)), f = __builtin_amdgcn_fractf(steps);
        const float u = (float)(k & 1 ? rnd.w[k >> 1] >> 16 : rnd.w[k >> 1] & 0xFFFFu);
        z[k] = with_sign((steps - f + (f > fmaf(u, 0x1p-16f, 0x1p-17f) ? 1.f : 0.f)) * p, x);
    }
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, z[0], z[1], 2.f, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, z[2], z[3], 2.f, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, z[4], z[5], 2.f, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, z[6], z[7], 2.f, 3);
}

// Codes of 8 elements of a block with scale byte s.  `group`: 4 * block + which
// quarter they are, for the random bits.
template <bool STOCHASTIC, class R>
__device__ __forceinline__ uint32_t encode8_at(const R &r, uint32_t s, uint64_t seed, uint64_t group, uint32_t orientation) {
    if (s == 255) return 0;
    if (STOCHASTIC) return encode_stochastic(r, s, philox8(seed, group, orientation));
    return encode_nearest(r, scale_value(s));
}
// The same and the scale byte, for a quad's block, each lane with its quarter.
template <bool STOCHASTIC, class R>
__device__ __forceinline__ uint32_t encode8(const R &r, uint64_t seed, uint64_t group, uint32_t orientation, uint32_t *s) {
    *s = scale_byte<STOCHASTIC>(quad_max(amax8(r)));
    return encode8_at<STOCHASTIC>(r, *s, seed, group, orientation);
}

__device__ __forceinline__ void decode8(float *v, uint32_t c, float scale) {
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 0);
    const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 1);
    const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 2);
    const f32x2 e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 3);
    v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y, v[4] = d.x, v[5] = d.y, v[6] = e.x, v[7] = e.y;
}
__device__ __forceinline__ u32x4 decode8_bf16(uint32_t c, float scale) {
    return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 0)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 1)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 2)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 3))};
}

// The values of a unit's codes, the low bits of c.
__device__ __forceinline__ u32x4 decode_unit(uint16_t, uint32_t c, float scale) { return decode8_bf16(c, scale); }
__device__ __forceinline__ u32x4 decode_unit(float, uint32_t c, float scale) {
    const f32x2 v[2] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 0), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 1)};
    return __builtin_bit_cast(u32x4, v);
}
// Those codes, of unit `unit` from p on.
template <class T>
__device__ __forceinline__ uint32_t unit_codes(const uint8_t *p, int64_t unit) {
    if (sizeof(T) == 2) return ld(reinterpret_cast<const uint32_t *>(p) + unit);
    return ld(reinterpret_cast<const uint16_t *>(p) + unit);
}

// A matrix of blocks, by value.  Rows fit in 31 bits, so a row's chunk comes
// from a multiplication: with l = ceil(log2(chunk_rows)) and
// mul = floor(2^(31+l) / chunk_rows) + 1, which is under 2^32,
// r / chunk_rows = r * mul >> (31 + l) for every r under 2^31.
struct Mx4Mat {
    const uint8_t *codes, *scales;
    int64_t code_stride, scale_stride, chunk_stride;
    uint32_t chunk_rows, chunk_mul, chunk_shift;   // chunk_rows 0: the rows are one run

    // Byte offsets of a row's codes and scales.
    __device__ __forceinline__ void row(uint32_t r, int64_t *code, int64_t *scale) const {
        int64_t base = 0;
        if (chunk_rows) {
            const uint32_t c = (uint32_t)((uint64_t)r * chunk_mul >> chunk_shift);
            base = c * chunk_stride;
            r -= c * chunk_rows;
        }
        *code = base + r * code_stride;
        *scale = base + r * scale_stride;
    }
};

// ------------------------------------------------------------ host side --

inline int64_t mx4_blocks(int64_t n) { return n / kMx4Block + (n % kMx4Block != 0); }

// Memory that a call reads or writes: runs of `width` bytes, `stride` apart (0: one run), `span` bytes from the first
// one's start to the last one's end.  A chunked matrix counts as one run, its gaps included.
struct Footprint {
    const void *p;
    int64_t span, stride, width;
    const char *name;
};
// Whether two meet.  Rows of one stride may lie between each other's, as a row's codes and scales side by side, and a
// single run between rows; rows of two strides whose spans meet are taken to meet.
inline bool meet(const Footprint &a, const Footprint &b) {
    if (!ranges_overlap(a.p, a.span, b.p, b.span)) return false;
    const int64_t s = a.stride ? a.stride : b.stride;
    if (s == 0 || (b.stride && b.stride != s)) return true;
    const int64_t off = (int64_t)(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p)) % s, d = off < 0 ? off + s : off;
    return d < a.width || b.width > s - d;   // a's rows reach into the next of b's, or b's into the next of a's
}

// Checks a matrix argument (`m` not NULL) and gives its kernel form and what
// its codes and its scales cover.
int check_matrix(const char *what, const char *name, const fs_mx4_matrix_t *m, Mx4Mat *out, Footprint (&covers)[2]);

}  // namespace fsi
