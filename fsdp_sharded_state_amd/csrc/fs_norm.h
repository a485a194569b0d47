// fs_norm.h -- the gradient norm's "total" as the kernels of both HIP sources
// make and use it.  Not part of the public ABI.
//
// The total is one double: the sum of squares (FS_NORM_L2) or the largest
// magnitude (FS_NORM_INF) of a set of gradients.  It is exact enough to be
// added up over calls, groups and ranks in any order: the square of a bf16 or
// fp32 value is exact in a double and cannot overflow it, so a total of n
// values is off by at most (n + joins) * 2^-53 relative, whatever the order,
// and in fact far less.  Every kernel writes its partial totals to fixed
// places of a workspace, and one workgroup joins them in a fixed order, so a
// call's result does not depend on which workgroup ends first.
#pragma once
#include "fs_device.h"

namespace fsi {

enum NormKind { kNoNorm = 0, kL2 = FS_NORM_L2, kInf = FS_NORM_INF };

// Join two partial totals.  The larger magnitude, with NaN above everything.
template <int KIND>
__device__ __forceinline__ double norm_join(double a, double b) {
    if (KIND == kL2) return a + b;
    return a != a || a > b ? a : b;   // b if it is NaN: a > NaN is false
}

// A lane's running total.  L2: a double; the square of an fp32 value is exact
// in it (48 significant bits), so the fused multiply-add rounds only the sum.
// INF: the largest magnitude as fp32 bits, whose order as integers is that of
// the magnitudes, with the infinity above every number and NaN above it (two
// integer instructions a value; comparing doubles made the reduce 3% slower).
template <int KIND>
struct LaneTotal {
    double t = 0;
    __device__ __forceinline__ void add(float x) {
        const double d = x;
        t = fma(d, d, t);
    }
};
template <>
struct LaneTotal<kInf> {
    uint32_t m = 0;
    __device__ __forceinline__ void add(float x) { m = max(m, __float_as_uint(x) & 0x7FFFFFFFu); }
};

// The value that the lanes CTRL names hold (data parallel primitives: no LDS,
// a few cycles); zero, which adds nothing to either total, where there is none.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_or_zero(uint32_t x) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xF, true);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_or_zero(double x) {
    const uint64_t b = (uint64_t)__double_as_longlong(x);
    const uint64_t hi = dpp_or_zero<CTRL, ROWS>((uint32_t)(b >> 32));
    return __longlong_as_double((long long)((hi << 32) | dpp_or_zero<CTRL, ROWS>((uint32_t)b)));
}

// x joined over the wave, in lane 63.  A fixed tree: the same for every
// launch.  Shifts by 1, 2, 4 and 8 lanes join each row of 16, the broadcasts
// of lanes 15 and 31 carry the rows' results on.
template <class T, class F>
__device__ __forceinline__ T wave_join(T x, F &&join) {
    x = join(x, dpp_or_zero<0x111, 0xF>(x));   // row_shr:1
    x = join(x, dpp_or_zero<0x112, 0xF>(x));   // row_shr:2
    x = join(x, dpp_or_zero<0x114, 0xF>(x));   // row_shr:4
    x = join(x, dpp_or_zero<0x118, 0xF>(x));   // row_shr:8
    x = join(x, dpp_or_zero<0x142, 0xA>(x));   // row_bcast:15 into rows 1 and 3
    x = join(x, dpp_or_zero<0x143, 0xC>(x));   // row_bcast:31 into rows 2 and 3
    return x;
}
template <int KIND>
__device__ __forceinline__ double norm_wave_join(double t) {
    return wave_join(t, [](double a, double b) { return norm_join<KIND>(a, b); });
}
template <int KIND>
__device__ __forceinline__ double norm_wave_join(const LaneTotal<KIND> &t) {
    if constexpr (KIND == kInf)
        return (double)__uint_as_float(wave_join(t.m, [](uint32_t a, uint32_t b) { return max(a, b); }));
    else
        return norm_wave_join<KIND>(t.t);
}

// The workgroup's total, in thread 0 (the other threads get parts of it).
// `lds`: one double per wave.
template <int KIND, int THREADS, class T>
__device__ __forceinline__ double norm_block_join(const T &lane, double *lds) {
    double t = norm_wave_join<KIND>(lane);
    if ((threadIdx.x & 63) == 63) lds[threadIdx.x >> 6] = t;
    __syncthreads();
    if (threadIdx.x == 0) {
        t = lds[0];
#pragma unroll
        for (int w = 1; w < THREADS / 64; ++w) t = norm_join<KIND>(t, lds[w]);
    }
    return t;
}

// What a consumer needs of fs_clip_t, by value.
struct ClipArgs {
    const double *total;
    double max_norm, eps;
    int32_t inf;
};

__device__ __forceinline__ double norm_of(double total, int inf) { return inf ? total : sqrt(total); }

// Thread 0 writes the total (joined to the one that stood there, where the
// call accumulates) and the norm.
template <int KIND>
__device__ __forceinline__ void write_total(double t, double before, double *total, float *norm) {
    if (threadIdx.x == 0) {
        t = norm_join<KIND>(before, t);
        total[0] = t;
        if (norm) norm[0] = (float)norm_of(t, KIND == kInf);
    }
}

// min(1, max_norm / (norm + eps)), computed in double and rounded once.  A
// norm within the limit gives exactly 1; a NaN norm gives NaN, an infinite
// one 0 (or 1 where max_norm is infinite too).
__device__ __forceinline__ float clip_coef(const ClipArgs &c) {
    const double d = norm_of(c.total[0], c.inf) + c.eps;
    return d <= c.max_norm ? 1.0f : (float)(c.max_norm / d);
}

// ------------------------------------------------------------ host side --

int check_norm_out(const char *what, int type, const double *total, const float *norm);
int check_clip(const char *what, const fs_clip_t *clip, ClipArgs *out);
int check_workspace_range(const char *what, const void *workspace, size_t bytes, int64_t need, const double *total,
                          const float *norm);
// Workspace bytes for `count` partial totals: what launch_norm_finish needs.
int64_t norm_parts_bytes(int64_t count);
// Joins the partial totals into total and norm; parts has norm_parts_bytes(count) bytes.
int launch_norm_finish(const char *what, int type, int accumulate, double *parts, int64_t count, double *total,
                       float *norm, hipStream_t stream);

}  // namespace fsi
