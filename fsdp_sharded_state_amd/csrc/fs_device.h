// fs_device.h -- helpers that the kernels and launchers of both HIP sources
// share.  Not part of the public ABI.
#pragma once
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>

#include "fs_plan_impl.h"

namespace fsi {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__host__ __device__ __forceinline__ int64_t imax(int64_t a, int64_t b) { return a > b ? a : b; }
__host__ __device__ __forceinline__ int64_t imin(int64_t a, int64_t b) { return a < b ? a : b; }

__device__ __forceinline__ u32x4 ld16(const char *p) {
    return __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p));
}
__device__ __forceinline__ void st16(char *p, u32x4 v) {
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4 *>(p));
}

// Select mask of the elements [e_lo, e_hi) of a 16-byte block (W-byte elements).
template <int W>
__device__ __forceinline__ u32x4 elem_mask(int e_lo, int e_hi) {
    uint32_t m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (W == 4) {
            m[i] = (i >= e_lo && i < e_hi) ? 0xFFFFFFFFu : 0u;
        } else {
            uint32_t lo = (2 * i >= e_lo && 2 * i < e_hi) ? 0x0000FFFFu : 0u;
            uint32_t hi = (2 * i + 1 >= e_lo && 2 * i + 1 < e_hi) ? 0xFFFF0000u : 0u;
            m[i] = lo | hi;
        }
    }
    return u32x4{m[0], m[1], m[2], m[3]};
}

template <int W>
__device__ __forceinline__ void store_elems(char *dst, u32x4 v, int e_lo, int e_hi) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 16 / W; ++e) {
        if (e >= e_lo && e < e_hi) {
            if (W == 4)
                *reinterpret_cast<uint32_t *>(dst + 4 * e) = w[e];
            else
                *reinterpret_cast<uint16_t *>(dst + 2 * e) = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
        }
    }
}

__device__ __forceinline__ uint16_t bf16_rne_bits(uint32_t u) {
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (uint16_t)((u >> 16) | 0x40u);   // quiet NaN
    u += 0x7FFFu + ((u >> 16) & 1u);
    return (uint16_t)(u >> 16);
}

// ------------------------------------------------------------ host side --

// Grids shorter than this many rounds of resident workgroups run uncapped.
constexpr int64_t kCapMinRounds = 16;

struct CuLimits {
    int lds_per_cu = 0, lds_per_wg = 0, cus = 0;   // 0: unknown, no cap
};

inline CuLimits cu_limits() {
    constexpr int kMaxDev = 64;
    static std::atomic<int> lds_cu[kMaxDev], lds_wg[kMaxDev], ncu[kMaxDev];   // 0: not read yet, -1: failed
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDev) return {};
    if (lds_cu[dev].load(std::memory_order_acquire) == 0) {
        int a = 0, b = 0, c = 0;
        const bool ok = hipDeviceGetAttribute(&a, hipDeviceAttributeMaxSharedMemoryPerMultiprocessor, dev) ==
                            hipSuccess &&
                        hipDeviceGetAttribute(&b, hipDeviceAttributeMaxSharedMemoryPerBlock, dev) == hipSuccess &&
                        hipDeviceGetAttribute(&c, hipDeviceAttributeMultiprocessorCount, dev) == hipSuccess &&
                        a > 0 && b > 0 && c > 0;
        lds_wg[dev].store(ok ? b : -1, std::memory_order_relaxed);
        ncu[dev].store(ok ? c : -1, std::memory_order_relaxed);
        lds_cu[dev].store(ok ? a : -1, std::memory_order_release);
    }
    CuLimits L;
    if (lds_cu[dev].load(std::memory_order_acquire) < 0) return L;
    L.lds_per_cu = lds_cu[dev].load(std::memory_order_relaxed);
    L.lds_per_wg = lds_wg[dev].load(std::memory_order_relaxed);
    L.cus = ncu[dev].load(std::memory_order_relaxed);
    return L;
}

// Dynamic LDS bytes for a grid of `grid` workgroups capped at k per CU, for a
// kernel that already uses `static_bytes` of LDS (0: no cap).
inline uint32_t lds_cap(int k, int64_t grid, int64_t static_bytes = 0, int64_t min_rounds = kCapMinRounds) {
    const CuLimits L = cu_limits();
    if (L.lds_per_cu <= 0 || k < 1) return 0;
    if (grid < min_rounds * k * (int64_t)L.cus) return 0;
    const int64_t per_wg = L.lds_per_cu / (k + 1) + 1;   // k of these fit in a CU, k + 1 do not
    if (per_wg > L.lds_per_wg || per_wg * k > L.lds_per_cu || per_wg <= static_bytes) return 0;
    return (uint32_t)(per_wg - static_bytes);
}

inline bool misaligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

inline int check_launch(const char *what) {
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fsi::fail(FS_E_HIP, "%s: kernel launch failed: %s", what, hipGetErrorString(e));
    return FS_OK;
}

inline bool ranges_overlap(const void *a, int64_t abytes, const void *b, int64_t bbytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return abytes > 0 && bbytes > 0 && x < y + (uintptr_t)bbytes && y < x + (uintptr_t)abytes;
}

}  // namespace fsi
