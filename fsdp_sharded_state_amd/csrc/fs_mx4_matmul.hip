// fs_mx4_matmul.hip -- the product of two matrices of 4-bit blocks.
#include <string.h>

#include "fs_mx4.h"

using namespace fsi;

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

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

__device__ __forceinline__ void store4(float *p, f32x4 v, int64_t valid) {
    if (valid >= 4) {
        __builtin_memcpy(p, &v, 16);
    } else {
        for (int k = 0; k < 4; ++k)
            if (k < valid) p[k] = v[k];
    }
}
__device__ __forceinline__ void store4(uint16_t *p, f32x4 v, int64_t valid) {
    uint16_t h[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = bf16_rne_bits(__float_as_uint(v[k]));
    if (valid >= 4) {
        __builtin_memcpy(p, h, 8);
    } else {
        for (int k = 0; k < 4; ++k)
            if (k < valid) p[k] = h[k];
    }
}

// Each wave takes 32 by 32 outputs, a workgroup 64 by 64, fragments straight
// from memory.  Rows beyond the matrices read the last one, and are not stored.
template <class T>
__global__ __launch_bounds__(256) void matmul_mx4_kernel(Mx4Mat a, Mx4Mat b, int64_t m, int64_t n, int64_t nb,
                                                         T *__restrict__ out, int64_t ldo, uint32_t tiles_n) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, kb = lane >> 4;
    const int64_t m0 = (int64_t)(blockIdx.x / tiles_n) * 64 + (wave >> 1) * 32;
    const int64_t n0 = (int64_t)(blockIdx.x % tiles_n) * 64 + (wave & 1) * 32;
    int64_t ac[2], as[2], bc[2], bs[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        a.row(imin(m0 + 16 * i + r, m - 1), &ac[i], &as[i]);
        b.row(imin(n0 + 16 * i + r, n - 1), &bc[i], &bs[i]);
    }
    f32x4 acc[2][2] = {};
    for (int64_t k = kb; k - kb < nb; k += 4) {
        u32x4 x[2], y[2];
        uint32_t sx[2], sy[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            x[i] = y[i] = u32x4{0, 0, 0, 0};
            sx[i] = sy[i] = 127;
            if (k < nb) {
                x[i] = *reinterpret_cast<const u32x4 *>(b.codes + bc[i] + k * kMx4BlockBytes);
                y[i] = *reinterpret_cast<const u32x4 *>(a.codes + ac[i] + k * kMx4BlockBytes);
                sx[i] = b.scales[bs[i] + k];
                sy[i] = a.scales[as[i] + k];
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[i][j] = mfma16(x[i], sx[i], y[j], sy[j], acc[i][j]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int64_t row = m0 + 16 * j + r, col = n0 + 16 * i + 4 * kb;
            if (row < m && col < n) store4(out + row * ldo + col, acc[i][j], n - col);
        }
}

int check_sizes(const char *what, int64_t m, int64_t n, int64_t k) {
    if (m < 0 || n < 0 || k < 0) return fail(FS_E_INVAL, "%s: negative size", what);
    if (m > INT32_MAX || n > INT32_MAX || k > INT32_MAX)
        return fail(FS_E_OVERFLOW, "%s: more than 2^31 - 1 rows or columns", what);
    return FS_OK;
}

}  // namespace

extern "C" int fs_mx4_matmul_workspace(int64_t m, int64_t n, int64_t k, int64_t *bytes) {
    clear_error();
    const char *what = "fs_mx4_matmul_workspace";
    if (!bytes) return fail(FS_E_INVAL, "%s: bytes is NULL", what);
    if (int rc = check_sizes(what, m, n, k)) return rc;
    *bytes = 0;
    return FS_OK;
}

extern "C" int fs_mx4_matmul(const fs_mx4_matrix_t *a, const fs_mx4_matrix_t *b, void *out, fs_dtype dtype, int64_t ldo,
                             void *workspace, size_t bytes, hipStream_t stream) {
    clear_error();
    const char *what = "fs_mx4_matmul";
    if (!a || !b) return fail(FS_E_INVAL, "%s: a matrix is NULL", what);
    if (dtype != FS_BF16 && dtype != FS_FP32) return fail(FS_E_DTYPE, "%s: unknown dtype %d", what, (int)dtype);
    Mx4Mat ka, kb;
    int64_t ac, as, bc, bs;
    if (int rc = check_matrix(what, "a", a, &ka, &ac, &as)) return rc;
    if (int rc = check_matrix(what, "b", b, &kb, &bc, &bs)) return rc;
    if (a->cols != b->cols)
        return fail(FS_E_INVAL, "%s: a has %lld columns, b %lld", what, (long long)a->cols, (long long)b->cols);
    const int64_t m = a->rows, n = b->rows, k = a->cols, w = dtype == FS_BF16 ? 2 : 4;
    int64_t need = 0;
    if (int rc = fs_mx4_matmul_workspace(m, n, k, &need)) return rc;
    if (m == 0 || n == 0) return FS_OK;
    if (!out) return fail(FS_E_INVAL, "%s: out is NULL", what);
    if (misaligned(out, w)) return fail(FS_E_ALIGN, "%s: out not aligned to its element size", what);
    if (m > 1 && ldo < n) return fail(FS_E_INVAL, "%s: the rows of out overlap", what);
    if (m > 1 && ldo > ((int64_t)1 << 56) / m) return fail(FS_E_OVERFLOW, "%s: out is too large", what);
    const int64_t span = ((m > 1 ? (m - 1) * ldo : 0) + n) * w;
    struct { const void *p; int64_t bytes; } in[] = {{ka.codes, ac}, {ka.scales, as}, {kb.codes, bc}, {kb.scales, bs}};
    for (const auto &s : in)
        if (ranges_overlap(out, span, s.p, s.bytes)) return fail(FS_E_INVAL, "%s: out overlaps a matrix", what);
    if (need > 0) {
        if (!workspace) return fail(FS_E_INVAL, "%s: workspace is NULL", what);
        if (misaligned(workspace, 16)) return fail(FS_E_ALIGN, "%s: workspace not 16-byte aligned", what);
        if ((int64_t)bytes < need)
            return fail(FS_E_INVAL, "%s: workspace too small (%zu < %lld bytes)", what, bytes, (long long)need);
        if (ranges_overlap(workspace, need, out, span)) return fail(FS_E_INVAL, "%s: workspace overlaps out", what);
        for (const auto &s : in)
            if (ranges_overlap(workspace, need, s.p, s.bytes))
                return fail(FS_E_INVAL, "%s: workspace overlaps a matrix", what);
    }
    const int64_t tn = (n + 63) / 64, tiles = tn * ((m + 63) / 64);
    if (tiles > UINT32_MAX / 256) return fail(FS_E_OVERFLOW, "%s: too many outputs for one launch", what);
    const int64_t nb = mx4_blocks(k), ld = m > 1 ? ldo : 0;
    (void)hipGetLastError();
    if (dtype == FS_BF16)
        hipLaunchKernelGGL(matmul_mx4_kernel<uint16_t>, dim3((uint32_t)tiles), dim3(256), 0, stream, ka, kb, m, n, nb,
                           static_cast<uint16_t *>(out), ld, (uint32_t)tn);
    else
        hipLaunchKernelGGL(matmul_mx4_kernel<float>, dim3((uint32_t)tiles), dim3(256), 0, stream, ka, kb, m, n, nb,
                           static_cast<float *>(out), ld, (uint32_t)tn);
    return check_launch(what);
}
