// mx4_calls_sanitize.cpp -- host-only driver for an UndefinedBehaviorSanitizer
// build of the 4-bit calls' host side (fs_mx4.hip, fs_mx4_matmul.hip): their
// checks and launch shapes, with arguments from the ends of every range.  The
// HIP calls are stubs that launch nothing and note the grid.  Exit status 0 and
// a final "ok" line mean clean.
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "../../include/fs.h"

static int g_fail = 0;
static long g_launches = 0;
static dim3 g_grid;

#define EXPECT(cond, ...)                                            \
    do {                                                             \
        if (!(cond) && g_fail++ < 20) {                              \
            fprintf(stderr, "FAIL %s:%d: ", __FILE__, __LINE__);     \
            fprintf(stderr, __VA_ARGS__);                            \
            fputc('\n', stderr);                                     \
        }                                                            \
    } while (0)

// ---- stubs of what the calls use of HIP
extern "C" {
hipError_t hipGetDevice(int *d) { return *d = 0, hipSuccess; }
hipError_t hipGetLastError() { return hipSuccess; }
const char *hipGetErrorString(hipError_t) { return ""; }
hipError_t hipDeviceGetAttribute(int *v, hipDeviceAttribute_t a, int) {
    *v = a == hipDeviceAttributeMultiprocessorCount ? 256 : a == hipDeviceAttributeMaxSharedMemoryPerMultiprocessor ? 163840 : 65536;
    return hipSuccess;
}
hipError_t hipPointerGetAttributes(hipPointerAttribute_t *, const void *) { return hipErrorInvalidValue; }
hipError_t hipMemcpyAsync(void *, const void *, size_t, hipMemcpyKind, hipStream_t) { return hipErrorInvalidValue; }
hipError_t hipStreamSynchronize(hipStream_t) { return hipErrorInvalidValue; }
hipError_t hipLaunchKernel(const void *, dim3 grid, dim3, void **, size_t, hipStream_t) {
    ++g_launches;
    g_grid = grid;
    return hipSuccess;
}
static dim3 g_config[2];
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t, hipStream_t) { return g_config[0] = grid, g_config[1] = block, hipSuccess; }
hipError_t __hipPopCallConfiguration(dim3 *grid, dim3 *block, size_t *lds, hipStream_t *s) {
    return *grid = g_config[0], *block = g_config[1], *lds = 0, *s = nullptr, hipSuccess;
}
static void *g_module;
void **__hipRegisterFatBinary(const void *) { return &g_module; }
void __hipRegisterFunction(void **, const void *, char *, const char *, unsigned, void *, void *, void *, void *, int *) {}
void __hipRegisterVar(void **, void *, char *, char *, int, size_t, int, int) {}
void __hipUnregisterFatBinary(void **) {}
}

static uint64_t g_state = 88172645463325252ull;
static uint64_t next() {
    g_state ^= g_state << 13;
    g_state ^= g_state >> 7;
    return g_state ^= g_state << 17;
}
template <class T, size_t N>
static T pick(const T (&of)[N]) {
    return of[next() % N];
}

static const int64_t kCounts[] = {0, 1, 2, 31, 32, 33, 255, 256, 257, 4095, 70000, 1 << 24, INT32_MAX - 1, INT32_MAX, (int64_t)1 << 31, (int64_t)1 << 40, INT64_MAX, -1, INT64_MIN};
static const int64_t kSmall[] = {1, 2, 31, 32, 33, 255, 256, 257, 4095, 70000};
static const int64_t kStrides[] = {0, 1, 16, 48, 64, 4096, 1 << 20, (int64_t)1 << 31, (int64_t)1 << 45, ((int64_t)1 << 56) - 16, (int64_t)1 << 56, INT64_MAX - 15, INT64_MAX, -16, INT64_MIN};
static const uint64_t kAddresses[] = {0, 16, 1 << 12, 1 << 20, (uint64_t)1 << 40, (uint64_t)1 << 46, (uint64_t)3 << 46, (uint64_t)5 << 45, ((uint64_t)1 << 40) + 8, ((uint64_t)1 << 40) + 1};

static void *address() { return reinterpret_cast<void *>(pick(kAddresses)); }
static int64_t count(bool odd) { return odd ? pick(kCounts) : pick(kSmall); }

static fs_mx4_matrix_t matrix(int64_t rows, int64_t cols) {
    fs_mx4_matrix_t m;
    memset(&m, 0, sizeof m);
    const bool odd = next() % 2;
    m.codes = address();
    m.scales = address();
    m.rows = rows;
    m.cols = cols;
    const int64_t nb = cols > 0 && cols <= INT32_MAX ? (cols + 31) / 32 : 1;
    m.code_stride = odd ? pick(kStrides) : 16 * nb + (int64_t)(next() % 3) * 16;
    m.scale_stride = odd ? pick(kStrides) : nb + (int64_t)(next() % 3);
    m.chunk_rows = next() % 2 ? 0 : pick(kCounts);
    m.chunk_stride = next() % 2 ? pick(kStrides) : (int64_t)1 << 32;
    return m;
}

// Rows of codes and of scales side by side in one buffer share no byte, and are not refused; rows that do, are.
static void rows_between_rows() {
    char *buf = reinterpret_cast<char *>(1ll << 30);
    for (int64_t stride = 48; stride <= 80; stride += 16)
        for (int64_t at = 0; at < stride; ++at) {
            fs_mx4_matrix_t m = {buf, buf + at, 5, 70, stride, stride, 0, 0};      // 48 bytes of codes, 3 of scales
            const int rc = fs_mx4_quantize(5, 70, reinterpret_cast<void *>(1 << 20), FS_FP32, 70, &m, nullptr, nullptr, nullptr);
            EXPECT(rc == (at >= 48 && at + 3 <= stride ? FS_OK : FS_E_INVAL), "stride %lld, scales at %lld: %d %s", (long long)stride, (long long)at, rc, fs_last_error());
        }
    // the plain matrix and its codes in one buffer, and a product's output beside its operand's rows
    fs_mx4_matrix_t m = {buf + 288, reinterpret_cast<void *>(1ll << 35), 5, 70, 336, 3, 0, 0};
    EXPECT(fs_mx4_quantize(5, 70, buf, FS_FP32, 84, &m, nullptr, nullptr, nullptr) == FS_OK, "%s", fs_last_error());
    EXPECT(fs_mx4_dequantize(&m, buf, FS_FP32, 84, nullptr) == FS_OK, "%s", fs_last_error());
    EXPECT(fs_mx4_dequantize(&m, buf + 12, FS_FP32, 84, nullptr) == FS_E_INVAL, "out reaches into the codes");
    EXPECT(fs_mx4_dequantize(&m, buf + 56, FS_FP32, 84, nullptr) == FS_E_INVAL, "the codes reach into out");
    EXPECT(fs_mx4_dequantize(&m, buf, FS_FP32, 85, nullptr) == FS_E_INVAL, "another stride");
    fs_mx4_matrix_t b = {reinterpret_cast<void *>(1ll << 36), reinterpret_cast<void *>(1ll << 37), 72, 70, 48, 3, 0, 0};
    EXPECT(fs_mx4_matmul(&m, &b, buf, FS_FP32, 84, nullptr) == FS_OK, "%s", fs_last_error());
    EXPECT(fs_mx4_matmul(&m, &b, buf + 4, FS_FP32, 84, nullptr) == FS_E_INVAL, "out reaches into the codes");
    // a seed between rows
    EXPECT(fs_mx4_quantize(5, 70, buf, FS_FP32, 84, &m, nullptr, reinterpret_cast<const uint64_t *>(buf + 280), nullptr) == FS_OK, "%s", fs_last_error());
    EXPECT(fs_mx4_quantize(5, 70, buf, FS_FP32, 84, &m, nullptr, reinterpret_cast<const uint64_t *>(buf + 336 + 328), nullptr) == FS_E_INVAL, "a seed in the codes");
}

int main() {
    long done = 0;
    for (int i = 0; i < 400000; ++i) {
        const bool odd = next() % 3 == 0;
        const int64_t rows = count(odd), cols = count(odd);
        const fs_dtype dt = next() % 2 ? FS_BF16 : FS_FP32;
        fs_mx4_matrix_t a = matrix(rows, cols), b = matrix(next() % 8 ? count(odd) : rows, cols), c = matrix(cols, rows);
        const int64_t ld = next() % 2 ? pick(kStrides) : cols > 0 && cols <= INT32_MAX ? cols + (int64_t)(next() % 9) : cols;
        if (next() % 2) a.chunk_rows = c.chunk_rows = 0;
        const long before = g_launches;
        const uint64_t *seed = next() % 2 ? nullptr : static_cast<const uint64_t *>(address());
        int rc;
        switch (next() % 3) {
        case 0: rc = fs_mx4_quantize(rows, cols, address(), dt, ld, next() % 3 ? &a : nullptr, next() % 3 ? &c : nullptr, seed, nullptr); break;
        case 1: rc = fs_mx4_dequantize(&a, address(), dt, ld, nullptr); break;
        default: rc = fs_mx4_matmul(&a, &b, address(), dt, next() % 2 ? ld : b.rows, nullptr); break;
        }
        EXPECT(rc <= 0 && rc >= -7, "status %d", rc);
        EXPECT(rc == FS_OK || g_launches == before, "a refused call has launched");
        if (g_launches != before) {
            ++done;
            EXPECT(g_grid.x > 0 && g_grid.y == 1 && g_grid.z == 1, "grid %u %u %u", g_grid.x, g_grid.y, g_grid.z);
        }
    }
    // chunks longer than any matrix are one run
    const int64_t longest[] = {41, INT32_MAX, INT64_MAX - 40, INT64_MAX - 1, INT64_MAX};
    for (int64_t n : longest) {
        fs_mx4_matrix_t m = {reinterpret_cast<void *>(1 << 20), reinterpret_cast<void *>(1 << 24), 40, 70, 48, 3, n, 0};
        EXPECT(fs_mx4_dequantize(&m, reinterpret_cast<void *>(1ll << 30), FS_FP32, 70, nullptr) == FS_OK, "chunks of %lld rows: %s", (long long)n, fs_last_error());
    }
    rows_between_rows();
    EXPECT(done > 1000, "only %ld calls came to a launch", done);
    if (g_fail) return 1;
    printf("ok: %ld calls came to a launch\n", done);
    return 0;
}
