// fs_norm.hip -- gfx950 (CDNA4) kernels of the gradient norm over many
// tensors and of clipping them in place, and their C-ABI launchers.
//
// Both are HBM-bound streams over a list of tensors: the norm reads every
// element once (2 or 4 bytes), the clip reads and writes it once.  A list is
// cut into tiles of 16-byte blocks, each inside one tensor; the list itself
// (addresses, sizes, tile counts) travels in the kernel arguments, so a call
// copies nothing to the GPU and can be captured into a graph, and kListMax
// tensors fit one launch.  Tensors start on any element (views of a flat
// shard): blocks are counted from the cache line that a tensor starts in, so
// that no two tiles share a line of it, and elements outside the tensor are
// masked.  Loads stay inside the lines that the tensor touches, so only mapped
// memory is read; stores write its elements only.
#include <hip/hip_runtime.h>
#include <math.h>
#include <string.h>

#include <algorithm>
#include <new>
#include <vector>

#include "fs_norm.h"

using namespace fsi;

namespace {

constexpr int kListMax = 192;   // tensors of one launch: the list takes 3840 of the 4096 argument bytes
constexpr int kListFew = 16;    // shorter lists take 320

template <int CAP>
struct ListArgs {
    char *ptr[CAP];            // first element
    int64_t size[CAP];         // bytes * 2, + 1 for fp32
    uint32_t tile_end[CAP];    // tiles of this tensor and those before it; UINT32_MAX past the last tensor
};

constexpr int kLine = 128;   // bytes of a cache line

// A tile's place: blocks [first, first + nblk) of the tensor whose bytes are
// [lo, hi) from the line-aligned address `base`.
struct TileAt {
    char *base;
    int64_t first, lo, hi;
    int nblk;
    bool f32, whole;   // whole: no element of any of the blocks lies outside the tensor
};

// The place of tile `tile` (of `blocks` blocks), which is one of tensor a's.
template <int CAP>
__device__ __forceinline__ TileAt tile_of(const ListArgs<CAP> &L, int a, uint32_t tile, int blocks) {
    const uint32_t before = a ? L.tile_end[a - 1] : 0;
    const uintptr_t p = reinterpret_cast<uintptr_t>(L.ptr[a]);
    const int64_t size = L.size[a];
    TileAt t;
    t.f32 = size & 1;
    t.lo = (int64_t)(p & (kLine - 1));
    t.hi = t.lo + (size >> 1);
    t.base = reinterpret_cast<char *>(p - (uintptr_t)t.lo);
    t.first = (int64_t)(tile - before) * blocks;
    t.nblk = (int)imin(blocks, ((t.hi + 15) >> 4) - t.first);
    t.whole = 16 * t.first >= t.lo && 16 * (t.first + t.nblk) <= t.hi;
    return t;
}

// Find a workgroup's tile: a binary search in scalar registers.  It waits for
// four to eight loads in turn, but costs few instructions and no vector
// loads, and over a long list the wait does no harm: with the tensor found
// in two loads (a table of hints) the 7B shard's norm took 492 us for 478,
// with all ends compared at once in scalar or vector registers 492 and 500.
template <int CAP>
__device__ __forceinline__ TileAt tile_at(const ListArgs<CAP> &L, uint32_t tile, int blocks) {
    int a = 0, b = CAP - 1;   // the first tensor whose tile_end lies above `tile`
    while (a < b) {
        const int mid = (a + b) >> 1;
        if (L.tile_end[mid] <= tile) a = mid + 1; else b = mid;
    }
    return tile_of<CAP>(L, a, tile, blocks);
}

// Whether block b of the tile (below its nblk) overlaps the tensor: blocks of
// the first line may lie before it.
__device__ __forceinline__ bool overlaps(const TileAt &t, int b) { return t.whole || 16 * (t.first + b + 1) > t.lo; }

// Elements [*e_lo, *e_hi) of block b (of the tensor) lie inside the tensor.
template <int W>
__device__ __forceinline__ void block_range(const TileAt &t, int64_t b, int *e_lo, int *e_hi) {
    *e_lo = (int)imax(0, (t.lo - 16 * b) / W);
    *e_hi = (int)imin(16 / W, (t.hi - 16 * b) / W);
}

// ------------------------------------------------------------------ norm --

constexpr int kNormUnroll = 2;                     // 16-byte blocks per lane
constexpr int kNormTile = kThreads * kNormUnroll;  // blocks of a tile (8 KB): one per workgroup

// bf16 lanes as fp32 bits
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

template <int KIND, int W>
__device__ __forceinline__ void add_block(LaneTotal<KIND> &t, u32x4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (W == 4) {
            t.add(__uint_as_float(w[i]));
        } else {
            t.add(bf_lo(w[i]));
            t.add(bf_hi(w[i]));
        }
    }
}

// Block b of the tile; elements outside the tensor are zero.
template <int W>
__device__ __forceinline__ u32x4 load_block(const TileAt &at, int b) {
    u32x4 v = ld16(at.base + 16 * (at.first + b));
    if (!at.whole) {
        int e_lo, e_hi;
        block_range<W>(at, at.first + b, &e_lo, &e_hi);
        v &= elem_mask<W>(e_lo, e_hi);
    }
    return v;
}

template <int KIND, int W>
__device__ __forceinline__ void add_tile(LaneTotal<KIND> &t, const TileAt &at) {
    u32x4 v[kNormUnroll];
#pragma unroll
    for (int u = 0; u < kNormUnroll; ++u) {
        const int b = u * kThreads + threadIdx.x;
        v[u] = u32x4{0u, 0u, 0u, 0u};   // zeros add nothing to either total
        if (b < at.nblk) v[u] = load_block<W>(at, b);
    }
#pragma unroll
    for (int u = 0; u < kNormUnroll; ++u) add_block<KIND, W>(t, v[u]);
}

template <int KIND, int CAP>
__global__ __launch_bounds__(kThreads) void list_norm_kernel(ListArgs<CAP> L, double *parts) {
    __shared__ double lds[kThreads / 64];
    LaneTotal<KIND> t;
    const TileAt at = tile_at<CAP>(L, blockIdx.x, kNormTile);
    if (at.f32) add_tile<KIND, 4>(t, at); else add_tile<KIND, 2>(t, at);
    const double sum = norm_block_join<KIND, kThreads>(t, lds);
    if (threadIdx.x == 0) parts[blockIdx.x] = sum;
}

// A lane's part of parts[lo, hi): every THREADS-th, eight loads in flight.
template <int KIND, int THREADS>
__device__ __forceinline__ double join_parts(const double *__restrict__ parts, int64_t lo, int64_t hi) {
    double t = 0;
    for (int64_t i = lo + threadIdx.x; i < hi; i += 8 * THREADS) {
        double v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = i + k * THREADS < hi ? parts[i + k * THREADS] : 0.0;
#pragma unroll
        for (int k = 0; k < 8; ++k) t = norm_join<KIND>(t, v[k]);
    }
    return t;
}

// Many partial totals are first joined to kJoinWgs, each workgroup's in a
// contiguous piece; one workgroup would read them at one CU's rate.
constexpr int kJoinWgs = 512;
constexpr int64_t kJoinMin = 16384;

template <int KIND>
__global__ __launch_bounds__(kThreads) void norm_join_kernel(const double *__restrict__ parts, int64_t count,
                                                             double *__restrict__ out) {
    __shared__ double lds[kThreads / 64];
    double t = join_parts<KIND, kThreads>(parts, count * blockIdx.x / kJoinWgs, count * (blockIdx.x + 1) / kJoinWgs);
    t = norm_block_join<KIND, kThreads>(t, lds);
    if (threadIdx.x == 0) out[blockIdx.x] = t;
}

// Joins the partial totals in a fixed order.
constexpr int kFinishThreads = 1024;

template <int KIND>
__global__ __launch_bounds__(kFinishThreads) void norm_finish_kernel(const double *__restrict__ parts, int64_t count,
                                                                     int accumulate, double *total, float *norm) {
    __shared__ double lds[kFinishThreads / 64];
    const double before = accumulate ? total[0] : 0.0;
    const double t = norm_block_join<KIND, kFinishThreads>(join_parts<KIND, kFinishThreads>(parts, 0, count), lds);
    write_total<KIND>(t, before, total, norm);
}

// A short list in one launch: the waves of one workgroup take tiles of one
// block per lane (1 KB) in turn, two of them in flight.
// The launch and the workspace that it saves are about 4 us of a caller's
// time; on the GPU it is ahead up to 80 KB (16 KB: 2.4 us for 3.9 of the two
// launches; 64 KB: 3.3 for 3.9; 128 KB: 5.0 for 4.0; one wave's tiles follow
// each other).
constexpr int kOneTile = 64;
constexpr int kOneUnroll = 2;
constexpr int kOneMaxTiles = 128;

template <int KIND, int CAP>
__global__ __launch_bounds__(kFinishThreads) void list_norm_one_kernel(ListArgs<CAP> L, int ntiles, int accumulate,
                                                                       double *total, float *norm) {
    constexpr int kWaves = kFinishThreads / 64;
    __shared__ double lds[kWaves];
    const double before = accumulate ? total[0] : 0.0;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // the tile ends, spread over the lanes: finding a tile then loads nothing
    uint32_t end[(CAP + 63) / 64];
#pragma unroll
    for (int k = 0; k < (CAP + 63) / 64; ++k) end[k] = 64 * k + lane < CAP ? L.tile_end[64 * k + lane] : UINT32_MAX;
    LaneTotal<KIND> t;
    for (int first = wave; first < ntiles; first += kWaves * kOneUnroll) {
        u32x4 v[kOneUnroll];
        bool f32[kOneUnroll];
#pragma unroll
        for (int u = 0; u < kOneUnroll; ++u) {
            v[u] = u32x4{0u, 0u, 0u, 0u};
            f32[u] = false;
            if (first + u * kWaves < ntiles) {
                const uint32_t tile = first + u * kWaves;
                int a = 0;
#pragma unroll
                for (int k = 0; k < (CAP + 63) / 64; ++k) a += __popcll(__ballot(end[k] <= tile));
                const TileAt at = tile_of<CAP>(L, a, tile, kOneTile);
                f32[u] = at.f32;
                if (lane < at.nblk) v[u] = f32[u] ? load_block<4>(at, lane) : load_block<2>(at, lane);
            }
        }
#pragma unroll
        for (int u = 0; u < kOneUnroll; ++u) {
            if (f32[u]) add_block<KIND, 4>(t, v[u]); else add_block<KIND, 2>(t, v[u]);
        }
    }
    write_total<KIND>(norm_block_join<KIND, kFinishThreads>(t, lds), before, total, norm);
}

// ------------------------------------------------------------------ clip --

// One tile per workgroup.  Over the 7B shard (3.37 GB in fp32, 1.68 in bf16)
// and 97 odd tensors of both types, 118 MB: 128 threads with two blocks each
// 1010 / 516 / 38.7 us, 64 threads with two 1016 / 521 / 39.1, 64 with one
// 1028 / 568 / 41.8, 128 with one 1058 / 589 / 42.7; with tiles counted from
// the tensor's first 16-byte block, which share lines, 1057 / 524 / 41.6, and
// there 256 threads with four blocks 1102 / 586 / 44.8, workgroups that walk
// several tiles 1034 to 1340 and residency caps 1045 to 1690 over the 7B shard
// in fp32.  A call whose coefficient is 1 costs its workgroups' launches, 183
// us over that shard.
constexpr int kClipThreads = 128;
constexpr int kClipUnroll = 2;
constexpr int kClipTile = kClipThreads * kClipUnroll;   // 16-byte blocks of a tile (4 KB)

template <int W>
__device__ __forceinline__ u32x4 scale_block(u32x4 v, float c) {
    if (W == 4)
        return u32x4{__float_as_uint(__uint_as_float(v.x) * c), __float_as_uint(__uint_as_float(v.y) * c),
                     __float_as_uint(__uint_as_float(v.z) * c), __float_as_uint(__uint_as_float(v.w) * c)};
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = (uint32_t)bf16_rne_bits(__float_as_uint(bf_lo(w[i]) * c)) |
               ((uint32_t)bf16_rne_bits(__float_as_uint(bf_hi(w[i]) * c)) << 16);
    return u32x4{w[0], w[1], w[2], w[3]};
}

template <int W>
__device__ __forceinline__ void clip_tile(const TileAt &at, float c) {
    u32x4 v[kClipUnroll];
#pragma unroll
    for (int u = 0; u < kClipUnroll; ++u) {
        const int b = u * kClipThreads + threadIdx.x;
        if (b < at.nblk && overlaps(at, b)) v[u] = ld16(at.base + 16 * (at.first + b));
    }
#pragma unroll
    for (int u = 0; u < kClipUnroll; ++u) {
        const int b = u * kClipThreads + threadIdx.x;
        if (b >= at.nblk || !overlaps(at, b)) continue;
        char *p = at.base + 16 * (at.first + b);
        const u32x4 x = scale_block<W>(v[u], c);
        int e_lo = 0, e_hi = 16 / W;
        if (!at.whole) block_range<W>(at, at.first + b, &e_lo, &e_hi);
        if (e_lo == 0 && e_hi == 16 / W)
            st16(p, x);
        else
            store_elems<W>(p, x, e_lo, e_hi);   // a neighbour in the same block may belong to another tensor
    }
}

template <int CAP>
__global__ __launch_bounds__(kClipThreads) void list_clip_kernel(ListArgs<CAP> L, ClipArgs clip, float *norm) {
    const float c = clip_coef(clip);
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) norm[0] = (float)norm_of(clip.total[0], clip.inf);
    if (c == 1.0f || L.tile_end[0] == 0) return;   // times one: the gradients stay as they are, unread
    const TileAt at = tile_at<CAP>(L, blockIdx.x, kClipTile);
    if (at.f32) clip_tile<4>(at, c); else clip_tile<2>(at, c);
}

// -------------------------------------------------------------- launchers --

int elem_bytes(fs_dtype d) { return d == FS_BF16 ? 2 : 4; }

// Tiles of `tile` 16-byte blocks that cover nb > 0 bytes at p and what precedes them in p's line.
int64_t tiles_of(const void *p, int64_t nb, int tile) {
    const int64_t blocks = ((int64_t)(reinterpret_cast<uintptr_t>(p) & (kLine - 1)) + nb + 15) >> 4;
    return (blocks + tile - 1) / tile;
}

// Tiles of one launch: its grid counts threads in 32 bits, one thread for two
// blocks (137 GB of tensors).
static_assert(kNormUnroll == 2 && kClipUnroll == 2, "threads of a tile");
int64_t max_tiles(int tile) { return UINT32_MAX / (tile / 2); }

// Shared argument checks of the list calls, whose tiles are of `tile` blocks.
int check_list(const char *what, int32_t n_tensors, const void *const *grads, const int64_t *numel,
               const fs_dtype *dtypes, int tile, const void *total, const void *norm) {
    if (n_tensors < 0) return fail(FS_E_INVAL, "%s: n_tensors < 0", what);
    if (n_tensors > 0 && (!grads || !numel || !dtypes)) return fail(FS_E_INVAL, "%s: NULL list", what);
    for (int i = 0; i < n_tensors; ++i) {
        if (numel[i] < 0) return fail(FS_E_INVAL, "%s: tensor %d has a negative element count", what, i);
        if (dtypes[i] != FS_BF16 && dtypes[i] != FS_FP32) return fail(FS_E_DTYPE, "%s: tensor %d has an unknown dtype", what, i);
        if (numel[i] > (INT64_MAX >> 4)) return fail(FS_E_OVERFLOW, "%s: tensor %d is too large", what, i);
        if (numel[i] == 0) continue;
        const int64_t nb = numel[i] * elem_bytes(dtypes[i]);
        if (!grads[i]) return fail(FS_E_INVAL, "%s: tensor %d is NULL", what, i);
        if (misaligned(grads[i], elem_bytes(dtypes[i])))
            return fail(FS_E_ALIGN, "%s: tensor %d not aligned to its element size", what, i);
        if (tiles_of(grads[i], nb, tile) > max_tiles(tile))
            return fail(FS_E_OVERFLOW, "%s: tensor %d is too large for one launch", what, i);
        if (ranges_overlap(total, 8, grads[i], nb) || (norm && ranges_overlap(norm, 4, grads[i], nb)))
            return fail(FS_E_INVAL, "%s: total or norm overlaps tensor %d", what, i);
    }
    return FS_OK;
}

// Cut the list into launches of at most CAP tensors and call
// f(args, tiles) for each; tensors without elements are left out.
template <int CAP, class F>
void launches_of(int32_t n_tensors, const void *const *grads, const int64_t *numel, const fs_dtype *dtypes, int tile,
                 F &&f) {
    ListArgs<CAP> L;
    int count = 0;
    int64_t tiles = 0;
    auto go = [&] {
        for (int k = count; k < CAP; ++k) {
            L.ptr[k] = nullptr;
            L.size[k] = 0;
            L.tile_end[k] = UINT32_MAX;
        }
        f(L, (uint32_t)tiles);
        count = 0;
        tiles = 0;
    };
    for (int i = 0; i < n_tensors; ++i) {
        if (numel[i] == 0) continue;
        const int64_t nb = numel[i] * elem_bytes(dtypes[i]), t = tiles_of(grads[i], nb, tile);
        if (count == CAP || tiles + t > max_tiles(tile)) go();
        tiles += t;
        L.ptr[count] = static_cast<char *>(const_cast<void *>(grads[i]));
        L.size[count] = nb * 2 + (dtypes[i] == FS_FP32);
        L.tile_end[count++] = (uint32_t)tiles;
    }
    if (count) go();
}

template <class F>
void for_each_launch(int32_t n_tensors, const void *const *grads, const int64_t *numel, const fs_dtype *dtypes, int tile,
                     F &&f) {
    if (n_tensors <= kListFew)
        launches_of<kListFew>(n_tensors, grads, numel, dtypes, tile, f);
    else
        launches_of<kListMax>(n_tensors, grads, numel, dtypes, tile, f);
}

// A norm goes in one launch where its list has at most kOneMaxTiles tiles, and
// so no more tensors with elements than one launch takes.  A tensor's tiles
// are counted as if it started on the last byte of a line, so that the choice
// and the workspace go by the sizes alone.
static_assert(kOneMaxTiles <= kListMax, "a tensor has a tile at least");
const void *const anywhere = reinterpret_cast<const void *>(kLine - 1);

// Two tensors that share memory would be scaled twice, or raced on.
int check_disjoint(const char *what, int32_t n_tensors, const void *const *grads, const int64_t *numel,
                   const fs_dtype *dtypes) {
    struct Range { uintptr_t lo, hi; };
    try {
        std::vector<Range> r;
        r.reserve((size_t)n_tensors);
        for (int i = 0; i < n_tensors; ++i)
            if (numel[i] > 0) {
                const uintptr_t a = reinterpret_cast<uintptr_t>(grads[i]);
                r.push_back({a, a + (uintptr_t)(numel[i] * elem_bytes(dtypes[i]))});
            }
        std::sort(r.begin(), r.end(), [](const Range &a, const Range &b) { return a.lo < b.lo; });
        for (size_t i = 1; i < r.size(); ++i)
            if (r[i].lo < r[i - 1].hi) return fail(FS_E_INVAL, "%s: two tensors share memory", what);
    } catch (const std::bad_alloc &) {
        return fail(FS_E_NOMEM, "%s: out of host memory", what);
    }
    return FS_OK;
}

}  // namespace

namespace fsi {

int check_norm_out(const char *what, int type, const double *total, const float *norm) {
    if (type != FS_NORM_L2 && type != FS_NORM_INF) return fail(FS_E_UNSUPPORTED, "%s: unknown norm type %d", what, type);
    if (!total) return fail(FS_E_INVAL, "%s: total is NULL", what);
    if (misaligned(total, 8) || misaligned(norm, 4))
        return fail(FS_E_ALIGN, "%s: total or norm not aligned to its element size", what);
    if (norm && ranges_overlap(total, 8, norm, 4)) return fail(FS_E_INVAL, "%s: norm overlaps total", what);
    return FS_OK;
}

int check_clip(const char *what, const fs_clip_t *clip, ClipArgs *out) {
    if (!clip) return fail(FS_E_INVAL, "%s: clip is NULL", what);
    if (int rc = check_norm_out(what, clip->norm_type, clip->total, nullptr)) return rc;
    if (!(clip->max_norm >= 0.f)) return fail(FS_E_INVAL, "%s: max_norm must be >= 0", what);
    if (!(clip->eps >= 0.f) || isinf(clip->eps)) return fail(FS_E_INVAL, "%s: eps must be >= 0 and finite", what);
    *out = ClipArgs{clip->total, clip->max_norm, clip->eps, clip->norm_type == FS_NORM_INF};
    return FS_OK;
}

int check_workspace_range(const char *what, const void *workspace, size_t bytes, int64_t need, const double *total,
                          const float *norm) {
    if (need == 0) return FS_OK;
    if (!workspace) return fail(FS_E_INVAL, "%s: workspace is NULL", what);
    if (misaligned(workspace, 8)) return fail(FS_E_ALIGN, "%s: workspace not 8-byte aligned", what);
    if ((int64_t)bytes < need)
        return fail(FS_E_INVAL, "%s: workspace too small (%zu < %lld bytes)", what, bytes, (long long)need);
    if (ranges_overlap(workspace, need, total, 8) || (norm && ranges_overlap(workspace, need, norm, 4)))
        return fail(FS_E_INVAL, "%s: workspace overlaps total or norm", what);
    return FS_OK;
}

int64_t norm_parts_bytes(int64_t count) {
    return (count + (count > kJoinMin ? kJoinWgs : 0)) * (int64_t)sizeof(double);
}

int launch_norm_finish(const char *what, int type, int accumulate, double *parts, int64_t count, double *total,
                       float *norm, hipStream_t stream) {
    if (count > kJoinMin) {
        double *joined = parts + count;
        if (type == FS_NORM_L2)
            hipLaunchKernelGGL(norm_join_kernel<kL2>, dim3(kJoinWgs), dim3(kThreads), 0, stream, parts, count, joined);
        else
            hipLaunchKernelGGL(norm_join_kernel<kInf>, dim3(kJoinWgs), dim3(kThreads), 0, stream, parts, count, joined);
        parts = joined;
        count = kJoinWgs;
    }
    if (type == FS_NORM_L2)
        hipLaunchKernelGGL(norm_finish_kernel<kL2>, dim3(1), dim3(kFinishThreads), 0, stream, parts, count, accumulate,
                           total, norm);
    else
        hipLaunchKernelGGL(norm_finish_kernel<kInf>, dim3(1), dim3(kFinishThreads), 0, stream, parts, count,
                           accumulate, total, norm);
    return check_launch(what);
}

}  // namespace fsi

// Partial totals: one per tile; none where the list goes in one launch.
extern "C" int fs_grad_norm_workspace(int32_t n_tensors, const int64_t *numel, const fs_dtype *dtypes,
                                      int64_t *bytes) {
    clear_error();
    const char *what = "fs_grad_norm_workspace";
    if (!bytes) return fail(FS_E_INVAL, "%s: bytes is NULL", what);
    if (n_tensors < 0) return fail(FS_E_INVAL, "%s: n_tensors < 0", what);
    if (n_tensors > 0 && (!numel || !dtypes)) return fail(FS_E_INVAL, "%s: NULL list", what);
    int64_t tiles = 0, one_tiles = 0;
    for (int i = 0; i < n_tensors; ++i) {
        if (numel[i] < 0) return fail(FS_E_INVAL, "%s: tensor %d has a negative element count", what, i);
        if (numel[i] > (INT64_MAX >> 4)) return fail(FS_E_OVERFLOW, "%s: tensor %d is too large", what, i);
        if (numel[i] == 0) continue;
        const int64_t nb = numel[i] * elem_bytes(dtypes[i]);
        const int64_t t = tiles_of(anywhere, nb, kNormTile);
        if (t > max_tiles(kNormTile)) return fail(FS_E_OVERFLOW, "%s: tensor %d is too large for one launch", what, i);
        tiles += t;
        one_tiles = std::min<int64_t>(one_tiles + tiles_of(anywhere, nb, kOneTile), INT32_MAX);
    }
    *bytes = one_tiles <= kOneMaxTiles ? 0 : norm_parts_bytes(tiles);
    return FS_OK;
}

namespace {

int check_grad_norm(const char *what, int32_t n_tensors, const void *const *grads, const int64_t *numel,
                    const fs_dtype *dtypes, fs_norm_type type, const double *total, const float *norm,
                    const void *workspace, size_t bytes, int64_t *need_out) {
    if (int rc = check_norm_out(what, type, total, norm)) return rc;
    if (int rc = check_list(what, n_tensors, grads, numel, dtypes, kNormTile, total, norm)) return rc;
    int64_t need = 0;
    if (int rc = fs_grad_norm_workspace(n_tensors, numel, dtypes, &need)) return rc;
    if (int rc = check_workspace_range(what, workspace, bytes, need, total, norm)) return rc;
    *need_out = need;
    for (int i = 0; i < n_tensors; ++i)
        if (ranges_overlap(workspace, need, grads[i], numel[i] * elem_bytes(dtypes[i])))
            return fail(FS_E_INVAL, "%s: workspace overlaps tensor %d", what, i);
    return FS_OK;
}

}  // namespace

extern "C" int fs_grad_norm(int32_t n_tensors, const void *const *grads, const int64_t *numel, const fs_dtype *dtypes,
                            fs_norm_type type, int32_t accumulate, double *total, float *norm, void *workspace,
                            size_t bytes, hipStream_t stream) {
    clear_error();
    const char *what = "fs_grad_norm";
    int64_t need = 0;
    if (int rc = check_grad_norm(what, n_tensors, grads, numel, dtypes, type, total, norm, workspace, bytes, &need))
        return rc;
    (void)hipGetLastError();
    if (need == 0) {   // one launch, which also covers an empty list
        bool empty = true;
        auto one = [&](const auto &L, uint32_t tiles) {
            constexpr int kCap = sizeof(L.ptr) / sizeof(L.ptr[0]);
            empty = false;
            if (type == FS_NORM_L2)
                hipLaunchKernelGGL((list_norm_one_kernel<kL2, kCap>), dim3(1), dim3(kFinishThreads), 0, stream, L,
                                   (int)tiles, accumulate != 0, total, norm);
            else
                hipLaunchKernelGGL((list_norm_one_kernel<kInf, kCap>), dim3(1), dim3(kFinishThreads), 0, stream, L,
                                   (int)tiles, accumulate != 0, total, norm);
        };
        for_each_launch(n_tensors, grads, numel, dtypes, kOneTile, one);
        if (!empty) return check_launch(what);
        return launch_norm_finish(what, type, accumulate != 0, nullptr, 0, total, norm, stream);
    }
    double *parts = static_cast<double *>(workspace);
    int64_t count = 0;
    for_each_launch(n_tensors, grads, numel, dtypes, kNormTile, [&](const auto &L, uint32_t tiles) {
        constexpr int kCap = sizeof(L.ptr) / sizeof(L.ptr[0]);
        if (type == FS_NORM_L2)
            hipLaunchKernelGGL((list_norm_kernel<kL2, kCap>), dim3(tiles), dim3(kThreads), 0, stream, L, parts + count);
        else
            hipLaunchKernelGGL((list_norm_kernel<kInf, kCap>), dim3(tiles), dim3(kThreads), 0, stream, L, parts + count);
        count += tiles;
    });
    if (int rc = check_launch(what)) return rc;
    return launch_norm_finish(what, type, accumulate != 0, parts, count, total, norm, stream);
}

extern "C" int fs_clip_grads(int32_t n_tensors, void *const *grads, const int64_t *numel, const fs_dtype *dtypes,
                             const fs_clip_t *clip, float *norm, hipStream_t stream) {
    clear_error();
    const char *what = "fs_clip_grads";
    ClipArgs c;
    if (int rc = check_clip(what, clip, &c)) return rc;
    if (int rc = check_norm_out(what, clip->norm_type, clip->total, norm)) return rc;
    if (int rc = check_list(what, n_tensors, grads, numel, dtypes, kClipTile, clip->total, norm)) return rc;
    if (int rc = check_disjoint(what, n_tensors, grads, numel, dtypes)) return rc;
    (void)hipGetLastError();
    float *out = norm;   // the first launch writes it
    for_each_launch(n_tensors, grads, numel, dtypes, kClipTile, [&](const auto &L, uint32_t tiles) {
        constexpr int kCap = sizeof(L.ptr) / sizeof(L.ptr[0]);
        hipLaunchKernelGGL(list_clip_kernel<kCap>, dim3(tiles), dim3(kClipThreads), 0, stream, L, c, out);
        out = nullptr;
    });
    if (out) {   // no tensor has elements
        ListArgs<kListFew> none;
        memset(&none, 0, sizeof none);
        hipLaunchKernelGGL(list_clip_kernel<kListFew>, dim3(1), dim3(kClipThreads), 0, stream, none, c, out);
    }
    return check_launch(what);
}
