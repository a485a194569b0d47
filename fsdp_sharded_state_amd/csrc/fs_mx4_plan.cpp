// fs_mx4_plan.cpp -- host planner of the quantised shards: where each
// parameter's run on a rank lies in the rank's blocks, cut into tiles of one
// workgroup's work, and what of a shard belongs to no run.
#include <string.h>

#include <algorithm>
#include <new>

#include "fs_mx4_plan.h"

using fsi::fail;
using fsi::Mx4Run;
using fsi::Mx4Tile;

namespace {

constexpr int64_t kMaxBlocks = INT64_MAX / 64;   // of a gathered buffer: its bytes and elements fit in int64

int64_t blocks_of(int64_t numel) { return numel / fsi::kMx4Block + (numel % fsi::kMx4Block != 0); }
int64_t align_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

void add_runs(std::vector<Mx4Run> &out, int64_t lo, int64_t hi, int64_t most, int32_t rank) {
    for (; lo < hi; lo += most) out.push_back(Mx4Run{lo, (int32_t)std::min(most, hi - lo), rank});
}

// One rank's tables; `pieces` are its segments in shard order, whose first
// blocks stand in p->piece_blk.
void rank_tables(fs_mx4_plan_s *p, int32_t rank, const fsi::Segment *pieces, size_t count) {
    const int64_t base = (int64_t)rank * p->shard_numel, blocks = p->info.shard_blocks;
    int64_t blk = 0, elem = 0;   // covered so far
    for (size_t k = 0; k < count; ++k) {
        const fsi::Segment &s = pieces[k];
        const int64_t b0 = p->piece_blk[(size_t)rank * p->n_params + s.buf], e0 = s.vx - base;
        add_runs(p->pads, blk, b0, fsi::kMx4TileBlocks, rank);
        add_runs(p->gaps, elem, e0, fsi::kMx4Tile, rank);
        for (int64_t at = 0; at < s.len; at += fsi::kMx4Tile) {
            Mx4Tile t;
            memset(&t, 0, sizeof t);
            t.src = s.src_off + at;
            t.blk = b0 + at / fsi::kMx4Block;
            t.elem = e0 + at;
            t.n = (int32_t)std::min<int64_t>(fsi::kMx4Tile, s.len - at);
            t.nblk = (int32_t)align_up(blocks_of(t.n), fsi::kMx4PieceAlign);
            t.param = s.buf;
            t.rank = rank;
            p->tiles.push_back(t);
        }
        blk = b0 + align_up(blocks_of(s.len), fsi::kMx4PieceAlign);
        elem = e0 + s.len;
        // a short gap after the piece goes with its last tile
        const int64_t next = k + 1 < count ? pieces[k + 1].vx - base : p->shard_numel;
        if (next - elem <= fsi::kMx4Fill) {
            p->tiles.back().fill = (int32_t)(next - elem);
            elem = next;
        }
    }
    add_runs(p->pads, blk, blocks, fsi::kMx4TileBlocks, rank);
    if (p->info.shard_bytes > 17 * blocks) p->pads.push_back(Mx4Run{blocks, 0, rank});
    add_runs(p->gaps, elem, p->shard_numel, fsi::kMx4Tile, rank);
    p->tile_off.push_back((int64_t)p->tiles.size());
    p->pad_off.push_back((int64_t)p->pads.size());
    p->gap_off.push_back((int64_t)p->gaps.size());
}

int build(fs_plan_t plan, fs_mx4_plan_s *p) {
    const fs_plan_info_t &I = plan->info;
    p->world = I.world;
    p->n_params = I.n_params;
    p->mode = I.mode;
    p->shard_numel = I.shard_numel;
    p->params = plan->params;
    const size_t np = (size_t)I.n_params, entries = (size_t)I.world * np;
    p->piece_blk.assign(entries, 0);
    p->piece_numel.assign(entries, 0);
    int64_t blocks = 0;
    // every sum below stays under shard_numel + 9 blocks a piece
    if (I.shard_numel > kMaxBlocks || (int64_t)np > kMaxBlocks / 16) return fail(FS_E_OVERFLOW, "fs_mx4_plan: the shard is too large");
    if (I.mode == FS_FSDP2_PER_PARAM) {
        for (size_t i = 0; i < np; ++i) {
            for (int32_t r = 0; r < I.world; ++r) p->piece_blk[r * np + i] = blocks;
            blocks += align_up(blocks_of(p->params[i].chunk_rows * p->params[i].row), fsi::kMx4PieceAlign);
        }
        for (const fsi::Segment &s : plan->pack_segs) p->piece_numel[s.rank * np + s.buf] = s.len;
    } else {
        int64_t at = 0;
        int32_t rank = 0;
        for (const fsi::Segment &s : plan->pack_segs) {   // gathered order: rank by rank
            if (s.rank != rank) at = 0;
            rank = s.rank;
            p->piece_blk[s.rank * np + s.buf] = at;
            p->piece_numel[s.rank * np + s.buf] = s.len;
            at += align_up(blocks_of(s.len), fsi::kMx4PieceAlign);
            blocks = std::max(blocks, at);
        }
    }
    if (blocks > kMaxBlocks / I.world) return fail(FS_E_OVERFLOW, "fs_mx4_plan: the gathered buffer is too large");
    p->info.shard_blocks = blocks;
    p->info.shard_bytes = align_up(17 * blocks, fsi::kMx4ShardAlign);
    p->info.gathered_bytes = I.world * p->info.shard_bytes;

    p->tile_off.push_back(0);
    p->pad_off.push_back(0);
    p->gap_off.push_back(0);
    size_t k = 0;
    for (int32_t r = 0; r < I.world; ++r) {
        const size_t first = k;
        while (k < plan->pack_segs.size() && plan->pack_segs[k].rank == r) ++k;
        rank_tables(p, r, plan->pack_segs.data() + first, k - first);
    }
    p->ws_tiles = 0;
    p->ws_pads = align_up((int64_t)(p->tiles.size() * sizeof(Mx4Tile)), 256);
    p->ws_gaps = p->ws_pads + align_up((int64_t)(p->pads.size() * sizeof(Mx4Run)), 256);
    p->info.workspace_bytes = std::max<int64_t>(256, p->ws_gaps + align_up((int64_t)(p->gaps.size() * sizeof(Mx4Run)), 256));
    return FS_OK;
}

}  // namespace

extern "C" int fs_mx4_plan(fs_plan_t plan, fs_mx4_plan_t *out) {
    fsi::clear_error();
    if (!plan || !out) return fail(FS_E_INVAL, "fs_mx4_plan: NULL argument");
    *out = nullptr;
    fs_mx4_plan_s *p = new (std::nothrow) fs_mx4_plan_s();
    if (!p) return fail(FS_E_NOMEM, "fs_mx4_plan: out of host memory");
    int rc;
    try {
        rc = build(plan, p);
    } catch (const std::exception &) {   // bad_alloc, or a length beyond what a vector holds
        rc = fail(FS_E_NOMEM, "fs_mx4_plan: out of host memory");
    }
    if (rc != FS_OK) {
        delete p;
        return rc;
    }
    *out = p;
    return FS_OK;
}

extern "C" int fs_mx4_plan_info(fs_mx4_plan_t p, fs_mx4_plan_info_t *out) {
    fsi::clear_error();
    if (!p || !out) return fail(FS_E_INVAL, "fs_mx4_plan_info: NULL argument");
    *out = p->info;
    return FS_OK;
}

extern "C" int fs_mx4_plan_piece(fs_mx4_plan_t p, int32_t i, int32_t rank, int64_t *first_block, int64_t *numel) {
    fsi::clear_error();
    if (!p || !first_block || !numel) return fail(FS_E_INVAL, "fs_mx4_plan_piece: NULL argument");
    if (i < 0 || i >= p->n_params) return fail(FS_E_INVAL, "fs_mx4_plan_piece: index %d out of range", i);
    if (rank < 0 || rank >= p->world)
        return fail(FS_E_INVAL, "fs_mx4_plan_piece: rank %d out of range [0, %d)", rank, p->world);
    const size_t at = (size_t)rank * p->n_params + i;
    *first_block = p->piece_blk[at];
    *numel = p->piece_numel[at];
    return FS_OK;
}

extern "C" void fs_mx4_plan_destroy(fs_mx4_plan_t p) { delete p; }

extern "C" int fs_mx4_plan_matrix(fs_mx4_plan_t p, void *gathered, int32_t i, fs_mx4_matrix_t *out) {
    fsi::clear_error();
    if (!p || !out) return fail(FS_E_INVAL, "fs_mx4_plan_matrix: NULL argument");
    if (i < 0 || i >= p->n_params) return fail(FS_E_INVAL, "fs_mx4_plan_matrix: index %d out of range", i);
    if (p->mode != FS_FSDP2_PER_PARAM)
        return fail(FS_E_UNSUPPORTED, "fs_mx4_plan_matrix: FSDP1's shards do not hold whole rows; unpack them");
    const fs_param_layout_t &L = p->params[i];
    if (L.row % fsi::kMx4Block != 0)
        return fail(FS_E_UNSUPPORTED, "fs_mx4_plan_matrix: parameter %d has rows of %lld elements, not whole blocks", i,
                    (long long)L.row);
    const int64_t rows = L.row ? L.numel / L.row : 0;
    if (rows > 0 && !gathered) return fail(FS_E_INVAL, "fs_mx4_plan_matrix: gathered is NULL");
    if ((reinterpret_cast<uintptr_t>(gathered) & 15) != 0)
        return fail(FS_E_ALIGN, "fs_mx4_plan_matrix: gathered not 16-byte aligned");
    char *base = static_cast<char *>(gathered);
    const int64_t blk = p->piece_blk[i];
    memset(out, 0, sizeof *out);
    out->rows = rows;
    out->cols = L.row;
    out->codes = base ? base + blk * fsi::kMx4BlockBytes : nullptr;
    out->scales = base ? base + p->info.shard_blocks * fsi::kMx4BlockBytes + blk : nullptr;
    out->scale_stride = L.row / fsi::kMx4Block;
    out->code_stride = out->scale_stride * fsi::kMx4BlockBytes;
    out->chunk_rows = L.chunk_rows;
    out->chunk_stride = p->info.shard_bytes;
    return FS_OK;
}
