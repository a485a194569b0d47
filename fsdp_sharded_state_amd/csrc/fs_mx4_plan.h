// fs_mx4_plan.h -- the plan of a group's quantised shards behind the opaque
// fs_mx4_plan_t, shared by its host planner (fs_mx4_plan.cpp) and the
// launchers (fs_mx4.hip).  Not part of the public ABI.
#pragma once
#include <stdint.h>

#include <vector>

#include "fs_plan_impl.h"

namespace fsi {

constexpr int kMx4Block = 32;        // elements of a block
constexpr int kMx4BlockBytes = 16;   // of codes
constexpr int kMx4PieceAlign = 8;    // blocks a piece starts on: 128 bytes of codes
constexpr int kMx4ShardAlign = 128;  // bytes a shard is a multiple of
constexpr int kMx4TileBlocks = 256;  // blocks of a tile: one workgroup's work
constexpr int kMx4Tile = kMx4TileBlocks * kMx4Block;

// A tile lies in one piece (one parameter's run on one rank), so that no
// kernel looks for piece boundaries inside it.
struct Mx4Tile {        // 48 bytes
    int64_t src;        // first parameter element
    int64_t blk;        // first block in the rank's quantised shard, a multiple of 8
    int64_t elem;       // first element in the rank's plain shard
    int32_t n;          // elements, 1..kMx4Tile
    int32_t nblk;       // blocks to write, those beyond the elements as zeros: a multiple of 8, at most kMx4TileBlocks
    int32_t param;
    int32_t rank;
    int32_t fill;       // elements of the plain shard after the last one that belong to no piece (0..kMx4Fill)
    int32_t unused;
};
static_assert(sizeof(Mx4Tile) == 48, "tile layout");
static_assert(kMx4TileBlocks % kMx4PieceAlign == 0, "tiles end where pieces may start");
constexpr int kMx4Fill = 64;

// What no tile covers: `n` blocks of a quantised shard from `at` on (a run of
// n = 0 stands for the bytes after the last scale), or `n` elements of a plain one.
struct Mx4Run {         // 16 bytes
    int64_t at;
    int32_t n;
    int32_t rank;
};
static_assert(sizeof(Mx4Run) == 16, "run layout");

}  // namespace fsi

struct fs_mx4_plan_s {
    fs_mx4_plan_info_t info;
    int32_t world = 0, n_params = 0, mode = 0;
    int64_t shard_numel = 0;                     // of the plain shard
    std::vector<fs_param_layout_t> params;
    std::vector<int64_t> piece_blk, piece_numel; // [N][n_params]
    // tables sorted by rank, with N + 1 offsets each
    std::vector<fsi::Mx4Tile> tiles;
    std::vector<fsi::Mx4Run> pads;               // quantised shards
    std::vector<fsi::Mx4Run> gaps;               // plain shards
    std::vector<int64_t> tile_off, pad_off, gap_off;
    int64_t ws_tiles = 0, ws_pads = 0, ws_gaps = 0;
    void *dev_ws = nullptr;                      // bound by fs_mx4_plan_upload
    int dev_id = -1;
};
