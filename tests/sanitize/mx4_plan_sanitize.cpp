// mx4_plan_sanitize.cpp -- host-only driver for a sanitizer build
// (AddressSanitizer and UndefinedBehaviorSanitizer) of the planner of
// quantised shards (fs_mx4_plan.cpp, over fs_plan.cpp).  For tiny and random
// parameter lists and the workload shapes it checks that the tables which the kernels
// index by cover every block and every element of every shard exactly once,
// inside the buffers.  Exit status 0 and a final "ok" line mean clean.
#include <stdint.h>
#include <stdio.h>

#include <vector>

#include "../../fsdp_sharded_state_amd/csrc/fs_mx4_plan.h"
#include "../../include/fs.h"

static long g_plans = 0;
static int g_fail = 0;

#define EXPECT(cond, ...)                                            \
    do {                                                             \
        if (!(cond) && g_fail++ < 20) {                              \
            fprintf(stderr, "FAIL %s:%d: ", __FILE__, __LINE__);     \
            fprintf(stderr, __VA_ARGS__);                            \
            fputc('\n', stderr);                                     \
        }                                                            \
    } while (0)

struct Shapes {
    std::vector<int32_t> ndim;
    std::vector<int64_t> dims;
    void add(int64_t a) { ndim.push_back(1), dims.push_back(a); }
    void add(int64_t a, int64_t b) { ndim.push_back(2), dims.push_back(a), dims.push_back(b); }
};

// A cover of [0, size) by ranges in any order, each place once.
struct Cover {
    std::vector<uint8_t> seen;   // of small shards; of large ones the sum alone
    int64_t size, sum = 0;
    explicit Cover(int64_t n) : seen(n <= (1 << 22) ? n : 0), size(n) {}
    void add(int64_t at, int64_t n) {
        EXPECT(at >= 0 && n >= 0 && at <= size - n, "range [%lld, +%lld) outside %lld", (long long)at, (long long)n, (long long)size);
        sum += n;
        if (!seen.empty() && at >= 0 && at <= size - n)
            for (int64_t k = at; k < at + n; ++k) EXPECT(seen[k]++ == 0, "place %lld twice", (long long)k);
    }
    void done() { EXPECT(sum == size, "%lld of %lld covered", (long long)sum, (long long)size); }
};

static void check(const Shapes &sh, fs_dtype dt, int32_t world, int32_t uo, fs_mode mode) {
    fs_plan_t plan = nullptr;
    const int rc = fs_plan((int32_t)sh.ndim.size(), sh.ndim.data(), sh.dims.data(), dt, world, uo, mode, 1, &plan);
    EXPECT(rc == FS_OK, "fs_plan rc %d", rc);
    if (rc != FS_OK) return;
    fs_mx4_plan_t p = nullptr;
    EXPECT(fs_mx4_plan(plan, &p) == FS_OK, "fs_mx4_plan: %s", fs_last_error());
    fs_plan_info_t P;
    fs_plan_info(plan, &P);
    if (p) {
        fs_mx4_plan_info_t I;
        fs_mx4_plan_info(p, &I);
        std::vector<int64_t> numel(P.n_params), got(P.n_params, 0);
        for (int32_t i = 0; i < P.n_params; ++i) {
            fs_param_layout_t L;
            fs_plan_param(plan, i, &L);
            numel[i] = L.numel;
        }
        EXPECT(I.shard_bytes % 128 == 0 && I.shard_bytes >= 17 * I.shard_blocks && I.shard_bytes < 17 * I.shard_blocks + 128 &&
               I.gathered_bytes == world * I.shard_bytes, "sizes");
        EXPECT((int32_t)p->tile_off.size() == world + 1 && (int32_t)p->pad_off.size() == world + 1 &&
               (int32_t)p->gap_off.size() == world + 1, "offsets");
        for (int32_t r = 0; r < world; ++r) {
            Cover blocks(I.shard_blocks), elems(P.shard_numel);
            for (int64_t k = p->tile_off[r]; k < p->tile_off[r + 1]; ++k) {
                const fsi::Mx4Tile &t = p->tiles[k];
                EXPECT(t.rank == r && t.param >= 0 && t.param < P.n_params && t.n >= 1 && t.n <= fsi::kMx4Tile &&
                       t.src >= 0 && t.src + t.n <= numel[t.param], "tile %lld", (long long)k);
                EXPECT(t.blk % 8 == 0 && t.nblk % 8 == 0 && t.nblk <= fsi::kMx4TileBlocks && 32 * (int64_t)t.nblk >= t.n &&
                       t.fill >= 0 && t.fill <= fsi::kMx4Fill, "tile %lld", (long long)k);
                blocks.add(t.blk, t.nblk);
                elems.add(t.elem, t.n + t.fill);
                got[t.param] += t.n;
            }
            bool tail = false;
            for (int64_t k = p->pad_off[r]; k < p->pad_off[r + 1]; ++k) {
                const fsi::Mx4Run &u = p->pads[k];
                EXPECT(u.rank == r && u.n <= fsi::kMx4TileBlocks, "pad");
                if (u.n == 0) tail = true;
                else blocks.add(u.at, u.n);
            }
            for (int64_t k = p->gap_off[r]; k < p->gap_off[r + 1]; ++k) elems.add(p->gaps[k].at, p->gaps[k].n);
            blocks.done();
            elems.done();
            EXPECT(tail == (I.shard_bytes > 17 * I.shard_blocks), "bytes after the scales");
            for (int32_t i = 0; i < P.n_params; ++i) {
                int64_t b, n;
                EXPECT(fs_mx4_plan_piece(p, i, r, &b, &n) == FS_OK && b >= 0 && b + (n + 31) / 32 <= I.shard_blocks, "piece");
            }
        }
        for (int32_t i = 0; i < P.n_params; ++i) {
            EXPECT(got[i] == numel[i], "parameter %d: %lld of %lld", i, (long long)got[i], (long long)numel[i]);
            fs_mx4_matrix_t m;
            alignas(16) static char somewhere[16];
            fs_mx4_plan_matrix(p, somewhere, i, &m);   // any answer; it reads nothing
        }
        EXPECT((int64_t)(p->tiles.size() * sizeof(fsi::Mx4Tile)) <= p->ws_pads &&
               p->ws_pads + (int64_t)(p->pads.size() * sizeof(fsi::Mx4Run)) <= p->ws_gaps &&
               p->ws_gaps + (int64_t)(p->gaps.size() * sizeof(fsi::Mx4Run)) <= I.workspace_bytes, "workspace");
        ++g_plans;
    }
    fs_plan_destroy(plan);
    fs_mx4_plan_destroy(p);
}

static void every_mode(const Shapes &sh, int32_t world) {
    for (fs_dtype dt : {FS_BF16, FS_FP32}) {
        check(sh, dt, world, 0, FS_FSDP2_PER_PARAM);
        check(sh, dt, world, 0, FS_FSDP1_FLAT);
        check(sh, dt, world, 1, FS_FSDP1_FLAT);
    }
}

int main() {
    for (int32_t world : {1, 2, 3, 8, 64}) {
        every_mode(Shapes(), world);
        for (int64_t a = 0; a <= 40; ++a)
            for (int64_t b : {0, 1, 31, 32, 33, 8192, 8193}) {
                Shapes sh;
                sh.add(a, b);
                sh.add(b);
                sh.add(a);
                every_mode(sh, world);
            }
    }
    uint64_t x = 7;
    auto next = [&](uint64_t n) { return (int64_t)((x = x * 6364136223846793005ull + 1442695040888963407ull) >> 33) % (int64_t)n; };
    for (int k = 0; k < 60; ++k) {
        Shapes sh;
        for (int64_t i = next(12); i >= 0; --i) {
            if (next(2)) sh.add(next(300), next(200));
            else sh.add(next(40000));
        }
        every_mode(sh, (int32_t)(1 + next(20)));
    }
    const int64_t d = 4096, f = 11008;
    Shapes block;
    for (int i = 0; i < 4; ++i) block.add(d, d);
    block.add(f, d);
    block.add(f, d);
    block.add(d, f);
    block.add(d);
    block.add(d);
    every_mode(block, 8);
    {   // refusals leave nothing behind
        fs_mx4_plan_t p = nullptr;
        EXPECT(fs_mx4_plan(nullptr, &p) == FS_E_INVAL && !p, "NULL plan");
        EXPECT(fs_mx4_plan_info(nullptr, nullptr) == FS_E_INVAL, "NULL info");
        fs_mx4_plan_destroy(nullptr);
    }
    if (g_fail) {
        fprintf(stderr, "%d failures over %ld plans\n", g_fail, g_plans);
        return 1;
    }
    printf("ok: %ld plans\n", g_plans);
    return 0;
}
