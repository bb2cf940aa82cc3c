// How a beam step's rows are cut into parts: on the host the plan, on both sides a part's columns.
#pragma once

#include <algorithm>

#include "vocab_common.cuh"

namespace lmloss {
namespace {

constexpr int kThreads = 256;
constexpr int kDepths = 8;                   // lists (parts of a sequence's rows) a thread
constexpr int kMaxLists = kDepths * kThreads;

// Where the part that begins at column `begin` ends.  A row's parts reach up to a whole part past
// its end, in all past 2^31 where V is near that, so the end is compared without their sum.
__host__ __device__ inline int part_end(int begin, int tiles, int tile_cols, int V)
{
    const int size = tiles * tile_cols;   // at most V rounded up to tiles
    return size < V - begin ? begin + size : V;
}

struct BeamPlan {
    int vpt, tiles, slices;
    size_t keys, stats, total;
};

// Tiles of four vectors a thread, or of one where those would not give every SM a
// block.  The parts of a row: a block costs its tiles and about eight more (the
// thresholds' barriers, the ranking, the count; tiles of one are a quarter as long),
// and an SM's blocks run together up to about three, one after another beyond.
// Measured at 512 rows of 262144 bf16: one part 52 us, two 57; 32 rows: eleven parts 23.6
// us, thirty-two 34.
lmloss_status plan_beam(const lmloss_beam_args* a, int num_sms, BeamPlan& P)
{
    const int64_t rows = a->B * a->K, E = 16 / float_bytes(a->dtype);
    auto tiles_of = [&](int vpt) { return (a->V + vpt * kThreads * E - 1) / (vpt * kThreads * E); };
    P.vpt = rows * tiles_of(4) >= num_sms ? 4 : 1;
    const int64_t all = tiles_of(P.vpt), fixed = P.vpt == 4 ? 8 : 32;
    // at most kMaxLists parts in a sequence's rows
    const int64_t most = kMaxLists / a->K, least = (all + most - 1) / most;
    int64_t tiles = all, best = INT64_MAX;
    for (int64_t t = least; t <= all && t <= least + 63; ++t) {
        const int64_t blocks = rows * ((all + t - 1) / t);
        const int64_t cost = std::max<int64_t>((blocks + num_sms - 1) / num_sms, 3) * (t + fixed);
        if (cost < best) {
            best = cost;
            tiles = t;
        }
    }
    const int64_t slices = (all + tiles - 1) / tiles;
    if (tiles > (1 << 30) || rows * slices >= (int64_t(1) << 31)) return LMLOSS_ERR_UNSUPPORTED;
    P.tiles = static_cast<int>(tiles);
    P.slices = static_cast<int>(slices);
    P.keys = 0;
    P.stats = vocab_align(sizeof(uint64_t) * static_cast<size_t>(rows * slices * a->M));
    P.total = P.stats + vocab_align(sizeof(float2) * static_cast<size_t>(rows * slices));
    return LMLOSS_OK;
}

}  // namespace
}  // namespace lmloss
