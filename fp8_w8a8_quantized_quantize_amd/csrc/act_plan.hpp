// How the products with an epilogue are divided into tiles and k ranges: plain host
// arithmetic on sizes, with no device code.
//
// A workgroup works on one output tile, 128 k (a stage) at a time.  Large tiles move
// the fewest bytes per output, but there are few of them, and a lone workgroup on a
// compute unit waits for each stage's load; small ones fill the card and hide loads
// behind each other.  The estimate below is linear in the stages and in the
// workgroups of a compute unit, with slopes measured on MI355X (us; weights in cache;
// bf16 output unless said):
//   tile                64        128       256
//   512 x 4096 x 4096   18.9      19.2      52.4
//   1024 x 4096 x 4096  30.9      24.1      52.8
//   2048 x 4096 x 4096  57        38        55
//   4096 x 4096 x 4096  109       72        65
//   fp32 output         162       127       -      (4096 x 4096 x 4096)
// With weights from HBM, 17 to 64 rows of 28672 x 8192 and 8192 x 28672 take 46 to 57 us
// by these plans, 235 MB at 4.2 to 5.1 TB/s, and 60 to 66 with an fp32 output.
// A k range is split when there are too few tiles of 64 for the card: 100 x 512 x
// 16384 takes 28.6 us in 16 workgroups and 12.4 us in 128, the addition included.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

namespace fp8k {

// Workgroups of a launch: the runtime takes less than 2^32 threads along an axis.
// The entry points refuse outputs of more than this many tiles of 128, so that one
// of the tile sizes always fits.
constexpr int64_t kMaxActTiles = ((int64_t(1) << 32) - 1) / 256 - 8;

struct ActPlan {
    int tile;     // output tiles of tile x tile, one workgroup each
    int stages;   // stages of a workgroup's ring in LDS
    int splits;   // workgroups sharing a tile's k; more than one: their sums are added by a second kernel
    int split_k;  // k of each, a multiple of 128
};

// Nanoseconds of `wgs` workgroups of a tile size over `kt` stages, and the ring that
// goes with it: deep where a compute unit has so few workgroups that nothing else
// hides the loads (and LDS to spare).  half: products in fp16, half the rate.
inline int64_t act_cost(int tile, int64_t wgs, int64_t kt, bool half, int* stages) {
    const int64_t n = (wgs + 255) / 256;  // of a compute unit
    *stages = 2;
    if (tile == 64) {
        if (half) {
            if (n == 1) *stages = 4;
            return 4500 + kt * (n == 1 ? 390 : 60 + 320 * n);
        }
        if (n <= 2) *stages = 4;
        return 4500 + kt * (n == 1 ? 200 : n == 2 ? 430 : 240 * n);
    }
    if (tile == 128) {
        if (half) return 6000 + kt * 930 * n;
        if (n == 1) *stages = 4;
        return 6000 + kt * (n == 1 ? 400 + 180 * wgs / 256 : 520 * n);
    }
    return 12000 + kt * 1550 * n;
}

// Dense products.
inline ActPlan act_plan(int64_t M, int64_t N, int64_t K, bool half) {
    const int64_t kt = (K + 127) / 128;
    ActPlan best{64, 2, 1, (int)std::max<int64_t>(K, 1)};
    int64_t least = INT64_MAX;
    for (int tile = 64; tile <= (half ? 128 : 256); tile *= 2) {
        const int64_t wgs = ((M + tile - 1) / tile) * ((N + tile - 1) / tile);
        if (wgs > kMaxActTiles) continue;
        int stages;
        const int64_t cost = act_cost(tile, wgs, kt, half, &stages);
        if (cost < least) {
            least = cost;
            best.tile = tile, best.stages = stages;
        }
        if (tile > 64) continue;
        // splits of at least four stages; the addition: a launch, and the sums written and read once
        for (int64_t s = 2; s <= 16 && wgs * s <= 512 && kt / s >= 4; s *= 2) {
            const int64_t per = (kt + s - 1) / s, used = (kt + per - 1) / per;
            const int64_t split = act_cost(tile, wgs * used, per, half, &stages) + 2500 + 100 * used + used * M * N * 8 / 3000;
            if (split < least) {
                least = split;
                best = ActPlan{tile, stages, (int)used, (int)per * 128};
            }
        }
    }
    if (best.tile > 64) best.splits = 1, best.split_k = (int)std::max<int64_t>(K, 1);
    return best;
}

// Bytes of a plan's partial sums.
inline size_t act_plan_ws_bytes(const ActPlan& p, int64_t M, int64_t N) {
    return p.splits > 1 ? (size_t)p.splits * (size_t)M * (size_t)N * sizeof(float) : 0;
}

// Products per expert, R rows of E experts; the rows of one are not known here, and
// taken to leave half a tile empty.  With few of them the weights' stream from memory
// is what counts, and small tiles with deep rings keep most of it under way (64
// experts of 2048 x 7168, 16 tokens of 8 choices: tiles of 64 122 us, of 128 150, of
// 256 182; 4096 tokens: 905, 610 and 505).  As planned, 16, 64, 256, 1000 and 4096
// tokens take 122, 159, 193, 274 and 520 us, with an fp32 output 133, 184, 221, 360 and
// 935.
inline ActPlan grouped_act_plan(int64_t R, int64_t E, int64_t N, int64_t K, bool half) {
    auto most = [&](int tile) { return ((R + tile - 1) / tile + E) * ((N + tile - 1) / tile); };  // tiles
    if (R <= (half ? 64 : 32) * E && most(64) <= kMaxActTiles) return ActPlan{64, 4, 1, 0};
    ActPlan best{64, 2, 1, 0};
    int64_t least = INT64_MAX;
    for (int tile = 64; tile <= (half ? 128 : 256); tile *= 2) {
        if (most(tile) > kMaxActTiles) continue;
        const int64_t wgs = ((R + tile - 1) / tile + (E + 1) / 2) * ((N + tile - 1) / tile);
        int stages;
        const int64_t cost = act_cost(tile, wgs, (K + 127) / 128, half, &stages);
        if (cost < least) {
            least = cost;
            best.tile = tile;
        }
    }
    return best;
}

}  // namespace fp8k
