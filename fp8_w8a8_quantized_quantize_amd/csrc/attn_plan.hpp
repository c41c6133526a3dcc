// How the attention calls over the paged cache are divided among workgroups:
// plain host arithmetic, with no device code, on sizes and launch hints alone.
#pragma once

#include <algorithm>
#include <cstdint>

namespace fp8k {

// Workgroups along a grid axis: the runtime takes less than 2^32 threads there,
// and the attention kernels have 256 a workgroup.
constexpr int64_t kMaxGrid = ((int64_t(1) << 32) - 1) / 256;

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// launch(first, n) for all of `units` workgroups, as many at a time as a grid
// holds; its first result that is not 0 (success) ends them.
template <typename Launch>
inline auto in_launches(int64_t units, Launch launch) {
    auto e = launch(int64_t(0), std::min(units, kMaxGrid));
    for (int64_t first = kMaxGrid; first < units && static_cast<int>(e) == 0; first += kMaxGrid)
        e = launch(first, std::min(units - first, kMaxGrid));
    return e;
}

// ---- which form ----

// Whether the tiled kernel takes a call, by the query rows of a sequence that
// share a KV head.  The streaming kernel walks over the keys once per 16 of
// them, the tiled one once per 128, but has its products wait on LDS.
// Streaming / tiled, us, 64 / 8 heads of 128, bf16, 16384 keys:
//     rows            24          32          64          128         512
//     1 sequence      22.2/22.8   21.1/20.9   25.3/26.5   35.5/37.6   89/63
//     8 sequences     99/84       100/66      115/84      197/111     622/348
//     32 sequences    270/289     250/230     420/289     838/382     3980/1322
// Two-term products (fp16, fp32, lse) fill the tiled kernel's matrix cores twice,
// and D = 256 leaves it one workgroup a CU; two sequences, 16384 keys:
//     rows                    12      24      32      48      64      96     128    256
//     fp16, D = 128                   34/41                   48/46   57/52  97/62  130/91
//     bf16, D = 256 (32/8)    39/73           50/64   74/76   74/68          115/81
//     fp16, D = 256 (32/8)                    43/61   53/68   56/64          89/74
inline bool attn_tiled(int64_t Hq, int64_t Hkv, int64_t D, int64_t new_rows, bool two_terms) {
    const int64_t columns = new_rows * (Hq / Hkv);
    return two_terms || D == 256 ? columns > 64 : columns >= 32;
}

// ---- the streaming form ----

constexpr int kTile = 32;     // keys per step of a wave
constexpr int kWaves = 4;     // waves of a workgroup
constexpr int kCols = 16;     // query columns of a tile

// Cost of an item's start (page and length look-ups, the first tiles' latency,
// the join of its waves) in rounds: measured about 6 us against 1.5 us a round.
constexpr int kItemCost = 4;

struct StreamPlan {
    int hw, shares, min_share;
    int64_t col_tiles;
    int64_t units, rows_y;  // workgroups: whole items (sequences times head groups) or shares, and column tiles
};

inline StreamPlan stream_plan(int64_t B, int64_t rows, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_q, int64_t max_len,
                              int64_t all_len) {
    StreamPlan s;
    B = std::max<int64_t>(B, 1);
    s.col_tiles = ceil_div(std::max<int64_t>(max_q, 1) * (Hq / Hkv), kCols);
    const int most = Hkv % 4 == 0 ? 4 : Hkv % 2 == 0 ? 2 : 1;
    const int64_t fill = D == 256 ? 256 : 512;  // workgroups that are resident at once
    // Where max_q is far from most sequences' new rows, a grid of it would be empty for the most part: some more column
    // tiles than the mean (a few rounds of the card's workgroups at the least), and the others in turn.
    const int64_t least = rows * (Hq / Hkv) / kCols + B;  // column tiles of all sequences, B fewer at the least
    const bool uneven = B * s.col_tiles > 4 * least;
    if (uneven) s.col_tiles = std::min(s.col_tiles, std::max(4 * ceil_div(least, B), 4 * fill * most / (B * Hkv)));
    s.col_tiles = std::max<int64_t>(1, std::min<int64_t>({s.col_tiles, kMaxGrid / (B * Hkv), 65535}));
    s.hw = most;
    s.shares = 0;
    s.min_share = 2;
    auto whole = [&]() {
        s.units = B * (Hkv / s.hw);
        s.rows_y = s.col_tiles;
        return s;
    };
    // Short sequences go whole, with as many heads a workgroup as still fill the card: shares cost a scan and a second
    // kernel.  Whole / shares, us, 64 / 8 heads of 128, bf16:  1 x 640 keys 11.5 / 12.5, 1 x 1000 14.8 / 12.4, 16 x 700
    // 13.6 / 17.4, 32 x 1000 16.3 / 23.9, 256 x 500 54 / 73; 16 x 2000 23.8 / 22.9, 16 x 8000 75 / 67, 1 x 8000 68 / 15.
    if (max_len <= 1024) {
        while (s.hw > 1 && B * (Hkv / s.hw) * s.col_tiles < fill) s.hw /= 2;
        if (max_len <= 640 || (!uneven && B * (Hkv / s.hw) * s.col_tiles >= fill / 4)) return whole();
    }
    // costs of all sequences are added up in 32 bits
    const int64_t cost = (ceil_div(all_len, kTile) + kItemCost) * least;
    if (cost >= (int64_t(1) << 30)) return whole();
    s.hw = most;
    // Several heads a workgroup read longer runs of a cache row; with few rounds a share, its four waves on one head
    // shorten the chain instead.  Four heads / one, us: 48 x 4096 ... 32768 keys 297 / 318, 64 x 1000 ... 8000 102 / 112,
    // 1 x 8000 17.2 / 14.7, 19 x 1 ... 9001 of 256 channels 25.8 / 23.9.
    const int64_t items = (uneven ? least : B * s.col_tiles) * (Hkv / most);
    if (items < 32 || items * max_len * most / (kTile * kWaves) < 16 * fill) s.hw = 1;
    s.shares = (int)std::max<int64_t>(1, fill / (Hkv / s.hw));
    s.units = s.shares * (Hkv / s.hw);
    s.rows_y = 1;
    return s;
}

// ---- the tiled form ----

constexpr int kTileKeys = 64;   // keys of a tile
constexpr int kTileCols = 128;  // query columns of a workgroup

// Workgroups that share a column tile's keys: as many as the card holds at once
// (two a CU, one with D = 256), where column tiles alone are fewer, each with at
// least 4 key tiles.  64 tokens over 16384 keys, 64 / 8 heads of 128: 59 us with
// one round of workgroups, 67 and 76 with one and a half and two (a second
// round that is not full), 367 without shares.  At 2048 keys: 27 us with 2 key
// tiles at least, 21 with 4, 25 with 8.  With long keys also two or three, where
// that leaves rounds fuller by a tenth or more (560 tokens: 527 us without, 404
// with 3; 1100: 903 and 749); at 2048 keys their parts cost what that gains (83
// and 85, 151 and 162).
inline int64_t tile_splits(int64_t B, int64_t rows, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_q, int64_t max_len) {
    const int64_t group = Hq / Hkv, planned = B * ceil_div(max_q * group, kTileCols);
    const int64_t full = rows * group / kTileCols;  // at least; `planned` may come from too small a max_q
    const int64_t tiles = std::max<int64_t>(1, std::max(full, std::min(planned, full + B)) * Hkv);
    const int64_t fill = D == 256 ? 256 : 512;
    int64_t s = std::max<int64_t>(1, std::min<int64_t>({fill / tiles, 64, max_len / (4 * kTileKeys)}));
    if (max_len >= 4096) {
        auto rounds = [&](int64_t n) { return (tiles * n + fill - 1) / fill; };
        for (int64_t n = s + 1; n <= 3; ++n)
            if (10 * rounds(n) * s < 9 * rounds(s) * n) s = n;
    }
    return s;
}

// Slots for the column tiles of a ragged batch, of which it has rows * group /
// kTileCols + B at the most, end to end whatever the sequences' new tokens are, so
// no hint is needed.  How a workgroup finds its tile, with 64/8 heads:
//   - the tiles of up to kMaxScan sequences added up, 64 of them at a time, the
//     empty slots last;
//   - or, of more than 64 with many workgroups, by the sequences' first columns,
//     with a slot to spare for each among the others.  Empty ones take CUs in turn
//     with full ones, which shows where the card is filled once or twice, but there
//     is less to look up: 32 x 16 tokens over 16384 keys 565 us so and 370 added
//     up, 300 x 64 over 100 keys 349 and 371;
//   - where by max_q one tile each will do, those come first and only the others,
//     if any, are looked for: 1024 x 8 over 512 keys 441 us, 465 by first columns,
//     473 all added up.
// One new token per sequence takes the same number of tiles everywhere.  A unit of
// work is a slot, a key share and a KV head.
constexpr int kMaxScan = 1024;

struct TilePlan {
    int64_t splits, col_tiles, slots, units;
    bool exact;
};

inline TilePlan tile_plan(int64_t B, int64_t rows, int64_t Hq, int64_t Hkv, int64_t D, bool decode, int64_t max_q,
                          int64_t max_len) {
    const int64_t group = Hq / Hkv, each = ceil_div(max_q * group, kTileCols);
    TilePlan t;
    t.splits = tile_splits(B, rows, Hq, Hkv, D, max_q, max_len);
    // each sequence's tiles but the first are fewer than its columns / kTileCols, so one tile each leaves slots for them
    t.slots = decode ? B * each : rows * group / kTileCols + B;
    t.col_tiles = decode ? each : each == 1 && B <= kMaxScan ? 1 : 0;
    t.units = t.slots * Hkv * t.splits;
    t.exact = B <= 64 || (B <= kMaxScan && (t.col_tiles > 0 || t.units <= 8 * 512));
    return t;
}

// ---- the join of rows whose keys were shared ----

// A unit is the 256 / (D / 4) / spread output rows of a workgroup, of
// which spread thread groups take one row together where rows are few.
struct JoinPlan {
    int64_t rows;  // new rows of a sequence (of all, for the tiled form's parts) that the units hold
    int spread, log_spread;
    int64_t units;
};

// max_q: the most new rows of a sequence; where most have far fewer, `typical`,
// units for some more than those, and for the rest in turn.
inline JoinPlan join_plan(int64_t heads, int64_t D, int64_t max_q, int64_t typical) {
    JoinPlan j;
    if (typical < max_q) max_q = std::min(max_q, std::max(2 * typical, (int64_t(1) << 17) / heads));
    j.rows = std::max<int64_t>(1, std::min<int64_t>(max_q, (int64_t(1) << 26) / heads));
    const int64_t groups = 256 / (D / 4);
    j.spread = 1, j.log_spread = 0;
    while (j.spread < groups && heads * j.rows * j.spread < 2048) j.spread *= 2, ++j.log_spread;
    j.units = ceil_div(heads * j.rows, groups / j.spread);
    return j;
}

}  // namespace fp8k
