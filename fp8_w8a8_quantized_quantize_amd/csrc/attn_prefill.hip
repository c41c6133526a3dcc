// Attention over the paged FP8 KV cache on gfx950, tiled form: many query rows
// per sequence, bound by the matrix cores.
//
// Mathematics, operand terms and visibility are those of the streaming form
// (attn_paged.hip): codes exact in fp16, key scales in the query, value scales
// at the output, scores transposed so that a lane's results belong to one query
// column, p straight from the scores' registers into the second product.  The
// sum of p, here on the vector unit, takes p as the product does: with one term
// rounded to fp16, with two as it is, which they give to 2^-22.
//
// Tile.  The columns are a KV head's query rows, token times group, so one pass
// over the keys serves all query heads of the group.  A workgroup of four waves
// takes 128 columns, 32 a wave, and walks over 64-key tiles that all its waves
// share in LDS: K as fp16 rows, V as fp16 transposed, eight keys of a channel in
// 16 bytes in the order in which a lane holds its p.  Codes become fp16 once per
// workgroup, on the way into LDS.  D = 128 takes 200 registers and 72 KB of LDS
// (two terms 255), two workgroups a CU: the softmax of one wave runs beside the
// matrix work of the other on its SIMD.  64 columns a wave (half the LDS reads per
// matrix instruction, one wave per SIMD) spilled and took 3.7 ms where this takes
// 1.15 to 1.24 by the card's clock (8192 tokens, 64 / 8 heads of 128, bf16: 890 to
// 960 TFLOP/s), and so did forming the next tile's scores during the softmax (2.3
// ms).  One workgroup does one unit of work: a loop around it cost up to 40 more
// registers and, with two terms, spills.  Two terms with D = 256 spill 9 registers,
// 27 under a bias or a cap.
//
// Bound: matrix cores 42 %, vector unit 48 % of the cycles (230 instructions per
// 32 columns x 64 keys, 32 of them exponentials, beside 32 matrix instructions
// of 32 cycles), LDS 42 %; the two waves of a SIMD seldom want different units
// (wave priorities around either phase changed nothing).
//
// One barrier per tile: step t writes K and V of tile t into the buffers last
// read in step t - 2, starts the loads of tile t + 1 into registers, and computes
// after the barrier.
//
// Column tiles of all sequences lie end to end in the grid, so its size is the
// batch's own whatever the hint says.  Where they are few, several
// workgroups share a tile's keys: each leaves its unscaled fp32 sums, its
// reference and its sum of p in the workspace, and the streaming form's join adds
// them in their order, row by row.
#include <algorithm>
#include <type_traits>

#include "attn_common.hpp"
#include "attn_plan.hpp"

namespace fp8k {

namespace {

typedef float v16f __attribute__((ext_vector_type(16)));

constexpr int kWavesT = 4;
constexpr int kThreadsT = kWavesT * kWave;
constexpr int kKeys = kTileKeys;
static_assert(kTileCols == kWavesT * 32, "32 columns a wave");

struct TileArgs {
    PagedAttn p;
    int group;
    int splits;     // workgroups that share a column tile's keys
    int col_tiles;  // column tiles laid out for every sequence, 0: none
    bool exact;     // no slot to spare among the others
    int slots;
    int unit0;      // the launch's first of the units (slot, split, KV head)
    float* part_o;    // [rows][Hq][splits][D], with splits > 1
    float2* part_ml;  // [rows][Hq][splits]: reference (log2), sum
    FastDiv by_block, by_group, by_kv_heads, by_splits, by_batch;
};

// The column tile of slot `slot`.  The first slots are for the tiles laid out for
// every sequence, the last ones, which see the most keys, first; then come all
// other tiles, the sequences' end to end.
struct TileAt {
    int b, ct;  // b < 0, or ct below 0 or past the sequence's tiles: none
};

__device__ __forceinline__ TileAt tile_at(const TileArgs& a, int slot, int lane) {
    const PagedAttn& p = a.p;
    if (slot < p.B * a.col_tiles) {
        const int tile = a.by_batch.of(slot);
        return TileAt{slot - tile * p.B, a.col_tiles - 1 - tile};
    }
    slot -= p.B * a.col_tiles;
    if (p.B == 1) {
        const Seq s = sequence(p, 0);
        const int ct = (s.nq * a.group + kTileCols - 1) / kTileCols - 1 - slot;
        return TileAt{ct >= a.col_tiles ? 0 : -1, ct};
    }
    if (a.exact) {
        auto others = [&](int b) {
            // past the last sequence both are its end; a branch would wait for every load by itself
            const int lo = min(max(p.cu_q[min(b, p.B)], 0), p.rows), hi = min(p.cu_q[min(b + 1, p.B)], p.rows);
            return max((int)(((uint32_t)max(hi - lo, 0) * a.group + kTileCols - 1) / kTileCols) - a.col_tiles, 0);
        };
        // lane l adds up the sequences 64 i + l, which come before lane l + 1's
        int mine = 0;
#pragma unroll 8
        for (int b0 = 0; b0 < p.B; b0 += kWave) mine += others(b0 + lane);
        int upto = wave_scan(mine);
        uint64_t past = __ballot(upto > slot);
        if (past == 0) return TileAt{-1, 0};
        const int l = __builtin_ctzll(past);
        if (p.B <= kWave) return TileAt{l, a.col_tiles + __builtin_amdgcn_readlane(upto, l) - 1 - slot};
        // and then lane i stands for sequence 64 i + l
        slot -= __builtin_amdgcn_readlane(upto - mine, l);
        upto = wave_scan(others(kWave * lane + l));
        past = __ballot(upto > slot);
        const int i = past ? __builtin_ctzll(past) : 0;
        return TileAt{kWave * i + l, a.col_tiles + __builtin_amdgcn_readlane(upto, i) - 1 - slot};
    }
    // Or not added up: sequence b's tiles start at slot floor(c / kTileCols) + b, c its first column, with one slot to
    // spare at the most.  Starts rise with b, so a wave finds b by 64 probes a step.
    auto start = [&](int b) { return (int)((uint32_t)min(max(p.cu_q[b], 0), p.rows) * a.group / kTileCols) + b; };
    slot = a.slots - 1 - slot;  // every sequence's last tile first
    int b = 0;
    for (int n = p.B; n > 1;) {  // one of n sequences from b on
        const int step = (n + kWave - 1) / kWave, at = lane * step;
        const uint64_t starts = __ballot(at < n && start(b + min(at, n - 1)) <= slot);
        const int last = starts ? (kWave - 1 - __builtin_clzll(starts)) * step : 0;
        b += last;
        n = min(step, n - last);
    }
    return TileAt{b, slot - start(b)};
}

// LDS rows are padded by 16 bytes, so that 32 neighbouring rows spread over the
// banks.  V's channel d, byte d % VB of the piece that lane d / VB stages, is
// row 32 (d % VB) + d / VB: writes and operand reads both take neighbouring
// rows, and the output blocks hold a lane's channels in order.
// LDS: two K tiles, two V tiles, cache offsets of 16 rows per wave for two
// tiles, and which keys of four tiles are there.
template <int D>
struct TileLds {
    static constexpr int kKRow = 2 * D + 16, kVRow = 2 * kKeys + 16;  // bytes; padded off the banks
    static constexpr int kKTile = kKeys * kKRow, kVTile = D * kVRow;
    static constexpr int kV = 2 * kKTile;
    static constexpr int kRows = kV + 2 * kVTile;
    static constexpr int kMask = kRows + 2 * kKeys * 8;
    static constexpr int kBytes = kMask + 4 * kWavesT * 4;
};

extern __shared__ __attribute__((aligned(1024))) uint8_t tile_smem[];

// Scheduling hint for N operand reads from LDS with M matrix instructions each:
// the first AHEAD reads at once, then a read per M instructions, so that an LDS
// round trip (about 150 cycles with eight waves reading) passes behind AHEAD
// instructions of 32 cycles.
template <int N, int M, int AHEAD>
__device__ __forceinline__ void reads_ahead() {
    __builtin_amdgcn_sched_group_barrier(0x100, AHEAD, 0);
#pragma unroll
    for (int i = 0; i < N - AHEAD; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, M, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, M * AHEAD, 0);
}

template <int D, int FMT, bool BIAS, int TERMS>
__global__ __launch_bounds__(kThreadsT, D == 256 ? 1 : 2) void attn_tile(TileArgs a) {
    const PagedAttn& p = a.p;
    constexpr int NK = D / 16;  // matrix instructions along the channels of K
    constexpr int DB = D / 32;  // 32-channel blocks of the output
    constexpr int VB = D / 32;  // V channels a thread stages
    using Lds = TileLds<D>;
    using P = PScale<TERMS>;
    typedef typename std::conditional<D == 64, uint16_t, typename std::conditional<D == 128, uint32_t, v2u>::type>::type vpiece;

    const int tid = threadIdx.x, lane = tid % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int c = lane % 32, h = lane / 32;
    // KV heads vary fastest: with 8 of them an XCD keeps to one head's keys.
    const int unit = a.unit0 + blockIdx.x;
    const int rest = a.by_kv_heads.of(unit), hk = unit - rest * p.Hkv;
    const int nth = a.by_splits.of(rest), split = rest - nth * a.splits;
    const TileAt at = tile_at(a, nth, lane);
    const int b = at.b, ct = at.ct;
    if (b < 0) return;
    const Seq seq = sequence(p, b);
    const int prefix = p.prefix ? p.prefix[b] : 0;
    const int cols = seq.nq * a.group;
    if ((uint32_t)ct >= (uint32_t)((cols + kTileCols - 1) / kTileCols)) return;
    const uint32_t C = 2u * p.Hkv * D;
    const int32_t* table = p.block_table + (int64_t)b * p.ld_table;
    const int last_page = max(p.max_blocks - 1, 0);
    uint64_t* const rows = reinterpret_cast<uint64_t*>(tile_smem + Lds::kRows) + wave * 16;  // [tile % 2][4 waves][16]
    uint32_t* const there = reinterpret_cast<uint32_t*>(tile_smem + Lds::kMask);             // [tile % 4][4 waves]

    // the keys any column of the workgroup sees
    int tlo, thi, unused;
    visible(p, seq, prefix, a.by_group.of(ct * kTileCols), tlo, unused);
    visible(p, seq, prefix, a.by_group.of(min(cols - 1, ct * kTileCols + kTileCols - 1)), unused, thi);
    thi = max(thi, 0);
    tlo = min(tlo, thi);
    const int base = p.window > 0 ? tlo / kKeys * kKeys : 0;
    const int all = thi > base ? (thi - base + kKeys - 1) / kKeys : 0;
    const int first = a.by_splits.of(all * split), tiles = a.by_splits.of(all * (split + 1));  // 2^24 tiles, 64 shares at most
    // this lane's column
    const int col = ct * kTileCols + wave * 32 + c;
    const bool has = col < cols;
    const int qi = has ? a.by_group.of(col) : 0;
    const int head = hk * a.group + (has ? col - qi * a.group : 0);
    const int64_t row = seq.row0 + qi;
    const int pos = seq.len - seq.nq + qi;
    const float slope = p.alibi ? p.alibi[head] * kLog2e : 0.0f;
    int lo, hi;
    visible(p, seq, prefix, qi, lo, hi);
    if (!has) lo = 0x7FFFFFFF, hi = 0;
    int wlo = lo, whi = hi;  // the keys any column of this wave sees
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        wlo = min(wlo, __shfl_xor(wlo, off, kWave));
        whi = max(whi, __shfl_xor(whi, off, kWave));
    }
    wlo = __builtin_amdgcn_readfirstlane(wlo);
    whi = __builtin_amdgcn_readfirstlane(whi);

    // q times the key scales, in fp16 terms
    v8h qt[TERMS][NK];
    float cs;
    {
        float x[NK][8], top = 0.0f;
#pragma unroll
        for (int st = 0; st < NK; ++st) {
            v4u raw[2];
            load_q8<TERMS>(p, row * p.ldq + (int64_t)head * D + 16 * st + 8 * h, raw);
            unpack_q8<TERMS>(p, raw, x[st]);
            const float4* ks = reinterpret_cast<const float4*>(p.scales + hk * D + 16 * st + 8 * h);
            const float4 k0 = ks[0], k1 = ks[1];
            const float k[8] = {k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[st][e] *= fmaxf(k[e], kScaleFloor);
                top = fmaxf(top, fabsf(x[st][e]));
            }
        }
        top = fmaxf(top, swap32(top));
        const int shift = 15 - __builtin_amdgcn_frexp_expf(top);
#pragma unroll
        for (int st = 0; st < NK; ++st)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float y = __builtin_amdgcn_ldexpf(x[st][e], shift);
                qt[0][st][e] = (_Float16)y;
                if constexpr (TERMS == 2) qt[TERMS - 1][st][e] = (_Float16)(y - (float)qt[0][st][e]);
            }
        cs = __builtin_amdgcn_ldexpf(p.scale, -shift);
    }
    if (p.softcap > 0.0f) cs *= kLn2;  // the cap takes the natural score
    const float cap_in = cap_factor(p.softcap);

    float m = 0.0f, l = 0.0f, l2 = 0.0f, limit = kNoRef;
    v16f o[DB];
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;

    // ---- staging.  A wave stages keys 16 wave .. + 15 of a tile: K, a quarter row per thread; V, the eight keys of
    // two lane groups, VB channels per thread.
    auto page_of = [&](int t) { return table[min(a.by_block.of(base + t * kKeys + 16 * wave + lane % 16), last_page)]; };
    // cache offsets of the wave's 16 rows of tile t, 0 for keys that are not there
    auto rows_of = [&](int t, int page) {
        const int key = base + t * kKeys + 16 * wave + lane % 16;
        const bool ok = key >= tlo && key < thi && page >= 0 && page < p.num_blocks;
        const uint32_t r = ok ? (page - a.by_block.of(key)) * p.block + key : 0;
        if (lane < 16) rows[t % 2 * kKeys + lane] = (uint64_t)r * C;
        const uint32_t mask = (uint32_t)__ballot(ok) & 0xFFFFu;
        if (lane == 0) there[t % 4 * kWavesT + wave] = mask;
        __builtin_amdgcn_wave_barrier();
        return mask;
    };
    v4u kreg[D / 64];
    vpiece vreg[8];
    auto load_k = [&](int t) {
        const uint8_t* src = p.cache + rows[t % 2 * kKeys + lane / 4] + hk * D + lane % 4 * (D / 4);
#pragma unroll
        for (int i = 0; i < D / 64; ++i) kreg[i] = *reinterpret_cast<const v4u*>(src + 16 * i);
    };
    auto load_v = [&](int t) {
        const uint8_t* src = p.cache + (int64_t)(p.Hkv + hk) * D + c * VB;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            vreg[e] = *reinterpret_cast<const vpiece*>(src + rows[t % 2 * kKeys + 8 * (e / 4) + 4 * h + e % 4]);
    };
    auto store_k = [&](int t) {
        uint8_t* dst = tile_smem + t % 2 * Lds::kKTile + (16 * wave + lane / 4) * Lds::kKRow;
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int unit = (lane % 4 * (D / 64) + i) * 2 + k;
                *reinterpret_cast<v8h*>(dst + unit * 16) =
                    row_f16<FMT>(kreg[i][2 * k], kreg[i][2 * k + 1]);
            }
    };
    auto vword = [&](int e, int i) -> uint32_t {
        if constexpr (D == 256)
            return vreg[e][i];
        else
            return vreg[e];
    };
    auto store_v = [&](int t, uint32_t mask) {
        uint8_t* const dst = tile_smem + Lds::kV + t % 2 * Lds::kVTile;
        if (mask != 0xFFFFu) {
            // a code behind the sequence may be anything, NaN too: 0 * NaN must not reach the sum
#pragma unroll
            for (int e = 0; e < 8; ++e)
                vreg[e] = ((mask >> (8 * (e / 4) + 4 * h + e % 4)) & 1u) ? vreg[e] : vpiece(0);
        }
#pragma unroll
        for (int j = 0; j < VB; ++j) {
            v4u r;
#pragma unroll
            for (int i = 0; i < 4; ++i) r[i] = pair_f16<FMT>(vword(2 * i, j / 4), vword(2 * i + 1, j / 4), j % 4);
            *reinterpret_cast<v4u*>(dst + (32 * j + c) * Lds::kVRow + (2 * wave + h) * 16) = r;
        }
    };
    v16f s[2];
    auto scores = [&](int t) {
        const uint8_t* src = tile_smem + t % 2 * Lds::kKTile + c * Lds::kKRow + h * 16;
#pragma unroll
        for (int j = 0; j < 32; ++j) s[j / 16][j % 16] = 0.0f;
#pragma unroll
        for (int st = 0; st < NK; ++st)
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                const v8h k = *reinterpret_cast<const v8h*>(src + 32 * kb * Lds::kKRow + 32 * st);
#pragma unroll
                for (int x = 0; x < TERMS; ++x) s[kb] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k, qt[x][st], s[kb], 0, 0, 0);
            }
        reads_ahead<2 * NK, TERMS, 4>();
    };
    // key of a lane's score j, less 4 h
    auto key_of = [](int j) { return 32 * (j / 16) + 8 * (j % 16 / 4) + j % 4; };
    // Scores of tile t above the reference, in place.
    auto above = [&](int t, uint64_t mask) {
        const int key0 = base + t * kKeys;
        if constexpr (BIAS) {
            auto capped = [&](auto series) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    s[j / 16][j % 16] = kLog2e * soft_cap<decltype(series)::value>(s[j / 16][j % 16] * cs, p.softcap, cap_in);
            };
            if (p.softcap > 0.0f) {
                if (cap_by_series<TERMS>(p.softcap)) capped(std::true_type());
                else capped(std::false_type());
            }
            const float by = p.softcap > 0.0f ? 1.0f : cs, dist = (float)(key0 + 4 * h - pos);
#pragma unroll
            for (int j = 0; j < 32; ++j)
                s[j / 16][j % 16] = __builtin_fmaf(slope, dist + (float)key_of(j), __builtin_fmaf(s[j / 16][j % 16], by, -m));
        } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) s[j / 16][j % 16] = __builtin_fmaf(s[j / 16][j % 16], cs, -m);
        }
        if (mask != ~0ull || __any(key0 < lo || key0 + kKeys > hi)) {
            const uint64_t mine = mask >> (4 * h);
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                const int key = key0 + 4 * h + key_of(j);
                const bool see = ((mine >> key_of(j)) & 1u) & (key >= lo) & (key < hi);
                s[j / 16][j % 16] = see ? s[j / 16][j % 16] : -INFINITY;
            }
        }
        float top = s[0][0];
#pragma unroll
        for (int j = 1; j < 32; ++j) top = fmaxf(top, s[j / 16][j % 16]);
        if (__any(top > limit)) {
            // Move the references of the columns that need it to the largest score, less the shift (scores past 2^24
            // are themselves too coarse for it).  A column without a reference has m = 0 and no sum yet.
            top = fmaxf(top, swap32(top));
            const bool move = top > limit;
            const float by = move ? (fabsf(top + m) < 16777216.0f ? top - P::kShift : top) : 0.0f;
            const float f = limit == P::kLimit ? __builtin_amdgcn_exp2f(-by) : 1.0f;
            m += by;
            limit = move ? P::kLimit : limit;
            l *= f;
            l2 *= f;
#pragma unroll
            for (int d = 0; d < DB; ++d) o[d] *= f;
#pragma unroll
            for (int j = 0; j < 32; ++j) s[j / 16][j % 16] -= by;
        }
    };
    // p and its product with V, 16 keys at a time
    auto product = [&](int t) {
        const uint8_t* src = tile_smem + Lds::kV + t % 2 * Lds::kVTile + c * Lds::kVRow + h * 16;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            v8h ph[TERMS];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float y = P::p(s[u / 2][8 * (u % 2) + e]);
                if constexpr (TERMS == 2) l += y;
                ph[0][e] = (_Float16)y;
                if constexpr (TERMS == 2) ph[TERMS - 1][e] = (_Float16)(y - (float)ph[0][e]);
            }
            if constexpr (TERMS == 1) {
                // The sum takes p as the product does, rounded to fp16, or the rounding would not cancel.  Two at a time,
                // fp16 subnormals kept, off by 3 2^-24 of the result at most and without bias (measured on random sums);
                // converted back and added one by one the 8192-token prompt took 1233 us, so 1176.  Two running sums: with
                // one, 1200 tokens over 2048 keys took 165 us, with four 157, so 156.
                const v2h one = {1, 1};
#pragma unroll
                for (int e = 0; e < 8; e += 4) {
                    l = __builtin_amdgcn_fdot2(v2h{ph[0][e], ph[0][e + 1]}, one, l, false);
                    l2 = __builtin_amdgcn_fdot2(v2h{ph[0][e + 2], ph[0][e + 3]}, one, l2, false);
                }
            }
#pragma unroll
            for (int db = 0; db < DB; ++db) {
                const v8h v = *reinterpret_cast<const v8h*>(src + 32 * db * Lds::kVRow + 32 * u);
#pragma unroll
                for (int x = 0; x < TERMS; ++x) o[db] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, ph[x], o[db], 0, 0, 0);
            }
        }
        reads_ahead<4 * DB, TERMS, 4>();
    };
    auto mask_of = [&](int t) {
        const uint32_t* w = there + t % 4 * kWavesT;
        const uint32_t lo32 = w[0] | (w[1] << 16), hi32 = w[2] | (w[3] << 16);
        return ((uint64_t)__builtin_amdgcn_readfirstlane(hi32) << 32) | (uint32_t)__builtin_amdgcn_readfirstlane(lo32);
    };

    if (tiles > first) {
        auto sees = [&](int t) { return base + t * kKeys < whi && base + (t + 1) * kKeys > wlo; };
        uint32_t m0 = rows_of(first, page_of(first));
        int page = page_of(first + 1);
        load_k(first);
        load_v(first);
        for (int t = first; t < tiles; ++t) {
            store_k(t);
            store_v(t, m0);
            m0 = rows_of(t + 1, page);
            page = page_of(t + 2);
            load_k(t + 1);
            load_v(t + 1);
            __syncthreads();
            if (sees(t)) {
                scores(t);
                above(t, mask_of(t));
                product(t);
            }
        }
    }

    // ---- results
    l += l2;
    l += swap32(l);
    if (has) {
        const int64_t at = (row * p.Hq + head) * a.splits + split;
        if (a.splits > 1 && h == 0) a.part_ml[at] = make_float2(limit == P::kLimit ? m : kNoRef, l);
#pragma unroll
        for (int x = 0; x < 16 * DB; x += 4) {
            // four channels in a row: elements x .. x + 3 of [row][block]
            const float4 r = make_float4(o[x % DB][x / DB], o[(x + 1) % DB][(x + 1) / DB], o[(x + 2) % DB][(x + 2) / DB],
                                         o[(x + 3) % DB][(x + 3) / DB]);
            const int i = x / DB, d = (8 * (i / 4) + 4 * h + i % 4) * VB + x % DB;
            if (a.splits > 1)
                *reinterpret_cast<float4*>(a.part_o + at * D + d) = r;
            else
                write_row(p, row, head, hk, D, d, m, l, r);
        }
    }
}

template <int D, int FMT, bool BIAS, int TERMS>
hipError_t launch_tile(TileArgs a, int64_t units, hipStream_t stream) {
    constexpr int lds = TileLds<D>::kBytes;
    if constexpr (lds > 64 * 1024) {
        const hipError_t e = FP8K_SET_LDS((attn_tile<D, FMT, BIAS, TERMS>), lds);
        if (e != hipSuccess) return e;
    }
    return in_launches(units, [&](int64_t first, int64_t n) {
        a.unit0 = (int)first;
        hipLaunchKernelGGL((attn_tile<D, FMT, BIAS, TERMS>), dim3((unsigned)n), dim3(kThreadsT), lds, stream, a);
        return hipGetLastError();
    });
}

template <int D, int TERMS>
hipError_t launch(const TileArgs& a, int64_t units, int fmt, hipStream_t stream) {
    const bool bias = a.p.softcap > 0.0f || a.p.alibi != nullptr;
    if (fmt == kKvE5M2)
        return bias ? launch_tile<D, kKvE5M2, true, TERMS>(a, units, stream) : launch_tile<D, kKvE5M2, false, TERMS>(a, units, stream);
    return bias ? launch_tile<D, kKvE4M3, true, TERMS>(a, units, stream) : launch_tile<D, kKvE4M3, false, TERMS>(a, units, stream);
}

}  // namespace

size_t attn_tiled_ws_bytes(int64_t B, int64_t rows, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_q, int64_t max_len) {
    const int64_t splits = tile_splits(B, rows, Hq, Hkv, D, max_q, max_len);
    return splits > 1 ? (size_t)(splits * rows * Hq) * ((size_t)D * 4 + 8) : 0;
}

hipError_t launch_attn_tiled(const PagedAttn& p, int D, int fmt, int64_t max_q, int64_t max_len, void* ws,
                             hipStream_t stream) {
    TileArgs a = {};
    a.p = p;
    a.group = p.Hq / p.Hkv;
    const TilePlan t = tile_plan(p.B, p.rows, p.Hq, p.Hkv, D, p.cu_q == nullptr, max_q, max_len);
    a.splits = (int)t.splits;
    a.col_tiles = (int)t.col_tiles;
    a.exact = t.exact;
    a.slots = (int)t.slots;
    a.part_o = static_cast<float*>(ws);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + (int64_t)a.splits * p.rows * p.Hq * D);
    a.by_block = FastDiv(p.block);
    a.by_group = FastDiv(a.group);
    a.by_kv_heads = FastDiv(p.Hkv);
    a.by_splits = FastDiv(a.splits);
    a.by_batch = FastDiv(p.B);
    const bool one = !two_terms(p);
    hipError_t e;
    switch (D) {
        case 64: e = one ? launch<64, 1>(a, t.units, fmt, stream) : launch<64, 2>(a, t.units, fmt, stream); break;
        case 128: e = one ? launch<128, 1>(a, t.units, fmt, stream) : launch<128, 2>(a, t.units, fmt, stream); break;
        default: e = one ? launch<256, 1>(a, t.units, fmt, stream) : launch<256, 2>(a, t.units, fmt, stream);
    }
    if (e != hipSuccess || a.splits == 1) return e;
    return launch_attn_join(p, D, a.splits, a.part_o, a.part_ml, stream);
}

}  // namespace fp8k
