// Attention over the paged FP8 KV cache on gfx950, streaming form: the cache
// is read once and that is the time it takes.
//
// Rows.  The query rows of a sequence that share a KV head -- its new tokens
// times the `group` query heads of that KV head -- are the columns of one
// matrix, 16 to a tile, so a wave reads a key once for all of them.
//
// Mathematics, per column with query q, keys k_j, values v_j (codes times
// channel scales ks, vs):
//     s_j = scale * sum_c (q_c ks_c) code(k_j)_c        [cap, bias]
//     out_c = vs_c * sum_j p_j code(v_j)_c / sum_j p_j,  p_j = exp(s_j - max s)
// so the codes go into the matrix instruction as they are: every E4M3 and E5M2
// value is exact in fp16, the key scales move to the query and the value scales
// to the output.  q_c ks_c and p_j are rounded to fp16 (off by 2^-11 at most),
// scaled by a power of two first so that nothing underflows that matters (q per
// column to 2^15, p to 2^8): each an eighth of the rounding that bf16 outputs get
// at the end, together, in the outputs' mean square, about a quarter of it.  For
// fp16 and fp32 outputs and for lse, which is fp32 (two_terms), where it would
// show, each is fed as two fp16 terms, high part and rest (2^-22), at the cost of
// a second matrix instruction; a call that asks for lse has its output from two
// terms too.  Scores, references, sums and outputs are fp32; the sum of p is a
// product with ones, so numerator and denominator see the same p.
//
// One pass with a running reference m.  p is 2^8 at the largest score of the
// first tile, and m moves only when p would pass 2^12 (p stays below 2^13 in
// fp16, and the result does not depend on m beyond rounding), so most tiles
// need no other lane.  Scores are formed transposed, S^T = K Q^T, so that a
// lane's four results belong to one column: its reference and rescale need no
// lane but the three others of that column, and its p are, as they stand, the
// operand of O^T = V^T P^T.  The k index of that second product may be any
// order as long as both operands share it: slot (g, e) of a 32-key tile is key
// 16 (e / 4) + 4 g + e % 4, the keys whose scores the lane group g holds.  Its
// V operand wants, per lane, one channel of 8 keys: a lane reads D / 16
// channels of its 8 keys and turns bytes around in registers (v_perm_b32; for
// E5M2, a cut-off fp16, the same instruction decodes).
//
// The codes come through LDS: whole rows by DMA (16 bytes a lane, D / 16
// adjacent lanes a row), into a ring of two tiles per wave (four of 64 channels),
// each wave its own ring and its own waits.  Read straight into the operand's registers, a key's row
// is touched by lanes 16 apart: every lane is a request of its own, and with
// about 70 of them outstanding per CU the kernel stood at 4.4 TB/s whatever it
// computed (131072 tokens x 8 heads of 128: 72 us with the arithmetic taken out;
// by DMA with it 50 us, 5.3 TB/s, and 48 sequences of 4096 to 32768 tokens 281,
// 5.5 TB/s, where plain reads reach 6.1).
// In LDS the 16-byte units of row r sit at u ^ swizzle(r), so that neither the
// 16 rows of a K operand nor the row pieces of V meet in a bank.
//
// Split.  A workgroup's four waves are `hw` neighbouring KV heads (4, 2 or 1)
// times 4 / hw key interleaves; a round is a 32-key tile for each of them, and
// waves of one head are joined in LDS.  An item -- one sequence and column tile
// -- is a run of rounds.  Either a workgroup takes whole items, or the runs of
// all items, laid end to end, are cut into equal shares, whatever the lengths
// are: every workgroup adds up the rounds of all sequences (a scan) and finds
// its own share.  Workgroups of the same share and neighbouring heads are
// neighbours in the grid: together they read whole cache rows.  A share's first
// and last item may be part of one; those parts go to the workspace, and a second
// kernel joins them, in order, into the rows that were cut (4 to 8 us a call).  No
// wave waits for another workgroup.
#include <algorithm>
#include <type_traits>

#include "attn_common.hpp"
#include "attn_plan.hpp"

namespace fp8k {

namespace {

constexpr int kLogRound = 7;   // of kTile * kWaves
struct StreamArgs {
    PagedAttn p;
    int group;         // query heads per KV head
    int hw, log_hw;    // KV heads of a workgroup
    int head_groups;   // workgroups that share a sequence's rows
    int item0;         // whole items (sequence, head group): the first one of this launch
    int col_tiles;     // whole items: column tiles a KV head is planned for
    int shares;        // equal shares: their number for every head group, 0 for whole items
    int min_share;     // and their least cost
    float* part_o;     // [workgroups][2][hw][kCols][D]: parts of rows, a share's first and last
    float2* part_ml;   // [workgroups][2][hw][kCols]: reference (log2), sum
    int* starts;       // [B + 1]: cost before every sequence, cost of all
    int splits;        // the join of parts: parts of every row, laid out [rows][Hq][splits]
    int spread, log_spread;  // the join's thread groups per output row
    int join_rows;     // and the new rows of a sequence it takes at a time
    int join_batch;    // of the p.B sequences; 1 for parts, which go by row
    int join_unit0;    // the first workgroup's worth of rows of this launch
    FastDiv by_block, by_group, by_head_groups, by_heads, by_batch;

    __device__ __forceinline__ int page(int key) const { return by_block.of(key); }
    __device__ __forceinline__ int round_keys() const { return (kTile * kWaves) >> log_hw; }
    __device__ __forceinline__ int share_of(int total) const { return max((total + shares - 1) / shares, min_share); }
};

// Keys [lo, hi) that some column of tile ct sees.
__device__ __forceinline__ void tile_keys(const StreamArgs& a, const Seq& s, int prefix, int ct, int& lo, int& hi) {
    const int first = a.by_group.of(ct * kCols);
    const int last = a.by_group.of(min(s.nq * a.group - 1, ct * kCols + kCols - 1));
    int unused;
    visible(a.p, s, prefix, first, lo, unused);
    visible(a.p, s, prefix, last, unused, hi);
    hi = max(hi, 0);
    lo = min(lo, hi);
}

// The keys any row of a sequence sees start at `base`, whole tiles of them; its
// items' rounds, and its items (column tiles).
struct Run {
    int base, rounds, items;
};

__device__ __forceinline__ Run run_of(const StreamArgs& a, const Seq& s, int prefix) {
    int lo, hi, unused;
    visible(a.p, s, prefix, 0, lo, unused);
    visible(a.p, s, prefix, s.nq - 1, unused, hi);
    Run r;
    // without a window every sequence starts at key 0
    r.base = a.p.window > 0 ? min(lo, max(hi, 0)) / kTile * kTile : 0;
    r.rounds = s.nq > 0 && hi > r.base ? (hi - r.base + a.round_keys() - 1) >> (kLogRound - a.log_hw) : 0;
    r.items = r.rounds > 0 ? (s.nq * a.group + kCols - 1) / kCols : 0;
    return r;
}

// The sequence in which this workgroup's share starts, the cost before that
// sequence, and the cost of all: thread i scans sequence i, 256 at a time.
// Workgroup 0 leaves the starts for the join.
struct Found {
    int b, before, total;
};

__device__ __forceinline__ Found find_share(const StreamArgs& a, int* lds) {
    const PagedAttn& p = a.p;
    constexpr int kThreads = kWaves * kWave;
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    auto cost = [&](int b) {
        const Run r = run_of(a, sequence(p, b), p.prefix ? p.prefix[b] : 0);
        return (r.rounds + kItemCost) * r.items;
    };
    if (p.B == 1) {
        const int total = cost(0);
        if (blockIdx.x == 0 && tid == 0) a.starts[0] = 0, a.starts[1] = total;
        return Found{0, 0, total};
    }
    if (p.B <= kWave) {
        // every wave for itself
        const int mine = lane < p.B ? cost(lane) : 0, upto = wave_scan(mine);
        const int total = __builtin_amdgcn_readlane(upto, kWave - 1);
        const int64_t start = (int64_t)a.by_head_groups.of(blockIdx.x) * a.share_of(total);
        const uint64_t past = __ballot(upto > start);
        if (blockIdx.x == 0 && wave == 0) {
            if (lane < p.B) a.starts[lane] = upto - mine;
            if (lane == 0) a.starts[p.B] = total;
        }
        const int b = past ? __builtin_ctzll(past) : 0;
        return Found{b, __builtin_amdgcn_readlane(upto - mine, b), total};
    }
    int* const wave_sum = lds;       // [2][kWaves], by turns
    int* const found = lds + 2 * kWaves;
    int total = 0, before = 0, mine = 0, turn = 0;
    const bool once = p.B <= kThreads;
    for (int pass = 0; pass < 2; ++pass) {
        const int share = a.share_of(total);
        const int64_t start = (int64_t)(a.by_head_groups.of(blockIdx.x)) * share;  // of the second pass
        int run = 0;
        for (int b0 = 0; b0 < p.B; b0 += kThreads) {
            const int b = b0 + tid;
            if (pass == 0 || !once) {
                mine = b < p.B ? cost(b) : 0;
                const int sum = wave_scan(mine);
                int* const sums = wave_sum + turn * kWaves;
                turn ^= 1;
                if (lane == kWave - 1) sums[wave] = sum;
                __syncthreads();
                before = run + sum - mine;
#pragma unroll
                for (int w = 0; w < kWaves; ++w) {
                    if (w < wave) before += sums[w];
                    run += sums[w];
                }
            }
            if (pass == 1 && b < p.B) {
                if (start >= before && start < before + mine) found[0] = b, found[1] = before;
                if (blockIdx.x == 0) a.starts[b] = before;
            }
        }
        if (pass == 0) total = run;
    }
    if (blockIdx.x == 0 && tid == 0) a.starts[p.B] = total;
    __syncthreads();
    return Found{found[0], found[1], total};  // nothing is found past the end: the caller looks at total
}

template <int D>
__device__ __forceinline__ int swizzle(int row) {
    if constexpr (D == 64) return ((row >> 1) ^ (row >> 3)) & 3;
    if constexpr (D == 128) return (row ^ (row >> 3)) & 7;
    return row & 15;
}

__device__ __forceinline__ void compiler_fence() { asm volatile("" ::: "memory"); }

// 16 bytes per lane into LDS: lane i's land at lds + 16 i (lds is wave-uniform).
__device__ __forceinline__ void dma16(const uint8_t* src, uint8_t* lds) {
    __builtin_amdgcn_global_load_lds(src, lds, 16, 0, 0);
}

// LDS of a workgroup: every wave's ring of kStages tiles (K rows, then V rows),
// the rows' cache offsets and page numbers, and the waves' references and sums;
// the ring is free again when the waves' outputs are joined in it.
template <int D>
struct StreamLds {
    static constexpr int kStages = D == 64 ? 4 : 2;
    static constexpr int kRing = kStages * 2 * kTile * D;  // bytes of a wave
    static constexpr int kRows = kWaves * kRing;
    static constexpr int kPages = kRows + kWaves * kTile * 8;
    static constexpr int kMl = kPages + kWaves * kStages * kWave * 4;
    static constexpr int kBytes = kMl + kWaves * kCols * 8;
};

extern __shared__ __attribute__((aligned(1024))) uint8_t attn_smem[];

__device__ __forceinline__ uint32_t word(uint32_t v, int) { return v; }
__device__ __forceinline__ uint32_t word(const v2u& v, int i) { return v[i]; }
__device__ __forceinline__ uint32_t word(const v4u& v, int i) { return v[i]; }

// BIAS: the score cap and the distance bias are compiled in.  TERMS: fp16 terms
// of the scaled query and of p.
template <int D, int FMT, bool BIAS, int TERMS>
__global__ __launch_bounds__(kWaves* kWave, D == 256 ? 1 : 2) void attn_stream(StreamArgs a) {
    const PagedAttn& p = a.p;
    constexpr int NJ = D / 32;           // matrix instructions along the channels of K
    constexpr int VB = D / 16;           // V channels of a lane
    constexpr int UR = D / 16;           // 16-byte units of a row
    constexpr int RI = kWave / UR;       // rows of one DMA instruction
    constexpr int NI = kTile / RI;       // DMA instructions of a tile's K, and of its V
    using Lds = StreamLds<D>;
    using P = PScale<TERMS>;
    constexpr int S = Lds::kStages;
    constexpr int kTileBytes = 2 * kTile * D;
    constexpr int kOutRow = D + 4;       // floats of a joined row, padded off the banks
    static_assert(kCols * kOutRow * 4 <= Lds::kRing, "a wave's outputs fit its ring");

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
    uint8_t* const ring = attn_smem + wave * Lds::kRing;
    uint64_t* const rows = reinterpret_cast<uint64_t*>(attn_smem + Lds::kRows) + wave * kTile;
    int* const pages = reinterpret_cast<int*>(attn_smem + Lds::kPages) + wave * S * kWave;
    float2* const ml = reinterpret_cast<float2*>(attn_smem + Lds::kMl);
    const int n = lane % 16, g = lane / 16;
    const uint32_t C = 2u * p.Hkv * D;
    const int last_page = max(p.max_blocks - 1, 0);

    // the first item: a whole one, or where this workgroup's share starts
    int b = 0, ct = 0, hg = 0, at_item = 0;  // at_item: cost of the item before this share
    int left = 0;                            // cost left of the share
    if (a.shares > 0) {
        const Found f = find_share(a, reinterpret_cast<int*>(attn_smem));
        const int share = a.share_of(f.total), nth = a.by_head_groups.of(blockIdx.x);
        const int64_t start = (int64_t)nth * share;
        left = (int)min((int64_t)share, f.total - start);
        if (left <= 0) return;
        hg = blockIdx.x - nth * a.head_groups;
        b = __builtin_amdgcn_readfirstlane(f.b);
        const Run r = run_of(a, sequence(p, b), p.prefix ? p.prefix[b] : 0);
        const int at = (int)start - f.before;
        ct = __builtin_amdgcn_readfirstlane(at / (r.rounds + kItemCost));
        at_item = __builtin_amdgcn_readfirstlane(at - ct * (r.rounds + kItemCost));
        __syncthreads();
    } else {
        const int item = a.item0 + blockIdx.x;
        b = a.by_head_groups.of(item);
        hg = item - b * a.head_groups;
        ct = blockIdx.y;
    }

    while (b < p.B) {
        const Seq seq = sequence(p, b);
        const int prefix = p.prefix ? p.prefix[b] : 0;
        const Run run = run_of(a, seq, prefix);
        int r0 = 0, r1 = run.rounds;  // its rounds that are this workgroup's
        bool mine = true;
        if (a.shares == 0) {
            if (ct * kCols >= seq.nq * a.group) break;
        } else {
            if (run.items == 0 || ct * kCols >= seq.nq * a.group) {
                ct = 0, ++b;  // the next sequence
                continue;
            }
            const int taken = min(left, run.rounds + kItemCost - at_item);
            r0 = max(at_item - kItemCost, 0);
            r1 = max(at_item + taken - kItemCost, 0);
            mine = r1 > r0;  // else the share ends in the item's start, which the next one then pays for
            left -= taken;
            at_item = 0;
        }
        // where the result goes: the rows, or the share's first or last part
        const int part = r0 == 0 && r1 == run.rounds ? -1 : 2 * (int)blockIdx.x + (r0 == 0);
        const int hk0 = hg * a.hw, hk = hk0 + (wave & (a.hw - 1));
        const int32_t* table = p.block_table + (int64_t)b * p.ld_table;

        if (!mine) break;

        // this lane's column
        const int col = ct * kCols + n;
        const bool has_col = col < seq.nq * a.group;
        const int qi = has_col ? a.by_group.of(col) : 0;
        const int head = hk * a.group + (has_col ? col - qi * a.group : 0);
        const int64_t row = seq.row0 + qi;
        int lo, hi, tlo, thi;
        visible(p, seq, prefix, qi, lo, hi);
        if (!has_col) hi = 0;
        tile_keys(a, seq, prefix, ct, tlo, thi);

        const float slope = p.alibi ? p.alibi[head] * kLog2e : 0.0f;
        const int pos = seq.len - seq.nq + qi;
        const float cap_in = cap_factor(p.softcap);

        float m = kNoRef;
        v4f o[VB], l = {0.0f, 0.0f, 0.0f, 0.0f};  // the sum of p, four times over
#pragma unroll
        for (int j = 0; j < VB; ++j) o[j] = l;
        const v8h ones = {1, 1, 1, 1, 1, 1, 1, 1};

        // this wave's tiles: keys k0 + stride i and on, up to `end`
        const int stride = a.round_keys();
        const int k0 = run.base + r0 * stride + (wave >> a.log_hw) * kTile;
        const int end = (int)min((int64_t)thi, (int64_t)run.base + (int64_t)r1 * stride);

        // Page numbers of keys key0 + lane % 32, by DMA into LDS: as a load into a register the compiler would wait for
        // it, and with it for the row DMA issued after it.  The index does not wait for the sequence's length: it is
        // held inside the table, and rows_of drops what lies outside the visible keys of these rounds.
        auto fetch_pages = [&](int i) {
            __builtin_amdgcn_global_load_lds(table + min(a.page(k0 + i * stride + lane % kTile), last_page),
                                             pages + i % S * kWave, 4, 0, 0);
        };
        // byte offsets of the tile's cache rows into LDS, 0 for none; returns the mask of those that are there
        auto rows_of = [&](int i) {
            const int key = k0 + i * stride + lane % kTile, page = pages[i % S * kWave + lane];
            const bool ok = key >= tlo && key < end && page >= 0 && page < p.num_blocks;
            const uint32_t row = ok ? (page - a.page(key)) * p.block + key : 0;
            if (lane < kTile) rows[lane] = (uint64_t)row * C;
            __builtin_amdgcn_wave_barrier();  // read below by this wave's other lanes; a wave's LDS accesses are in order
            return (uint32_t)__ballot(ok);
        };
        const uint8_t* const kbase = p.cache + hk * D;
        auto fetch = [&](int i) {
            uint8_t* const tile = ring + i % S * kTileBytes;
            uint64_t row[NI];
#pragma unroll
            for (int j = 0; j < NI; ++j) row[j] = rows[RI * j + lane / UR];
#pragma unroll
            for (int j = 0; j < NI; ++j) {
                const int r = RI * j + lane / UR;
                const uint8_t* src = kbase + row[j] + ((lane % UR) ^ swizzle<D>(r)) * 16;
                dma16(src, tile + j * 1024);
                dma16(src + p.Hkv * D, tile + kTile * D + j * 1024);
            }
        };
        // The ring holds S tiles.  Step i issues the rows of tile i + S - 1, and before them the page numbers of tile
        // i + 2 S - 1: once tile i has landed, so have the page numbers that the next step needs, and one counter wait
        // that leaves S - 1 tiles in flight covers both.
        uint32_t masks[S];
        auto fill = [&]() {
#pragma unroll
            for (int i = 0; i < S - 1; ++i) {
                masks[i] = rows_of(i);
                compiler_fence();
                fetch_pages(i + S);
                fetch(i);
            }
        };
#pragma unroll
        for (int i = 0; i < S; ++i) fetch_pages(i);
        // the query and its scales, on their way while the pages are
        v4u raw[NJ][2];
        float4 ks[NJ][2];
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int e0 = 64 * (j / 2) + 16 * g + 8 * (j % 2);
            load_q8<TERMS>(p, row * p.ldq + (int64_t)head * D + e0, raw[j]);
#pragma unroll
            for (int i = 0; i < 2; ++i) ks[j][i] = *reinterpret_cast<const float4*>(p.scales + hk * D + e0 + 4 * i);
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        fill();

        // meanwhile: q times the key scales, in fp16 terms
        v8h qt[TERMS][NJ];
        float c;  // score (log2 units, or natural ones under a cap) per unit of the product
        {
            float x[NJ][8], top = 0.0f;
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                unpack_q8<TERMS>(p, raw[j], x[j]);
                const float s[8] = {ks[j][0].x, ks[j][0].y, ks[j][0].z, ks[j][0].w,
                                    ks[j][1].x, ks[j][1].y, ks[j][1].z, ks[j][1].w};
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[j][e] *= fmaxf(s[e], kScaleFloor);
                    top = fmaxf(top, fabsf(x[j][e]));
                }
            }
            top = max_over_groups(top);
            const int shift = 15 - __builtin_amdgcn_frexp_expf(top);
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float y = __builtin_amdgcn_ldexpf(x[j][e], shift);
                    qt[0][j][e] = (_Float16)y;
                    if constexpr (TERMS == 2) qt[1][j][e] = (_Float16)(y - (float)qt[0][j][e]);
                }
            c = __builtin_amdgcn_ldexpf(p.scale, -shift);
        }
        if (p.softcap > 0.0f) c *= kLn2;  // the cap takes the natural score

        auto step = [&](const uint8_t* tile, int key0, uint32_t mask) {
            // Both reads are typed vector loads: read as bytes they might alias the DMA's writes, and the compiler
            // would wait for the next tile's here.
            v4u kw[2][D / 64];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < D / 64; ++i) {
                    const int r = 16 * t + n;
                    kw[t][i] = *reinterpret_cast<const v4u*>(tile + r * D + ((4 * i + g) ^ swizzle<D>(r)) * 16);
                }
            typedef typename std::conditional<D == 64, uint32_t, typename std::conditional<D == 128, v2u, v4u>::type>::type vrow;
            vrow v[8];  // the V codes of this lane's 8 keys, channels n * VB ..
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int r = 16 * (e / 4) + 4 * g + e % 4;
                v[e] = *reinterpret_cast<const vrow*>(tile + kTile * D + r * D + ((n * VB / 16) ^ swizzle<D>(r)) * 16 +
                                                      n * VB % 16);
            }
            v4f s[2];  // products; under BIAS scores
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                v4f acc = {0.0f, 0.0f, 0.0f, 0.0f}, rest = acc;
#pragma unroll
                for (int i = 0; i < D / 64; ++i) {
                    const v4u w = kw[t][i];
#pragma unroll
                    for (int j = 2 * i; j < 2 * i + 2; ++j) {
                        const v8h k = row_f16<FMT>(w[2 * (j % 2)], w[2 * (j % 2) + 1]);
                        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, qt[0][j], acc, 0, 0, 0);
                        if constexpr (TERMS == 2) rest = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, qt[1][j], rest, 0, 0, 0);
                    }
                }
                s[t] = TERMS == 2 ? acc + rest : acc;
            }
            if constexpr (BIAS) {
                auto capped = [&](auto series) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        s[j / 4][j % 4] = kLog2e * soft_cap<decltype(series)::value>(s[j / 4][j % 4] * c, p.softcap, cap_in);
                };
                if (p.softcap > 0.0f) {
                    if (cap_by_series<TERMS>(p.softcap)) capped(std::true_type());
                    else capped(std::false_type());
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) s[j / 4][j % 4] *= c;
                }
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[t][i] += slope * (float)(key0 + 16 * t + 4 * g + i - pos);
            }
            const bool whole = mask == 0xFFFFFFFFu && !__any(key0 < lo || key0 + kTile > hi);
            float x[8];  // scores above the reference
            auto above = [&]() {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    x[e] = BIAS ? s[e / 4][e % 4] - m : __builtin_fmaf(s[e / 4][e % 4], c, -m);
            };
            auto hide = [&]() {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int j = 16 * (e / 4) + 4 * g + e % 4;
                    const bool there = (mask >> j) & 1u;
                    x[e] = (there & (key0 + j >= lo) & (key0 + j < hi)) ? x[e] : -INFINITY;
                    // a code behind the sequence may be anything, NaN too: 0 * NaN must not reach the sum
                    v[e] &= there ? ~0u : 0u;
                }
            };
            above();
            if (!whole) hide();
            float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
            if (__any(top > P::kLimit)) {
                // move the references of the columns that need it to the largest score, less the shift; scores past 2^24
                // are themselves too coarse for the shift, and one of them takes all the weight
                const float old = m;
                m = 0.0f;
                above();
                if (!whole) hide();
                top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
                top = max_over_groups(top);
                m = top > old + P::kLimit ? (fabsf(top) < 16777216.0f ? top - P::kShift : top) : old;
                const float f = __builtin_amdgcn_exp2f(old - m);
                l *= f;
#pragma unroll
                for (int j = 0; j < VB; ++j) o[j] *= f;
                above();
                if (!whole) hide();
            }
            v8h ph, pl;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float y = P::p(x[e]);
                ph[e] = (_Float16)y;
                if constexpr (TERMS == 2) pl[e] = (_Float16)(y - (float)ph[e]);
            }
            l = __builtin_amdgcn_mfma_f32_16x16x32_f16(ones, ph, l, 0, 0, 0);
            if constexpr (TERMS == 2) l = __builtin_amdgcn_mfma_f32_16x16x32_f16(ones, pl, l, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < VB; ++j) {
                v4u r;
#pragma unroll
                for (int i = 0; i < 4; ++i) r[i] = pair_f16<FMT>(word(v[2 * i], j / 4), word(v[2 * i + 1], j / 4), j % 4);
                const v8h vt = __builtin_bit_cast(v8h, r);
                o[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vt, ph, o[j], 0, 0, 0);
                if constexpr (TERMS == 2) o[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vt, pl, o[j], 0, 0, 0);
            }
        };

        for (int i = 0; k0 + i * stride < end; ++i) {
            masks[S - 1] = rows_of(i + S - 1);
            compiler_fence();
            fetch_pages(i + 2 * S - 1);
            fetch(i + S - 1);  // past the last tile: row 0, unused
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"((S - 1) * (2 * NI + 1)) : "memory");
            step(ring + i % S * kTileBytes, k0 + i * stride, masks[0]);
            compiler_fence();
#pragma unroll
            for (int j = 0; j < S - 1; ++j) masks[j] = masks[j + 1];
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // nothing lands in the ring any more
        if (a.hw == kWaves) {
            // a wave has its head to itself: results go from its registers
            if (has_col) {
                const int64_t at = part >= 0 ? ((int64_t)part * a.hw + wave) * kCols + n : 0;
                if (part >= 0 && g == 0) a.part_ml[at] = make_float2(m, l[0]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < VB; j += 4) {
                        const int d = (4 * g + i) * VB + j;
                        const float4 r = make_float4(o[j][i], o[j + 1][i], o[j + 2][i], o[j + 3][i]);
                        if (part >= 0)
                            *reinterpret_cast<float4*>(a.part_o + at * D + d) = r;
                        else
                            write_row(p, row, head, hk, D, d, m, l[0], r);
                    }
            }
            if (a.shares == 0) {
                ct += a.col_tiles;
            } else {
                if (left <= 0) break;
                ++ct;
            }
            continue;
        }

        // the waves of a head joined in wave order
        if (g == 0) ml[wave * kCols + n] = make_float2(m, l[0]);
        float* const outs = reinterpret_cast<float*>(ring);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < VB; j += 4)
                *reinterpret_cast<float4*>(outs + n * kOutRow + (4 * g + i) * VB + j) =
                    make_float4(o[j][i], o[j + 1][i], o[j + 2][i], o[j + 3][i]);
        __syncthreads();
        for (int x = threadIdx.x; x < a.hw * kCols * D / 4; x += kWaves * kWave) {
            const int d = x % (D / 4) * 4, cc = x / (D / 4) % kCols, hs = x / (D / 4 * kCols);
            const int ccol = ct * kCols + cc;
            if (ccol >= seq.nq * a.group) continue;
            float M = kNoRef, L = 0.0f;
            for (int w = hs; w < kWaves; w += a.hw) M = fmaxf(M, ml[w * kCols + cc].x);
            float4 r = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int w = hs; w < kWaves; w += a.hw) {
                const float2 y = ml[w * kCols + cc];
                const float f = __builtin_amdgcn_exp2f(y.x - M);
                const float4 v = *reinterpret_cast<const float4*>(attn_smem + w * Lds::kRing + (cc * kOutRow + d) * 4);
                L += f * y.y;
                r = make_float4(r.x + f * v.x, r.y + f * v.y, r.z + f * v.z, r.w + f * v.w);
            }
            const int i = a.by_group.of(ccol), h = (hk0 + hs) * a.group + ccol - i * a.group;
            const int64_t orow = seq.row0 + i;
            if (part >= 0) {
                const int64_t at = ((int64_t)part * a.hw + hs) * kCols + cc;
                if (d == 0) a.part_ml[at] = make_float2(M, L);
                *reinterpret_cast<float4*>(a.part_o + at * D + d) = r;
            } else {
                write_row(p, orow, h, hk0 + hs, D, d, M, L, r);
            }
        }
        __syncthreads();

        // the next item
        if (a.shares == 0) {
            ct += a.col_tiles;
        } else {
            if (left <= 0) break;
            ++ct;
        }
    }
}

// Joins the key shares of the output rows.  A group of D / 4 threads adds up a
// row's weighted shares, four channels a thread, every `spread`-th of them when
// several groups of the workgroup take one row; LDS joins those in order.
// PARTS: of all rows, each in `splits` parts; else of those that equal shares cut.
template <int D, bool PARTS>
__global__ __launch_bounds__(kWaves* kWave) void attn_join(StreamArgs a) {
    const PagedAttn& p = a.p;
    constexpr int kThreads = kWaves * kWave;
    constexpr int kLanes = D / 4;                // threads of a group
    constexpr int kGroups = kThreads / kLanes;
    constexpr int kBatch = 8;
    __shared__ float4 sums[kThreads];
    __shared__ float2 group_ml[kGroups];
    const int tid = threadIdx.x, d4 = tid % kLanes, grp = tid / kLanes, part = grp & (a.spread - 1);
    const int nth = (a.join_unit0 + blockIdx.x) * (kGroups >> a.log_spread) + (grp >> a.log_spread);  // row of the launch: (i0, b, h)
    const int rest = a.by_heads.of(nth), i0 = a.by_batch.of(rest);
    const int h = nth - rest * p.Hq, b = rest - i0 * a.join_batch;
    const int hk = a.by_group.of(h);
    Seq seq = {0, p.rows, 0};
    int prefix = 0, first_row = 0, start = 0, share = 1;
    if constexpr (PARTS) {
        // the rows of all sequences, without regard to whose they are
        if (p.cu_q) first_row = p.cu_q[0], seq.nq = min(p.cu_q[p.B], p.rows);
    } else {
        // looked up together and before the barrier: one trip to memory
        start = a.starts[b];
        share = a.starts[p.B];
        seq = sequence(p, b);
        prefix = p.prefix ? p.prefix[b] : 0;
        share = a.share_of(share);
    }
    if (i0 >= a.join_rows) seq.nq = 0;
    // Every thread goes through as many rounds as the longest sequence of its workgroup: the barriers are for all.
    for (int i = i0; __syncthreads_or(i < seq.nq); i += a.join_rows) {
        float M = kNoRef, L = 0.0f;
        float4 r = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        int shares = 0;
        bool cut = false;  // else the first kernel has written the row
        if (i >= first_row && i < seq.nq) {
            const int col = i * a.group + h - hk * a.group;
            int first = 0;
            shares = a.splits;
            if constexpr (!PARTS) {
                // the shares that its item was cut into, as the first kernel dealt them out
                const Run run = run_of(a, seq, prefix);
                const int at = start + col / kCols * (run.rounds + kItemCost) + kItemCost;
                first = at / share;
                shares = run.rounds == 0 ? 0 : (at + run.rounds - 1) / share - first + 1;
            }
            cut = shares != 1;
            if (cut) {
                // the item's first round is in its first share; kBatch shares at a time, so that their loads travel together
                for (int s0 = part; s0 < shares; s0 += kBatch * a.spread) {
                    float2 y[kBatch];
                    float4 v[kBatch];
                    float top = M;
#pragma unroll
                    for (int k = 0; k < kBatch; ++k) {
                        const int s = min(s0 + k * a.spread, shares - 1);
                        const int group = (first + s) * a.head_groups + (hk >> a.log_hw);
                        const int64_t x = PARTS ? ((int64_t)i * p.Hq + h) * a.splits + s
                                                : ((2 * group + (s == 0)) * a.hw + (hk & (a.hw - 1))) * kCols + col % kCols;
                        y[k] = a.part_ml[x];
                        v[k] = *reinterpret_cast<const float4*>(a.part_o + x * D + 4 * d4);
                        if (s0 + k * a.spread >= shares) y[k].x = kNoRef;
                        top = fmaxf(top, y[k].x);
                    }
                    const float g = __builtin_amdgcn_exp2f(M - top);
                    M = top;
                    L *= g;
                    r = make_float4(r.x * g, r.y * g, r.z * g, r.w * g);
#pragma unroll
                    for (int k = 0; k < kBatch; ++k) {
                        // by a weight of zero: a branch would sink the loads into it, one after the other
                        const float f = s0 + k * a.spread < shares ? __builtin_amdgcn_exp2f(y[k].x - M) : 0.0f;
                        L += f * y[k].y;
                        r = make_float4(r.x + f * v[k].x, r.y + f * v[k].y, r.z + f * v[k].z, r.w + f * v[k].w);
                    }
                }
            }
        }
        if (a.spread > 1) {
            sums[tid] = r;
            if (d4 == 0) group_ml[grp] = make_float2(M, L);
            __syncthreads();
            if (part == 0) {
                for (int k = 1; k < a.spread; ++k) {
                    const float4 v = sums[tid + k * kLanes];
                    const float2 y = group_ml[grp + k];
                    const float top = fmaxf(M, y.x), f = __builtin_amdgcn_exp2f(M - top), g = __builtin_amdgcn_exp2f(y.x - top);
                    M = top;
                    L = L * f + y.y * g;
                    r = make_float4(r.x * f + v.x * g, r.y * f + v.y * g, r.z * f + v.z * g, r.w * f + v.w * g);
                }
            }
        }
        if (part == 0 && cut) write_row(p, seq.row0 + i, h, hk, D, 4 * d4, M, L, r);
    }
}

template <int D, int FMT, bool BIAS, int TERMS>
hipError_t launch_stream(StreamArgs a, const StreamPlan& s, hipStream_t stream) {
    constexpr int lds = StreamLds<D>::kBytes;
    if constexpr (lds > 64 * 1024) {
        const hipError_t e = FP8K_SET_LDS((attn_stream<D, FMT, BIAS, TERMS>), lds);
        if (e != hipSuccess) return e;
    }
    return in_launches(s.units, [&](int64_t first, int64_t n) {
        a.item0 = (int)first;
        hipLaunchKernelGGL((attn_stream<D, FMT, BIAS, TERMS>), dim3((unsigned)n, (unsigned)s.rows_y), dim3(kWaves * kWave),
                           lds, stream, a);
        return hipGetLastError();
    });
}

template <int D, bool PARTS>
hipError_t launch_join(StreamArgs a, int64_t max_q, int64_t typical, hipStream_t stream) {
    const JoinPlan j = join_plan((int64_t)a.join_batch * a.p.Hq, D, max_q, typical);
    a.join_rows = (int)j.rows;
    a.spread = j.spread, a.log_spread = j.log_spread;
    a.by_batch = FastDiv(a.join_batch);
    return in_launches(j.units, [&](int64_t first, int64_t n) {
        a.join_unit0 = (int)first;
        hipLaunchKernelGGL((attn_join<D, PARTS>), dim3((unsigned)n), dim3(kWaves * kWave), 0, stream, a);
        return hipGetLastError();
    });
}

template <int D>
hipError_t launch(const StreamArgs& a, const StreamPlan& s, int fmt, int64_t max_q, int64_t typical, hipStream_t stream) {
    const bool bias = a.p.softcap > 0.0f || a.p.alibi != nullptr, one = !two_terms(a.p);
    hipError_t e;
    if (fmt == kKvE5M2)
        e = bias ? (one ? launch_stream<D, kKvE5M2, true, 1>(a, s, stream) : launch_stream<D, kKvE5M2, true, 2>(a, s, stream))
                 : (one ? launch_stream<D, kKvE5M2, false, 1>(a, s, stream) : launch_stream<D, kKvE5M2, false, 2>(a, s, stream));
    else
        e = bias ? (one ? launch_stream<D, kKvE4M3, true, 1>(a, s, stream) : launch_stream<D, kKvE4M3, true, 2>(a, s, stream))
                 : (one ? launch_stream<D, kKvE4M3, false, 1>(a, s, stream) : launch_stream<D, kKvE4M3, false, 2>(a, s, stream));
    if (e != hipSuccess || a.shares == 0) return e;
    return launch_join<D, false>(a, max_q, typical, stream);
}

}  // namespace

size_t attn_paged_ws_bytes(int64_t B, int64_t rows, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_q, int64_t max_len,
                           int64_t all_len) {
    const StreamPlan s = stream_plan(B, rows, Hq, Hkv, D, max_q, max_len, all_len);
    if (B == 0 || rows == 0 || s.shares == 0) return 0;
    return (size_t)s.shares * Hkv * 2 * kCols * ((size_t)D * 4 + 8) + ((size_t)B + 1) * 4;
}

hipError_t launch_attn_join(const PagedAttn& p, int D, int splits, float* part_o, float2* part_ml, hipStream_t stream) {
    StreamArgs a = {};
    a.p = p;
    a.group = p.Hq / p.Hkv;
    a.splits = splits;
    a.part_o = part_o;
    a.part_ml = part_ml;
    a.join_batch = 1;
    a.by_group = FastDiv(a.group);
    a.by_heads = FastDiv(p.Hq);
    switch (D) {
        case 64: return launch_join<64, true>(a, p.rows, p.rows, stream);
        case 128: return launch_join<128, true>(a, p.rows, p.rows, stream);
        default: return launch_join<256, true>(a, p.rows, p.rows, stream);
    }
}

hipError_t launch_attn_paged(const PagedAttn& p, int D, int fmt, int64_t max_q, int64_t typical, int64_t max_len, void* ws,
                             hipStream_t stream) {
    const StreamPlan s = stream_plan(p.B, p.rows, p.Hq, p.Hkv, D, max_q, max_len, (int64_t)p.max_blocks * p.block);
    StreamArgs a = {};
    a.p = p;
    a.group = p.Hq / p.Hkv;
    a.hw = s.hw;
    a.col_tiles = (int)s.col_tiles;
    a.shares = s.shares;
    a.min_share = s.min_share;
    if (s.shares > 0) {
        const size_t cols = (size_t)s.shares * p.Hkv * 2 * kCols;
        a.part_o = static_cast<float*>(ws);
        a.part_ml = reinterpret_cast<float2*>(a.part_o + cols * D);
        a.starts = reinterpret_cast<int*>(a.part_ml + cols);
    }
    a.log_hw = s.hw == 4 ? 2 : s.hw == 2 ? 1 : 0;
    a.head_groups = p.Hkv / s.hw;
    a.by_block = FastDiv(p.block);
    a.by_group = FastDiv(a.group);
    a.by_heads = FastDiv(p.Hq);
    a.join_batch = p.B;
    a.by_head_groups = FastDiv(a.head_groups);
    switch (D) {
        case 64: return launch<64>(a, s, fmt, max_q, typical, stream);
        case 128: return launch<128>(a, s, fmt, max_q, typical, stream);
        default: return launch<256>(a, s, fmt, max_q, typical, stream);
    }
}

}  // namespace fp8k
