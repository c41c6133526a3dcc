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
// to the output.  q_c ks_c and p_j are not exact in fp16; each is fed as two
// fp16 terms, high part and rest (22 bits), scaled by a power of two first so
// that neither part underflows where it matters (q per column to 2^15, p to
// 2^14).  The second term costs a second matrix instruction, which is free
// here: a CU needs about 12 bytes of codes a cycle to keep up with HBM and the
// matrix cores take 64 with both terms.  Scores, maxima, sums and outputs are
// fp32.
//
// One pass with running maximum and sum.  Scores are formed transposed,
// S^T = K Q^T, so that a lane's four results belong to one column: its maximum,
// sum and rescale need no lane but the three others of that column, and its p
// are, as they stand, the operand of O^T = V^T P^T.  The k index of that second
// product may be any order as long as both operands share it: slot (g, e) of a
// 32-key tile is key 16 (e / 4) + 4 g + e % 4, the keys whose scores the lane
// group g holds.  Its V operand wants, per lane, one channel of 8 keys: a lane
// loads D / 16 channels of its 8 keys and turns bytes around in registers
// (v_perm_b32; for E5M2, a cut-off fp16, the same instruction decodes).
//
// Split.  A workgroup is one KV head of one sequence and a share of its keys;
// its four waves take 32-key tiles in turn and are joined in LDS.  Shares
// beyond one per sequence go to the workspace and a second kernel joins them in
// a fixed order.  No wave waits for another workgroup.
#include <algorithm>

#include "kv_common.hpp"

namespace fp8k {

namespace {

typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));

constexpr int kTile = 32;      // keys per step of a wave
constexpr int kWaves = 4;      // waves of a workgroup
constexpr int kCols = 16;      // query columns of a tile
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kPShift = 14.0f;  // p is held as p * 2^14

struct StreamArgs {
    PagedAttn p;
    int group;         // query heads per KV head
    int col_tiles;     // column tiles a KV head is planned for
    int splits;        // key shares per (sequence, column tile)
    int chunk;         // keys of a share per round, a multiple of kTile * kWaves
    float* part_o;     // [splits][rows][Hq][D]
    float2* part_ml;   // [splits][rows][Hq]: running maximum (log2), sum
};

// A sequence's new rows and length, held inside the buffers whatever the
// device arrays say.
struct Seq {
    int row0, nq, len;
};

__device__ __forceinline__ Seq sequence(const PagedAttn& p, int b) {
    Seq s;
    if (p.cu_q == nullptr) {
        s.row0 = b;
        s.nq = 1;
    } else {
        const int64_t lo = max(p.cu_q[b], 0);
        const int64_t hi = min(p.cu_q[b + 1], p.rows);
        s.row0 = (int)min(lo, (int64_t)p.rows);
        s.nq = (int)max(hi - lo, (int64_t)0);
    }
    s.len = min(max(p.seq_lens[b], 0), p.max_blocks * p.block);
    return s;
}

// Keys [lo, hi) that new token i of a sequence sees.
__device__ __forceinline__ void visible(const PagedAttn& p, const Seq& s, int prefix, int i, int& lo, int& hi) {
    const int pos = s.len - s.nq + i;
    hi = p.causal ? min(s.len, max(pos + 1, prefix)) : s.len;
    lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
}

// Keys [lo, hi) that some column of tile ct sees.
__device__ __forceinline__ void tile_keys(const PagedAttn& p, const Seq& s, int prefix, int group, int ct, int& lo,
                                          int& hi) {
    const int first = ct * kCols / group;
    const int last = min(s.nq * group - 1, ct * kCols + kCols - 1) / group;
    int unused;
    visible(p, s, prefix, first, lo, unused);
    visible(p, s, prefix, last, unused, hi);
    lo = min(lo, hi);
}

// Two codes (bytes j of even and odd) -> packed fp16, exact.
template <int FMT>
__device__ __forceinline__ uint32_t pair_f16(uint32_t even, uint32_t odd, uint32_t j) {
    if constexpr (FMT == kKvE5M2) {
        return __builtin_amdgcn_perm(odd, even, 0x040C000Cu + 0x01000100u * j);
    } else {
        const uint32_t w = __builtin_amdgcn_perm(odd, even, 0x0C0C0400u + 0x00000101u * j);
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false));
    }
}

// Eight codes in a row -> 8 fp16, exact.
template <int FMT>
__device__ __forceinline__ v8h row_f16(uint32_t lo, uint32_t hi) {
    v4u r;
    if constexpr (FMT == kKvE5M2) {
        r = v4u{__builtin_amdgcn_perm(lo, lo, 0x010C000Cu), __builtin_amdgcn_perm(lo, lo, 0x030C020Cu),
                __builtin_amdgcn_perm(hi, hi, 0x010C000Cu), __builtin_amdgcn_perm(hi, hi, 0x030C020Cu)};
    } else {
        r = v4u{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true))};
    }
    return __builtin_bit_cast(v8h, r);
}

// 8 consecutive elements of a query row as fp32.
__device__ __forceinline__ void load_q8(const PagedAttn& p, int64_t e, float (&x)[8]) {
    if (p.dtype == kKvF32) {
        const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + e);
        const float4 a = f[0], b = f[1];
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    } else {
        const v4u w = *reinterpret_cast<const v4u*>(static_cast<const uint16_t*>(p.q) + e);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (p.dtype == kKvBF16) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            } else {
                x[2 * i] = half_to_float(w[i] & 0xFFFFu);
                x[2 * i + 1] = half_to_float(w[i] >> 16);
            }
        }
    }
}

// 4 fp32 values to consecutive elements of an output row, rounded once (RNE).
__device__ __forceinline__ void store_o4(const PagedAttn& p, int64_t e, const float4& x) {
    if (p.dtype == kKvF32) {
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + e) = x;
    } else {
        const v2u w = p.dtype == kKvBF16 ? v2u{round_bf16x2(x.x, x.y), round_bf16x2(x.z, x.w)}
                                         : v2u{round_f16x2(x.x, x.y), round_f16x2(x.z, x.w)};
        *reinterpret_cast<v2u*>(static_cast<uint16_t*>(p.out) + e) = w;
    }
}

__device__ __forceinline__ float max_over_groups(float v) {
    v = fmaxf(v, __shfl_xor(v, 16, kWave));
    return fmaxf(v, __shfl_xor(v, 32, kWave));
}

__device__ __forceinline__ float sum_over_groups(float v) {
    v += __shfl_xor(v, 16, kWave);
    return v + __shfl_xor(v, 32, kWave);
}

// cap * tanh(x / cap) in fp32: 1 - 2 / (exp(2 x / cap) + 1), whose absolute
// error is that of a few roundings at the cap's magnitude.
__device__ __forceinline__ float soft_cap(float x, float cap, float two_log2e_over_cap) {
    const float e = __builtin_amdgcn_exp2f(x * two_log2e_over_cap);
    return cap * (1.0f - 2.0f * __builtin_amdgcn_rcpf(e + 1.0f));
}

// Four channels of an output row from its sum r of p_j code(v_j), maximum M
// and sum L of p_j; an empty row (L == 0) is zeros, its log-sum-exp -inf.
__device__ __forceinline__ void write_row(const PagedAttn& p, int64_t row, int h, int group, int D, int d, float M,
                                          float L, const float4& r) {
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    const float4 sc = *reinterpret_cast<const float4*>(p.scales + (int64_t)(p.Hkv + h / group) * D + d);
    store_o4(p, row * p.ldo + (int64_t)h * D + d,
             make_float4(r.x * inv * fmaxf(sc.x, kScaleFloor), r.y * inv * fmaxf(sc.y, kScaleFloor),
                         r.z * inv * fmaxf(sc.z, kScaleFloor), r.w * inv * fmaxf(sc.w, kScaleFloor)));
    if (p.lse && d == 0) p.lse[row * p.Hq + h] = L == 0.0f ? -INFINITY : kLn2 * (M - kPShift + __builtin_amdgcn_logf(L));
}

// Codes of one 32-key tile as a wave holds them.
template <int D>
struct Codes {
    v4u k[2][D / 64];   // K: keys 16 t + lane % 16, channels 64 i + 16 g ..
    uint32_t v[8][D / 64];  // V: keys of slot (g, e), channels lane % 16 * D / 16 ..
};

template <int D, int FMT>
__global__ __launch_bounds__(kWaves* kWave, D == 256 ? 1 : 2) void attn_stream(StreamArgs a) {
    const PagedAttn& p = a.p;
    constexpr int kParts = D == 256 ? 2 : 1;  // rounds of the waves' join (34 KB of LDS)
    constexpr int kI = 4 / kParts;
    constexpr int NJ = D / 32;  // matrix instructions along the channels of K
    constexpr int VB = D / 16;  // V channels of a lane
    __shared__ int slots_lds[kWaves][kTile];
    __shared__ float2 ml_lds[kWaves][kCols];
    __shared__ float o_lds[kWaves][kCols][D / kParts + 4];

    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    const int n = lane % 16, g = lane / 16;
    int id = blockIdx.x;
    const int hk = id % p.Hkv;
    id /= p.Hkv;
    const int ct0 = id % a.col_tiles;
    id /= a.col_tiles;
    const int split = id % a.splits;
    const int b = id / a.splits;
    const Seq seq = sequence(p, b);
    const int prefix = p.prefix ? p.prefix[b] : 0;
    const int64_t C = 2 * (int64_t)p.Hkv * D;
    const int32_t* table = p.block_table + (int64_t)b * p.ld_table;

    for (int ct = ct0; ct * kCols < seq.nq * a.group; ct += a.col_tiles) {
        // this lane's column
        const int col = ct * kCols + n;
        const bool has_col = col < seq.nq * a.group;
        const int qi = has_col ? col / a.group : 0;
        const int head = hk * a.group + (has_col ? col - qi * a.group : 0);
        const int64_t row = seq.row0 + qi;
        int lo, hi, tlo, thi;
        visible(p, seq, prefix, qi, lo, hi);
        if (!has_col) hi = 0;
        tile_keys(p, seq, prefix, a.group, ct, tlo, thi);
        const int base = tlo / kTile * kTile;
        const int chunk_tiles = a.chunk / (kTile * kWaves);  // tiles a wave takes of one chunk

        // q times the key scales, as two fp16 terms
        v8h qh[NJ], ql[NJ];
        float c;  // score (log2 units, or natural ones under a cap) per unit of the product
        {
            float x[NJ][8], top = 0.0f;
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const int e0 = 64 * (j / 2) + 16 * g + 8 * (j % 2);
                load_q8(p, row * p.ldq + (int64_t)head * D + e0, x[j]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[j][e] *= fmaxf(p.scales[hk * D + e0 + e], kScaleFloor);
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
                    qh[j][e] = (_Float16)y;
                    ql[j][e] = (_Float16)(y - (float)qh[j][e]);
                }
            c = __builtin_amdgcn_ldexpf(p.scale, -shift);
        }
        const float slope = p.alibi ? p.alibi[head] * kLog2e : 0.0f;
        const int pos = seq.len - seq.nq + qi;
        const float cap_in = p.softcap > 0.0f ? 2.0f * kLog2e / p.softcap : 0.0f;
        if (p.softcap > 0.0f) c *= kLn2;  // the cap takes the natural score

        float m = -INFINITY, l = 0.0f;
        v4f o[VB];
#pragma unroll
        for (int j = 0; j < VB; ++j) o[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

        // this wave's tiles: number i of it is tile chunk_tiles * kWaves * c + kWaves * (i % chunk_tiles) + wave of
        // chunk c = split + splits * (i / chunk_tiles)
        int in_chunk = 0, first = base + (split * chunk_tiles * kWaves + wave) * kTile;
        const int64_t next_chunk = (int64_t)a.splits * chunk_tiles * kWaves * kTile - (int64_t)chunk_tiles * kWaves * kTile;
        auto advance = [&](int key) {
            int64_t k = (int64_t)key + kWaves * kTile;
            if (++in_chunk == chunk_tiles) {
                in_chunk = 0;
                k += next_chunk;
            }
            return (int)min(k, (int64_t)0x7FFFFF00);
        };
        // page of key key0 + lane % 32, -1 outside the visible keys
        auto page_of = [&](int key0) {
            const int key = key0 + lane % kTile;
            return key >= tlo && key < thi ? table[key / p.block] : -1;
        };
        // cache rows of the tile's keys into LDS, -1 for none; returns their mask
        auto rows_of = [&](int key0, int page) {
            const int key = key0 + lane % kTile;
            const bool ok = page >= 0 && page < p.num_blocks;
            const int r = ok ? page * p.block + key % p.block : -1;
            if (lane < kTile) slots_lds[wave][lane] = r;
            __builtin_amdgcn_wave_barrier();  // read below by this wave's other lanes; a wave's LDS accesses are in order
            return (uint32_t)__ballot(ok);
        };
        auto fetch = [&](Codes<D>& w) {
            const uint8_t* kbase = p.cache + hk * D + 16 * g;
            const uint8_t* vbase = p.cache + (int64_t)(p.Hkv + hk) * D + n * VB;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int64_t at = (int64_t)max(slots_lds[wave][16 * t + n], 0) * C;
#pragma unroll
                for (int i = 0; i < D / 64; ++i) w.k[t][i] = *reinterpret_cast<const v4u*>(kbase + at + 64 * i);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int64_t at = (int64_t)max(slots_lds[wave][16 * (e / 4) + 4 * g + e % 4], 0) * C;
                __builtin_memcpy(w.v[e], __builtin_assume_aligned(vbase + at, VB), VB);
            }
        };
        auto step = [&](Codes<D>& w, int key0, uint32_t mask) {
            float s[2][4];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    const v8h k = row_f16<FMT>(w.k[t][j / 2][2 * (j % 2)], w.k[t][j / 2][2 * (j % 2) + 1]);
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, qh[j], acc, 0, 0, 0);
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, ql[j], acc, 0, 0, 0);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) s[t][i] = acc[i] * c;
            }
            if (p.softcap > 0.0f) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[t][i] = kLog2e * soft_cap(s[t][i], p.softcap, cap_in);
            }
            if (p.alibi) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[t][i] += slope * (float)(key0 + 16 * t + 4 * g + i - pos);
            }
            const bool whole = mask == 0xFFFFFFFFu && !__any(key0 < lo || key0 + kTile > hi);
            if (!whole) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int j = 16 * t + 4 * g + i;
                        const bool see = ((mask >> j) & 1u) && key0 + j >= lo && key0 + j < hi;
                        s[t][i] = see ? s[t][i] : -INFINITY;
                        // a code behind the sequence may be anything, NaN too: 0 * NaN must not reach the sum
                        if (!((mask >> j) & 1u)) {
#pragma unroll
                            for (int q = 0; q < D / 64; ++q) w.v[4 * t + i][q] = 0u;
                        }
                    }
            }
            float top = fmaxf(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3])),
                              fmaxf(fmaxf(s[1][0], s[1][1]), fmaxf(s[1][2], s[1][3])));
            top = max_over_groups(top);
            if (__any(top > m)) {
                const float up = fmaxf(top, m);
                const float f = up == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - up);
                m = up;
                l *= f;
#pragma unroll
                for (int j = 0; j < VB; ++j) o[j] *= f;
            }
            const float mm = m == -INFINITY ? 0.0f : m;
            v8h ph, pl;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // the shift is added last: m - kPShift would round for scores past 2^24 and p pass fp16's range
                const float x = __builtin_amdgcn_exp2f((s[e / 4][e % 4] - mm) + kPShift);
                l += x;
                ph[e] = (_Float16)x;
                pl[e] = (_Float16)(x - (float)ph[e]);
            }
#pragma unroll
            for (int j = 0; j < VB; ++j) {
                v4u r;
#pragma unroll
                for (int i = 0; i < 4; ++i) r[i] = pair_f16<FMT>(w.v[2 * i][j / 4], w.v[2 * i + 1][j / 4], j % 4);
                const v8h v = __builtin_bit_cast(v8h, r);
                o[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, ph, o[j], 0, 0, 0);
                o[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, pl, o[j], 0, 0, 0);
            }
        };

        // Two tiles' codes are in flight: while one is used the next is on its way, and the page numbers of the
        // one after that.
        Codes<D> w[2];
        int k0 = first;
        if (k0 < thi) {
            uint32_t mask0 = rows_of(k0, page_of(k0));
            fetch(w[0]);
            int k1 = advance(k0);
            int page = page_of(k1);
            while (true) {
                uint32_t mask1 = rows_of(k1, page);
                int k2 = 0;
                if (k1 < thi) {
                    fetch(w[1]);
                    k2 = advance(k1);
                    page = page_of(k2);
                }
                step(w[0], k0, mask0);
                if (k1 >= thi) break;
                mask0 = rows_of(k2, page);
                if (k2 < thi) {
                    fetch(w[0]);
                    k0 = k2;
                    const int k3 = advance(k2);
                    page = page_of(k3);
                    step(w[1], k1, mask1);
                    k1 = k3;
                } else {
                    step(w[1], k1, mask1);
                    break;
                }
            }
        }
        l = sum_over_groups(l);

        // The waves' results joined in wave order, the channels in kParts rounds.
        if (g == 0) ml_lds[wave][n] = make_float2(m, l);
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
#pragma unroll
            for (int i = 0; i < kI; ++i)
#pragma unroll
                for (int j = 0; j < VB; j += 4)
                    *reinterpret_cast<float4*>(&o_lds[wave][n][(kI * g + i) * VB + j]) =
                        make_float4(o[j][kI * part + i], o[j + 1][kI * part + i], o[j + 2][kI * part + i],
                                    o[j + 3][kI * part + i]);
            __syncthreads();
            for (int x = threadIdx.x; x < kCols * D / kParts / 4; x += kWaves * kWave) {
                const int cc = x / (D / kParts / 4), y = x % (D / kParts / 4) * 4;
                const int ccol = ct * kCols + cc;
                if (ccol >= seq.nq * a.group) continue;
                const int d = y / (kI * VB) * (4 * VB) + part * kI * VB + y % (kI * VB);
                float M = -INFINITY, L = 0.0f;
#pragma unroll
                for (int w = 0; w < kWaves; ++w) M = fmaxf(M, ml_lds[w][cc].x);
                float4 r = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int w = 0; w < kWaves; ++w) {
                    const float f = ml_lds[w][cc].x == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(ml_lds[w][cc].x - M);
                    const float4 v = *reinterpret_cast<const float4*>(&o_lds[w][cc][y]);
                    L += f * ml_lds[w][cc].y;
                    r = make_float4(r.x + f * v.x, r.y + f * v.y, r.z + f * v.z, r.w + f * v.w);
                }
                const int i = ccol / a.group, h = hk * a.group + ccol % a.group;
                const int64_t orow = seq.row0 + i;
                if (a.splits > 1) {
                    const int64_t at = ((int64_t)split * p.rows + orow) * p.Hq + h;
                    if (d == 0) a.part_ml[at] = make_float2(M, L);
                    *reinterpret_cast<float4*>(a.part_o + at * D + d) = r;
                } else {
                    write_row(p, orow, h, a.group, D, d, M, L, r);
                }
            }
            __syncthreads();
        }
    }
}

// Joins the key shares of every output row, in share order: four waves take
// shares in turn, then their sums meet in LDS.
template <int D>
__global__ __launch_bounds__(kWaves* kWave) void attn_join(StreamArgs a) {
    const PagedAttn& p = a.p;
    constexpr int V = D / kWave;  // channels of a lane
    __shared__ float sums[kWaves][D];
    __shared__ float weight[kWaves];
    const int h = blockIdx.x % p.Hq;
    const int by = blockIdx.x / p.Hq;
    const int b = by % p.B, i0 = by / p.B;
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    const Seq seq = sequence(p, b);
    const int prefix = p.prefix ? p.prefix[b] : 0;
    const int per_pass = gridDim.x / (p.Hq * p.B);
    for (int i = i0; i < seq.nq; i += per_pass) {
        // the shares that have keys, as the first kernel dealt them out
        int lo, hi;
        tile_keys(p, seq, prefix, a.group, (i * a.group + h % a.group) / kCols, lo, hi);
        const int keys = max(0, hi - lo / kTile * kTile);
        const int shares = (int)min((int64_t)a.splits, ((int64_t)keys + a.chunk - 1) / a.chunk);
        const int64_t at = (int64_t)(seq.row0 + i) * p.Hq + h;
        const int64_t stride = (int64_t)p.rows * p.Hq;
        float M = -INFINITY;
        for (int s = lane; s < shares; s += kWave) M = fmaxf(M, a.part_ml[s * stride + at].x);
        M = wave_max(M);
        float L = 0.0f, r[V];
#pragma unroll
        for (int v = 0; v < V; ++v) r[v] = 0.0f;
        for (int s = wave; s < shares; s += kWaves) {
            const float2 ml = a.part_ml[s * stride + at];
            const float f = ml.x == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(ml.x - M);
            L += f * ml.y;
#pragma unroll
            for (int v = 0; v < V; ++v) r[v] += f * a.part_o[(s * stride + at) * D + lane * V + v];
        }
#pragma unroll
        for (int v = 0; v < V; ++v) sums[wave][lane * V + v] = r[v];
        if (lane == 0) weight[wave] = L;
        __syncthreads();
        static_assert(kWaves == 4, "four sums");
        L = weight[0] + weight[1] + weight[2] + weight[3];
        if (threadIdx.x < D / 4) {
            const int d = 4 * threadIdx.x;
            float y[4];
#pragma unroll
            for (int v = 0; v < 4; ++v) y[v] = (sums[0][d + v] + sums[1][d + v]) + (sums[2][d + v] + sums[3][d + v]);
            write_row(p, seq.row0 + i, h, a.group, D, d, M, L, make_float4(y[0], y[1], y[2], y[3]));
        }
        __syncthreads();
    }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Workgroups of one launch; rows beyond what they are planned for are taken in turn.
constexpr int64_t kMaxGrid = 1 << 26;

struct StreamPlan {
    int64_t col_tiles, splits, chunk;
};

// Key shares: enough workgroups to fill the card (two of four waves on each
// of 256 CUs), none with fewer than 256 keys.
StreamPlan stream_plan(int64_t B, int64_t Hq, int64_t Hkv, int64_t max_q, int64_t max_len) {
    constexpr int64_t kTarget = 1024, kMinKeys = 256, kRound = kTile * kWaves;
    StreamPlan s;
    s.col_tiles = std::max<int64_t>(1, ceil_div(std::max<int64_t>(max_q, 1) * (Hq / Hkv), kCols));
    s.col_tiles = std::max<int64_t>(1, std::min(s.col_tiles, kMaxGrid / std::max<int64_t>(1, B * Hkv)));
    const int64_t units = std::max<int64_t>(1, B * Hkv * s.col_tiles);
    s.splits = std::min(ceil_div(kTarget, units), std::max<int64_t>(1, max_len / kMinKeys));
    s.chunk = std::max<int64_t>(kRound, ceil_div(ceil_div(max_len, s.splits), kRound) * kRound);
    s.splits = std::max<int64_t>(1, std::min(s.splits, ceil_div(max_len, s.chunk)));
    return s;
}

template <int D>
hipError_t launch(const StreamArgs& a, int fmt, unsigned grid, int64_t max_q, hipStream_t stream) {
    if (fmt == kKvE5M2)
        hipLaunchKernelGGL((attn_stream<D, kKvE5M2>), dim3(grid), dim3(kWaves * kWave), 0, stream, a);
    else
        hipLaunchKernelGGL((attn_stream<D, kKvE4M3>), dim3(grid), dim3(kWaves * kWave), 0, stream, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1) return e;
    const int64_t heads = (int64_t)a.p.B * a.p.Hq;
    const int64_t per_head = std::max<int64_t>(1, std::min(max_q, kMaxGrid / heads));
    hipLaunchKernelGGL((attn_join<D>), dim3((unsigned)(heads * per_head)), dim3(kWaves * kWave), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

size_t attn_paged_ws_bytes(int64_t B, int64_t rows, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_q,
                           int64_t max_len) {
    const StreamPlan s = stream_plan(B, Hq, Hkv, max_q, max_len);
    return s.splits > 1 ? (size_t)(s.splits * rows * Hq) * ((size_t)D * 4 + 8) : 0;
}

hipError_t launch_attn_paged(const PagedAttn& p, int D, int fmt, int64_t max_q, int64_t max_len, void* ws,
                             hipStream_t stream) {
    const StreamPlan s = stream_plan(p.B, p.Hq, p.Hkv, max_q, max_len);
    StreamArgs a;
    a.p = p;
    a.group = p.Hq / p.Hkv;
    a.col_tiles = (int)s.col_tiles;
    a.splits = (int)s.splits;
    a.chunk = (int)s.chunk;
    a.part_o = static_cast<float*>(ws);
    a.part_ml = reinterpret_cast<float2*>(static_cast<float*>(ws) + s.splits * p.rows * p.Hq * D);
    const unsigned grid = (unsigned)((int64_t)p.B * p.Hkv * s.col_tiles * s.splits);
    const int64_t q = std::max<int64_t>(1, max_q);
    switch (D) {
        case 64: return launch<64>(a, fmt, grid, q, stream);
        case 128: return launch<128>(a, fmt, grid, q, stream);
        default: return launch<256>(a, fmt, grid, q, stream);
    }
}

}  // namespace fp8k
