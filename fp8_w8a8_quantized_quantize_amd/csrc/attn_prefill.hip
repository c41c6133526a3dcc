// Attention over the paged FP8 KV cache on gfx950, tiled form: many query rows
// per sequence, bound by the matrix cores.
//
// Mathematics, operand terms and visibility are those of the streaming form
// (attn_paged.hip): codes exact in fp16, key scales in the query, value scales
// at the output, scores transposed so that a lane's results belong to one query
// column, p straight from the scores' registers into the second product.
//
// Tile.  The columns are a KV head's query rows, token times group, so one pass
// over the keys serves all query heads of the group.  A workgroup of four waves
// takes 128 NC columns, 32 NC a wave, and walks over 64-key tiles that all its
// waves share in LDS: K as fp16 rows, V as fp16 transposed, eight keys of a
// channel in 16 bytes in the order in which a lane holds its p.  Codes become
// fp16 once per workgroup, on the way into LDS.  NC = 2 halves the LDS bytes per
// matrix instruction (64 columns a wave: each 1 KB operand read feeds two
// 32x32x16 instructions of 32 cycles; four waves then need 64 of the 128 bytes
// a cycle that LDS gives); it takes the registers of one wave per SIMD, so the
// overlap of softmax and matrix work is inside the wave: scores of tile i + 1
// are formed while the softmax of tile i runs.
//
// One barrier per tile: step i writes V of tile i and K of tile i + 1 into the
// buffers last read in steps i - 2 and i - 1, loads K of tile i + 2 and V of
// tile i + 1 into registers, and after the barrier forms S(i + 1) = Q K(i + 1),
// p of tile i, and adds p V(i).
#include <algorithm>

#include "attn_common.hpp"

namespace fp8k {

namespace {

typedef float v16f __attribute__((ext_vector_type(16)));

constexpr int kWavesT = 4;
constexpr int kThreadsT = kWavesT * kWave;
constexpr int kKeys = 64;  // keys of a tile

struct TileArgs {
    PagedAttn p;
    int group;
    int col_tiles;  // planned per KV head; further ones are taken in turn
    FastDiv by_block, by_group, by_kv_heads;
};

template <int D, int TERMS>
constexpr int col_groups() {
    return TERMS == 1 && D <= 128 ? 2 : 1;
}

template <int D, int TERMS>
constexpr int tile_cols() {
    return kWavesT * 32 * col_groups<D, TERMS>();
}

// LDS: two K tiles, two V tiles, cache offsets of 16 rows per wave for three
// tiles, and which keys of two tiles are there.
template <int D>
struct TileLds {
    static constexpr int kK = kKeys * D * 2;
    static constexpr int kV = 2 * kK;
    static constexpr int kRows = 4 * kK;
    static constexpr int kMask = kRows + 3 * kKeys * 8;
    static constexpr int kBytes = kMask + 2 * kWavesT * 4;
};

extern __shared__ __attribute__((aligned(1024))) uint8_t tile_smem[];

// Place of the 16-byte units of a K row (2 D bytes) and of a V channel (128
// bytes) such that neighbouring rows' units lie in different banks.
template <int D>
__device__ __forceinline__ int swz_k(int key) {
    return D == 64 ? (key ^ (key >> 3)) & 7 : key & 15;
}
__device__ __forceinline__ int swz_v(int d) { return (d ^ (d >> 3)) & 7; }

template <int D, int FMT, bool BIAS, int TERMS>
__global__ __launch_bounds__(kThreadsT, 1) void attn_tile(TileArgs a) {
    const PagedAttn& p = a.p;
    constexpr int NC = col_groups<D, TERMS>();
    constexpr int COLS = tile_cols<D, TERMS>();
    constexpr int NK = D / 16;  // matrix instructions along the channels of K
    constexpr int DB = D / 32;  // 32-channel blocks of the output
    constexpr int VB = D / 32;  // V channels a thread stages
    using Lds = TileLds<D>;
    typedef typename std::conditional<D == 64, uint16_t, typename std::conditional<D == 128, uint32_t, v2u>::type>::type vpiece;

    const int tid = threadIdx.x, lane = tid % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int c = lane % 32, h = lane / 32;
    const int nth = a.by_kv_heads.of(blockIdx.x), hk = blockIdx.x - nth * p.Hkv;
    const int b = blockIdx.y;
    const Seq seq = sequence(p, b);
    const int prefix = p.prefix ? p.prefix[b] : 0;
    const int cols = seq.nq * a.group;
    const uint32_t C = 2u * p.Hkv * D;
    const int32_t* table = p.block_table + (int64_t)b * p.ld_table;
    const int last_page = max(p.max_blocks - 1, 0);
    uint64_t* const rows = reinterpret_cast<uint64_t*>(tile_smem + Lds::kRows) + wave * 16;  // [tile % 3][4 waves][16]
    uint32_t* const there = reinterpret_cast<uint32_t*>(tile_smem + Lds::kMask);             // [tile % 2][4 waves]

    // the last column tiles see the most keys: they go first
    for (int ct = a.col_tiles - 1 - nth + (cols > a.col_tiles * COLS ? (cols - 1) / (a.col_tiles * COLS) * a.col_tiles : 0);
         ct >= 0; ct -= a.col_tiles) {
        if (ct * COLS >= cols) continue;
        // this lane's columns
        int lo[NC], hi[NC], pos[NC], head[NC];
        int64_t row[NC];
        bool has[NC];
        float slope[NC];
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            const int col = ct * COLS + (wave * NC + n) * 32 + c;
            has[n] = col < cols;
            const int qi = has[n] ? a.by_group.of(col) : 0;
            head[n] = hk * a.group + (has[n] ? col - qi * a.group : 0);
            row[n] = seq.row0 + qi;
            pos[n] = seq.len - seq.nq + qi;
            visible(p, seq, prefix, qi, lo[n], hi[n]);
            if (!has[n]) lo[n] = 0x7FFFFFFF, hi[n] = 0;
            slope[n] = p.alibi ? p.alibi[head[n]] * kLog2e : 0.0f;
        }
        // the keys any column of the workgroup sees, and of this wave
        int tlo, thi, unused;
        visible(p, seq, prefix, a.by_group.of(ct * COLS), tlo, unused);
        visible(p, seq, prefix, a.by_group.of(min(cols - 1, ct * COLS + COLS - 1)), unused, thi);
        thi = max(thi, 0);
        tlo = min(tlo, thi);
        const int base = p.window > 0 ? tlo / kKeys * kKeys : 0;
        const int tiles = thi > base ? (thi - base + kKeys - 1) / kKeys : 0;
        int wlo = lo[0], whi = hi[0];
#pragma unroll
        for (int n = 1; n < NC; ++n) wlo = min(wlo, lo[n]), whi = max(whi, hi[n]);
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            wlo = min(wlo, __shfl_xor(wlo, off, kWave));
            whi = max(whi, __shfl_xor(whi, off, kWave));
        }
        wlo = __builtin_amdgcn_readfirstlane(wlo);
        whi = __builtin_amdgcn_readfirstlane(whi);

        // q times the key scales, in fp16 terms
        v8h qt[TERMS][NC][NK];
        float cs[NC];
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            v4u raw[NK][2];
            float top = 0.0f;
#pragma unroll
            for (int s = 0; s < NK; ++s)
                load_q8<TERMS>(p, row[n] * p.ldq + (int64_t)head[n] * D + 16 * s + 8 * h, raw[s]);
            float x[NK][8];
#pragma unroll
            for (int s = 0; s < NK; ++s) {
                unpack_q8<TERMS>(p, raw[s], x[s]);
                const float4* ks = reinterpret_cast<const float4*>(p.scales + hk * D + 16 * s + 8 * h);
                const float4 k0 = ks[0], k1 = ks[1];
                const float k[8] = {k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w};
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[s][e] *= fmaxf(k[e], kScaleFloor);
                    top = fmaxf(top, fabsf(x[s][e]));
                }
            }
            top = fmaxf(top, swap32(top));
            const int shift = 15 - __builtin_amdgcn_frexp_expf(top);
#pragma unroll
            for (int s = 0; s < NK; ++s)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float y = __builtin_amdgcn_ldexpf(x[s][e], shift);
                    qt[0][n][s][e] = (_Float16)y;
                    if constexpr (TERMS == 2) qt[TERMS - 1][n][s][e] = (_Float16)(y - (float)qt[0][n][s][e]);
                }
            cs[n] = __builtin_amdgcn_ldexpf(p.scale, -shift);
            if (p.softcap > 0.0f) cs[n] *= kLn2;  // the cap takes the natural score
        }
        const float cap_in = p.softcap > 0.0f ? 2.0f * kLog2e / p.softcap : 0.0f;

        float m[NC], l[NC];
        v16f o[NC][DB];
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            m[n] = kNoRef;
            l[n] = 0.0f;
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[n][d][i] = 0.0f;
        }

        // ---- staging.  A wave stages keys 16 wave .. + 15 of a tile: K, a quarter row per thread; V, the eight keys of
        // two lane groups, VB channels per thread.
        auto page_of = [&](int t) { return table[min(a.by_block.of(base + t * kKeys + 16 * wave + lane % 16), last_page)]; };
        // cache offsets of the wave's 16 rows of tile t, 0 for keys that are not there
        auto rows_of = [&](int t, int page) {
            const int key = base + t * kKeys + 16 * wave + lane % 16;
            const bool ok = key >= tlo && key < thi && page >= 0 && page < p.num_blocks;
            const uint32_t r = ok ? (page - a.by_block.of(key)) * p.block + key : 0;
            if (lane < 16) rows[t % 3 * kKeys + lane] = (uint64_t)r * C;
            const uint32_t mask = (uint32_t)__ballot(ok) & 0xFFFFu;
            if (lane == 0) there[t % 2 * kWavesT + wave] = mask;
            __builtin_amdgcn_wave_barrier();
            return mask;
        };
        v4u kreg[D / 64];
        vpiece vreg[8];
        auto load_k = [&](int t) {
            const uint8_t* src = p.cache + rows[t % 3 * kKeys + lane / 4] + hk * D + lane % 4 * (D / 4);
#pragma unroll
            for (int i = 0; i < D / 64; ++i) kreg[i] = *reinterpret_cast<const v4u*>(src + 16 * i);
        };
        auto load_v = [&](int t) {
            const uint8_t* src = p.cache + (int64_t)(p.Hkv + hk) * D + c * VB;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                vreg[e] = *reinterpret_cast<const vpiece*>(src + rows[t % 3 * kKeys + 8 * (e / 4) + 4 * h + e % 4]);
        };
        auto store_k = [&](int t) {
            uint8_t* dst = tile_smem + t % 2 * Lds::kK + (16 * wave + lane / 4) * 2 * D;
#pragma unroll
            for (int i = 0; i < D / 64; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int unit = (lane % 4 * (D / 64) + i) * 2 + k;
                    *reinterpret_cast<v8h*>(dst + (unit ^ swz_k<D>(16 * wave + lane / 4)) * 16) =
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
            uint8_t* const dst = tile_smem + Lds::kV + t % 2 * Lds::kK;
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
                const int d = c * VB + j;
                *reinterpret_cast<v4u*>(dst + d * 128 + ((2 * wave + h) ^ swz_v(d)) * 16) = r;
            }
        };
        v16f s[NC][2];
        auto scores = [&](int t) {
            const uint8_t* src = tile_smem + t % 2 * Lds::kK;
#pragma unroll
            for (int n = 0; n < NC; ++n)
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                    for (int i = 0; i < 16; ++i) s[n][kb][i] = 0.0f;
#pragma unroll
            for (int st = 0; st < NK; ++st)
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) {
                    const int key = 32 * kb + c;
                    const v8h k = *reinterpret_cast<const v8h*>(src + key * 2 * D + ((2 * st + h) ^ swz_k<D>(key)) * 16);
#pragma unroll
                    for (int n = 0; n < NC; ++n)
#pragma unroll
                        for (int x = 0; x < TERMS; ++x)
                            s[n][kb] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k, qt[x][n][st], s[n][kb], 0, 0, 0);
                }
        };
        // p of tile t from its scores z
        v8h ph[TERMS][NC][4];
        auto softmax = [&](int t, v16f (&z)[NC][2], uint64_t mask) {
            const int key0 = base + t * kKeys;
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                if constexpr (BIAS) {
#pragma unroll
                    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float x = z[n][kb][i] * cs[n];
                            if (p.softcap > 0.0f) x = kLog2e * soft_cap(x, p.softcap, cap_in);
                            z[n][kb][i] = x + slope[n] * (float)(key0 + 32 * kb + 8 * (i / 4) + 4 * h + i % 4 - pos[n]);
                        }
                }
                const bool whole = mask == ~0ull && !__any(key0 < lo[n] || key0 + kKeys > hi[n]);
                if (!whole) {
#pragma unroll
                    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int j = 32 * kb + 8 * (i / 4) + 4 * h + i % 4;
                            const bool see = ((mask >> j) & 1u) & (key0 + j >= lo[n]) & (key0 + j < hi[n]);
                            // below every reference: exp2 gives 0 (the scale's sign would turn an infinity round)
                            z[n][kb][i] = see ? z[n][kb][i] : __uint_as_float(0x7FC00000u);
                        }
                }
                auto above = [&](int kb, int i) {
                    const float x = BIAS ? z[n][kb][i] - m[n] : __builtin_fmaf(z[n][kb][i], cs[n], -m[n]);
                    return whole ? x : z[n][kb][i] == z[n][kb][i] ? x : -INFINITY;
                };
                float top = -INFINITY;
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                    for (int i = 0; i < 16; ++i) top = fmaxf(top, above(kb, i));
                if (__any(top > kPLimit)) {
                    // move the references of the columns that need it, as in the streaming form
                    const float old = m[n];
                    m[n] = 0.0f;
                    top = -INFINITY;
#pragma unroll
                    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                        for (int i = 0; i < 16; ++i) top = fmaxf(top, above(kb, i));
                    top = fmaxf(top, swap32(top));
                    m[n] = top > old + kPLimit ? (fabsf(top) < 16777216.0f ? top - kPShift : top) : old;
                    const float f = __builtin_amdgcn_exp2f(old - m[n]);
                    l[n] *= f;
#pragma unroll
                    for (int d = 0; d < DB; ++d) o[n][d] *= f;
                }
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float y = __builtin_amdgcn_exp2f(above(u / 2, 8 * (u % 2) + e));
                        l[n] += y;
                        ph[0][n][u][e] = (_Float16)y;
                        if constexpr (TERMS == 2) ph[TERMS - 1][n][u][e] = (_Float16)(y - (float)ph[0][n][u][e]);
                    }
            }
        };
        auto product = [&](int t) {
            const uint8_t* src = tile_smem + Lds::kV + t % 2 * Lds::kK;
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int db = 0; db < DB; ++db) {
                    const int d = 32 * db + c;
                    const v8h v = *reinterpret_cast<const v8h*>(src + d * 128 + ((2 * u + h) ^ swz_v(d)) * 16);
#pragma unroll
                    for (int n = 0; n < NC; ++n)
#pragma unroll
                        for (int x = 0; x < TERMS; ++x)
                            o[n][db] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, ph[x][n][u], o[n][db], 0, 0, 0);
                }
        };
        auto mask_of = [&](int t) {
            const uint32_t* w = there + t % 2 * kWavesT;
            const uint32_t lo32 = w[0] | (w[1] << 16), hi32 = w[2] | (w[3] << 16);
            return ((uint64_t)__builtin_amdgcn_readfirstlane(hi32) << 32) | (uint32_t)__builtin_amdgcn_readfirstlane(lo32);
        };

        if (tiles > 0) {
            auto sees = [&](int t) { return base + t * kKeys < whi && base + (t + 1) * kKeys > wlo; };
            uint32_t m0 = rows_of(0, page_of(0));
            int page = page_of(1);
            load_k(0);
            load_v(0);
            store_k(0);
            uint32_t m1 = rows_of(1, page);
            page = page_of(2);
            load_k(1);
            __syncthreads();
            uint64_t mask = mask_of(0);
            if (sees(0)) scores(0);
            for (int t = 0; t < tiles; ++t) {
                store_v(t, m0);
                store_k(t + 1);
                const uint32_t m2 = rows_of(t + 2, page);
                page = page_of(t + 3);
                load_k(t + 2);
                load_v(t + 1);
                __syncthreads();
                const bool now = sees(t);
                v16f z[NC][2];
#pragma unroll
                for (int n = 0; n < NC; ++n) z[n][0] = s[n][0], z[n][1] = s[n][1];
                const uint64_t next_mask = mask_of(t + 1);
                if (t + 1 < tiles && sees(t + 1)) scores(t + 1);
                if (now) {
                    softmax(t, z, mask);
                    product(t);
                }
                mask = next_mask;
                m0 = m1, m1 = m2;
            }
        }

        // ---- results
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            const float L = l[n] + swap32(l[n]);
            if (has[n]) {
#pragma unroll
                for (int db = 0; db < DB; ++db)
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        write_row(p, row[n], head[n], hk, D, 32 * db + 2 * i + 4 * h, m[n], L,
                                  make_float4(o[n][db][i], o[n][db][i + 1], o[n][db][i + 2], o[n][db][i + 3]));
            }
        }
        __syncthreads();
    }
}

template <int D, int FMT, bool BIAS, int TERMS>
hipError_t launch_tile(const TileArgs& a, dim3 grid, hipStream_t stream) {
    constexpr int lds = TileLds<D>::kBytes;
    if constexpr (lds > 64 * 1024) {
        const hipError_t e = FP8K_SET_LDS((attn_tile<D, FMT, BIAS, TERMS>), lds);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((attn_tile<D, FMT, BIAS, TERMS>), grid, dim3(kThreadsT), lds, stream, a);
    return hipGetLastError();
}

template <int D, int TERMS>
hipError_t launch(TileArgs a, int fmt, int64_t max_q, hipStream_t stream) {
    const int64_t tiles = (max_q * a.group + tile_cols<D, TERMS>() - 1) / tile_cols<D, TERMS>();
    a.col_tiles = (int)std::max<int64_t>(1, std::min<int64_t>(tiles, (int64_t(1) << 30) / a.p.Hkv));
    const dim3 grid((unsigned)(a.col_tiles * a.p.Hkv), (unsigned)a.p.B);
    const bool bias = a.p.softcap > 0.0f || a.p.alibi != nullptr;
    if (fmt == kKvE5M2)
        return bias ? launch_tile<D, kKvE5M2, true, TERMS>(a, grid, stream) : launch_tile<D, kKvE5M2, false, TERMS>(a, grid, stream);
    return bias ? launch_tile<D, kKvE4M3, true, TERMS>(a, grid, stream) : launch_tile<D, kKvE4M3, false, TERMS>(a, grid, stream);
}

}  // namespace

hipError_t launch_attn_tiled(const PagedAttn& p, int D, int fmt, int64_t max_q, hipStream_t stream) {
    TileArgs a = {};
    a.p = p;
    a.group = p.Hq / p.Hkv;
    a.by_block = FastDiv(p.block);
    a.by_group = FastDiv(a.group);
    a.by_kv_heads = FastDiv(p.Hkv);
    const bool one = p.dtype == kKvBF16;
    switch (D) {
        case 64: return one ? launch<64, 1>(a, fmt, max_q, stream) : launch<64, 2>(a, fmt, max_q, stream);
        case 128: return one ? launch<128, 1>(a, fmt, max_q, stream) : launch<128, 2>(a, fmt, max_q, stream);
        default: return one ? launch<256, 1>(a, fmt, max_q, stream) : launch<256, 2>(a, fmt, max_q, stream);
    }
}

}  // namespace fp8k
