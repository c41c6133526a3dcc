// Device helpers shared by the attention kernels over the paged FP8 cache: what
// a query sees, codes as matrix operands, query rows in, output rows out.
#pragma once

#include "kv_common.hpp"

namespace fp8k {

typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));

constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kNoRef = -3.0e38f;

// p in fp16: a new reference leaves the largest at 2^8 and stays until one
// passes 2^12.  With one term the reference itself is 2^8 below the largest
// score; with two, scores next to the largest keep their last bits (their
// distance to 2^8 would round at 2^-21), and p is multiplied instead.
constexpr float kPUnit = 256.0f;
template <int TERMS>
struct PScale {
    static constexpr float kShift = TERMS == 1 ? 8.0f : 0.0f;
    static constexpr float kLimit = kShift + 4.0f;

    static __device__ __forceinline__ float p(float x) {
        const float y = __builtin_amdgcn_exp2f(x);
        return TERMS == 1 ? y : y * kPUnit;
    }
};

// n / d for 0 <= n < 2^31 by a product: magic = ceil(2^shift / d) with shift =
// 31 + ceil(log2(d)) is off by e < 1, which adds n e / 2^shift < 1 / d.
struct FastDiv {
    uint32_t magic;
    int shift;

    FastDiv(int64_t d = 1) : shift(31) {
        while ((int64_t(1) << (shift - 31)) < d) ++shift;
        magic = (uint32_t)(((uint64_t(1) << shift) + d - 1) / d);
    }
    __device__ __forceinline__ int of(int n) const { return (int)(((uint64_t)(uint32_t)n * magic) >> shift); }
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

// 8 consecutive elements of a query row, as they are and as fp32.
template <int TERMS>  // 1: bf16 rows alone
__device__ __forceinline__ void load_q8(const PagedAttn& p, int64_t e, v4u (&raw)[2]) {
    if (TERMS == 2 && p.dtype == kKvF32) {
        const v4u* f = reinterpret_cast<const v4u*>(static_cast<const float*>(p.q) + e);
        raw[0] = f[0];
        raw[1] = f[1];
    } else {
        raw[0] = *reinterpret_cast<const v4u*>(static_cast<const uint16_t*>(p.q) + e);
        raw[1] = raw[0];
    }
}

template <int TERMS>
__device__ __forceinline__ void unpack_q8(const PagedAttn& p, const v4u (&raw)[2], float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (TERMS == 1 || p.dtype == kKvBF16) {
            x[2 * i] = __uint_as_float(raw[0][i] << 16);
            x[2 * i + 1] = __uint_as_float(raw[0][i] & 0xFFFF0000u);
        } else if (p.dtype == kKvF32) {
            x[i] = __uint_as_float(raw[0][i]);
            x[4 + i] = __uint_as_float(raw[1][i]);
        } else {
            x[2 * i] = half_to_float(raw[0][i] & 0xFFFFu);
            x[2 * i + 1] = half_to_float(raw[0][i] >> 16);
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

// v of the lane 16 (32) away: gfx950's row and half swaps, no trip through LDS.
__device__ __forceinline__ float swap16(float v) {
    const uint32_t u = __float_as_uint(v);
    const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    return __uint_as_float((threadIdx.x & 16) ? r[0] : r[1]);
}

__device__ __forceinline__ float swap32(float v) {
    const uint32_t u = __float_as_uint(v);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return __uint_as_float((threadIdx.x & 32) ? r[0] : r[1]);
}

// Inclusive sums over the lanes of a wave.
__device__ __forceinline__ int wave_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);   // row_shr:1
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);   // row_shr:2
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);   // row_shr:4
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);   // row_shr:8
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast:15 into rows 1 and 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast:31 into rows 2 and 3
    return v;
}

// Over the four lanes of a column (16 and 32 apart).
__device__ __forceinline__ float max_over_groups(float v) {
    v = fmaxf(v, swap16(v));
    return fmaxf(v, swap32(v));
}

// cap * tanh(x / cap) in fp32: 1 - 2 / (exp(2 x / cap) + 1), whose absolute
// error is that of a few roundings at the cap's magnitude.  In scores far below
// the cap that shows beside two terms, and beside one (2^-11 of the operands)
// from caps of some hundreds on, where a score below 2^-23 of the cap would
// vanish: there x (1 + t), t from the series of tanh(y) / y - 1 up to y^10, off
// by 3e-8 of the score at most.
constexpr float kSmallCap = 256.0f;
template <int TERMS>
__device__ __forceinline__ bool cap_by_series(float cap) { return TERMS == 2 || cap > kSmallCap; }

// 2 log2(e) / cap, finite for the smallest caps too (0 times it is 0).
__device__ __forceinline__ float cap_factor(float cap) { return cap > 0.0f ? fminf(2.0f * kLog2e / cap, 3.4e38f) : 0.0f; }

template <bool SERIES>
__device__ __forceinline__ float soft_cap(float x, float cap, float two_log2e_over_cap) {
    const float u = x * two_log2e_over_cap;
    const float e = __builtin_amdgcn_exp2f(u);
    const float far = cap * (1.0f - 2.0f * __builtin_amdgcn_rcpf(e + 1.0f));
    if constexpr (!SERIES) return far;
    const float y = u * (0.5f * kLn2), z = y * y;
    float t = __builtin_fmaf(z, -1382.0f / 155925.0f, 62.0f / 2835.0f);
    t = __builtin_fmaf(z, t, -17.0f / 315.0f);
    t = __builtin_fmaf(z, t, 2.0f / 15.0f);
    t = __builtin_fmaf(z, t, -1.0f / 3.0f) * z;
    return z < 0.14f ? __builtin_fmaf(x, t, x) : far;
}

// Four channels of an output row from its sum r of p_j code(v_j), reference M
// and sum L of p_j; an empty row (L == 0) is zeros, its log-sum-exp -inf.  Where
// lse is wanted there are two terms, and M is the score at which p is kPUnit.
__device__ __forceinline__ void write_row(const PagedAttn& p, int64_t row, int h, int hk, int D, int d, float M,
                                          float L, const float4& r) {
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    const float4 sc = *reinterpret_cast<const float4*>(p.scales + (int64_t)(p.Hkv + hk) * D + d);
    store_o4(p, row * p.ldo + (int64_t)h * D + d,
             make_float4(r.x * inv * fmaxf(sc.x, kScaleFloor), r.y * inv * fmaxf(sc.y, kScaleFloor),
                         r.z * inv * fmaxf(sc.z, kScaleFloor), r.w * inv * fmaxf(sc.w, kScaleFloor)));
    if (p.lse && d == 0) p.lse[row * p.Hq + h] = L == 0.0f ? -INFINITY : kLn2 * (M + __builtin_amdgcn_logf(L * (1.0f / kPUnit)));
}

}  // namespace fp8k
