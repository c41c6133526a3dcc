// Device helpers shared by the kernels that read or write the FP8 KV cache:
// row element types, the E4M3 / E5M2 codec and the per-channel scales.
#pragma once

#include "device_common.hpp"
#include "kernels.hpp"

namespace fp8k {

constexpr float kE5M2Max = 57344.0f;  // largest finite E5M2 value

__device__ __forceinline__ float4 load_nt(const float4* p) {
    const v4f t = __builtin_nontemporal_load(reinterpret_cast<const v4f*>(p));
    return make_float4(t[0], t[1], t[2], t[3]);
}

__device__ __forceinline__ void store_nt(const float4& v, float4* p) {
    const v4f t = {v.x, v.y, v.z, v.w};
    __builtin_nontemporal_store(t, reinterpret_cast<v4f*>(p));
}

typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float half_to_float(uint32_t h) {
    _Float16 f;
    const uint16_t b = (uint16_t)h;
    __builtin_memcpy(&f, &b, 2);
    return (float)f;
}

__device__ __forceinline__ uint32_t float_to_half_bits(float x) {
    const _Float16 f = (_Float16)x;  // round to nearest even
    uint16_t b;
    __builtin_memcpy(&b, &f, 2);
    return b;
}

// Quads (4 consecutive channels) per thread: one 16-byte load covers 4
// fp32 or 8 bf16 / fp16 channels.
template <int DT>
constexpr int kv_quads() {
    return DT == kKvF32 ? 1 : 2;
}

// The 4 * Q elements of a KV row at element offset `e` from `base`, as fp32
// quads; DT: kKvF32, kKvBF16 or kKvF16.  Read once: nontemporal.
template <int DT>
__device__ __forceinline__ void kv_load(const void* base, int64_t e, float4 (&v)[kv_quads<DT>()]) {
    if constexpr (DT == kKvF32) {
        v[0] = load_nt(reinterpret_cast<const float4*>(static_cast<const float*>(base) + e));
    } else {
        const v4u w = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(static_cast<const uint16_t*>(base) + e));
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const uint32_t a = w[2 * q], b = w[2 * q + 1];
            if constexpr (DT == kKvBF16)
                v[q] = make_float4(__uint_as_float(a << 16), __uint_as_float(a & 0xFFFF0000u), __uint_as_float(b << 16),
                                   __uint_as_float(b & 0xFFFF0000u));
            else
                v[q] = make_float4(half_to_float(a & 0xFFFFu), half_to_float(a >> 16), half_to_float(b & 0xFFFFu),
                                   half_to_float(b >> 16));
        }
    }
}

// 4 * Q fp32 values to consecutive output elements (written once).
template <int DT>
__device__ __forceinline__ void kv_store(void* base, int64_t e, const float4 (&v)[kv_quads<DT>()]) {
    if constexpr (DT == kKvF32) {
        store_nt(v[0], reinterpret_cast<float4*>(static_cast<float*>(base) + e));
    } else {
        v4u w;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            if constexpr (DT == kKvBF16) {
                w[2 * q] = pack_bf16x2(v[q].x, v[q].y);
                w[2 * q + 1] = pack_bf16x2(v[q].z, v[q].w);
            } else {
                w[2 * q] = float_to_half_bits(v[q].x) | (float_to_half_bits(v[q].y) << 16);
                w[2 * q + 1] = float_to_half_bits(v[q].z) | (float_to_half_bits(v[q].w) << 16);
            }
        }
        __builtin_nontemporal_store(w, reinterpret_cast<v4u*>(static_cast<uint16_t*>(base) + e));
    }
}

// Two fp32 -> FP8 codes in bytes [2*HI, 2*HI+1] of `old`, clamped to the
// format's largest finite value first so the conversion saturates; the
// hardware convert rounds to nearest even.
template <int FMT, bool HI>
__device__ __forceinline__ int kv_cvt2(float a, float b, int old) {
    constexpr float m = FMT == kKvE5M2 ? kE5M2Max : kE4M3Max;
    a = __builtin_amdgcn_fmed3f(a, -m, m);
    b = __builtin_amdgcn_fmed3f(b, -m, m);
    if constexpr (FMT == kKvE5M2)
        return __builtin_amdgcn_cvt_pk_bf8_f32(a, b, old, HI);
    else
        return __builtin_amdgcn_cvt_pk_fp8_f32(a, b, old, HI);
}

// Four codes (bytes, little-endian) -> four exact fp32 values.
template <int FMT>
__device__ __forceinline__ float4 kv_decode4(uint32_t w) {
    typedef float v2f __attribute__((ext_vector_type(2)));
    v2f lo, hi;
    if constexpr (FMT == kKvE5M2) {
        lo = __builtin_amdgcn_cvt_pk_f32_bf8((int)w, false);
        hi = __builtin_amdgcn_cvt_pk_f32_bf8((int)w, true);
    } else {
        lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
        hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    }
    return make_float4(lo[0], lo[1], hi[0], hi[1]);
}

__device__ __forceinline__ RowScale channel_scale(float s) {
    s = fmaxf(s, kScaleFloor);
    return RowScale{s, __fdiv_rn(1.0f, s)};
}

template <int FMT>
__device__ __forceinline__ uint32_t kv_encode4(const float4& v, const RowScale& r0, const RowScale& r1,
                                               const RowScale& r2, const RowScale& r3) {
    int w = kv_cvt2<FMT, false>(div_by_scale(v.x, r0), div_by_scale(v.y, r1), 0);
    w = kv_cvt2<FMT, true>(div_by_scale(v.z, r2), div_by_scale(v.w, r3), w);
    return (uint32_t)w;
}

template <int FMT>
__device__ __forceinline__ uint32_t kv_encode4(const float4& v, const RowScale (&rs)[4]) {
    return kv_encode4<FMT>(v, rs[0], rs[1], rs[2], rs[3]);
}

// Two fp32 values rounded to nearest even to a packed pair, NaN kept (the
// KV codec's pack_bf16x2 takes finite values only).
__device__ __forceinline__ uint32_t round_bf16x2(float lo, float hi) {
    typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
    const v2bf p = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, p);
}

__device__ __forceinline__ uint32_t round_f16x2(float lo, float hi) {
    typedef _Float16 v2h __attribute__((ext_vector_type(2)));
    const v2h p = {(_Float16)lo, (_Float16)hi};
    return __builtin_bit_cast(uint32_t, p);
}

}  // namespace fp8k
