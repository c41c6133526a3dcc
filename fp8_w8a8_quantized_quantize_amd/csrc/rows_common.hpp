// Device helpers of the kernels around the products (expert rows, epilogues,
// the activation quantizer): elements of rows at any alignment, codes as fp16,
// the activation functions and the epilogue of four outputs.
#pragma once

#include <type_traits>

#include "device_common.hpp"
#include "kernels.hpp"

namespace fp8k {

// Runs of row elements need not be aligned (an odd row length moves every row):
// gfx950's global loads and stores take any byte address, so these types only
// keep the compiler from assuming more.
typedef uint32_t u32x1_any __attribute__((aligned(1)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));

// W words (4 W bytes) at p.
template <int W>
__device__ __forceinline__ void load_words(const void* p, uint32_t (&w)[W]) {
    static_assert(W == 1 || W == 2 || W % 4 == 0, "1, 2 or a multiple of 4 words");
    if constexpr (W == 1) {
        w[0] = *static_cast<const u32x1_any*>(p);
    } else if constexpr (W == 2) {
        const u32x2_any v = *static_cast<const u32x2_any*>(p);
        w[0] = v[0], w[1] = v[1];
    } else {
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
            const u32x4_any v = static_cast<const u32x4_any*>(p)[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[4 * i + j] = v[j];
        }
    }
}

template <int W>
__device__ __forceinline__ void store_words(void* p, const uint32_t (&w)[W]) {
    static_assert(W == 1 || W == 2 || W % 4 == 0, "1, 2 or a multiple of 4 words");
    if constexpr (W == 1) {
        *static_cast<u32x1_any*>(p) = w[0];
    } else if constexpr (W == 2) {
        *static_cast<u32x2_any*>(p) = u32x2_any{w[0], w[1]};
    } else {
#pragma unroll
        for (int i = 0; i < W / 4; ++i)
            static_cast<u32x4_any*>(p)[i] = u32x4_any{w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
    }
}

template <int DT>
constexpr int elem_size() {
    return DT == kKvF32 ? 4 : 2;
}

__device__ __forceinline__ float half_value(uint32_t bits) {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
}

// The V elements of type DT that `w` holds, as fp32 (exact).
template <int DT, int V>
__device__ __forceinline__ void unpack(const uint32_t (&w)[V * elem_size<DT>() / 4], float (&x)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if constexpr (DT == kKvF32)
            x[i] = __uint_as_float(w[i]);
        else if constexpr (DT == kKvBF16)
            x[i] = __uint_as_float((i & 1) ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
        else
            x[i] = half_value((i & 1) ? w[i / 2] >> 16 : w[i / 2] & 0xFFFFu);
    }
}

// fp32 rounded to nearest even to DT's bits; NaN stays NaN.
template <int DT>
__device__ __forceinline__ uint32_t round_bits(float x) {
    if constexpr (DT == kKvF32)
        return __float_as_uint(x);
    else if constexpr (DT == kKvBF16)
        return __builtin_bit_cast(uint16_t, (__bf16)x);
    else
        return __builtin_bit_cast(uint16_t, (_Float16)x);
}

template <int DT>
__device__ __forceinline__ uint32_t round_pair(float lo, float hi) {
    if constexpr (DT == kKvBF16) {
        typedef __bf16 v2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, (v2{(__bf16)lo, (__bf16)hi}));
    } else {
        typedef _Float16 v2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, (v2{(_Float16)lo, (_Float16)hi}));
    }
}

template <int DT, int V>
__device__ __forceinline__ void pack(const float (&x)[V], uint32_t (&w)[V * elem_size<DT>() / 4]) {
    if constexpr (DT == kKvF32) {
#pragma unroll
        for (int i = 0; i < V; ++i) w[i] = __float_as_uint(x[i]);
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) w[i] = round_pair<DT>(x[2 * i], x[2 * i + 1]);
    }
}

template <int DT>
__device__ __forceinline__ float load_elem(const void* base, int64_t e) {
    if constexpr (DT == kKvF32)
        return static_cast<const float*>(base)[e];
    else if constexpr (DT == kKvBF16)
        return __uint_as_float((uint32_t) static_cast<const uint16_t*>(base)[e] << 16);
    else
        return half_value(static_cast<const uint16_t*>(base)[e]);
}

template <int DT>
__device__ __forceinline__ void store_elem(void* base, int64_t e, float x) {
    if constexpr (DT == kKvF32)
        static_cast<float*>(base)[e] = x;
    else
        static_cast<uint16_t*>(base)[e] = (uint16_t)round_bits<DT>(x);
}

// V elements at element offset e, the first n of them in the row (others 0).
template <int DT, int V>
__device__ __forceinline__ void load_run(const void* base, int64_t e, int n, float (&x)[V]) {
    if (n >= V) {
        uint32_t w[V * elem_size<DT>() / 4];
        load_words(static_cast<const uint8_t*>(base) + e * elem_size<DT>(), w);
        unpack<DT, V>(w, x);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = i < n ? load_elem<DT>(base, e + i) : 0.0f;
    }
}

template <int DT, int V>
__device__ __forceinline__ void store_run(void* base, int64_t e, int n, const float (&x)[V]) {
    if (n >= V) {
        uint32_t w[V * elem_size<DT>() / 4];
        pack<DT, V>(x, w);
        store_words(static_cast<uint8_t*>(base) + e * elem_size<DT>(), w);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < n) store_elem<DT>(base, e + i, x[i]);
    }
}

// Eight E4M3 codes (two words) as the fp16 values they are, exactly.
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
__device__ __forceinline__ v8h half8_of(int lo, int hi) {
    typedef _Float16 v2h __attribute__((ext_vector_type(2)));
    const v2h a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
    const v2h b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
    const v2h c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
    const v2h d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
    return v8h{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Activation functions on fp32, each in a form that keeps its relative accuracy in
// the tails (no 1 - x of nearly equal values) down to 2^-126 (|x| + 1): there the
// hardware's 2^t and reciprocal are past their range and give 0:
//   silu(x)      = x / (1 + e^-x)
//   gelu(x)      = x Phi(x), Phi(-a) = erfc(a / sqrt 2) / 2 and Phi(a) = 1 - Phi(-a) for a >= 0
//   gelu_tanh(x) = x / (1 + e^-2u), u = sqrt(2 / pi) (x + 0.044715 x^3):
//                  the same as x (1 + tanh u) / 2.
// FINE, for fp32 outputs (the activation quantizer's scales among them) and where other
// work hides it: within a few units of 2^-24 (gelu 5e-7).  Otherwise, for the tiled
// products' 16-bit outputs, which round by 2^-12 or more themselves: an exponent's
// argument t costs |t| 2^-23 and gelu's fit 4.7e-6, for half the instructions (these
// epilogues run while the matrix units wait).

// 1 / x, to one step of fp32; 0 for inf.
__device__ __forceinline__ float fast_recip(float x) { return __builtin_amdgcn_rcpf(x); }

// 2^(x c), c_low being what the constant c leaves out: the rounding error of the
// product (and the constant's) goes into a first-order factor, so large |x| keep the
// accuracy of the hardware's 2^t.  Past the range the error term is NaN (inf - inf);
// the clamp turns it into a number, the factor stays above 0.3, and 2^t is 0 or inf
// whatever it is.
__device__ __forceinline__ float exp2_fine(float x, float c, float c_low, float more = 0.0f) {
    const float t = x * c;
    const float low = __builtin_amdgcn_fmed3f(__builtin_fmaf(x, c, -t) + __builtin_fmaf(x, c_low, more), -1.0f, 1.0f);
    return __builtin_amdgcn_exp2f(t) * __builtin_fmaf(0.693147182f, low, 1.0f);
}

constexpr float kLog2e = 1.44269502f, kLog2eLow = 1.92596303e-8f;

template <bool FINE>
__device__ __forceinline__ float silu(float x) {
    const float e = FINE ? exp2_fine(x, -kLog2e, -kLog2eLow) : __builtin_amdgcn_exp2f(x * -kLog2e);
    return x * fast_recip(1.0f + e);
}

template <bool FINE>
__device__ __forceinline__ float gelu(float x) {
    // erfc(a / sqrt 2) / 2 = e^(-a^2 / 2) t P(t), t = 1 / (1 + q a), P fitted over
    // 0 <= a <= 13.5 (past it the value is below fp32's range): to 1.4e-8 with nine
    // coefficients, to 4.7e-6 with six.
    const float a = fabsf(x);
    const float t = fast_recip(__builtin_fmaf(FINE ? 0.21f : 0.31f, a, 1.0f));
    float p, e;
    const float s = x * x;
    if constexpr (FINE) {
        p = -0.07203391939401627f;
        p = __builtin_fmaf(p, t, 0.28545311093330383f);
        p = __builtin_fmaf(p, t, -0.3341890871524811f);
        p = __builtin_fmaf(p, t, 0.3540330231189728f);
        p = __builtin_fmaf(p, t, -0.09724528342485428f);
        p = __builtin_fmaf(p, t, 0.12635496258735657f);
        p = __builtin_fmaf(p, t, 0.06879008561372757f);
        p = __builtin_fmaf(p, t, 0.08512940257787704f);
        p = __builtin_fmaf(p, t, 0.08370770514011383f);
        // the square's rounding error goes along
        constexpr float kHalf = -0.5f * kLog2e;
        e = exp2_fine(s, kHalf, -0.5f * kLog2eLow, __builtin_fmaf(x, x, -s) * kHalf);
    } else {
        p = -0.07392915338277817f;
        p = __builtin_fmaf(p, t, 0.18045033514499664f);
        p = __builtin_fmaf(p, t, 0.015744805335998535f);
        p = __builtin_fmaf(p, t, 0.13342967629432678f);
        p = __builtin_fmaf(p, t, 0.12044132500886917f);
        p = __builtin_fmaf(p, t, 0.12386069446802139f);
        e = __builtin_amdgcn_exp2f(s * (-0.5f * kLog2e));
    }
    // the minimum: phi is 0 at +inf, and inf - inf 0 would be NaN
    const float phi = p * t * e;
    return x < 0.0f ? x * phi : __builtin_fmaf(-fminf(x, 3.40282347e38f), phi, x);
}

template <bool FINE>
__device__ __forceinline__ float gelu_tanh(float x) {
    // -2u = x (-2 sqrt(2 / pi) - 2 sqrt(2 / pi) 0.044715 x^2), times log2(e) right away when not FINE
    constexpr float kA = -1.59576912f, kB = -0.0713548163f;
    if constexpr (FINE) {
        const float e = exp2_fine(x * __builtin_fmaf(kB, x * x, kA), kLog2e, kLog2eLow);
        return x * fast_recip(1.0f + e);
    } else {
        const float e = __builtin_amdgcn_exp2f(x * __builtin_fmaf(kB * kLog2e, x * x, kA * kLog2e));
        return x * fast_recip(1.0f + e);
    }
}

// act of V values; `act` is the same for the whole launch, so the branch is uniform.
template <bool FINE, int V>
__device__ __forceinline__ void activate(float (&x)[V], int act) {
    if (act == kActNone) return;
    if (act == kActRelu) {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = x[i] < 0.0f ? 0.0f : x[i];  // NaN stays
    } else if (act == kActSilu) {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = silu<FINE>(x[i]);
    } else if (act == kActGelu) {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = gelu<FINE>(x[i]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = gelu_tanh<FINE>(x[i]);
    }
}

// The epilogue of four neighbouring outputs from their sums (decode and split k, whose
// memory traffic hides the activation).  A missing bias enters as -0, which leaves every
// value as it is, signed zeros included.
template <int DT>
__device__ __forceinline__ void finish4_typed(const Epilogue& e, const v4f& sum, float st,
                                              const float* __restrict__ s_ch, int m, int nb, int N) {
    const int left = N - nb;
    float sc[4], x[4];
    load_run<kKvF32, 4>(s_ch, nb, left, sc);
    if (e.bias != nullptr) {
        load_run<kKvF32, 4>(e.bias, nb, left, x);
    } else {
#pragma unroll
        for (int v = 0; v < 4; ++v) x[v] = -0.0f;
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) x[v] = __builtin_fmaf(sum[v], st * sc[v], x[v]);
    activate<true, 4>(x, e.act);
    if (e.residual != nullptr) {
        float r[4];
        load_run<DT, 4>(e.residual, (int64_t)m * e.ldr + nb, left, r);
#pragma unroll
        for (int v = 0; v < 4; ++v) x[v] += r[v];
    }
    store_run<DT, 4>(e.y, (int64_t)m * e.ldy + nb, left, x);
}

__device__ __forceinline__ void finish4(const Epilogue& e, const v4f& sum, float st, const float* __restrict__ s_ch,
                                        int m, int nb, int N) {
    if (e.type == kKvBF16)
        finish4_typed<kKvBF16>(e, sum, st, s_ch, m, nb, N);
    else if (e.type == kKvF16)
        finish4_typed<kKvF16>(e, sum, st, s_ch, m, nb, N);
    else
        finish4_typed<kKvF32>(e, sum, st, s_ch, m, nb, N);
}

// kernel<DT>(...) of a runtime element type: f(std::integral_constant<int, DT>).
template <typename F>
hipError_t with_type(int dtype, F&& f) {
    switch (dtype) {
        case kKvF32: return f(std::integral_constant<int, kKvF32>{});
        case kKvBF16: return f(std::integral_constant<int, kKvBF16>{});
        default: return f(std::integral_constant<int, kKvF16>{});
    }
}

}  // namespace fp8k
