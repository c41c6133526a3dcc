// Activation and per-token E4M3 quantization in one pass on gfx950: the step
// between a feed-forward layer's two FP8 products.
//
//   v = act(g) * u (gated: a row holds F of g, then F of u), or act(h)
//   s = max(fl32(max |v| / 448), 1e-12f), codes E4M3(fl32(v / s)), RNE
//
// in fp32 from the row's own type, so the product of the activation is never
// rounded to 16 bits.  A row is read once: its values stay in registers between
// the maximum and the cast.  WPR waves share a row; one wave per row needs no
// LDS and no barrier, and takes over as soon as there are rows enough.  Memory bounds
// many rows (32768 x 2048 gated bf16, silu: 60 us, 5.5 TB/s), the vector unit gelu on
// 16-bit rows (74 us) and the few compute units in use few long ones (64 x 28672, silu:
// 7.1 us for 9 MB).  The activation is that of fp32 outputs, for the scales are fp32 and
// a value's error moves codes across their borders; with that of 16-bit outputs these
// three took 61, 64 and 6.2 us, and gelu's scales were 4.7e-6 off.
#include <type_traits>

#include "rows_common.hpp"

namespace fp8k {

namespace {

template <int DT>
constexpr int piece() {  // elements of a 16-byte piece
    return 16 / elem_size<DT>();
}

// The bytes of a piece of the row: of h, and of the gate's partner.
template <bool GATED>
struct Raw {
    uint32_t g[4], u[GATED ? 4 : 1];
};

template <int DT, bool GATED>
__device__ __forceinline__ void load_raw(const void* h, int64_t e, int64_t F, Raw<GATED>& r) {
    load_words(static_cast<const uint8_t*>(h) + e * elem_size<DT>(), r.g);
    if constexpr (GATED) load_words(static_cast<const uint8_t*>(h) + (e + F) * elem_size<DT>(), r.u);
}

template <int DT, bool GATED, int ACT>
__device__ __forceinline__ void value_of(const Raw<GATED>& r, float (&v)[piece<DT>()]) {
    constexpr int V = piece<DT>();
    unpack<DT, V>(r.g, v);
    activate<true, V>(v, ACT);
    if constexpr (GATED) {
        float u[V];
        unpack<DT, V>(r.u, u);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] *= u[i];
    }
}

// f(std::integral_constant<int, act>): one branch around a row's whole work, not one
// per piece, which costs registers up to spills.
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
    switch (act) {
        case kActNone: f(std::integral_constant<int, kActNone>{}); break;
        case kActRelu: f(std::integral_constant<int, kActRelu>{}); break;
        case kActSilu: f(std::integral_constant<int, kActSilu>{}); break;
        case kActGelu: f(std::integral_constant<int, kActGelu>{}); break;
        default: f(std::integral_constant<int, kActGeluTanh>{}); break;
    }
}

template <int V>
__device__ __forceinline__ float absmax(float m, const float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) m = fmaxf(m, fabsf(v[i]));
    return m;
}

// The codes of fl32(v / s), as cast4 forms them, without its clamps: |v| <= max |v|
// makes no quotient larger than 448 (1 + 2^-23), which rounds to 448, and none of the
// steps overflows.
__device__ __forceinline__ float quotient(float x, const RowScale& rs) {
    const float q0 = x * rs.r;
    return __builtin_fmaf(__builtin_fmaf(q0, rs.s, -x), -rs.r, q0);
}

template <int V>
__device__ __forceinline__ void store_codes(uint8_t* q, const float (&v)[V], const RowScale& rs) {
    uint32_t w[V / 4];
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
        int c = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(v[4 * i], rs), quotient(v[4 * i + 1], rs), 0, false);
        c = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(v[4 * i + 2], rs), quotient(v[4 * i + 3], rs), c, true);
        w[i] = (uint32_t)c;
    }
    store_words(q, w);
}

// The maximum over the WPR waves of a row.
template <int WPR>
__device__ __forceinline__ float row_max(float m, float* red) {
    m = wave_max(m);
    if constexpr (WPR > 1) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
        __syncthreads();
        m = red[0];
#pragma unroll
        for (int w = 1; w < WPR; ++w) m = fmaxf(m, red[w]);
        __syncthreads();
    }
    return m;
}

constexpr int threads_of(int wpr) { return wpr > 4 ? 64 * wpr : 256; }

// P pieces per lane hold the row: F <= 64 WPR P piece<DT>().  P == 0: any F, the
// values computed once for the maximum and once more for the cast.
template <int DT, bool GATED, int WPR, int P>
__global__ __launch_bounds__(threads_of(WPR)) void act_quantize(const void* __restrict__ h, int64_t ldh, int64_t rows,
                                                                int64_t F, int act, uint8_t* __restrict__ q, int64_t ldq,
                                                                float* __restrict__ scales,
                                                                const int32_t* __restrict__ live_rows) {
    constexpr int V = piece<DT>();
    constexpr int ROWS = threads_of(WPR) / (64 * WPR);  // rows of a workgroup: 4, or 1
    __shared__ float red[WPR];
    if (live_rows != nullptr) rows = min(rows, (int64_t)max(*live_rows, 0));
    const int l = threadIdx.x % (64 * WPR);
    for (int64_t r = (int64_t)blockIdx.x * ROWS + threadIdx.x / (64 * WPR); r < rows; r += (int64_t)gridDim.x * ROWS) {
        float m = 0.0f;
        if constexpr (P > 0) {
            // Pieces past the row's end read its last one again (it changes no maximum) and
            // are not stored: all loads go out with no branch between them.
            Raw<GATED> raw[P];
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int64_t n = (int64_t)(i * 64 * WPR + l) * V;
                load_raw<DT, GATED>(h, r * ldh + min(n, F - V), F, raw[i]);
            }
            float v[P][V];
            with_act(act, [&](auto a) {
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    value_of<DT, GATED, decltype(a)::value>(raw[i], v[i]);
                    m = absmax<V>(m, v[i]);
                }
            });
            const RowScale rs = make_row_scale(row_max<WPR>(m, red));
            if (l == 0) scales[r] = rs.s;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int64_t n = (int64_t)(i * 64 * WPR + l) * V;
                if (n < F) store_codes<V>(q + r * ldq + n, v[i], rs);
            }
        } else {
            Raw<GATED> raw;
            float v[V];
            with_act(act, [&](auto a) {
                for (int64_t n = (int64_t)l * V; n < F; n += 64 * WPR * V) {
                    load_raw<DT, GATED>(h, r * ldh + n, F, raw);
                    value_of<DT, GATED, decltype(a)::value>(raw, v);
                    m = absmax<V>(m, v);
                }
            });
            const RowScale rs = make_row_scale(row_max<WPR>(m, red));
            if (l == 0) scales[r] = rs.s;
            with_act(act, [&](auto a) {
                for (int64_t n = (int64_t)l * V; n < F; n += 64 * WPR * V) {
                    load_raw<DT, GATED>(h, r * ldh + n, F, raw);
                    value_of<DT, GATED, decltype(a)::value>(raw, v);
                    store_codes<V>(q + r * ldq + n, v, rs);
                }
            });
        }
    }
}

// Rows of no elements: their scale alone.
__global__ __launch_bounds__(256) void act_quantize_empty(int64_t rows, float* __restrict__ scales,
                                                          const int32_t* __restrict__ live_rows) {
    if (live_rows != nullptr) rows = min(rows, (int64_t)max(*live_rows, 0));
    for (int64_t r = (int64_t)blockIdx.x * 256 + threadIdx.x; r < rows; r += (int64_t)gridDim.x * 256) scales[r] = kScaleFloor;
}

struct ActQuantize {
    const void* h;
    int64_t ldh, rows, F;
    int act;
    uint8_t* q;
    int64_t ldq;
    float* scales;
    const int32_t* live_rows;
};

template <int DT, bool GATED, int WPR, int P>
hipError_t launch_one(const ActQuantize& a, hipStream_t stream) {
    constexpr int ROWS = threads_of(WPR) / (64 * WPR);
    const int64_t groups = (a.rows + ROWS - 1) / ROWS;
    const dim3 grid((unsigned)(groups < (1 << 20) ? groups : 1 << 20));
    hipLaunchKernelGGL((act_quantize<DT, GATED, WPR, P>), grid, dim3(threads_of(WPR)), 0, stream, a.h, a.ldh, a.rows, a.F,
                       a.act, a.q, a.ldq, a.scales, a.live_rows);
    return hipGetLastError();
}

// From this many rows on the rows fill the card, and a wave takes as much of one as
// its registers hold; below it a row is spread over as many lanes as it has pieces
// (2048 bf16 elements, gated: 400 rows 4.4 us with 1024 threads a row, 2.9 with 256).
constexpr int64_t kManyRows = 512;

template <int DT, bool GATED>
hipError_t launch_typed(const ActQuantize& a, hipStream_t stream) {
    const int64_t pieces = a.F / piece<DT>();
    if (pieces <= 64) return launch_one<DT, GATED, 1, 1>(a, stream);
    if (a.rows >= kManyRows) {
        if (pieces <= 64 * 2) return launch_one<DT, GATED, 1, 2>(a, stream);
        if (pieces <= 64 * 4) return launch_one<DT, GATED, 1, 4>(a, stream);
        if (pieces <= 256 * 2) return launch_one<DT, GATED, 4, 2>(a, stream);
        if (pieces <= 256 * 4) return launch_one<DT, GATED, 4, 4>(a, stream);
        if (pieces <= 256 * 8) return launch_one<DT, GATED, 4, 8>(a, stream);
    } else if (pieces <= 256) {
        return launch_one<DT, GATED, 4, 1>(a, stream);
    }
    if (pieces <= 1024) return launch_one<DT, GATED, 16, 1>(a, stream);
    if (pieces <= 1024 * 2) return launch_one<DT, GATED, 16, 2>(a, stream);
    if (pieces <= 1024 * 4) return launch_one<DT, GATED, 16, 4>(a, stream);
    return launch_one<DT, GATED, 16, 0>(a, stream);
}

}  // namespace

hipError_t launch_act_quantize(const void* h, int64_t ldh, int dtype, int64_t rows, int64_t F, int act, bool gated,
                               uint8_t* q, int64_t ldq, float* scales, const int32_t* live_rows, hipStream_t stream) {
    if (rows <= 0) return hipSuccess;
    if (F == 0) {
        const int64_t groups = (rows + 255) / 256;
        hipLaunchKernelGGL(act_quantize_empty, dim3((unsigned)(groups < (1 << 20) ? groups : 1 << 20)), dim3(256), 0, stream,
                           rows, scales, live_rows);
        return hipGetLastError();
    }
    const ActQuantize a{h, ldh, rows, F, act, q, ldq, scales, live_rows};
    return with_type(dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        return gated ? launch_typed<DT, true>(a, stream) : launch_typed<DT, false>(a, stream);
    });
}

}  // namespace fp8k
