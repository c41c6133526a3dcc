// Activation and per-token E4M3 quantization in one pass on gfx950: the step
// between a feed-forward layer's two FP8 products.
//
//   v = act(g) * u (gated: a row holds F of g, then F of u), or act(h)
//   s = max(fl32(max |v| / 448), 1e-12f), codes E4M3(fl32(v / s)), RNE
//
// in fp32 from the row's own type, so the product of the activation is never
// rounded to 16 bits.  A row is read once: its values stay in registers between
// the maximum and the cast.  WPR waves share a row; one wave per row needs no
// LDS and no barrier, and takes over as soon as there are rows enough.
#include <type_traits>

#include "rows_common.hpp"

namespace fp8k {

namespace {

template <int DT>
constexpr int piece() {  // elements of a 16-byte piece
    return 16 / elem_size<DT>();
}

template <int DT, bool GATED>
__device__ __forceinline__ void load_value(const void* h, int64_t e, int64_t F, int act, float (&v)[piece<DT>()]) {
    constexpr int V = piece<DT>();
    load_run<DT, V>(h, e, V, v);
    activate<V>(v, act);
    if constexpr (GATED) {
        float u[V];
        load_run<DT, V>(h, e + F, V, u);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] *= u[i];
    }
}

template <int V>
__device__ __forceinline__ float absmax(float m, const float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) m = fmaxf(m, fabsf(v[i]));
    return m;
}

template <int V>
__device__ __forceinline__ void store_codes(uint8_t* q, const float (&v)[V], const RowScale& rs) {
    uint32_t w[V / 4];
#pragma unroll
    for (int i = 0; i < V / 4; ++i)
        w[i] = cast4(make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]), rs);
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
            float v[P][V];
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int64_t n = (int64_t)(i * 64 * WPR + l) * V;
                if (n < F) {
                    load_value<DT, GATED>(h, r * ldh + n, F, act, v[i]);
                    m = absmax<V>(m, v[i]);
                }
            }
            const RowScale rs = make_row_scale(row_max<WPR>(m, red));
            if (l == 0) scales[r] = rs.s;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int64_t n = (int64_t)(i * 64 * WPR + l) * V;
                if (n < F) store_codes<V>(q + r * ldq + n, v[i], rs);
            }
        } else {
            float v[V];
            for (int64_t n = (int64_t)l * V; n < F; n += 64 * WPR * V) {
                load_value<DT, GATED>(h, r * ldh + n, F, act, v);
                m = absmax<V>(m, v);
            }
            const RowScale rs = make_row_scale(row_max<WPR>(m, red));
            if (l == 0) scales[r] = rs.s;
            for (int64_t n = (int64_t)l * V; n < F; n += 64 * WPR * V) {
                load_value<DT, GATED>(h, r * ldh + n, F, act, v);
                store_codes<V>(q + r * ldq + n, v, rs);
            }
        }
    }
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

// Below this many rows a row is shared by 16 waves: fewer waves would leave most
// of the card idle.
constexpr int64_t kWideRowsBelow = 512;

template <int DT, bool GATED>
hipError_t launch_typed(const ActQuantize& a, hipStream_t stream) {
    const int64_t pieces = a.F / piece<DT>();
#define FP8K_ACT_Q(WPR)                                                            \
    if (pieces <= 64 * WPR) return launch_one<DT, GATED, WPR, 1>(a, stream);       \
    if (pieces <= 64 * WPR * 2) return launch_one<DT, GATED, WPR, 2>(a, stream);   \
    if (pieces <= 64 * WPR * 4) return launch_one<DT, GATED, WPR, 4>(a, stream);   \
    if (pieces <= 64 * WPR * 8) return launch_one<DT, GATED, WPR, 8>(a, stream);
    if (a.rows >= kWideRowsBelow) {
        FP8K_ACT_Q(1)
        FP8K_ACT_Q(4)
    }
    FP8K_ACT_Q(16)
#undef FP8K_ACT_Q
    return launch_one<DT, GATED, 16, 0>(a, stream);
}

}  // namespace

hipError_t launch_act_quantize(const void* h, int64_t ldh, int dtype, int64_t rows, int64_t F, int act, bool gated,
                               uint8_t* q, int64_t ldq, float* scales, const int32_t* live_rows, hipStream_t stream) {
    if (rows <= 0) return hipSuccess;
    const ActQuantize a{h, ldh, rows, F, act, q, ldq, scales, live_rows};
    return with_type(dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        return gated ? launch_typed<DT, true>(a, stream) : launch_typed<DT, false>(a, stream);
    });
}

}  // namespace fp8k
