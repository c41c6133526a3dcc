// Rows of a mixture of experts on gfx950: the order of the tokens' choices by
// expert, tokens moved into that order, and the experts' rows brought back with
// their weights, with the gradient of that.
//
// Everything but the sort is a stream over rows, seen from the tokens: a token's
// row is read once and written to its topk places (permute), or its topk rows
// are read once and summed (combine).  No place is written twice and every sum
// runs over j = 0, 1, .. in fp32, so results do not depend on timing.
#include <algorithm>
#include <type_traits>

#include "rows_common.hpp"

namespace fp8k {

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ---------------------------------------------------------------- sort ----
//
// A stable counting sort of R = T * topk choices by expert.  Choices outside
// [0, E) take the key E: they come last and get no row.

template <typename ID>
__device__ __forceinline__ int key_of(ID id, int E) {
    return id >= 0 && id < (ID)E ? (int)id : E;
}

// Few choices: workgroup e of E + 1 reads them all, counts those below e (its
// first row) and those of e in front of each of its waves, and places its own in
// a second reading.  One launch and no workspace; E + 1 readings of the ids.
constexpr int kSortOneThreads = 1024;

template <typename ID, int T>
__global__ __launch_bounds__(T) void moe_sort_one(const ID* __restrict__ ids, int R, int topk, int E,
                                                  int32_t* __restrict__ offsets, int32_t* __restrict__ row_token,
                                                  int32_t* __restrict__ row_of) {
    constexpr int W = T / kWave;
    __shared__ int below[W], equal[W];
    const int e = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int per = ((R + W - 1) / W + 63) & ~63;  // choices of a wave, contiguous
    const int begin = min(R, wave * per), end = min(R, begin + per);
    int lt = 0, eq = 0;
    for (int i0 = begin; i0 < end; i0 += 64) {
        const int i = i0 + lane;
        const int key = i < end ? key_of(ids[i], E) : E + 1;
        lt += __popcll(__ballot(key < e));
        eq += __popcll(__ballot(key == e));
    }
    if (lane == 0) below[wave] = lt, equal[wave] = eq;
    __syncthreads();
    int row = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) row += below[w];
    if (threadIdx.x == 0) offsets[e] = row;
    for (int w = 0; w < wave; ++w) row += equal[w];
    for (int i0 = begin; i0 < end; i0 += 64) {
        const int i = i0 + lane;
        const bool mine = i < end && key_of(ids[i], E) == e;
        const unsigned long long all = __ballot(mine);
        if (mine) {
            const int r = row + __popcll(all & ((1ull << lane) - 1));
            row_of[i] = e < E ? r : -1;
            row_token[r] = e < E ? i / topk : -1;
        }
        row += __popcll(all);
    }
}

// Many choices: chunks of them, one per workgroup.  The first kernel counts each
// chunk's keys; the second adds up the chunks' counts to every key's first row in
// its own chunk, and places the chunk's choices in order.
constexpr int kSortThreads = 512;
constexpr int kSortWaves = kSortThreads / kWave;
constexpr int kSortKeys = 1025;  // E <= 1024 and the key of choices without an expert
constexpr int kSortPerKey = (kSortKeys + kSortThreads - 1) / kSortThreads;

template <typename ID>
__global__ __launch_bounds__(kSortThreads) void moe_sort_count(const ID* __restrict__ ids, int R, int chunk, int E,
                                                               int* __restrict__ counts) {
    __shared__ int cnt[kSortKeys];
    for (int k = threadIdx.x; k <= E; k += kSortThreads) cnt[k] = 0;
    __syncthreads();
    const int64_t begin = (int64_t)blockIdx.x * chunk, end = min((int64_t)R, begin + chunk);
    for (int64_t i = begin + threadIdx.x; i < end; i += kSortThreads) atomicAdd(&cnt[key_of(ids[i], E)], 1);
    __syncthreads();
    for (int k = threadIdx.x; k <= E; k += kSortThreads) counts[(int64_t)blockIdx.x * (E + 1) + k] = cnt[k];
}

template <typename ID>
__global__ __launch_bounds__(kSortThreads) void moe_sort_place(const ID* __restrict__ ids, int R, int chunk, int topk,
                                                               int E, int key_bits, const int* __restrict__ counts,
                                                               int32_t* __restrict__ offsets,
                                                               int32_t* __restrict__ row_token,
                                                               int32_t* __restrict__ row_of) {
    __shared__ int next[kSortWaves][kSortKeys];  // the next row of a key in a wave's part of the chunk
    __shared__ int wave_sum[kSortWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int keys = E + 1;
    for (int k = threadIdx.x; k < kSortWaves * kSortKeys; k += kSortThreads) (&next[0][0])[k] = 0;
    __syncthreads();
    const int64_t base = (int64_t)blockIdx.x * chunk;
    const int64_t chunk_end = min((int64_t)R, base + chunk);
    const int per = chunk / kSortWaves;  // a multiple of 64
    const int64_t begin = min(chunk_end, base + (int64_t)wave * per), end = min(chunk_end, begin + per);
    for (int64_t i = begin + lane; i < end; i += 64) atomicAdd(&next[wave][key_of(ids[i], E)], 1);

    // Every key's count in all chunks and in those before this one; thread t takes
    // the keys t * kSortPerKey + j, so that the scan over keys is one over threads.
    int total[kSortPerKey], before[kSortPerKey], sum = 0;
#pragma unroll
    for (int j = 0; j < kSortPerKey; ++j) {
        total[j] = before[j] = 0;
        const int k = threadIdx.x * kSortPerKey + j;
        if (k < keys)
            for (int b = 0; b < (int)gridDim.x; ++b) {
                const int c = counts[(int64_t)b * keys + k];
                total[j] += c;
                before[j] += b < (int)blockIdx.x ? c : 0;
            }
        sum += total[j];
    }
    int incl = sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int v = __shfl_up(incl, off, 64);
        if (lane >= off) incl += v;
    }
    if (lane == 63) wave_sum[wave] = incl;
    __syncthreads();  // also: next[] holds the counts of every wave
    int first = incl - sum;
    for (int w = 0; w < wave; ++w) first += wave_sum[w];
#pragma unroll
    for (int j = 0; j < kSortPerKey; ++j) {
        const int k = threadIdx.x * kSortPerKey + j;
        if (k < keys) {
            if (blockIdx.x == 0) offsets[k] = first;
            int row = first + before[j];
#pragma unroll
            for (int w = 0; w < kSortWaves; ++w) {
                const int c = next[w][k];
                next[w][k] = row;
                row += c;
            }
        }
        first += total[j];
    }
    __syncthreads();

    for (int64_t i0 = begin; i0 < end; i0 += 64) {
        const int64_t i = i0 + lane;
        const bool live = i < end;
        const int key = live ? key_of(ids[i], E) : E;
        // the lanes of the same key
        unsigned long long same = __ballot(live);
        for (int b = 0; b < key_bits; ++b) {
            const unsigned long long set = __ballot((key >> b) & 1);
            same &= (key >> b) & 1 ? set : ~set;
        }
        if (live) {
            const int r = next[wave][key] + __popcll(same & ((1ull << lane) - 1));
            row_of[i] = key < E ? r : -1;
            row_token[r] = key < E ? (int32_t)((uint32_t)i / (uint32_t)topk) : -1;
            if ((same >> lane) == 1) next[wave][key] = r + 1;  // the last of them
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// ---------------------------------------------------------------- permute ----
//
// A workgroup's threads cover `lanes` 16-byte pieces of 256 / lanes tokens.

constexpr int kRowThreads = 256;

__global__ __launch_bounds__(kRowThreads) void moe_permute(const uint8_t* __restrict__ x, int64_t ldx,
                                                           const float* __restrict__ s_tok,
                                                           const int32_t* __restrict__ row_of, int T, int topk, int R,
                                                           int64_t row_bytes, int lane_bits, uint8_t* __restrict__ out,
                                                           int64_t ldo, float* __restrict__ s_out) {
    const int lanes = 1 << lane_bits;
    const int l = threadIdx.x & (lanes - 1);
    const int per_block = kRowThreads >> lane_bits;
    for (int64_t t = (int64_t)blockIdx.x * per_block + (threadIdx.x >> lane_bits); t < T;
         t += (int64_t)gridDim.x * per_block) {
        const int32_t* rows = row_of + t * topk;
        const uint8_t* src = x + t * ldx;
        if (s_tok != nullptr)
            for (int j = l; j < topk; j += lanes)
                if ((uint32_t)rows[j] < (uint32_t)R) s_out[rows[j]] = s_tok[t];
        for (int64_t b = 16 * (int64_t)l; b < row_bytes; b += 16 * (int64_t)lanes) {
            if (b + 16 <= row_bytes) {
                uint32_t w[4];
                load_words(src + b, w);
                for (int j = 0; j < topk; ++j)
                    if ((uint32_t)rows[j] < (uint32_t)R) store_words(out + (int64_t)rows[j] * ldo + b, w);
            } else {
                for (int64_t i = b; i < row_bytes; ++i) {
                    const uint8_t v = src[i];
                    for (int j = 0; j < topk; ++j)
                        if ((uint32_t)rows[j] < (uint32_t)R) out[(int64_t)rows[j] * ldo + i] = v;
                }
            }
        }
    }
}

// ---------------------------------------------------------------- combine ----

template <int DT, int ODT, int U>
__global__ __launch_bounds__(kRowThreads) void moe_combine(MoeCombine p, int lane_bits) {
    constexpr int V = 16 / elem_size<DT>();
    const int lanes = 1 << lane_bits;
    const int l = threadIdx.x & (lanes - 1);
    const int per_block = kRowThreads >> lane_bits;
    for (int64_t t = (int64_t)blockIdx.x * per_block + (threadIdx.x >> lane_bits); t < p.T;
         t += (int64_t)gridDim.x * per_block) {
        for (int64_t n = (int64_t)V * l; n < p.H; n += (int64_t)V * lanes) {
            const int left = (int)min((int64_t)V, p.H - n);
            float acc[V];
            if (p.residual != nullptr) {
                load_run<ODT, V>(p.residual, t * p.ldr + n, left, acc);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] = 0.0f;
            }
            for (int j0 = 0; j0 < p.topk; j0 += U) {
                float v[U][V], w[U];
                bool live[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int j = min(j0 + u, p.topk - 1);
                    const int r = p.row_of[t * p.topk + j];
                    live[u] = j0 + u < p.topk && (uint32_t)r < (uint32_t)p.R;
                    w[u] = p.weights != nullptr ? p.weights[t * p.topk + j] : 1.0f;
                    // a choice without a row reads row 0 and leaves it unused
                    load_run<DT, V>(p.y, (live[u] ? (int64_t)r : 0) * p.ldy + n, left, v[u]);
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (live[u]) {
#pragma unroll
                        for (int i = 0; i < V; ++i) acc[i] = __builtin_fmaf(w[u], v[u][i], acc[i]);
                    }
            }
            store_run<ODT, V>(p.out, t * p.ldo + n, left, acc);
        }
    }
}

// The gradient: choice (t, j) of row r writes dy[r] = w dout[t] and its weight's
// gradient <dout[t], y[r]>.  `lanes` neighbouring threads take a choice, so the
// topk readings of dout[t] happen side by side and all but one come from cache.
template <int DT, int YDT>
__global__ __launch_bounds__(kRowThreads) void moe_combine_grad(MoeCombineGrad p, int lane_bits) {
    constexpr int V = 16 / elem_size<YDT>();
    __shared__ float part[kRowThreads / kWave];
    const int lanes = 1 << lane_bits;
    const int l = threadIdx.x & (lanes - 1);
    const int per_block = kRowThreads >> lane_bits;
    const int64_t choices = (int64_t)p.T * p.topk;
    for (int64_t c0 = (int64_t)blockIdx.x * per_block; c0 < choices; c0 += (int64_t)gridDim.x * per_block) {
        const int64_t c = c0 + (threadIdx.x >> lane_bits);
        const int r = c < choices ? p.row_of[c] : -1;
        float dot = 0.0f;
        if ((uint32_t)r < (uint32_t)p.R) {
            const int64_t t = c / p.topk;
            const float w = p.weights != nullptr ? p.weights[c] : 1.0f;
            for (int64_t n = (int64_t)V * l; n < p.H; n += (int64_t)V * lanes) {
                const int left = (int)min((int64_t)V, p.H - n);
                float d[V], y[V];
                load_run<DT, V>(p.dout, t * p.ldd + n, left, d);
                if (p.dweights != nullptr) {
                    load_run<YDT, V>(p.y, (int64_t)r * p.ldy + n, left, y);
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (i < left) dot = __builtin_fmaf(d[i], y[i], dot);
                }
                if (p.dy != nullptr) {
#pragma unroll
                    for (int i = 0; i < V; ++i) d[i] *= w;
                    store_run<YDT, V>(p.dy, (int64_t)r * p.lddy + n, left, d);
                }
            }
        }
        if (p.dweights != nullptr) {
            for (int off = min(lanes, 64) >> 1; off > 0; off >>= 1) dot += __shfl_xor(dot, off, kWave);
            if (lanes > kWave) {  // a choice of several waves: their sums in order
                if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = dot;
                __syncthreads();
                const int first = (threadIdx.x >> lane_bits) << (lane_bits - 6);
                dot = part[first];
                for (int w = 1; w < lanes / kWave; ++w) dot += part[first + w];
                __syncthreads();
            }
            if (l == 0 && c < choices) p.dweights[c] = dot;
        }
    }
}

int bits_for(int64_t pieces, int most) {
    int b = 0;
    while (b < most && (int64_t(1) << b) < pieces) ++b;
    return b;
}

// Workgroups for `groups` of them, further ones by looping.
dim3 row_grid(int64_t groups) { return dim3((unsigned)std::min<int64_t>(std::max<int64_t>(groups, 1), 1 << 20)); }

}  // namespace

// One launch up to here: the ids are read E + 1 times.
constexpr int64_t kSortOneWork = 4 << 20;
constexpr int64_t kSortOneMax = 65536;

static bool sort_one(int64_t R, int64_t E) { return R <= kSortOneMax && R * (E + 1) <= kSortOneWork; }

// Chunks of whole waves' steps, at least 4096 choices and at most 256 of them.
static int64_t sort_chunk(int64_t R) {
    const int64_t step = kSortWaves * kWave;
    return std::max<int64_t>(4096, ceil_div(ceil_div(R, 256), step) * step);
}

size_t moe_sort_ws_bytes(int64_t R, int64_t E) {
    return sort_one(R, E) ? 0 : (size_t)ceil_div(R, sort_chunk(R)) * (size_t)(E + 1) * sizeof(int);
}

template <typename ID>
static hipError_t launch_sort(const ID* ids, int64_t R, int64_t topk, int64_t E, int32_t* offsets, int32_t* row_token,
                              int32_t* row_of, void* ws, hipStream_t stream) {
    if (sort_one(R, E)) {
        if (R <= 4096)
            hipLaunchKernelGGL((moe_sort_one<ID, 256>), dim3((unsigned)(E + 1)), dim3(256), 0, stream, ids, (int)R,
                               (int)topk, (int)E, offsets, row_token, row_of);
        else
            hipLaunchKernelGGL((moe_sort_one<ID, kSortOneThreads>), dim3((unsigned)(E + 1)), dim3(kSortOneThreads), 0,
                               stream, ids, (int)R, (int)topk, (int)E, offsets, row_token, row_of);
        return hipGetLastError();
    }
    const int64_t chunk = sort_chunk(R);
    const dim3 grid((unsigned)ceil_div(R, chunk));
    int* counts = static_cast<int*>(ws);
    hipLaunchKernelGGL((moe_sort_count<ID>), grid, dim3(kSortThreads), 0, stream, ids, (int)R, (int)chunk, (int)E, counts);
    hipLaunchKernelGGL((moe_sort_place<ID>), grid, dim3(kSortThreads), 0, stream, ids, (int)R, (int)chunk, (int)topk,
                       (int)E, bits_for(E + 1, 31), counts, offsets, row_token, row_of);
    return hipGetLastError();
}

hipError_t launch_moe_sort(const void* ids, bool wide, int64_t R, int64_t topk, int64_t E, int32_t* offsets,
                           int32_t* row_token, int32_t* row_of, void* ws, hipStream_t stream) {
    return wide ? launch_sort(static_cast<const int64_t*>(ids), R, topk, E, offsets, row_token, row_of, ws, stream)
                : launch_sort(static_cast<const int32_t*>(ids), R, topk, E, offsets, row_token, row_of, ws, stream);
}

hipError_t launch_moe_permute(const void* x, int64_t ldx_bytes, const float* s_tok, const int32_t* row_of, int64_t T,
                              int64_t topk, int64_t R, int64_t row_bytes, void* out, int64_t ldo_bytes, float* s_out,
                              hipStream_t stream) {
    const int bits = bits_for(ceil_div(row_bytes, 16), 8);
    hipLaunchKernelGGL(moe_permute, row_grid(ceil_div(T, kRowThreads >> bits)), dim3(kRowThreads), 0, stream,
                       static_cast<const uint8_t*>(x), ldx_bytes, s_tok, row_of, (int)T, (int)topk, (int)R, row_bytes,
                       bits, static_cast<uint8_t*>(out), ldo_bytes, s_out);
    return hipGetLastError();
}

hipError_t launch_moe_combine(const MoeCombine& p, int dtype, int out_dtype, hipStream_t stream) {
    return with_type(dtype, [&](auto dt) {
        return with_type(out_dtype, [&](auto odt) {
            constexpr int DT = decltype(dt)::value, ODT = decltype(odt)::value;
            const int bits = bits_for(ceil_div(p.H, 16 / elem_size<DT>()), 8);
            const dim3 grid = row_grid(ceil_div(p.T, kRowThreads >> bits));
            if (p.topk <= 1)
                hipLaunchKernelGGL((moe_combine<DT, ODT, 1>), grid, dim3(kRowThreads), 0, stream, p, bits);
            else if (p.topk <= 2)
                hipLaunchKernelGGL((moe_combine<DT, ODT, 2>), grid, dim3(kRowThreads), 0, stream, p, bits);
            else if (p.topk <= 4)
                hipLaunchKernelGGL((moe_combine<DT, ODT, 4>), grid, dim3(kRowThreads), 0, stream, p, bits);
            else
                hipLaunchKernelGGL((moe_combine<DT, ODT, 8>), grid, dim3(kRowThreads), 0, stream, p, bits);
            return hipGetLastError();
        });
    });
}

hipError_t launch_moe_combine_grad(const MoeCombineGrad& p, int dtype, int y_dtype, hipStream_t stream) {
    return with_type(dtype, [&](auto dt) {
        return with_type(y_dtype, [&](auto ydt) {
            constexpr int DT = decltype(dt)::value, YDT = decltype(ydt)::value;
            const int64_t choices = (int64_t)p.T * p.topk;
            const int bits = bits_for(ceil_div(p.H, 16 / elem_size<YDT>()), choices < 1024 ? 8 : 6);
            hipLaunchKernelGGL((moe_combine_grad<DT, YDT>), row_grid(ceil_div(choices, kRowThreads >> bits)),
                               dim3(kRowThreads), 0, stream, p, bits);
            return hipGetLastError();
        });
    });
}

}  // namespace fp8k
