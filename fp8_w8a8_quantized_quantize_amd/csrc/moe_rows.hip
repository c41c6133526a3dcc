// Rows of a mixture of experts on gfx950: the order of the tokens' choices by
// expert, tokens moved into that order, and the experts' rows brought back with
// their weights, with the gradient of that.
//
// Everything but the sort is a stream over rows, seen from the tokens: a token's
// row is read once and written to its topk places (permute), or its topk rows
// are read once and summed (combine).  No place is written twice and every sum
// runs over j = 0, 1, .. in fp32, so results do not depend on timing.  Memory
// bounds them: 4096 x 8 rows of 7168, permute of codes 52 us (5.1 TB/s), combine of
// bf16 rows onto a residual 110 us (5.3 TB/s, a plain copy's rate), its gradient
// 197 us (5.1 TB/s); 1777 x 6 rows of 4999 fp16 elements, none of them aligned, 52 us
// (4.1 TB/s).
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

// Few choices: the workgroups of expert e (of E + 1) read them all, count those below
// e (its first row) and those of e in front of each of their waves, and place its
// own.  A wave holds its part of the choices in registers, KEYS per lane, so they
// are read once, with all loads in flight together.  `parts` workgroups of an expert
// do the same and share the placing, each taking every parts-th step of a wave: a
// step's scattered stores cost more than its counting.  One launch, no workspace.
constexpr int kSortOneThreads = 1024;

// Choices a lane takes side by side: 16 bytes.
template <typename ID>
constexpr int ids_per_load() {
    return 16 / (int)sizeof(ID);
}

template <typename ID, int T, int KEYS>
__global__ __launch_bounds__(T) void moe_sort_one(const ID* __restrict__ ids, int R, uint32_t per_topk, int E,
                                                  int parts, int32_t* __restrict__ offsets, int32_t* __restrict__ row_token,
                                                  int32_t* __restrict__ row_of) {
    constexpr int W = T / kWave, V = ids_per_load<ID>(), STEPS = KEYS / V;
    static_assert(KEYS % V == 0, "whole loads");
    typedef ID idv __attribute__((ext_vector_type(V)));
    __shared__ int below[W], equal[W];
    const int e = blockIdx.x / parts, part = blockIdx.x % parts;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int begin = wave * (64 * KEYS) + lane * V;  // of this lane's first load; further ones 64 V apart
    int key[STEPS][V];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const int i = begin + s * 64 * V;
        if (i + V <= R) {
            const idv id = *reinterpret_cast<const idv*>(ids + i);
#pragma unroll
            for (int v = 0; v < V; ++v) key[s][v] = key_of((ID)id[v], E);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) key[s][v] = i + v < R ? key_of(ids[i + v], E) : E + 1;
        }
    }
    int lt = 0, eq = 0;
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
        for (int v = 0; v < V; ++v) lt += key[s][v] < e, eq += key[s][v] == e;
    int sum = lt | eq << 16;  // a wave has fewer than 2^16 choices
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off, kWave);
    if (lane == 0) below[wave] = sum & 0xFFFF, equal[wave] = sum >> 16;
    __syncthreads();
    int row = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) row += below[w];
    if (threadIdx.x == 0 && part == 0) offsets[e] = row;
#pragma unroll
    for (int w = 0; w < W; ++w) row += w < wave ? equal[w] : 0;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        unsigned long long mine[V];
        unsigned long long any = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) mine[v] = __ballot(key[s][v] == e), any |= mine[v];
        int r = row;
#pragma unroll
        for (int v = 0; v < V; ++v) row += __popcll(mine[v]);
        if (any == 0 || s % parts != part) continue;
#pragma unroll
        for (int v = 0; v < V; ++v) r += __popcll(mine[v] & ((1ull << lane) - 1));
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (key[s][v] == e) {
                const uint32_t i = begin + s * 64 * V + v;
                row_of[i] = e < E ? r : -1;
                // i / topk: i topk < 2^32, so the rounded-up reciprocal gives the quotient
                row_token[r] = e < E ? (int32_t)(per_topk != 0 ? __umulhi(i, per_topk) : i) : -1;
                ++r;
            }
        }
    }
}

// Many choices: chunks of them, one per workgroup.  The first kernel counts each
// chunk's keys; the second adds up the chunks' counts to every key's first row in
// its own chunk, and places the chunk's choices in order.
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / kWave;
constexpr int kSortKeys = 1025;  // E <= 1024 and the key of choices without an expert
constexpr int kSortAhead = 4;    // steps of 64 choices loaded together
constexpr int kCountAhead = 4;   // choices of a thread counted together
constexpr int kChunksAhead = 32; // chunks' counts of a key added together

// cnt[key] += 1 for every lane with a key (not -1).  A wave of one key alone (the
// padding at a buffer's end) adds once: its lanes' additions would wait for each other.
__device__ __forceinline__ void count_key(int* cnt, int key) {
    const int one = __builtin_amdgcn_readfirstlane(key);
    const unsigned long long live = __ballot(key >= 0);
    if (one >= 0 && __ballot(key == one) == live) {
        if ((threadIdx.x & 63) == 0) atomicAdd(&cnt[one], __popcll(live));
    } else if (key >= 0) {
        atomicAdd(&cnt[key], 1);
    }
}

template <typename ID>
__global__ __launch_bounds__(kSortThreads) void moe_sort_count(const ID* __restrict__ ids, int R, int chunk, int E,
                                                               int* __restrict__ counts) {
    __shared__ int cnt[kSortKeys];
    for (int k = threadIdx.x; k <= E; k += kSortThreads) cnt[k] = 0;
    __syncthreads();
    const int64_t begin = (int64_t)blockIdx.x * chunk, end = min((int64_t)R, begin + chunk);
    for (int64_t i0 = begin; i0 < end; i0 += kCountAhead * kSortThreads) {
        const int64_t i = i0 + threadIdx.x;
        ID id[kCountAhead];  // read again past the end, and not counted: no branch between the loads
#pragma unroll
        for (int a = 0; a < kCountAhead; ++a) id[a] = ids[min(i + a * kSortThreads, end - 1)];
#pragma unroll
        for (int a = 0; a < kCountAhead; ++a)
            count_key(cnt, i + a * kSortThreads < end ? key_of(id[a], E) : -1);
    }
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
    __shared__ int total[kSortKeys], before[kSortKeys];
    __shared__ int wave_sum[kSortWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int keys = E + 1;
    for (int k = lane; k < keys; k += 64) next[wave][k] = 0;
    for (int k = threadIdx.x; k < keys; k += kSortThreads) total[k] = before[k] = 0;
    const int64_t base = (int64_t)blockIdx.x * chunk;
    const int64_t chunk_end = min((int64_t)R, base + chunk);
    const int per = chunk / kSortWaves;  // a multiple of 64 kSortAhead
    const int64_t begin = min(chunk_end, base + (int64_t)wave * per), end = min(chunk_end, begin + per);
    auto load_keys = [&](int64_t i0, int (&key)[kSortAhead]) {
        ID id[kSortAhead];  // no branch between the loads, as in the count
#pragma unroll
        for (int a = 0; a < kSortAhead; ++a) id[a] = ids[min(i0 + a * 64 + lane, end - 1)];
#pragma unroll
        for (int a = 0; a < kSortAhead; ++a) key[a] = i0 + a * 64 + lane < end ? key_of(id[a], E) : -1;
    };
    __syncthreads();
    for (int64_t i0 = begin; i0 < end; i0 += 64 * kSortAhead) {
        int key[kSortAhead];
        load_keys(i0, key);
#pragma unroll
        for (int a = 0; a < kSortAhead; ++a)
            count_key(next[wave], key[a]);
    }
    // Every key's count in all chunks and in those before this one.  Threads side by
    // side take neighbouring keys of one chunk; when the keys leave threads over,
    // groups of threads take every group-th chunk.
    const int wide = min(kSortThreads, (keys + 63) & ~63), groups = kSortThreads / wide;
    const int group = threadIdx.x / wide;
    if (group < groups) {
        for (int k = threadIdx.x - group * wide; k < keys; k += wide) {
            int all = 0, front = 0;
            for (int b0 = group; b0 < (int)gridDim.x; b0 += groups * kChunksAhead) {
                int c[kChunksAhead];
#pragma unroll
                for (int a = 0; a < kChunksAhead; ++a)
                    c[a] = counts[(int64_t)min(b0 + a * groups, (int)gridDim.x - 1) * keys + k];
#pragma unroll
                for (int a = 0; a < kChunksAhead; ++a) {
                    const int b = b0 + a * groups;
                    all += b < (int)gridDim.x ? c[a] : 0;
                    front += b < (int)blockIdx.x ? c[a] : 0;
                }
            }
            atomicAdd(&total[k], all);
            atomicAdd(&before[k], front);
        }
    }
    __syncthreads();
    // Keys' first rows: thread t scans the keys [t n, (t + 1) n).
    const int n = (keys + kSortThreads - 1) / kSortThreads;
    int sum = 0;
    for (int k = threadIdx.x * n; k < min(keys, ((int)threadIdx.x + 1) * n); ++k) sum += total[k];
    int incl = sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int v = __shfl_up(incl, off, 64);
        if (lane >= off) incl += v;
    }
    if (lane == 63) wave_sum[wave] = incl;
    __syncthreads();
    int first = incl - sum;
    for (int w = 0; w < wave; ++w) first += wave_sum[w];
    for (int k = threadIdx.x * n; k < min(keys, ((int)threadIdx.x + 1) * n); ++k) {
        if (blockIdx.x == 0) offsets[k] = first;
        int row = first + before[k];
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
            const int c = next[w][k];
            next[w][k] = row;
            row += c;
        }
        first += total[k];
    }
    __syncthreads();

    for (int64_t i0 = begin; i0 < end; i0 += 64 * kSortAhead) {
        int keys_ahead[kSortAhead];
        load_keys(i0, keys_ahead);
#pragma unroll
        for (int a = 0; a < kSortAhead; ++a) {
            const int64_t i = i0 + a * 64 + lane;
            const int key = keys_ahead[a];
            // the lanes of the same key
            unsigned long long same = __ballot(key >= 0);
            for (int b = 0; b < key_bits; ++b) {
                const unsigned long long set = __ballot((key >> b) & 1);
                same &= (key >> b) & 1 ? set : ~set;
            }
            if (key >= 0) {
                const int r = next[wave][key] + __popcll(same & ((1ull << lane) - 1));
                row_of[i] = key < E ? r : -1;
                row_token[r] = key < E ? (int32_t)((uint32_t)i / (uint32_t)topk) : -1;
                if ((same >> lane) == 1) next[wave][key] = r + 1;  // the last of them
            }
            __builtin_amdgcn_wave_barrier();
        }
    }
}

// ---------------------------------------------------------------- permute ----
//
// Lanes side by side take 16-byte pieces of a row: a wave 64 of one token's (a task
// is then a token and one of its 64-piece columns), or, where a row has fewer, its
// lanes 2^bits each of several tokens'.  A lane's piece is all it does, so its loads
// are in flight together and rows of any length leave no lanes idle but in their
// last column.

constexpr int kRowThreads = 256;

struct RowTasks {
    int bits;      // lanes of a task: 2^bits
    int64_t cols;  // tasks of a row
};

// Task `u` of this lane's group: its row and the lane's piece in it.
struct RowTask {
    int64_t row, piece;
};

__device__ __forceinline__ int64_t first_task(const RowTasks& k) {
    return (int64_t)blockIdx.x * (kRowThreads >> k.bits) + (threadIdx.x >> k.bits);
}
__device__ __forceinline__ int64_t task_stride(const RowTasks& k) {
    return (int64_t)gridDim.x * (kRowThreads >> k.bits);
}
// WAVE: k.bits is 6.  The task is then the same for the whole wave, and said to be
// so: its indices and weights come by scalar loads.
template <bool WAVE>
__device__ __forceinline__ RowTask row_task(const RowTasks& k, int64_t u) {
    if constexpr (WAVE)
        u = (int64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)u) |
            (int64_t)__builtin_amdgcn_readfirstlane((int)(u >> 32)) << 32;
    const int64_t row = k.cols == 1 ? u : u / k.cols;
    return {row, ((u - row * k.cols) << k.bits) + (threadIdx.x & ((1 << k.bits) - 1))};
}

template <bool WAVE>
__global__ __launch_bounds__(kRowThreads) void moe_permute(const uint8_t* __restrict__ x, int64_t ldx,
                                                           const float* __restrict__ s_tok,
                                                           const int32_t* __restrict__ row_of, int64_t tasks, int topk,
                                                           int R, int64_t row_bytes, RowTasks k,
                                                           uint8_t* __restrict__ out, int64_t ldo,
                                                           float* __restrict__ s_out) {
    for (int64_t u = first_task(k); u < tasks; u += task_stride(k)) {
        const RowTask at = row_task<WAVE>(k, u);
        const int32_t* rows = row_of + at.row * topk;
        const uint8_t* src = x + at.row * ldx;
        const int64_t b = 16 * at.piece;
        if (s_tok != nullptr && at.piece < topk)
            for (int64_t j = at.piece; j < topk; j += k.cols << k.bits)
                if ((uint32_t)rows[j] < (uint32_t)R) s_out[rows[j]] = s_tok[at.row];
        if (b >= row_bytes) continue;
        if (row_bytes >= 16) {
            // a row's last piece overlaps the one before it: both write the same bytes there
            const int64_t at0 = min(b, row_bytes - 16);
            uint32_t w[4];
            load_words(src + at0, w);
            for (int j = 0; j < topk; ++j)
                if ((uint32_t)rows[j] < (uint32_t)R) store_words(out + (int64_t)rows[j] * ldo + at0, w);
        } else {
            for (int64_t i = 0; i < row_bytes; ++i) {
                const uint8_t v = src[i];
                for (int j = 0; j < topk; ++j)
                    if ((uint32_t)rows[j] < (uint32_t)R) out[(int64_t)rows[j] * ldo + i] = v;
            }
        }
    }
}

// ---------------------------------------------------------------- combine ----

// U choices' pieces are in flight together: loads before anything that waits for
// one, and no branch between them.  A row's last piece reaches back over the one
// before it and stores only the elements that are its own (what it reads of the
// others may have been written already, where the residual is the output).  Rows
// shorter than a piece go element by element.
template <int DT, int ODT, int U, bool WAVE>
__global__ __launch_bounds__(kRowThreads) void moe_combine(MoeCombine p, int64_t tasks, RowTasks k) {
    constexpr int V = 16 / elem_size<DT>();
    for (int64_t u0 = first_task(k); u0 < tasks; u0 += task_stride(k)) {
        const RowTask at = row_task<WAVE>(k, u0);
        const int64_t t = at.row, own = V * at.piece;
        const int32_t* rows = p.row_of + t * p.topk;
        const float* weights = p.weights != nullptr ? p.weights + t * p.topk : nullptr;
        if (own >= p.H) continue;
        if (p.H >= V) {
            const int64_t n = min(own, p.H - V);
            uint32_t res[V * elem_size<ODT>() / 4];
            float acc[V];
            if (p.residual != nullptr) {
                load_words(static_cast<const uint8_t*>(p.residual) + (t * p.ldr + n) * elem_size<ODT>(), res);
            } else {
#pragma unroll
                for (int i = 0; i < V * elem_size<ODT>() / 4; ++i) res[i] = 0;
            }
            auto choices = [&](int j0, bool first) {
                int r[U];
                float w[U];
                uint32_t raw[U][4];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int j = min(j0 + u, p.topk - 1);
                    r[u] = rows[j];
                    r[u] = j0 + u < p.topk && (uint32_t)r[u] < (uint32_t)p.R ? r[u] : -1;
                }
                if (weights != nullptr) {
#pragma unroll
                    for (int u = 0; u < U; ++u) w[u] = weights[min(j0 + u, p.topk - 1)];
                }
                // a choice without a row reads row 0 and leaves it unused
#pragma unroll
                for (int u = 0; u < U; ++u)
                    load_words(static_cast<const uint8_t*>(p.y) + ((int64_t)max(r[u], 0) * p.ldy + n) * elem_size<DT>(), raw[u]);
                if (first) unpack<ODT, V>(res, acc);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (r[u] < 0) continue;
                    float v[V];
                    unpack<DT, V>(raw[u], v);
                    const float wu = weights != nullptr ? w[u] : 1.0f;
#pragma unroll
                    for (int i = 0; i < V; ++i) acc[i] = __builtin_fmaf(wu, v[i], acc[i]);
                }
            };
            if (p.topk > 0)
                choices(0, true);
            else
                unpack<ODT, V>(res, acc);
            for (int j0 = U; j0 < p.topk; j0 += U) choices(j0, false);
            if (n == own) {
                store_run<ODT, V>(p.out, t * p.ldo + n, V, acc);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (n + i >= own) store_elem<ODT>(p.out, t * p.ldo + n + i, acc[i]);
            }
        } else {
            for (int64_t i = 0; i < p.H; ++i) {
                float acc = p.residual != nullptr ? load_elem<ODT>(p.residual, t * p.ldr + i) : 0.0f;
                for (int j = 0; j < p.topk; ++j)
                    if ((uint32_t)rows[j] < (uint32_t)p.R)
                        acc = __builtin_fmaf(weights != nullptr ? weights[j] : 1.0f,
                                             load_elem<DT>(p.y, (int64_t)rows[j] * p.ldy + i), acc);
                store_elem<ODT>(p.out, t * p.ldo + i, acc);
            }
        }
    }
}

// The gradient: choice (t, j) of row r writes dy[r] = w dout[t] and its weight's
// gradient <dout[t], y[r]>.  `lanes` neighbouring threads take a choice, so the
// topk readings of dout[t] happen side by side and all but one come from cache.
template <int DT, int YDT>
__global__ __launch_bounds__(kRowThreads) void moe_combine_grad(MoeCombineGrad p, int lane_bits) {
    constexpr int V = 16 / elem_size<YDT>();
    constexpr int U = 4;  // pieces of a lane in flight
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
            const int64_t d0 = t * p.ldd, y0 = (int64_t)r * p.ldy, g0 = (int64_t)r * p.lddy;
            // M pieces of the lane, `lanes` apart, from element n0 on.  LAST: not all of them
            // whole and in the row.  The row's last piece reaches back over the one before
            // it, as in moe_combine, and one past it reads that too, so that all loads go out
            // together; what is not the lane's own counts nowhere.
            auto pieces = [&](auto many, auto last, int64_t n0) {
                constexpr int M = decltype(many)::value;
                constexpr bool LAST = decltype(last)::value;
                uint32_t dr[M][V * elem_size<DT>() / 4], yr[M][4];
                int64_t at[M];
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    at[m] = n0 + (int64_t)m * V * lanes;
                    if constexpr (LAST) at[m] = min(at[m], p.H - V);
                    load_words(static_cast<const uint8_t*>(p.dout) + (d0 + at[m]) * elem_size<DT>(), dr[m]);
                    if (p.dweights != nullptr)
                        load_words(static_cast<const uint8_t*>(p.y) + (y0 + at[m]) * elem_size<YDT>(), yr[m]);
                }
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    const int64_t own = n0 + (int64_t)m * V * lanes;
                    float d[V], y[V];
                    unpack<DT, V>(dr[m], d);
                    if (p.dweights != nullptr) {
                        unpack<YDT, V>(yr[m], y);
#pragma unroll
                        for (int i = 0; i < V; ++i)
                            if (!LAST || at[m] + i >= own) dot = __builtin_fmaf(d[i], y[i], dot);
                    }
                    if (p.dy != nullptr) {
#pragma unroll
                        for (int i = 0; i < V; ++i) d[i] *= w;
                        if (!LAST || at[m] == own) {
                            store_run<YDT, V>(p.dy, g0 + at[m], V, d);
                        } else {
#pragma unroll
                            for (int i = 0; i < V; ++i)
                                if (at[m] + i >= own) store_elem<YDT>(p.dy, g0 + at[m] + i, d[i]);
                        }
                    }
                }
            };
            const int64_t run = (int64_t)V * lanes;  // elements of the choice's lanes together
            int64_t n0 = 0;
            for (; n0 + U * run <= p.H; n0 += U * run)
                pieces(std::integral_constant<int, U>{}, std::false_type{}, n0 + (int64_t)V * l);
            if (p.H >= V) {
                const int64_t n = n0 + (int64_t)V * l;
                switch ((int)((p.H - n0 + run - 1) / run)) {
                    case 0: break;
                    case 1: pieces(std::integral_constant<int, 1>{}, std::true_type{}, n); break;
                    case 2: pieces(std::integral_constant<int, 2>{}, std::true_type{}, n); break;
                    case 3: pieces(std::integral_constant<int, 3>{}, std::true_type{}, n); break;
                    default: pieces(std::integral_constant<int, U>{}, std::true_type{}, n); break;
                }
            } else if (l == 0) {
                for (int64_t i = 0; i < p.H; ++i) {
                    const float d = load_elem<DT>(p.dout, d0 + i);
                    if (p.dweights != nullptr) dot = __builtin_fmaf(d, load_elem<YDT>(p.y, y0 + i), dot);
                    if (p.dy != nullptr) store_elem<YDT>(p.dy, g0 + i, d * w);
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

// The single launch, whose every workgroup reads all choices, against the two (in chunks
// of 4096 choices, so 8 workgroups for 32768; smaller ones were not measured), in us:
//   choices x experts   512 x 64   8192 x 256   32768 x 64   32768 x 256   16384 x 1024   32768 x 1024   40000 x 256
//   one                 2.4        4.3          7.7          9.7           12.2           23.3           16.8
//   two                 8.5        11.5         11.9         12.8          14.8           14.8           12.8
constexpr int64_t kSortOneMax = 32 * kSortOneThreads;
constexpr int64_t kSortOneWork = 20 << 20;

static bool sort_one(int64_t R, int64_t E) { return R <= kSortOneMax && R * (E + 1) <= kSortOneWork; }

// Chunks of whole waves' loads, at least 4096 choices and at most 256 of them.
static int64_t sort_chunk(int64_t R) {
    const int64_t step = kSortWaves * kWave * kSortAhead;
    return std::max<int64_t>(4096, ceil_div(ceil_div(R, 256), step) * step);
}

size_t moe_sort_ws_bytes(int64_t R, int64_t E) {
    return sort_one(R, E) ? 0 : (size_t)ceil_div(R, sort_chunk(R)) * (size_t)(E + 1) * sizeof(int);
}

template <typename ID>
static hipError_t launch_sort(const ID* ids, int64_t R, int64_t topk, int64_t E, int32_t* offsets, int32_t* row_token,
                              int32_t* row_of, void* ws, hipStream_t stream) {
    if (sort_one(R, E)) {
        // ceil(2^32 / topk); 0 for topk 1 (and for no choices at all)
        const uint32_t per_topk = topk > 1 ? (uint32_t)(((uint64_t(1) << 32) + topk - 1) / topk) : 0;
        const int parts = R <= 4 * 256 ? 1 : (int)std::max<int64_t>(1, std::min<int64_t>(4, 256 / (E + 1)));
#define FP8K_SORT_ONE(T, KEYS)                                                                                       \
    hipLaunchKernelGGL((moe_sort_one<ID, T, KEYS>), dim3((unsigned)((E + 1) * parts)), dim3(T), 0, stream, ids, (int)R, \
                       per_topk, (int)E, parts, offsets, row_token, row_of)
        if (R <= 4 * 256)
            FP8K_SORT_ONE(256, 4);
        else if (R <= 4 * kSortOneThreads)
            FP8K_SORT_ONE(kSortOneThreads, 4);
        else if (R <= 8 * kSortOneThreads)
            FP8K_SORT_ONE(kSortOneThreads, 8);
        else if (R <= 16 * kSortOneThreads)
            FP8K_SORT_ONE(kSortOneThreads, 16);
        else
            FP8K_SORT_ONE(kSortOneThreads, 32);
#undef FP8K_SORT_ONE
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

// Rows of `pieces` 16-byte pieces as tasks, and their workgroups.
static RowTasks row_tasks(int64_t pieces) {
    const int bits = bits_for(pieces, 6);
    return {bits, std::max<int64_t>(ceil_div(pieces, int64_t(1) << bits), 1)};
}
static dim3 task_grid(int64_t tasks, const RowTasks& k) { return row_grid(ceil_div(tasks, kRowThreads >> k.bits)); }

hipError_t launch_moe_permute(const void* x, int64_t ldx_bytes, const float* s_tok, const int32_t* row_of, int64_t T,
                              int64_t topk, int64_t R, int64_t row_bytes, void* out, int64_t ldo_bytes, float* s_out,
                              hipStream_t stream) {
    const RowTasks k = row_tasks(ceil_div(row_bytes, 16));
    const auto kernel = k.bits == 6 ? moe_permute<true> : moe_permute<false>;
    hipLaunchKernelGGL(kernel, task_grid(T * k.cols, k), dim3(kRowThreads), 0, stream, static_cast<const uint8_t*>(x),
                       ldx_bytes, s_tok, row_of, T * k.cols, (int)topk, (int)R, row_bytes, k, static_cast<uint8_t*>(out),
                       ldo_bytes, s_out);
    return hipGetLastError();
}

template <int DT, int ODT, int U>
static hipError_t launch_combine(const MoeCombine& p, hipStream_t stream) {
    const RowTasks k = row_tasks(ceil_div(p.H, 16 / elem_size<DT>()));
    const int64_t tasks = p.T * k.cols;
    const auto kernel = k.bits == 6 ? moe_combine<DT, ODT, U, true> : moe_combine<DT, ODT, U, false>;
    hipLaunchKernelGGL(kernel, task_grid(tasks, k), dim3(kRowThreads), 0, stream, p, tasks, k);
    return hipGetLastError();
}

hipError_t launch_moe_combine(const MoeCombine& p, int dtype, int out_dtype, hipStream_t stream) {
    return with_type(dtype, [&](auto dt) {
        return with_type(out_dtype, [&](auto odt) {
            constexpr int DT = decltype(dt)::value, ODT = decltype(odt)::value;
            if (p.topk <= 1) return launch_combine<DT, ODT, 1>(p, stream);
            if (p.topk <= 2) return launch_combine<DT, ODT, 2>(p, stream);
            if (p.topk <= 4) return launch_combine<DT, ODT, 4>(p, stream);
            return launch_combine<DT, ODT, 8>(p, stream);
        });
    });
}

hipError_t launch_moe_combine_grad(const MoeCombineGrad& p, int dtype, int y_dtype, hipStream_t stream) {
    return with_type(dtype, [&](auto dt) {
        return with_type(y_dtype, [&](auto ydt) {
            constexpr int DT = decltype(dt)::value, YDT = decltype(ydt)::value;
            const int64_t choices = (int64_t)p.T * p.topk;
            // Few choices: a lane a piece, up to a workgroup each.  Many: two to four pieces a
            // lane, up to a wave each (10000 choices of 333 fp16 elements: 14 us with a wave each, 6.4 with 16 lanes).
            const int64_t each = ceil_div(p.H, 16 / elem_size<YDT>());
            const int bits = choices < 1024 ? bits_for(each, 8) : bits_for(ceil_div(each, 4), 6);
            hipLaunchKernelGGL((moe_combine_grad<DT, YDT>), row_grid(ceil_div(choices, kRowThreads >> bits)),
                               dim3(kRowThreads), 0, stream, p, bits);
            return hipGetLastError();
        });
    });
}

}  // namespace fp8k
