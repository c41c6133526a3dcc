// Append to the paged FP8 KV cache on gfx950: rotate queries and keys by their
// positions, quantize keys and values into cache rows, in one pass over them.
//
// A pair (a, b) of a head turns by its angle t = position * frequency, whose
// cosine and sine come from the caller's fp32 table (so any frequency scaling
// is a table):
//     a' = fl(fl(a cos t) - fl(b sin t)),   b' = fl(fl(b cos t) + fl(a sin t)),
// each product and sum rounded to fp32 once, no fused multiply-add: the bits
// are those of the formula evaluated step by step, and a cache written here
// equals one written by rotating first and calling the codec.  Keys then take
// the codec's quotient and code; q is rounded once to its own type.
//
// The pass is a stream: it reads q, k, v and writes q and one byte per k / v
// element.  A thread owns 16 elements of a head, laid out so that a pair never
// leaves it: two runs of 8 half the rotated width apart (or 16 neighbours when
// pairs are interleaved), so every access is 16 bytes of a 16-bit row, and the
// same slot of two tokens, so its scales are read and inverted once and the
// loads of both are in flight together.  32768 tokens, 64 / 8 heads of 128, bf16:
// 227 us, 5.7 TB/s; one token: 2.7 us, a launch.  Workgroups of 128 threads: 256
// leave a sixth of the lanes without a slot there (229 us; 32 / 8 heads 79.7
// against 70.2 at 16384 tokens).
#include <algorithm>

#include "kv_common.hpp"

namespace fp8k {

namespace {

constexpr int kAppendThreads = 128;

// 8 consecutive row elements as fp32.
template <int DT>
__device__ __forceinline__ void load8(const void* base, int64_t e, float (&x)[8]) {
    float4 v[kv_quads<DT>()];
    if constexpr (DT == kKvF32) {
        kv_load<DT>(base, e, v);
        x[0] = v[0].x, x[1] = v[0].y, x[2] = v[0].z, x[3] = v[0].w;
        kv_load<DT>(base, e + 4, v);
        x[4] = v[0].x, x[5] = v[0].y, x[6] = v[0].z, x[7] = v[0].w;
    } else {
        kv_load<DT>(base, e, v);
#pragma unroll
        for (int q = 0; q < 2; ++q) x[4 * q] = v[q].x, x[4 * q + 1] = v[q].y, x[4 * q + 2] = v[q].z, x[4 * q + 3] = v[q].w;
    }
}

// 8 fp32 values rounded (RNE) to 8 consecutive row elements.
template <int DT>
__device__ __forceinline__ void store8(void* base, int64_t e, const float (&x)[8]) {
    if constexpr (DT == kKvF32) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + e);
        p[0] = make_float4(x[0], x[1], x[2], x[3]);
        p[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        v4u w;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = DT == kKvBF16 ? round_bf16x2(x[2 * i], x[2 * i + 1]) : round_f16x2(x[2 * i], x[2 * i + 1]);
        *reinterpret_cast<v4u*>(static_cast<uint16_t*>(base) + e) = w;
    }
}

// The pair's rotation, every step rounded to fp32: contraction is off, or the
// compiler would fuse one product of each sum.
__device__ __forceinline__ void rotate(float& a, float& b, float c, float s) {
#pragma clang fp contract(off)
    const float ac = a * c, bs = b * s, bc = b * c, as = a * s;
    a = ac - bs;
    b = bc + as;
}

template <int FMT, int DT, bool PAIRS, int U>
__global__ __launch_bounds__(kAppendThreads) void kv_append_rope(KvAppend p) {
    const int slots = p.D / 16;  // 16-element slots of a head
    const int u = blockIdx.x * kAppendThreads + threadIdx.x;
    const int head = u / slots;
    if (head >= p.Hq + 2 * p.Hkv) return;
    const int i = u - head * slots;
    const int half = p.rot / 2;
    const bool is_q = head < p.Hq, is_v = head >= p.Hq + p.Hkv;
    const bool turns = !is_v && i < p.rot / 16;
    // the slot's two runs of 8 elements
    const int e0 = PAIRS || !turns ? 16 * i : 8 * i;
    const int e1 = PAIRS || !turns ? 16 * i + 8 : half + 8 * i;
    const void* src = is_q ? p.q : is_v ? p.v : p.k;
    const int64_t ld = is_q ? p.ldq : is_v ? p.ldv : p.ldk;
    const int h = is_q ? head : is_v ? head - p.Hq - p.Hkv : head - p.Hq;
    const int ch = (is_v ? p.Hkv + h : h) * p.D;  // the head's first cache channel
    RowScale rs[16];
    if (!is_q) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            rs[j] = channel_scale(p.scales[ch + e0 + j]);
            rs[8 + j] = channel_scale(p.scales[ch + e1 + j]);
        }
    }
    const int64_t C = 2 * (int64_t)p.Hkv * p.D;
    const int64_t t0 = (int64_t)blockIdx.y * p.tokens_per_block;
    const int64_t t1 = min((int64_t)p.T, t0 + p.tokens_per_block);
    for (int64_t t = t0; t < t1; t += U) {
        float a[U][8], b[U][8], c[U][8], s[U][8];
        int slot[U];
        bool live[U];
#pragma unroll
        for (int n = 0; n < U; ++n) {
            const int64_t tt = min(t + n, t1 - 1);
            load8<DT>(src, tt * ld + (int64_t)h * p.D + e0, a[n]);
            load8<DT>(src, tt * ld + (int64_t)h * p.D + e1, b[n]);
            const int pos = p.positions[tt];
            slot[n] = is_q ? -1 : p.slot[tt];  // null without KV heads
            live[n] = t + n < t1 && pos >= 0 && pos < p.P;
            if (turns) {
                const float* row = p.cos_sin + (int64_t)(live[n] ? pos : 0) * p.rot + 8 * i;
#pragma unroll
                for (int j = 0; j < 8; j += 4) {
                    const float4 x = *reinterpret_cast<const float4*>(row + j);
                    const float4 y = *reinterpret_cast<const float4*>(row + half + j);
                    c[n][j] = x.x, c[n][j + 1] = x.y, c[n][j + 2] = x.z, c[n][j + 3] = x.w;
                    s[n][j] = y.x, s[n][j + 1] = y.y, s[n][j + 2] = y.z, s[n][j + 3] = y.w;
                }
            }
        }
#pragma unroll
        for (int n = 0; n < U; ++n) {
            if (turns) {
                if constexpr (PAIRS) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        rotate(a[n][2 * j], a[n][2 * j + 1], c[n][j], s[n][j]);
                        rotate(b[n][2 * j], b[n][2 * j + 1], c[n][4 + j], s[n][4 + j]);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) rotate(a[n][j], b[n][j], c[n][j], s[n][j]);
                }
            }
            if (is_q) {
                if (live[n]) {
                    const int64_t at = (t + n) * p.ldqo + (int64_t)h * p.D;
                    store8<DT>(p.q_out, at + e0, a[n]);
                    store8<DT>(p.q_out, at + e1, b[n]);
                }
            } else {
                // coded outside the test, as in kv_quantize_paged: only the store waits for the slot
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    w[j] = kv_encode4<FMT>(make_float4(a[n][4 * j], a[n][4 * j + 1], a[n][4 * j + 2], a[n][4 * j + 3]),
                                           rs[4 * j], rs[4 * j + 1], rs[4 * j + 2], rs[4 * j + 3]);
                    w[2 + j] = kv_encode4<FMT>(make_float4(b[n][4 * j], b[n][4 * j + 1], b[n][4 * j + 2], b[n][4 * j + 3]),
                                               rs[8 + 4 * j], rs[9 + 4 * j], rs[10 + 4 * j], rs[11 + 4 * j]);
                }
                if (live[n] && slot[n] >= 0 && slot[n] < p.num_slots) {
                    uint8_t* dst = p.cache + (int64_t)slot[n] * C + ch;
                    *reinterpret_cast<v2u*>(dst + e0) = v2u{w[0], w[1]};
                    *reinterpret_cast<v2u*>(dst + e1) = v2u{w[2], w[3]};
                }
            }
        }
    }
}

template <int FMT, int DT>
hipError_t launch(KvAppend p, bool pairs, hipStream_t stream) {
    const int64_t units = (int64_t)(p.Hq + 2 * p.Hkv) * (p.D / 16);
    const int64_t cols = (units + kAppendThreads - 1) / kAppendThreads;
    // Two tokens a thread, whose loads travel together; one where that leaves
    // CUs idle (latency is what counts there).  us for 512 / 1777 / 32768 tokens
    // (64 / 8 heads of 128, bf16; 1777: 24 / 3 of 256, fp16): one token 7.7 /
    // 16.0 / 257, two 6.4 / 14.5 / 227, four 7.6 / 16.0 / 266, two in a loop of
    // 2048 workgroups 7.7 / 14.4 / 279.
    const int64_t work = p.T * cols;
    p.tokens_per_block = work < 2048 ? 1 : 2;
    // more rows than a grid has: loops
    while ((p.T + p.tokens_per_block - 1) / p.tokens_per_block > 65535) p.tokens_per_block *= 2;
    const dim3 grid((unsigned)cols, (unsigned)((p.T + p.tokens_per_block - 1) / p.tokens_per_block));
    const bool many = p.tokens_per_block > 1;
    if (pairs) {
        if (many) hipLaunchKernelGGL((kv_append_rope<FMT, DT, true, 2>), grid, dim3(kAppendThreads), 0, stream, p);
        else hipLaunchKernelGGL((kv_append_rope<FMT, DT, true, 1>), grid, dim3(kAppendThreads), 0, stream, p);
    } else {
        if (many) hipLaunchKernelGGL((kv_append_rope<FMT, DT, false, 2>), grid, dim3(kAppendThreads), 0, stream, p);
        else hipLaunchKernelGGL((kv_append_rope<FMT, DT, false, 1>), grid, dim3(kAppendThreads), 0, stream, p);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append_rope(const KvAppend& p, int dtype, int fmt, bool interleaved, hipStream_t stream) {
#define FP8K_APPEND(D) \
    (fmt == kKvE5M2 ? launch<kKvE5M2, D>(p, interleaved, stream) : launch<kKvE4M3, D>(p, interleaved, stream))
    switch (dtype) {
        case kKvBF16: return FP8K_APPEND(kKvBF16);
        case kKvF16: return FP8K_APPEND(kKvF16);
        default: return FP8K_APPEND(kKvF32);
    }
#undef FP8K_APPEND
}

}  // namespace fp8k
