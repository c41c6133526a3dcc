// C ABI of the unified-FP8 linear layer: host-side validation and dispatch.
//
// Every entry point checks its arguments on the host first and returns a
// status without touching the device when they are invalid; only then does it
// enqueue kernels on the caller's stream.  No memory is allocated and no state
// is kept between calls.
#include "../../include/fp8w8a8.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "act_plan.hpp"
#include "attn_plan.hpp"
#include "kernels.hpp"

namespace {

constexpr int64_t kMaxDim = INT32_MAX;  // kernels index rows and columns with 32-bit ints
constexpr size_t kAlign = 256;          // workspace sub-buffer alignment
constexpr int64_t kMaxExperts = 1024;   // of the grouped products and of the sort
constexpr int64_t kMaxTiles = INT32_MAX - 8;  // launch grids count output tiles in 32 bits

// Output tiles of 128 x 128 (no GEMM kernel uses smaller tiles along both axes
// with one workgroup each), bounded so every grid and tile index fits 32 bits.
bool tiles_ok(int64_t row_tiles, int64_t N) { return row_tiles * ((N + 127) / 128) <= kMaxTiles; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

// a * b without int64 overflow (a, b >= 0)
bool mul_ok(int64_t a, int64_t b, int64_t* out) {
    if (a != 0 && b > INT64_MAX / a) return false;
    *out = a * b;
    return true;
}

fp8_status_t check_dims(int64_t M, int64_t N, int64_t K) {
    if (M < 0 || N < 0 || K < 0) return FP8_ERR_INVALID_ARGUMENT;
    if (M > kMaxDim || N > kMaxDim || K > kMaxDim) return FP8_ERR_UNSUPPORTED;
    if (K % 16 != 0) return FP8_ERR_UNSUPPORTED;
    if (!tiles_ok((M + 127) / 128, N)) return FP8_ERR_UNSUPPORTED;
    return FP8_OK;
}

// A row-major matrix argument: rows x cols elements of `elem` bytes, stride
// ld.  Input operands are read in 16-byte pieces, so their row stride must be
// a multiple of 16 bytes (strided_ok = false); the BF16 output may have any
// row stride (strided_ok = true).
fp8_status_t check_matrix(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t elem,
                          bool strided_ok = false) {
    if (rows > 0 && cols > 0 && p == nullptr) return FP8_ERR_INVALID_ARGUMENT;
    if (rows > 0 && ld < cols) return FP8_ERR_INVALID_ARGUMENT;
    int64_t span, bytes;
    if (!mul_ok(rows, ld, &span) || !mul_ok(span, elem, &bytes)) return FP8_ERR_INVALID_ARGUMENT;
    if (rows > 0 && cols > 0) {
        if (!aligned16(p)) return FP8_ERR_UNSUPPORTED;
        if (!strided_ok && (ld * elem) % 16 != 0) return FP8_ERR_UNSUPPORTED;
    }
    return FP8_OK;
}

fp8_status_t check_vector(const void* p, int64_t n) {
    if (n > 0 && p == nullptr) return FP8_ERR_INVALID_ARGUMENT;
    if (n > 0 && !aligned16(p)) return FP8_ERR_UNSUPPORTED;
    return FP8_OK;
}

#define FP8_TRY(expr)                          \
    do {                                       \
        fp8_status_t s_ = (expr);              \
        if (s_ != FP8_OK) return s_;           \
    } while (0)

static_assert(FP8_KV_E4M3 == fp8k::kKvE4M3 && FP8_KV_E5M2 == fp8k::kKvE5M2, "KV format ids");
static_assert(FP8_KV_F32 == fp8k::kKvF32 && FP8_KV_BF16 == fp8k::kKvBF16 && FP8_KV_F16 == fp8k::kKvF16, "KV dtype ids");

// KV batch extents: C channels in groups of 4 (one 32-bit word of codes).
fp8_status_t check_kv_dims(int64_t T, int64_t C) {
    if (T < 0 || C < 0) return FP8_ERR_INVALID_ARGUMENT;
    if (T > kMaxDim || C > kMaxDim) return FP8_ERR_UNSUPPORTED;
    if (C % 4 != 0) return FP8_ERR_UNSUPPORTED;
    return FP8_OK;
}

fp8_status_t check_kv_format(fp8_kv_format_t fmt) {
    return (fmt == FP8_KV_E4M3 || fmt == FP8_KV_E5M2) ? FP8_OK : FP8_ERR_INVALID_ARGUMENT;
}

// Element size of a KV row type, 0 when the type is unknown.
int64_t kv_elem_bytes(fp8_kv_dtype_t t) {
    switch (t) {
        case FP8_KV_F32: return 4;
        case FP8_KV_BF16:
        case FP8_KV_F16: return 2;
    }
    return 0;
}

// Element size of a KV row type and the channel rule that goes with it:
// 16-bit rows are read 8 channels (16 bytes) per thread, so C % 8 == 0.
fp8_status_t kv_row_type(fp8_kv_dtype_t t, int64_t C, int64_t* eb) {
    *eb = kv_elem_bytes(t);
    if (*eb == 0) return FP8_ERR_INVALID_ARGUMENT;
    if (*eb == 2 && C % 8 != 0) return FP8_ERR_UNSUPPORTED;
    return FP8_OK;
}

fp8_status_t from_hip(hipError_t e) { return e == hipSuccess ? FP8_OK : FP8_ERR_DEVICE; }

// Attention extents: positions, rows and row-head pairs are 32-bit in the kernels.
constexpr int64_t kMaxAttn = int64_t(1) << 30;

fp8_status_t check_attn_dims(int64_t rows, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t block_size,
                             int64_t max_blocks, int64_t max_q, int64_t max_len) {
    if (rows < 0 || B < 0 || Hq < 0 || Hkv < 0 || D < 0 || max_blocks < 0 || max_q < 0 || max_len < 0)
        return FP8_ERR_INVALID_ARGUMENT;
    if (block_size < 1 || Hkv < 1 || Hq % Hkv != 0) return FP8_ERR_INVALID_ARGUMENT;
    if (D != 64 && D != 128 && D != 256) return FP8_ERR_UNSUPPORTED;
    if (Hkv > 65535 || rows > kMaxAttn || B > kMaxAttn || Hq > kMaxAttn / D || block_size > kMaxAttn || max_blocks > kMaxAttn)
        return FP8_ERR_UNSUPPORTED;
    if (block_size * max_blocks > kMaxAttn || rows * Hq > kMaxAttn || B * Hq > kMaxAttn / 16) return FP8_ERR_UNSUPPORTED;
    return FP8_OK;
}

// Launch hints: unknown (0) or past what the buffers hold is taken as the most
// they hold.  A wrong hint changes no result.
int64_t hint(int64_t v, int64_t most) { return v > 0 ? std::min(v, most) : most; }

// The new rows of a sequence: the most to expect, by the hint or, without one, by
// the keys that rows past them would not have; and those of most sequences, by
// the hint or the mean.
struct NewRows {
    int64_t most, typical;

    NewRows(int64_t max_q, int64_t rows, int64_t B, int64_t max_len)
        : most(hint(max_q, rows)), typical(max_q > 0 ? most : fp8k::ceil_div(rows, std::max<int64_t>(B, 1))) {
        if (max_q == 0) most = std::max(typical, std::min(most, max_len));
    }
};

// Either way: the queries are not told the type, nor whether lse is wanted.
size_t attn_ws(int64_t rows, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t block_size, int64_t max_blocks,
               int64_t max_q, int64_t max_len) {
    const int64_t all_len = block_size * max_blocks;
    max_len = hint(max_len, all_len);
    if (B == 0 || rows == 0) return 0;
    const NewRows q(max_q, rows, B, max_len);
    const bool one = fp8k::attn_tiled(Hq, Hkv, D, q.typical, false), two = fp8k::attn_tiled(Hq, Hkv, D, q.typical, true);
    size_t need = 0;
    if (one || two) need = fp8k::attn_tiled_ws_bytes(B, rows, Hq, Hkv, D, q.most, max_len);
    if (!one || !two) need = std::max(need, fp8k::attn_paged_ws_bytes(B, rows, Hq, Hkv, D, q.most, max_len, all_len));
    return round_up(need, kAlign);
}

// Both attention entry points; cu_q null: one new row per sequence.
fp8_status_t attn(fp8k::PagedAttn p, fp8_kv_dtype_t dtype, fp8_kv_format_t fmt, int64_t rows, int64_t B, int64_t Hq,
                  int64_t Hkv, int64_t D, int64_t block_size, int64_t max_blocks, int64_t max_q, int64_t max_len,
                  int64_t window, float sm_scale, void* ws, size_t ws_bytes, hipStream_t stream) {
    FP8_TRY(check_attn_dims(rows, B, Hq, Hkv, D, block_size, max_blocks, max_q, max_len));
    FP8_TRY(check_kv_format(fmt));
    const int64_t eb = kv_elem_bytes(dtype);
    if (eb == 0) return FP8_ERR_INVALID_ARGUMENT;
    if (!std::isfinite(sm_scale) || !std::isfinite(p.softcap) || p.softcap < 0 || window < 0 || p.num_blocks < 0)
        return FP8_ERR_INVALID_ARGUMENT;
    if (p.num_blocks > kMaxDim / block_size) return FP8_ERR_UNSUPPORTED;
    const bool some = rows > 0 && B > 0 && Hq > 0;
    FP8_TRY(check_matrix(p.q, rows, Hq * D, p.ldq, eb));
    FP8_TRY(check_matrix(p.out, rows, Hq * D, p.ldo, eb));
    FP8_TRY(check_matrix(p.cache, p.num_blocks * block_size, 2 * Hkv * D, 2 * Hkv * D, 1, true));
    if (some) {
        FP8_TRY(check_vector(p.scales, 2 * Hkv * D));
        if (p.seq_lens == nullptr || (max_blocks > 0 && p.block_table == nullptr)) return FP8_ERR_INVALID_ARGUMENT;
        if (max_blocks > 0 && p.ld_table < max_blocks) return FP8_ERR_INVALID_ARGUMENT;
        const uintptr_t words = reinterpret_cast<uintptr_t>(p.seq_lens) | reinterpret_cast<uintptr_t>(p.block_table) |
                                reinterpret_cast<uintptr_t>(p.cu_q) | reinterpret_cast<uintptr_t>(p.prefix) |
                                reinterpret_cast<uintptr_t>(p.alibi) | reinterpret_cast<uintptr_t>(p.lse);
        if ((words & 3u) != 0) return FP8_ERR_UNSUPPORTED;
    }
    const size_t need = attn_ws(rows, B, Hq, Hkv, D, block_size, max_blocks, max_q, max_len);
    if (ws_bytes < need) return FP8_ERR_WORKSPACE;
    if (need > 0 && ws == nullptr) return FP8_ERR_INVALID_ARGUMENT;
    if (need > 0 && !aligned16(ws)) return FP8_ERR_UNSUPPORTED;
    if (!some) return FP8_OK;
    p.scale = sm_scale * 1.44269504088896341f;  // scores in powers of two
    // The kernels may read (never use) one page number and one cache row: there is one of each, even in an empty table
    // or pool.
    if (max_blocks == 0) p.block_table = p.seq_lens, p.ld_table = 0;
    if (p.num_blocks == 0) p.cache = reinterpret_cast<const uint8_t*>(p.scales);
    p.B = (int)B, p.rows = (int)rows, p.Hq = (int)Hq, p.Hkv = (int)Hkv;
    p.block = (int)block_size, p.max_blocks = (int)max_blocks;
    p.window = (int)std::min(window, kMaxAttn);  // no key is further back
    p.dtype = (int)dtype;
    max_len = hint(max_len, block_size * max_blocks);
    const NewRows n(max_q, rows, B, max_len);
    const bool tiled = fp8k::attn_tiled(Hq, Hkv, D, n.typical, fp8k::two_terms(p));
    return from_hip(tiled ? fp8k::launch_attn_tiled(p, (int)D, (int)fmt, n.most, max_len, ws, stream)
                          : fp8k::launch_attn_paged(p, (int)D, (int)fmt, n.most, n.typical, max_len, ws, stream));
}

// Bytes the GEMM path itself needs for an M x N x K problem: the skinny
// kernel's fp32 split-k partial sums when it splits k, else none.
size_t gemm_ws_bytes(int64_t M, int64_t N, int64_t K) {
    return M <= fp8k::kSkinnyMaxM ? round_up(fp8k::gemm_skinny_ws_bytes(M, N, K), kAlign) : 0;
}

// Bytes the fused path stages its activation codes and scales in.
size_t fused_stage_bytes(int64_t M, int64_t K) {
    return round_up((size_t)M * (size_t)K, kAlign) + round_up((size_t)M * sizeof(float), kAlign);
}

// BF16 output to y, or (y32 != nullptr) the fp32 value before rounding to y32.
fp8_status_t gemm_dispatch(const uint8_t* qa, int64_t lda, const float* s_tok, const uint8_t* qw, int64_t ldw,
                           const float* s_ch, uint16_t* y, float* y32, int64_t ldy, int64_t M, int64_t N, int64_t K,
                           void* ws, hipStream_t stream) {
    if (M <= fp8k::kSkinnyMaxM)
        return from_hip(fp8k::launch_gemm_skinny(qa, lda, s_tok, qw, ldw, s_ch, y, y32, ldy, M, N, K, ws, stream));
    if (K % 128 == 0)
        return from_hip(fp8k::launch_gemm_mfma(qa, lda, s_tok, qw, ldw, s_ch, y, y32, ldy, M, N, K, stream));
    return from_hip(fp8k::launch_gemm_tiled(qa, lda, s_tok, qw, ldw, s_ch, y, y32, ldy, M, N, K, stream));
}

static_assert(FP8_ACT_NONE == fp8k::kActNone && FP8_ACT_RELU == fp8k::kActRelu && FP8_ACT_SILU == fp8k::kActSilu &&
                  FP8_ACT_GELU == fp8k::kActGelu && FP8_ACT_GELU_TANH == fp8k::kActGeluTanh,
              "activation ids");

fp8_status_t check_act(fp8_act_t act) {
    return act >= FP8_ACT_NONE && act <= FP8_ACT_GELU_TANH ? FP8_OK : FP8_ERR_INVALID_ARGUMENT;
}

// Output tiles of 128 x 128 of the products with an epilogue.
bool act_tiles_ok(int64_t row_tiles, int64_t N) { return row_tiles * ((N + 127) / 128) <= fp8k::kMaxActTiles; }

// A vector of 32-bit words that is read one by one.
fp8_status_t check_words(const void* p, int64_t n) {
    if (n > 0 && p == nullptr) return FP8_ERR_INVALID_ARGUMENT;
    return n > 0 && (reinterpret_cast<uintptr_t>(p) & 3u) != 0 ? FP8_ERR_UNSUPPORTED : FP8_OK;
}

// A 16-byte aligned row-major matrix whose row stride is free.
fp8_status_t check_rows(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t elem) {
    return check_matrix(p, rows, cols, ld, elem, true);
}

// A matrix written in place of one read: the same rows at the same stride, or no
// element is where it was read.
bool in_place_ok(const void* in, int64_t ld_in, const void* out, int64_t ld_out, int64_t rows, int64_t cols) {
    return in != out || ld_in == ld_out || rows <= 1 || cols == 0;
}

// Whether an output is at the address of one of these inputs (or outputs).
bool at_any(const void* out, std::initializer_list<const void*> others) {
    return out != nullptr && std::find(others.begin(), others.end(), out) != others.end();
}

// Extents of the expert-row calls: T tokens of topk choices, R expert rows of H elements.
fp8_status_t check_choices(int64_t T, int64_t topk, int64_t R, int64_t H) {
    if (T < 0 || topk < 0 || R < 0 || H < 0) return FP8_ERR_INVALID_ARGUMENT;
    if (T > kMaxDim || topk > kMaxDim || R > kMaxDim || H > kMaxDim) return FP8_ERR_UNSUPPORTED;
    return T * topk > kMaxDim ? FP8_ERR_UNSUPPORTED : FP8_OK;
}

// The output and the residual of a product's epilogue.
fp8_status_t check_epilogue(const fp8k::Epilogue& e, fp8_act_t act, fp8_kv_dtype_t type, int64_t bias, int64_t M,
                            int64_t N) {
    FP8_TRY(check_act(act));
    const int64_t eb = kv_elem_bytes(type);
    if (eb == 0) return FP8_ERR_INVALID_ARGUMENT;
    FP8_TRY(check_rows(e.y, M, N, e.ldy, eb));
    if (e.residual != nullptr) {
        FP8_TRY(check_rows(e.residual, M, N, e.ldr, eb));
        if (!in_place_ok(e.residual, e.ldr, e.y, e.ldy, M, N)) return FP8_ERR_INVALID_ARGUMENT;
    }
    return e.bias != nullptr ? check_vector(e.bias, bias) : FP8_OK;
}

// Bytes of the fp32 output staged by the FP8-output GEMM.
size_t fp8out_stage_bytes(int64_t M, int64_t N) { return round_up((size_t)M * (size_t)N * sizeof(float), kAlign); }

}  // namespace

extern "C" {

const char* fp8_status_string(fp8_status_t status) {
    switch (status) {
        case FP8_OK: return "FP8_OK";
        case FP8_ERR_INVALID_ARGUMENT: return "FP8_ERR_INVALID_ARGUMENT";
        case FP8_ERR_UNSUPPORTED: return "FP8_ERR_UNSUPPORTED";
        case FP8_ERR_WORKSPACE: return "FP8_ERR_WORKSPACE";
        case FP8_ERR_DEVICE: return "FP8_ERR_DEVICE";
    }
    return "FP8_ERR_UNKNOWN";
}

size_t fp8_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (check_dims(M, N, K) == FP8_ERR_INVALID_ARGUMENT) return SIZE_MAX;
    int64_t mk;
    if (!mul_ok(M, K, &mk)) return SIZE_MAX;
    return fused_stage_bytes(M, K) + gemm_ws_bytes(M, N, K);
}

size_t fp8_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (check_dims(M, N, K) == FP8_ERR_INVALID_ARGUMENT) return SIZE_MAX;
    return gemm_ws_bytes(M, N, K);
}

size_t fp8_fp8out_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (check_dims(M, N, K) == FP8_ERR_INVALID_ARGUMENT) return SIZE_MAX;
    int64_t mn;
    if (!mul_ok(M, N, &mn) || mn > INT64_MAX / 8) return SIZE_MAX;
    return fp8out_stage_bytes(M, N) + gemm_ws_bytes(M, N, K);
}

size_t fp8_grouped_workspace_bytes(int64_t T, int64_t R, int64_t E, int64_t N, int64_t K) {
    if (T < 0 || R < 0 || E < 0 || N < 0 || K < 0) return SIZE_MAX;
    return 0;
}

fp8_status_t fp8_quantize_per_token(const float* x, int64_t rows, int64_t K, int64_t ldx, uint8_t* q,
                                    int64_t ldq, float* scales, hipStream_t stream) {
    FP8_TRY(check_dims(rows, 1, K));
    FP8_TRY(check_matrix(x, rows, K, ldx, 4));
    FP8_TRY(check_matrix(q, rows, K, ldq, 1));
    FP8_TRY(check_vector(scales, rows));
    if (rows == 0) return FP8_OK;
    return from_hip(fp8k::launch_quantize_rows(x, ldx, q, ldq, scales, rows, K, stream));
}

fp8_status_t fp8_quantize_static(const float* x, int64_t rows, int64_t K, int64_t ldx, const float* scale,
                                 uint8_t* q, int64_t ldq, float* scales_out, hipStream_t stream) {
    FP8_TRY(check_dims(rows, 1, K));
    FP8_TRY(check_matrix(x, rows, K, ldx, 4));
    FP8_TRY(check_matrix(q, rows, K, ldq, 1));
    FP8_TRY(check_vector(scales_out, rows));
    if (rows > 0 && scale == nullptr) return FP8_ERR_INVALID_ARGUMENT;
    if (rows > 0 && (reinterpret_cast<uintptr_t>(scale) & 3u) != 0) return FP8_ERR_UNSUPPORTED;
    if (rows == 0) return FP8_OK;
    return from_hip(fp8k::launch_quantize_static(x, ldx, scale, q, ldq, scales_out, rows, K, stream));
}

fp8_status_t fp8_quantize_per_token_clipped(const float* x, int64_t rows, int64_t K, int64_t ldx, const float* clip,
                                            uint8_t* q, int64_t ldq, float* scales, hipStream_t stream) {
    FP8_TRY(check_dims(rows, 1, K));
    FP8_TRY(check_matrix(x, rows, K, ldx, 4));
    FP8_TRY(check_matrix(q, rows, K, ldq, 1));
    FP8_TRY(check_vector(scales, rows));
    if (rows > 0 && clip == nullptr) return FP8_ERR_INVALID_ARGUMENT;
    if (rows > 0 && (reinterpret_cast<uintptr_t>(clip) & 3u) != 0) return FP8_ERR_UNSUPPORTED;
    if (rows == 0) return FP8_OK;
    return from_hip(fp8k::launch_quantize_clipped(x, ldx, clip, q, ldq, scales, rows, K, stream));
}

size_t fp8_calibrate_workspace_bytes(void) { return fp8k::kCalibrateWsBytes; }

fp8_status_t fp8_calibrate_percentile(const float* x, int64_t n, int64_t num, int64_t den, float* value_out,
                                      float* scale_out, void* ws, size_t ws_bytes, hipStream_t stream) {
    if (n <= 0 || num <= 0 || den <= 0 || num > den) return FP8_ERR_INVALID_ARGUMENT;
    if (n > (int64_t)UINT32_MAX) return FP8_ERR_UNSUPPORTED;  // 32-bit histogram bins
    if (x == nullptr || value_out == nullptr || ws == nullptr) return FP8_ERR_INVALID_ARGUMENT;
    if ((reinterpret_cast<uintptr_t>(x) & 3u) != 0 || (reinterpret_cast<uintptr_t>(value_out) & 3u) != 0 ||
        (reinterpret_cast<uintptr_t>(scale_out) & 3u) != 0)
        return FP8_ERR_UNSUPPORTED;
    if (!aligned16(ws)) return FP8_ERR_UNSUPPORTED;
    if (ws_bytes < fp8k::kCalibrateWsBytes) return FP8_ERR_WORKSPACE;
    // nearest rank: ceil(num * n / den), exact in 128-bit integers
    const unsigned __int128 prod = (unsigned __int128)num * (unsigned __int128)n;
    int64_t rank = (int64_t)((prod + (unsigned __int128)(den - 1)) / (unsigned __int128)den);
    if (rank < 1) rank = 1;
    if (rank > n) rank = n;
    return from_hip(fp8k::launch_calibrate_percentile(x, n, rank, value_out, scale_out, ws, stream));
}

fp8_status_t fp8_quantize_mx(const float* x, int64_t rows, int64_t K, int64_t ldx, uint8_t* q, int64_t ldq,
                             uint8_t* scales, hipStream_t stream) {
    FP8_TRY(check_dims(rows, 1, K));
    if (K % 128 != 0) return FP8_ERR_UNSUPPORTED;
    FP8_TRY(check_matrix(x, rows, K, ldx, 4));
    FP8_TRY(check_matrix(q, rows, K, ldq, 1));
    FP8_TRY(check_matrix(scales, K / 128, 4 * rows, 4 * rows, 1, true));
    if (rows == 0 || K == 0) return FP8_OK;
    return from_hip(fp8k::launch_quantize_mx(x, ldx, q, ldq, scales, rows, K, stream));
}

// The block-scaled GEMM's workspace: the skinny kernel's split-K partial
// sums (M <= 64); none for the MFMA kernel.
static size_t mx_ws_bytes(int64_t M, int64_t N, int64_t K) { return gemm_ws_bytes(M, N, K); }

size_t fp8_mx_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (check_dims(M, N, K) != FP8_OK || K % 128 != 0) return SIZE_MAX;
    return mx_ws_bytes(M, N, K);
}

fp8_status_t fp8_gemm_mx(const uint8_t* qa, int64_t lda, const uint8_t* sa, const uint8_t* qw, int64_t ldw,
                         const uint8_t* sw, uint16_t* y, int64_t ldy, int64_t M, int64_t N, int64_t K, void* ws,
                         size_t ws_bytes, hipStream_t stream) {
    FP8_TRY(check_dims(M, N, K));
    if (K % 128 != 0) return FP8_ERR_UNSUPPORTED;
    FP8_TRY(check_matrix(qa, M, K, lda, 1));
    FP8_TRY(check_matrix(qw, N, K, ldw, 1));
    FP8_TRY(check_matrix(y, M, N, ldy, 2, true));
    // block scales: unit-stride rows of K / 32 bytes, read as 32-bit words
    if (M > 0 && N > 0 && K > 0) {
        if (qa == nullptr || qw == nullptr || sa == nullptr || sw == nullptr) return FP8_ERR_INVALID_ARGUMENT;
        if ((reinterpret_cast<uintptr_t>(sa) & 3u) != 0 || (reinterpret_cast<uintptr_t>(sw) & 3u) != 0)
            return FP8_ERR_UNSUPPORTED;
    }
    const size_t need = mx_ws_bytes(M, N, K);
    if (ws_bytes < need) return FP8_ERR_WORKSPACE;
    if (need > 0 && ws == nullptr) return FP8_ERR_INVALID_ARGUMENT;
    if (need > 0 && !aligned16(ws)) return FP8_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return FP8_OK;
    if (M <= fp8k::kSkinnyMaxM)
        return from_hip(fp8k::launch_gemm_skinny_mx(qa, lda, sa, qw, ldw, sw, y, ldy, M, N, K, ws, stream));
    return from_hip(fp8k::launch_gemm_mfma_mx(qa, lda, sa, qw, ldw, sw, y, ldy, M, N, K, stream));
}

size_t fp8_kv_scales_workspace_bytes(int64_t T, int64_t C) {
    if (check_kv_dims(T, C) != FP8_OK) return SIZE_MAX;
    return round_up(fp8k::kv_scales_ws_bytes(T, C), kAlign);
}

fp8_status_t fp8_kv_channel_scales(const void* kv, fp8_kv_dtype_t kv_dtype, int64_t T, int64_t C, int64_t ldkv,
                                   fp8_kv_format_t fmt, float* scales, void* ws, size_t ws_bytes,
                                   hipStream_t stream) {
    FP8_TRY(check_kv_dims(T, C));
    FP8_TRY(check_kv_format(fmt));
    int64_t eb = 0;
    FP8_TRY(kv_row_type(kv_dtype, C, &eb));
    FP8_TRY(check_matrix(kv, T, C, ldkv, eb));
    FP8_TRY(check_vector(scales, C));
    if (C == 0) return FP8_OK;
    const size_t need = round_up(fp8k::kv_scales_ws_bytes(T, C), kAlign);
    if (ws_bytes < need) return FP8_ERR_WORKSPACE;
    if (ws == nullptr) return FP8_ERR_INVALID_ARGUMENT;
    if (!aligned16(ws)) return FP8_ERR_UNSUPPORTED;
    return from_hip(fp8k::launch_kv_channel_scales(kv, (int)kv_dtype, T, C, ldkv, (int)fmt, scales, ws, stream));
}

fp8_status_t fp8_kv_quantize_paged(const void* kv, fp8_kv_dtype_t kv_dtype, int64_t T, int64_t C, int64_t ldkv,
                                   const float* scales, fp8_kv_format_t fmt, const int32_t* slot_mapping,
                                   uint8_t* cache, int64_t num_slots, hipStream_t stream) {
    FP8_TRY(check_kv_dims(T, C));
    FP8_TRY(check_kv_format(fmt));
    int64_t eb = 0;
    FP8_TRY(kv_row_type(kv_dtype, C, &eb));
    if (num_slots < 0) return FP8_ERR_INVALID_ARGUMENT;
    if (num_slots > kMaxDim) return FP8_ERR_UNSUPPORTED;
    FP8_TRY(check_matrix(kv, T, C, ldkv, eb));
    FP8_TRY(check_vector(scales, T > 0 ? C : 0));
    FP8_TRY(check_matrix(cache, num_slots, C, C, 1, true));
    if (T > 0 && slot_mapping == nullptr) return FP8_ERR_INVALID_ARGUMENT;
    if (T > 0 && (reinterpret_cast<uintptr_t>(slot_mapping) & 3u) != 0) return FP8_ERR_UNSUPPORTED;
    if (T == 0 || C == 0 || num_slots == 0) return FP8_OK;
    return from_hip(fp8k::launch_kv_quantize_paged(kv, (int)kv_dtype, T, C, ldkv, scales, (int)fmt, slot_mapping,
                                                   cache, num_slots, stream));
}

fp8_status_t fp8_kv_dequantize_paged(const uint8_t* cache, int64_t num_slots, const int32_t* slot_mapping,
                                     int64_t T, int64_t C, const float* scales, fp8_kv_format_t fmt, void* out,
                                     fp8_kv_dtype_t out_dtype, int64_t ldo, hipStream_t stream) {
    FP8_TRY(check_kv_dims(T, C));
    FP8_TRY(check_kv_format(fmt));
    int64_t eb = 0;
    FP8_TRY(kv_row_type(out_dtype, C, &eb));
    if (num_slots < 0) return FP8_ERR_INVALID_ARGUMENT;
    if (num_slots > kMaxDim) return FP8_ERR_UNSUPPORTED;
    FP8_TRY(check_matrix(cache, num_slots, C, C, 1, true));
    FP8_TRY(check_matrix(out, T, C, ldo, eb));
    FP8_TRY(check_vector(scales, T > 0 ? C : 0));
    if (T > 0 && slot_mapping == nullptr) return FP8_ERR_INVALID_ARGUMENT;
    if (T > 0 && (reinterpret_cast<uintptr_t>(slot_mapping) & 3u) != 0) return FP8_ERR_UNSUPPORTED;
    if (T == 0 || C == 0) return FP8_OK;
    return from_hip(fp8k::launch_kv_dequantize_paged(cache, num_slots, slot_mapping, T, C, scales, (int)fmt, out,
                                                     (int)out_dtype, ldo, stream));
}

fp8_status_t fp8_kv_append_rope_paged(const void* q, int64_t ldq, void* q_out, int64_t ldqo, const void* k,
                                      int64_t ldk, const void* v, int64_t ldv, fp8_kv_dtype_t dtype, int64_t T,
                                      int64_t Hq, int64_t Hkv, int64_t D, const int32_t* positions,
                                      const float* cos_sin, int64_t P, int64_t rot_dim, int32_t interleaved,
                                      const float* scales, fp8_kv_format_t fmt, const int32_t* slot_mapping,
                                      uint8_t* cache, int64_t num_slots, hipStream_t stream) {
    if (T < 0 || Hq < 0 || Hkv < 0 || D < 0 || P < 0 || rot_dim < 0 || num_slots < 0) return FP8_ERR_INVALID_ARGUMENT;
    if (T > kMaxDim || D > kMaxDim || P > kMaxDim || num_slots > kMaxDim) return FP8_ERR_UNSUPPORTED;
    if (D % 16 != 0 || D == 0 || rot_dim % 16 != 0 || rot_dim == 0) return FP8_ERR_UNSUPPORTED;
    if (rot_dim > D) return FP8_ERR_INVALID_ARGUMENT;
    if (Hq > kMaxDim / D || Hkv > kMaxDim / (2 * D) || (Hq + 2 * Hkv) * D > kMaxDim - 4096) return FP8_ERR_UNSUPPORTED;
    FP8_TRY(check_kv_format(fmt));
    const int64_t eb = kv_elem_bytes(dtype);
    if (eb == 0) return FP8_ERR_INVALID_ARGUMENT;
    FP8_TRY(check_matrix(q, T, Hq * D, ldq, eb));
    FP8_TRY(check_matrix(q_out, T, Hq * D, ldqo, eb));
    FP8_TRY(check_matrix(k, T, Hkv * D, ldk, eb));
    FP8_TRY(check_matrix(v, T, Hkv * D, ldv, eb));
    FP8_TRY(check_matrix(cos_sin, T > 0 ? P : 0, rot_dim, rot_dim, 4));
    FP8_TRY(check_vector(scales, T > 0 ? 2 * Hkv * D : 0));
    FP8_TRY(check_matrix(cache, num_slots, 2 * Hkv * D, 2 * Hkv * D, 1, true));
    if (T > 0 && (positions == nullptr || (Hkv > 0 && slot_mapping == nullptr))) return FP8_ERR_INVALID_ARGUMENT;
    if (((reinterpret_cast<uintptr_t>(positions) | reinterpret_cast<uintptr_t>(slot_mapping)) & 3u) != 0)
        return FP8_ERR_UNSUPPORTED;
    if (T == 0 || P == 0 || Hq + Hkv == 0) return FP8_OK;
    fp8k::KvAppend p;
    p.q = q, p.k = k, p.v = v, p.q_out = q_out;
    p.ldq = ldq, p.ldk = ldk, p.ldv = ldv, p.ldqo = ldqo;
    p.positions = positions, p.cos_sin = cos_sin, p.scales = scales, p.slot = slot_mapping;
    p.cache = cache, p.num_slots = num_slots;
    p.T = (int)T, p.Hq = (int)Hq, p.Hkv = (int)Hkv, p.D = (int)D, p.rot = (int)rot_dim, p.P = (int)P;
    p.tokens_per_block = 1;
    return from_hip(fp8k::launch_kv_append_rope(p, (int)dtype, (int)fmt, interleaved != 0, stream));
}

size_t fp8_attn_decode_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t block_size,
                                       int64_t max_blocks, int64_t max_len) {
    if (check_attn_dims(B, B, Hq, Hkv, D, block_size, max_blocks, 1, max_len) != FP8_OK) return SIZE_MAX;
    return attn_ws(B, B, Hq, Hkv, D, block_size, max_blocks, 1, max_len);
}

fp8_status_t fp8_attn_decode_paged(const void* q, int64_t ldq, fp8_kv_dtype_t dtype, const uint8_t* cache,
                                   int64_t num_blocks, int64_t block_size, const float* scales, fp8_kv_format_t fmt,
                                   const int32_t* block_table, int64_t ld_table, int64_t max_blocks,
                                   const int32_t* seq_lens, int64_t B, int64_t Hq, int64_t Hkv, int64_t D,
                                   int64_t max_len, float sm_scale, float softcap, const float* alibi_slopes,
                                   int64_t window, void* out, int64_t ldo, float* lse, void* ws, size_t ws_bytes,
                                   hipStream_t stream) {
    fp8k::PagedAttn p = {};
    p.q = q, p.ldq = ldq, p.out = out, p.ldo = ldo, p.lse = lse;
    p.cache = cache, p.num_blocks = num_blocks, p.scales = scales;
    p.block_table = block_table, p.ld_table = ld_table, p.seq_lens = seq_lens;
    p.softcap = softcap, p.alibi = alibi_slopes, p.causal = 1;
    return attn(p, dtype, fmt, B, B, Hq, Hkv, D, block_size, max_blocks, 1, max_len, window, sm_scale, ws, ws_bytes,
                stream);
}

size_t fp8_attn_prefill_workspace_bytes(int64_t T, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t block_size,
                                        int64_t max_blocks, int64_t max_q, int64_t max_len) {
    if (check_attn_dims(T, B, Hq, Hkv, D, block_size, max_blocks, max_q, max_len) != FP8_OK) return SIZE_MAX;
    return attn_ws(T, B, Hq, Hkv, D, block_size, max_blocks, max_q, max_len);
}

fp8_status_t fp8_attn_prefill_paged(const void* q, int64_t ldq, fp8_kv_dtype_t dtype, const int32_t* cu_q, int64_t T,
                                    const uint8_t* cache, int64_t num_blocks, int64_t block_size, const float* scales,
                                    fp8_kv_format_t fmt, const int32_t* block_table, int64_t ld_table,
                                    int64_t max_blocks, const int32_t* seq_lens, int64_t B, int64_t Hq, int64_t Hkv,
                                    int64_t D, int64_t max_q, int64_t max_len, int32_t causal,
                                    const int32_t* prefix_lens, float sm_scale, float softcap,
                                    const float* alibi_slopes, int64_t window, void* out, int64_t ldo, float* lse,
                                    void* ws, size_t ws_bytes, hipStream_t stream) {
    if (T > 0 && B > 0 && cu_q == nullptr) return FP8_ERR_INVALID_ARGUMENT;
    fp8k::PagedAttn p = {};
    p.q = q, p.ldq = ldq, p.out = out, p.ldo = ldo, p.lse = lse, p.cu_q = cu_q;
    p.cache = cache, p.num_blocks = num_blocks, p.scales = scales;
    p.block_table = block_table, p.ld_table = ld_table, p.seq_lens = seq_lens, p.prefix = prefix_lens;
    p.softcap = softcap, p.alibi = alibi_slopes, p.causal = causal != 0;
    return attn(p, dtype, fmt, T, B, Hq, Hkv, D, block_size, max_blocks, max_q, max_len, window, sm_scale, ws, ws_bytes,
                stream);
}

fp8_status_t fp8_gemm_scaled(const uint8_t* qa, int64_t lda, const float* s_tok, const uint8_t* qw,
                             int64_t ldw, const float* s_ch, uint16_t* y, int64_t ldy, int64_t M, int64_t N,
                             int64_t K, void* ws, size_t ws_bytes, hipStream_t stream) {
    FP8_TRY(check_dims(M, N, K));
    FP8_TRY(check_matrix(qa, M, K, lda, 1));
    FP8_TRY(check_matrix(qw, N, K, ldw, 1));
    FP8_TRY(check_vector(s_tok, M));
    FP8_TRY(check_vector(s_ch, N));
    FP8_TRY(check_matrix(y, M, N, ldy, 2, true));
    // operands are read only when the output is non-empty
    if (M > 0 && N > 0 && K > 0 && (qa == nullptr || qw == nullptr)) return FP8_ERR_INVALID_ARGUMENT;
    const size_t need = gemm_ws_bytes(M, N, K);
    if (ws_bytes < need) return FP8_ERR_WORKSPACE;
    if (need > 0 && ws == nullptr) return FP8_ERR_INVALID_ARGUMENT;
    if (need > 0 && !aligned16(ws)) return FP8_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return FP8_OK;
    return gemm_dispatch(qa, lda, s_tok, qw, ldw, s_ch, y, nullptr, ldy, M, N, K, ws, stream);
}

fp8_status_t fp8_quant_gemm_fused(const float* x, int64_t ldx, const uint8_t* qw, int64_t ldw,
                                  const float* s_ch, uint16_t* y, int64_t ldy, int64_t M, int64_t N, int64_t K,
                                  uint8_t* qa_out, float* s_tok_out, void* ws, size_t ws_bytes,
                                  hipStream_t stream) {
    FP8_TRY(check_dims(M, N, K));
    FP8_TRY(check_matrix(x, M, K, ldx, 4));
    FP8_TRY(check_matrix(qw, N, K, ldw, 1));
    FP8_TRY(check_vector(s_ch, N));
    FP8_TRY(check_matrix(y, M, N, ldy, 2, true));
    if (qa_out) FP8_TRY(check_matrix(qa_out, M, K, K, 1));
    if (s_tok_out) FP8_TRY(check_vector(s_tok_out, M));
    if (M > 0 && N > 0 && K > 0 && qw == nullptr) return FP8_ERR_INVALID_ARGUMENT;
    const size_t need = fp8_workspace_bytes(M, N, K);
    if (ws_bytes < need) return FP8_ERR_WORKSPACE;
    if (need > 0 && ws == nullptr) return FP8_ERR_INVALID_ARGUMENT;
    if (need > 0 && !aligned16(ws)) return FP8_ERR_UNSUPPORTED;
    if (M == 0) return FP8_OK;
    if (N > 0 && fp8k::gemm_skinny_fused_fits(M, N, K))
        return from_hip(fp8k::launch_gemm_skinny_fused(x, ldx, qw, ldw, s_ch, y, ldy, M, N, K, qa_out, s_tok_out,
                                                       stream));
    uint8_t* base = static_cast<uint8_t*>(ws);
    uint8_t* qa = qa_out ? qa_out : base;
    float* s_tok = s_tok_out ? s_tok_out : reinterpret_cast<float*>(base + round_up((size_t)M * (size_t)K, kAlign));
    FP8_TRY(from_hip(fp8k::launch_quantize_rows(x, ldx, qa, K, s_tok, M, K, stream)));
    if (N == 0) return FP8_OK;
    return gemm_dispatch(qa, K, s_tok, qw, ldw, s_ch, y, nullptr, ldy, M, N, K, base + fused_stage_bytes(M, K),
                         stream);
}

fp8_status_t fp8_gemm_scaled_fp8out(const uint8_t* qa, int64_t lda, const float* s_tok, const uint8_t* qw,
                                    int64_t ldw, const float* s_ch, uint8_t* q_out, int64_t ldq, float* s_out,
                                    float* y32_out, int64_t M, int64_t N, int64_t K, void* ws, size_t ws_bytes,
                                    hipStream_t stream) {
    FP8_TRY(check_dims(M, N, K));
    if (N % 16 != 0) return FP8_ERR_UNSUPPORTED;  // output rows are quantized in 16-byte pieces
    FP8_TRY(check_matrix(qa, M, K, lda, 1));
    FP8_TRY(check_matrix(qw, N, K, ldw, 1));
    FP8_TRY(check_vector(s_tok, M));
    FP8_TRY(check_vector(s_ch, N));
    FP8_TRY(check_matrix(q_out, M, N, ldq, 1));
    FP8_TRY(check_vector(s_out, M));
    if (y32_out) FP8_TRY(check_matrix(y32_out, M, N, N, 4));
    if (M > 0 && N > 0 && K > 0 && (qa == nullptr || qw == nullptr)) return FP8_ERR_INVALID_ARGUMENT;
    int64_t mn;
    if (!mul_ok(M, N, &mn) || mn > INT64_MAX / 8) return FP8_ERR_INVALID_ARGUMENT;
    const size_t stage = y32_out ? 0 : fp8out_stage_bytes(M, N);
    const size_t need = stage + gemm_ws_bytes(M, N, K);
    if (ws_bytes < need) return FP8_ERR_WORKSPACE;
    if (need > 0 && ws == nullptr) return FP8_ERR_INVALID_ARGUMENT;
    if (need > 0 && !aligned16(ws)) return FP8_ERR_UNSUPPORTED;
    if (M == 0) return FP8_OK;
    float* y32 = y32_out ? y32_out : static_cast<float*>(ws);
    if (N > 0)
        FP8_TRY(gemm_dispatch(qa, lda, s_tok, qw, ldw, s_ch, nullptr, y32, N, M, N, K,
                              static_cast<uint8_t*>(ws) + stage, stream));
    return from_hip(fp8k::launch_quantize_rows(y32, N, q_out, ldq, s_out, M, N, stream));
}

fp8_status_t fp8_gemm_grouped_scaled(const uint8_t* qa, const float* s_tok, const int32_t* row_token,
                                     const int32_t* expert_offsets, const uint8_t* qw, const float* s_ch,
                                     uint16_t* y, int64_t T, int64_t R, int64_t E, int64_t N, int64_t K,
                                     void* ws, size_t ws_bytes, hipStream_t stream) {
    (void)ws;
    FP8_TRY(check_dims(T, N, K));
    if (R < 0 || E < 0) return FP8_ERR_INVALID_ARGUMENT;
    if (R > kMaxDim || E > 1024) return FP8_ERR_UNSUPPORTED;
    if (!tiles_ok((R + 127) / 128 + E, N)) return FP8_ERR_UNSUPPORTED;
    if (R > 0 && E == 0) return FP8_ERR_INVALID_ARGUMENT;
    if (R > 0 && T == 0) return FP8_ERR_INVALID_ARGUMENT;
    FP8_TRY(check_matrix(qa, T, K, K, 1));
    FP8_TRY(check_vector(s_tok, T));
    FP8_TRY(check_vector(row_token, R));
    FP8_TRY(check_vector(expert_offsets, R > 0 ? E + 1 : 0));
    int64_t en;
    if (!mul_ok(E, N, &en)) return FP8_ERR_INVALID_ARGUMENT;
    FP8_TRY(check_matrix(qw, en, K, K, 1));
    FP8_TRY(check_vector(s_ch, en));
    FP8_TRY(check_matrix(y, R, N, N, 2, true));
    if (R > 0 && N > 0 && K > 0 && (qa == nullptr || qw == nullptr)) return FP8_ERR_INVALID_ARGUMENT;
    if (ws_bytes < fp8_grouped_workspace_bytes(T, R, E, N, K)) return FP8_ERR_WORKSPACE;
    if (R == 0 || N == 0) return FP8_OK;
    if (K % 128 == 0)
        return from_hip(fp8k::launch_gemm_grouped_mfma(qa, s_tok, row_token, expert_offsets, qw, s_ch, y, T, R, E,
                                                       N, K, stream));
    return from_hip(fp8k::launch_gemm_grouped(qa, s_tok, row_token, expert_offsets, qw, s_ch, y, T, R, E, N, K,
                                              stream));
}

size_t fp8_gemm_act_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (check_dims(M, N, K) != FP8_OK || !act_tiles_ok((M + 127) / 128, N)) return SIZE_MAX;
    if (fp8k::skinny_act(M, N)) return 0;
    return round_up(std::max(fp8k::act_plan_ws_bytes(fp8k::act_plan(M, N, K, false), M, N),
                             fp8k::act_plan_ws_bytes(fp8k::act_plan(M, N, K, true), M, N)), kAlign);
}

fp8_status_t fp8_gemm_scaled_act(const uint8_t* qa, int64_t lda, const float* s_tok, const uint8_t* qw, int64_t ldw,
                                 const float* s_ch, const float* bias, fp8_act_t act, const void* residual, int64_t ldr,
                                 void* y, fp8_kv_dtype_t y_dtype, int64_t ldy, int64_t M, int64_t N, int64_t K, void* ws,
                                 size_t ws_bytes, hipStream_t stream) {
    FP8_TRY(check_dims(M, N, K));
    if (!act_tiles_ok((M + 127) / 128, N)) return FP8_ERR_UNSUPPORTED;
    FP8_TRY(check_matrix(qa, M, K, lda, 1));
    FP8_TRY(check_matrix(qw, N, K, ldw, 1));
    FP8_TRY(check_vector(s_tok, M));
    FP8_TRY(check_vector(s_ch, N));
    const fp8k::Epilogue epi{bias, residual, y, ldr, ldy, (int)act, (int)y_dtype};
    FP8_TRY(check_epilogue(epi, act, y_dtype, N, M, N));
    const size_t need = fp8_gemm_act_workspace_bytes(M, N, K);
    if (ws_bytes < need) return FP8_ERR_WORKSPACE;
    if (need > 0 && ws == nullptr) return FP8_ERR_INVALID_ARGUMENT;
    if (need > 0 && !aligned16(ws)) return FP8_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return FP8_OK;
    if (at_any(y, {qa, s_tok, qw, s_ch, bias})) return FP8_ERR_INVALID_ARGUMENT;
    if (fp8k::skinny_act(M, N))
        return from_hip(fp8k::launch_gemm_skinny_act(qa, lda, s_tok, qw, ldw, s_ch, epi, M, N, K, stream));
    return from_hip(fp8k::launch_gemm_mfma_act(qa, lda, s_tok, qw, ldw, s_ch, epi, M, N, K, ws, stream));
}

fp8_status_t fp8_gemm_grouped_scaled_act(const uint8_t* qa, const float* s_tok, const int32_t* row_token,
                                         const int32_t* expert_offsets, const uint8_t* qw, const float* s_ch,
                                         const float* bias, fp8_act_t act, void* y, fp8_kv_dtype_t y_dtype, int64_t ldy,
                                         int64_t T, int64_t R, int64_t E, int64_t N, int64_t K, void* ws,
                                         size_t ws_bytes, hipStream_t stream) {
    (void)ws;
    FP8_TRY(check_dims(T, N, K));
    if (R < 0 || E < 0) return FP8_ERR_INVALID_ARGUMENT;
    if (R > kMaxDim || E > kMaxExperts) return FP8_ERR_UNSUPPORTED;
    if (!act_tiles_ok((R + 127) / 128 + E, N)) return FP8_ERR_UNSUPPORTED;
    if (R > 0 && (E == 0 || T == 0)) return FP8_ERR_INVALID_ARGUMENT;
    FP8_TRY(check_matrix(qa, T, K, K, 1));
    FP8_TRY(check_vector(s_tok, T));
    FP8_TRY(check_vector(row_token, R));
    FP8_TRY(check_vector(expert_offsets, R > 0 ? E + 1 : 0));
    FP8_TRY(check_matrix(qw, E * N, K, K, 1));
    FP8_TRY(check_vector(s_ch, E * N));
    const fp8k::Epilogue epi{bias, nullptr, y, 0, ldy, (int)act, (int)y_dtype};
    FP8_TRY(check_epilogue(epi, act, y_dtype, E * N, R, N));
    if (ws_bytes < fp8_grouped_workspace_bytes(T, R, E, N, K)) return FP8_ERR_WORKSPACE;
    if (R == 0 || N == 0) return FP8_OK;
    if (at_any(y, {qa, s_tok, row_token, expert_offsets, qw, s_ch, bias})) return FP8_ERR_INVALID_ARGUMENT;
    return from_hip(fp8k::launch_gemm_grouped_mfma_act(qa, s_tok, row_token, expert_offsets, qw, s_ch, epi, T, R, E, N, K,
                                                       stream));
}

fp8_status_t fp8_act_quantize(const void* h, int64_t ldh, fp8_kv_dtype_t dtype, int64_t rows, int64_t F, fp8_act_t act,
                              int32_t gated, uint8_t* q, int64_t ldq, float* scales, const int32_t* live_rows,
                              hipStream_t stream) {
    FP8_TRY(check_dims(rows, 1, F));
    FP8_TRY(check_act(act));
    const int64_t eb = kv_elem_bytes(dtype);
    if (eb == 0) return FP8_ERR_INVALID_ARGUMENT;
    FP8_TRY(check_matrix(h, rows, gated ? 2 * F : F, ldh, eb));
    FP8_TRY(check_matrix(q, rows, F, ldq, 1));
    FP8_TRY(check_vector(scales, rows));
    if (live_rows != nullptr) FP8_TRY(check_words(live_rows, 1));
    if (rows == 0) return FP8_OK;
    if ((F > 0 && at_any(q, {h, live_rows, scales})) || at_any(scales, {F > 0 ? h : nullptr, live_rows}))
        return FP8_ERR_INVALID_ARGUMENT;
    return from_hip(fp8k::launch_act_quantize(h, ldh, (int)dtype, rows, F, (int)act, gated != 0, q, ldq, scales,
                                              live_rows, stream));
}

size_t fp8_moe_sort_workspace_bytes(int64_t T, int64_t topk, int64_t E) {
    if (check_choices(T, topk, 0, 0) != FP8_OK || E < 0 || E > kMaxExperts) return SIZE_MAX;
    return round_up(fp8k::moe_sort_ws_bytes(T * topk, E), kAlign);
}

fp8_status_t fp8_moe_sort(const void* expert_ids, int32_t ids_64, int64_t T, int64_t topk, int64_t E,
                          int32_t* expert_offsets, int32_t* row_token, int32_t* row_of, void* ws, size_t ws_bytes,
                          hipStream_t stream) {
    FP8_TRY(check_choices(T, topk, 0, 0));
    if (E < 0) return FP8_ERR_INVALID_ARGUMENT;
    if (E > kMaxExperts) return FP8_ERR_UNSUPPORTED;
    const int64_t R = T * topk;
    FP8_TRY(check_vector(expert_ids, R));
    FP8_TRY(check_vector(expert_offsets, E + 1));
    FP8_TRY(check_vector(row_token, R));
    FP8_TRY(check_vector(row_of, R));
    const size_t need = fp8_moe_sort_workspace_bytes(T, topk, E);
    if (ws_bytes < need) return FP8_ERR_WORKSPACE;
    if (need > 0 && ws == nullptr) return FP8_ERR_INVALID_ARGUMENT;
    if (need > 0 && !aligned16(ws)) return FP8_ERR_UNSUPPORTED;
    if (R > 0 && (at_any(expert_offsets, {expert_ids, row_token, row_of}) || at_any(row_token, {expert_ids, row_of}) ||
                  row_of == expert_ids))
        return FP8_ERR_INVALID_ARGUMENT;
    return from_hip(fp8k::launch_moe_sort(expert_ids, ids_64 != 0, R, topk, E, expert_offsets, row_token, row_of, ws,
                                          stream));
}

fp8_status_t fp8_moe_permute(const void* x, int64_t ldx, const float* s_tok, const int32_t* row_of, int64_t T,
                             int64_t topk, int64_t R, int64_t H, int64_t elem_bytes, void* out, int64_t ldo,
                             float* s_out, hipStream_t stream) {
    FP8_TRY(check_choices(T, topk, R, H));
    if (elem_bytes != 1 && elem_bytes != 2 && elem_bytes != 4) return FP8_ERR_INVALID_ARGUMENT;
    FP8_TRY(check_rows(x, T, H, ldx, elem_bytes));
    FP8_TRY(check_rows(out, R, H, ldo, elem_bytes));
    FP8_TRY(check_vector(row_of, T * topk));
    if ((s_tok == nullptr) != (s_out == nullptr)) return FP8_ERR_INVALID_ARGUMENT;
    if (s_tok != nullptr) {
        FP8_TRY(check_vector(s_tok, T));
        FP8_TRY(check_vector(s_out, R));
    }
    if (T == 0 || topk == 0 || R == 0 || (H == 0 && s_tok == nullptr)) return FP8_OK;
    if ((H > 0 && at_any(out, {x, row_of, s_tok, s_out})) || at_any(s_out, {H > 0 ? x : nullptr, row_of, s_tok}))
        return FP8_ERR_INVALID_ARGUMENT;
    return from_hip(fp8k::launch_moe_permute(x, ldx * elem_bytes, s_tok, row_of, T, topk, R, H * elem_bytes, out,
                                             ldo * elem_bytes, s_out, stream));
}

fp8_status_t fp8_moe_combine(const void* y, int64_t ldy, fp8_kv_dtype_t y_dtype, const int32_t* row_of,
                             const float* weights, const void* residual, int64_t ldr, void* out,
                             fp8_kv_dtype_t out_dtype, int64_t ldo, int64_t T, int64_t topk, int64_t R, int64_t H,
                             hipStream_t stream) {
    FP8_TRY(check_choices(T, topk, R, H));
    const int64_t yb = kv_elem_bytes(y_dtype), ob = kv_elem_bytes(out_dtype);
    if (yb == 0 || ob == 0) return FP8_ERR_INVALID_ARGUMENT;
    FP8_TRY(check_rows(y, R, H, ldy, yb));
    FP8_TRY(check_rows(out, T, H, ldo, ob));
    if (residual != nullptr) FP8_TRY(check_rows(residual, T, H, ldr, ob));
    FP8_TRY(check_vector(row_of, T * topk));
    if (weights != nullptr) FP8_TRY(check_vector(weights, T * topk));
    if (T == 0 || H == 0) return FP8_OK;
    if (at_any(out, {R > 0 ? y : nullptr, topk > 0 ? row_of : nullptr, topk > 0 ? weights : nullptr}) ||
        (residual != nullptr && !in_place_ok(residual, ldr, out, ldo, T, H)))
        return FP8_ERR_INVALID_ARGUMENT;
    fp8k::MoeCombine p = {};
    p.y = y, p.row_of = row_of, p.weights = weights, p.residual = residual, p.out = out;
    p.ldy = ldy, p.ldr = ldr, p.ldo = ldo, p.H = H;
    p.T = (int)T, p.R = (int)R;
    p.topk = R > 0 ? (int)topk : 0;  // without rows every choice is without one
    return from_hip(fp8k::launch_moe_combine(p, (int)y_dtype, (int)out_dtype, stream));
}

fp8_status_t fp8_moe_combine_grad(const void* dout, int64_t ldd, fp8_kv_dtype_t dout_dtype, const void* y, int64_t ldy,
                                  fp8_kv_dtype_t y_dtype, const int32_t* row_of, const float* weights, void* dy,
                                  int64_t lddy, float* dweights, int64_t T, int64_t topk, int64_t R, int64_t H,
                                  hipStream_t stream) {
    FP8_TRY(check_choices(T, topk, R, H));
    const int64_t db = kv_elem_bytes(dout_dtype), yb = kv_elem_bytes(y_dtype);
    if (db == 0 || yb == 0) return FP8_ERR_INVALID_ARGUMENT;
    FP8_TRY(check_rows(dout, T, H, ldd, db));
    if (dweights != nullptr) {
        FP8_TRY(check_rows(y, R, H, ldy, yb));
        FP8_TRY(check_vector(dweights, T * topk));
    }
    if (dy != nullptr) FP8_TRY(check_rows(dy, R, H, lddy, yb));
    FP8_TRY(check_vector(row_of, T * topk));
    if (weights != nullptr) FP8_TRY(check_vector(weights, T * topk));
    if (T == 0 || topk == 0 || (dy == nullptr && dweights == nullptr)) return FP8_OK;
    if (R > 0 && H > 0 && (at_any(dy, {dout, row_of, weights, dweights}) || at_any(dweights, {dout, y}) ||
                           (dy != nullptr && dweights != nullptr && !in_place_ok(y, ldy, dy, lddy, R, H))))
        return FP8_ERR_INVALID_ARGUMENT;
    if (at_any(dweights, {row_of, weights})) return FP8_ERR_INVALID_ARGUMENT;
    fp8k::MoeCombineGrad p = {};
    p.dout = dout, p.y = y, p.row_of = row_of, p.weights = weights, p.dy = dy, p.dweights = dweights;
    p.ldd = ldd, p.ldy = ldy, p.lddy = lddy, p.H = H;
    p.T = (int)T, p.topk = (int)topk, p.R = (int)R;
    return from_hip(fp8k::launch_moe_combine_grad(p, (int)dout_dtype, (int)y_dtype, stream));
}

fp8_status_t fp8_stream_read(const void* p, size_t bytes, int32_t workgroups, int32_t nontemporal, uint32_t* sink,
                             hipStream_t stream) {
    if (bytes % 16 != 0 || workgroups < 1 || workgroups > (1 << 20)) return FP8_ERR_INVALID_ARGUMENT;
    if (bytes > 0 && (p == nullptr || sink == nullptr)) return FP8_ERR_INVALID_ARGUMENT;
    if (bytes > 0 && (!aligned16(p) || (reinterpret_cast<uintptr_t>(sink) & 3u) != 0)) return FP8_ERR_UNSUPPORTED;
    if (bytes == 0) return FP8_OK;
    return from_hip(fp8k::launch_stream_read(p, bytes, workgroups, nontemporal != 0, sink, stream));
}

}  // extern "C"
