// Launchers of the gfx950 kernels (internal to the library; the C ABI in
// include/fp8w8a8.h validates arguments before calling these).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace fp8k {

// Per-row absmax quantization (quantize.hip).
hipError_t launch_quantize_rows(const float* x, int64_t ldx, uint8_t* q, int64_t ldq, float* scales,
                                int64_t rows, int64_t K, hipStream_t stream);
// Static per-tensor scale *scale (device, floored at 1e-12) for every row;
// scales[r] receives it for each row.
hipError_t launch_quantize_static(const float* x, int64_t ldx, const float* scale, uint8_t* q, int64_t ldq,
                                  float* scales, int64_t rows, int64_t K, hipStream_t stream);
// Per-row absmax scale with the absmax clipped at *clip (device).
hipError_t launch_quantize_clipped(const float* x, int64_t ldx, const float* clip, uint8_t* q, int64_t ldq,
                                   float* scales, int64_t rows, int64_t K, hipStream_t stream);
// Nearest-rank percentile of |x| over n values (calibrate.hip): value_out =
// the rank-th smallest |x| (1 <= rank <= n); scale_out (nullable) =
// max(fl32(value / 448), 1e-12f).  ws: kCalibrateWsBytes bytes.
constexpr size_t kCalibrateWsBytes = 2048;
hipError_t launch_calibrate_percentile(const float* x, int64_t n, int64_t rank, float* value_out, float* scale_out,
                                       void* ws, hipStream_t stream);

// FP8 KV-cache codec (kv_cache.hip).  fmt: kKvE4M3 or kKvE5M2; element
// types of the KV rows and of the read back: kKvF32, kKvBF16, kKvF16.
// C % 4 == 0, row strides in elements with 16-byte aligned rows, scales
// 16-byte aligned.
constexpr int kKvE4M3 = 0;
constexpr int kKvE5M2 = 1;
constexpr int kKvF32 = 0;
constexpr int kKvBF16 = 1;
constexpr int kKvF16 = 2;
// Row chunks of the per-channel maximum pass; its fp32 partials take
// kv_scales_ws_bytes(T, C) bytes of workspace (16-byte aligned).
struct KvChunks {
    int rows_per_chunk, chunks;
};
KvChunks kv_amax_chunks(int64_t T, int64_t C, int quads);
size_t kv_scales_ws_bytes(int64_t T, int64_t C);
hipError_t launch_kv_channel_scales(const void* kv, int dtype, int64_t T, int64_t C, int64_t ldkv, int fmt,
                                    float* scales, void* ws, hipStream_t stream);
hipError_t launch_kv_quantize_paged(const void* kv, int dtype, int64_t T, int64_t C, int64_t ldkv, const float* scales,
                                    int fmt, const int32_t* slot, uint8_t* cache, int64_t num_slots,
                                    hipStream_t stream);
hipError_t launch_kv_dequantize_paged(const uint8_t* cache, int64_t num_slots, const int32_t* slot, int64_t T,
                                      int64_t C, const float* scales, int fmt, void* out, int out_dtype, int64_t ldo,
                                      hipStream_t stream);

// Append with rotation (kv_append.hip): strides in elements, rows 16-byte
// aligned, D and rot multiples of 16; q and q_out may be null with Hq == 0, k,
// v, scales, slot and cache with Hkv == 0.
// tokens_per_block is the launcher's.
struct KvAppend {
    const void *q, *k, *v;
    void* q_out;
    int64_t ldq, ldk, ldv, ldqo;
    const int32_t* positions;
    const float* cos_sin;
    const float* scales;
    const int32_t* slot;
    uint8_t* cache;
    int64_t num_slots;
    int T, Hq, Hkv, D, rot, P, tokens_per_block;
};
hipError_t launch_kv_append_rope(const KvAppend& p, int dtype, int fmt, bool interleaved, hipStream_t stream);

// Attention over the paged cache (attn_paged.hip).  Sequence b owns q rows
// [cu_q[b], cu_q[b + 1]) (row b when cu_q is null) of `rows` rows in all;
// its key j lies in cache row block_table[b][j / block] * block + j % block.
// scale: the score scale times log2(e); softcap 0, window 0, alibi null and
// prefix null turn those off.  block_table holds one entry and
// cache one row at least.
struct PagedAttn {
    const void* q;
    void* out;
    float* lse;  // [rows, Hq], may be null
    int64_t ldq, ldo;
    const int32_t* cu_q;
    const uint8_t* cache;
    int64_t num_blocks;
    const float* scales;
    const int32_t* block_table;
    int64_t ld_table;
    const int32_t* seq_lens;
    const int32_t* prefix;
    const float* alibi;
    float scale, softcap;
    int B, rows, Hq, Hkv, block, max_blocks, window, causal, dtype;
};
// Whether the scaled query and p are fed as two fp16 terms: an fp16 or fp32
// output, or lse, would show the rounding of one.
inline bool two_terms(const PagedAttn& p) { return p.dtype != kKvBF16 || p.lse != nullptr; }

// The streaming form (attn_paged.hip), for few rows per sequence, and the tiled
// one (attn_prefill.hip), for many (attn_plan.hpp says which).  max_q, the most
// new rows of a sequence, typical, those of most, and max_len plan the launch;
// more rows and longer sequences are still computed whole.  ws: the matching
// *_ws_bytes bytes (all_len = max_blocks * block), 16-byte aligned.
size_t attn_paged_ws_bytes(int64_t B, int64_t rows, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_q, int64_t max_len,
                           int64_t all_len);
hipError_t launch_attn_paged(const PagedAttn& p, int D, int fmt, int64_t max_q, int64_t typical, int64_t max_len, void* ws,
                             hipStream_t stream);
size_t attn_tiled_ws_bytes(int64_t B, int64_t rows, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_q, int64_t max_len);
hipError_t launch_attn_tiled(const PagedAttn& p, int D, int fmt, int64_t max_q, int64_t max_len, void* ws,
                             hipStream_t stream);
// Output rows from `splits` parts each: part_o [rows][Hq][splits][D], part_ml
// (reference in log2, sum) [rows][Hq][splits].
hipError_t launch_attn_join(const PagedAttn& p, int D, int splits, float* part_o, float2* part_ml, hipStream_t stream);

// The dense GEMM launchers write BF16 y, or, when y32 is not null, the fp32
// value acc * (s_tok * s_ch) before rounding to y32 (same row stride ldy).

// Block-scaled quantization (block_scale.hip): K % 128 == 0; scales are
// chunk-major exponent bytes: word [K / 128][rows], byte j = block 4c + j.
hipError_t launch_quantize_mx(const float* x, int64_t ldx, uint8_t* q, int64_t ldq, uint8_t* scales, int64_t rows,
                              int64_t K, hipStream_t stream);

// Block ("MX") scales of both GEMM operands: exponent bytes, 2^(c - 127),
// one per 32 k of a row, chunk-major: 32-bit word [K / 128][rows] holds a
// row's 4 bytes of one 128-k chunk.  sa covers M rows, sw N rows.
struct MxScales {
    const uint8_t* sa;
    const uint8_t* sw;
};

// Largest M the skinny (decode) kernel takes.
constexpr int64_t kSkinnyMaxM = 64;

// Skinny-M scaled GEMM, M <= kSkinnyMaxM (gemm_skinny.hip).  Shapes with few
// weight rows and long k split k across workgroups; they need
// gemm_skinny_ws_bytes(M, N, K) bytes of workspace in ws (fp32 partial sums,
// fully overwritten by every call, no zero fill needed).
struct SkinnyPlan {
    int mt, nt, splits, split_chunks;
};
SkinnyPlan skinny_plan(int64_t M, int64_t N, int64_t K);
size_t gemm_skinny_ws_bytes(int64_t M, int64_t N, int64_t K);
hipError_t launch_gemm_skinny(const uint8_t* qa, int64_t lda, const float* s_tok, const uint8_t* qw,
                              int64_t ldw, const float* s_ch, uint16_t* y, float* y32, int64_t ldy, int64_t M, int64_t N,
                              int64_t K, void* ws, hipStream_t stream);

// Block-scaled skinny GEMM (K % 128 == 0): y = bf16_rne(sum over blocks of
// 2^(sa + sw - 254) * block dot); same plan and workspace as above.
hipError_t launch_gemm_skinny_mx(const uint8_t* qa, int64_t lda, const uint8_t* sa, const uint8_t* qw, int64_t ldw,
                                 const uint8_t* sw, uint16_t* y, int64_t ldy, int64_t M, int64_t N, int64_t K, void* ws,
                                 hipStream_t stream);

// Block-scaled MFMA GEMM for M > kSkinnyMaxM, K % 128 == 0 (gemm_mfma.hip).
hipError_t launch_gemm_mfma_mx(const uint8_t* qa, int64_t lda, const uint8_t* sa, const uint8_t* qw, int64_t ldw,
                               const uint8_t* sw, uint16_t* y, int64_t ldy, int64_t M, int64_t N, int64_t K,
                               hipStream_t stream);

// Quantize + skinny GEMM in one kernel, for M <= kSkinnyFusedMaxM rows whose
// codes fit in kSkinnyFusedLds bytes of LDS and N <= 8192 (gemm_skinny.hip).  qa_out and
// s_tok_out may be null; when given they receive the codes and scales.
constexpr int64_t kSkinnyFusedMaxM = 16;
constexpr int64_t kSkinnyFusedLds = 64 * 1024 + 16 * 16;
bool gemm_skinny_fused_fits(int64_t M, int64_t N, int64_t K);
hipError_t launch_gemm_skinny_fused(const float* x, int64_t ldx, const uint8_t* qw, int64_t ldw, const float* s_ch,
                                    uint16_t* y, int64_t ldy, int64_t M, int64_t N, int64_t K, uint8_t* qa_out,
                                    float* s_tok_out, hipStream_t stream);

// LDS-tiled MFMA scaled GEMM for larger M (gemm_tiled.hip).
hipError_t launch_gemm_tiled(const uint8_t* qa, int64_t lda, const float* s_tok, const uint8_t* qw,
                             int64_t ldw, const float* s_ch, uint16_t* y, float* y32, int64_t ldy, int64_t M, int64_t N,
                             int64_t K, hipStream_t stream);

// Two-stage DMA-fed MFMA GEMM, K % 128 == 0 (gemm_mfma.hip).
hipError_t launch_gemm_mfma(const uint8_t* qa, int64_t lda, const float* s_tok, const uint8_t* qw, int64_t ldw,
                            const float* s_ch, uint16_t* y, float* y32, int64_t ldy, int64_t M, int64_t N, int64_t K,
                            hipStream_t stream);

// Grouped (MoE) variant of the two-stage kernel, K % 128 == 0 (gemm_mfma.hip).
hipError_t launch_gemm_grouped_mfma(const uint8_t* qa, const float* s_tok, const int32_t* row_token,
                                    const int32_t* offsets, const uint8_t* qw, const float* s_ch, uint16_t* y,
                                    int64_t T, int64_t R, int64_t E, int64_t N, int64_t K, hipStream_t stream);

// Grouped (MoE) scaled GEMM, any K % 16 == 0 (gemm_tiled.hip).
hipError_t launch_gemm_grouped(const uint8_t* qa, const float* s_tok, const int32_t* row_token,
                               const int32_t* offsets, const uint8_t* qw, const float* s_ch, uint16_t* y,
                               int64_t T, int64_t R, int64_t E, int64_t N, int64_t K, hipStream_t stream);

// Plain streaming read of `bytes` bytes (multiple of 16, p 16-byte aligned)
// by about `workgroups` workgroups of 256 threads (stream_read.hip); sink: one
// uint32 that is written only when the folded data equals a magic value.
hipError_t launch_stream_read(const void* p, size_t bytes, int workgroups, bool nontemporal, uint32_t* sink,
                              hipStream_t stream);

}  // namespace fp8k
