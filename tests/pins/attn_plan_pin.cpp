/* The attention calls' division into workgroups, as the library computes it, for the CPU tests. */
#include "../../fp8_w8a8_quantized_quantize_amd/csrc/attn_plan.hpp"

extern "C" {

/* whether the tiled form takes the call */
void pin_form(int64_t Hq, int64_t Hkv, int64_t D, int64_t new_rows, int64_t two_terms, int64_t* out) {
    out[0] = fp8k::attn_tiled(Hq, Hkv, D, new_rows, two_terms != 0);
}

/* units, column tiles, equal shares or 0 */
void pin_stream(int64_t B, int64_t rows, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_q, int64_t max_len,
                int64_t all_len, int64_t* out) {
    const fp8k::StreamPlan s = fp8k::stream_plan(B, rows, Hq, Hkv, D, max_q, max_len, all_len);
    out[0] = s.units, out[1] = s.rows_y, out[2] = s.shares;
}

/* units, slots, splits, column tiles laid out for every sequence (and 1000 when the others are added up) */
void pin_tiled(int64_t B, int64_t rows, int64_t Hq, int64_t Hkv, int64_t D, int64_t decode, int64_t max_q, int64_t max_len,
               int64_t* out) {
    const fp8k::TilePlan t = fp8k::tile_plan(B, rows, Hq, Hkv, D, decode != 0, max_q, max_len);
    out[0] = t.units, out[1] = t.slots, out[2] = t.splits, out[3] = t.col_tiles + (t.exact ? 1000 : 0);
}

/* units, rows a sequence, thread groups a row */
void pin_join(int64_t heads, int64_t D, int64_t max_q, int64_t typical, int64_t* out) {
    const fp8k::JoinPlan j = fp8k::join_plan(heads, D, max_q, typical);
    out[0] = j.units, out[1] = j.rows, out[2] = j.spread;
}

/* launches of that many units, their units in all if they follow each other, and the largest */
void pin_launches(int64_t units, int64_t* out) {
    out[0] = out[1] = out[2] = 0;
    fp8k::in_launches(units, [&](int64_t first, int64_t n) {
        if (first == out[1]) out[1] += n;
        out[2] = n > out[2] ? n : out[2];
        ++out[0];
        return 0;
    });
}

}
