// rf_attn.h -- host-side interface between the attention entry point and its
// kernels.
#pragma once

#include "rf_kv.cuh"

namespace rf {

// One call, as the kernels see it.
struct AttnParams {
    rf_kv_cache c;
    rf_kv_batch b;
    const void *q;
    void *out;
    const float *sinks;
    int64_t q_lt, q_lh, o_lt, o_lh;
    int64_t window;          // 0: none
    float qk_scale;          // scale * log2(e): scores are powers of two
    int n_heads, group;      // query heads; query heads per K/V head
    bool q_vec, o_vec;       // aligned for four elements at a time
    bool q_vec8;             // queries aligned for eight
    bool o_sector;           // every 32 bytes of an output row are aligned to them
    int splits;              // parts of a row's positions, joined by a second launch
    int split_blocks;        // 32-token blocks per part
    float *part_o;           // [token][head][split][head_dim]
    float2 *part_ml;         // [token][head][split]: maximum, sum
};

// Tokens of a sequence, on average and rounded up.
inline int64_t tokens_per_seq(const AttnParams &p) { return ((int64_t)p.b.n_tok + p.b.n_seq - 1) / p.b.n_seq; }

// Softmax weights are 2^(x - m + w_shift), where m is the row's maximum or up
// to w_lazy below it: at most 2^15 (2^15.5), the top of fp16's range.  The
// factor cancels between numerator and denominator.  SPLIT (fp32, two terms):
// 22 bits of weights down to 2^-17 of the largest and an absolute 2^-39 of it
// below.  One term: 11 bits down to 2^-22 and an absolute 2^-33, which lets
// maxima lag further and sums be rescaled less often (8192-token prompt: 466
// against 486 us).
template <bool SPLIT> __host__ __device__ constexpr float w_shift() { return SPLIT ? 14.f : 8.f; }
template <bool SPLIT> __host__ __device__ constexpr float w_lazy() { return SPLIT ? 1.5f : 7.f; }
constexpr float kLog2e = 1.4426950408889634f;

// The path for long chunks (128-row tiles on tcgen05), its workspace and
// whether it takes the call.
bool attn_tile_takes(const AttnParams &p, int64_t max_len);
size_t attn_tile_workspace(const AttnParams &p, int dtype, int64_t max_len);
void attn_tile_plan(const AttnParams &p, int dtype, int64_t max_len, rf_attention_plan *out);
rf_status launch_attn_tile(AttnParams p, int dtype, int64_t max_len, void *workspace, cudaStream_t s,
                           bool chain);

// Joins the parts of each row (part_o, part_ml) into out.  Whether it takes
// the rows is asked before anything is enqueued.
bool attn_join_takes(const AttnParams &p);
rf_status launch_attn_join(const AttnParams &p, int dtype, cudaStream_t s);

}  // namespace rf
