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
    int splits;              // parts of a row's positions, joined by a second launch
    int split_blocks;        // 32-token blocks per part
    float *part_o;           // [token][head][split][head_dim]
    float2 *part_ml;         // [token][head][split]: maximum, sum
};

// Softmax weights are 2^(x - m + kWShift): the largest is 2^14, so that fp16
// keeps 11 bits of weights down to 2^-28 of the largest.  The factor cancels
// between numerator and denominator.
constexpr float kWShift = 14.f;
constexpr float kLog2e = 1.4426950408889634f;

// The path for long chunks (128-row tiles on tcgen05), its workspace and
// whether it takes the call.
bool attn_tile_takes(const AttnParams &p);
size_t attn_tile_workspace(const AttnParams &p, int dtype, int64_t max_len);
rf_status launch_attn_tile(AttnParams p, int dtype, int64_t max_len, void *workspace, cudaStream_t s,
                           bool chain);

// Joins the parts of each row (part_o, part_ml) into out.
rf_status launch_attn_join(const AttnParams &p, int dtype, cudaStream_t s);

}  // namespace rf
