// rf_chunk.h -- host-side interface between the chunk operators' entry points
// (rf_chunk.cu) and their product kernels (rf_chunk_mma.cu, rf_chunk_few.cu).
#pragma once

#include <algorithm>

#include "rf_internal.h"

namespace rf {

// A token tile: `cnt` rows of a group, from row `row0` of the call; its
// operand image starts `gran` granules into the images.
struct ChunkTile {
    int32_t group, row0, cnt, gran;
};
struct ChunkPlan {
    int32_t n_tiles;   // token tiles
    int32_t next;      // work items drawn
    int32_t pad[62];
};

// Raw chunk of each format: weights and bytes of a row that are copied at once.
__host__ __device__ constexpr int chunk_bytes(int fmt) { return fmt == RF_Q4_0 || fmt == RF_Q4_K ? 144 : 272; }
__host__ __device__ constexpr int chunk_weights(int fmt) { return fmt == RF_MXFP4 ? 512 : 256; }

constexpr int kSliceK = 64;                  // inputs per operand slice: two 32-weight blocks
constexpr int kGranRows = 16;                // operand rows per granule (the step of the MMA's N)
constexpr int kGranBytes = kGranRows * kSliceK * 2;   // ... and its bytes per slice

// Operands of one product.  xt: fp16 terms per activation (a granule holds
// kGranRows / xt tokens: 8 rows of high terms, then 8 of low ones, when there
// are two; tiles of eight operand rows have granules of eight).  wt: fp16 terms per weight.  nt: operand rows per token tile.
struct ChunkShape {
    int fmt, xt, wt, nt;
    bool few;                                // for rf_chunk_few.cu's kernel
    int64_t n_row, n_group, rows, in_dim;
    int nst;                                 // slices (few: whole chunks, the last ones zeros)
    int64_t cap_tiles, cap_gran;             // token tiles and granules at most
    int parts, part_chunks;                  // parts of a row's raw chunks, and chunks per part
    int segment;                             // slices after which 16-bit calls' sums leave the tensor cores (a power of two)
    bool segments;                           // a part has several such segments
    size_t at_tiles, at_inv, at_img, at_sums, at_held, bytes;   // workspace: plan, tiles, 1 / row scale, images, parts'
                                                                // sums, segments' sums (a tile for each CTA)
    size_t upto;                             // bytes that do for this call and every one of fewer rows
    int tile_tokens() const { return nt / xt; }
    int gran_rows() const { return std::min(nt, kGranRows); }   // (8: half a granule)
    int gran_tokens() const { return gran_rows() / xt; }
    int gran_bytes() const { return gran_rows() * kSliceK * 2; }
};

// One product, as the MMA kernel's launcher takes it.
struct ChunkGemm {
    ChunkShape sh;
    const uint8_t *W, *up;        // the stacked tensors (up: gated activations)
    int64_t row0;                 // first row of group 0's window
    int64_t group_rows;           // tensor rows from one group to the next
    int64_t total_rows;           // rows of the tensors that may be read
    rf_epilogue epi;
    int dtype;                    // of Y and the residual
    void *Y;
    int64_t ldy;
    uint8_t *ws;
};

rf_status launch_chunk_mma(const ChunkGemm &g, cudaStream_t s);

// Routing of a chunk (rf_route.cu).
size_t route_workspace(int64_t n_tok, int n_expert, int top_k);
rf_status launch_route_tokens(int dtype, const void *logits, int64_t ld, int64_t n_tok, int n_expert, int top_k,
                              int32_t *idx, float *w, int32_t *offsets, int32_t *order, int32_t *place, void *workspace,
                              cudaStream_t s);

}  // namespace rf
