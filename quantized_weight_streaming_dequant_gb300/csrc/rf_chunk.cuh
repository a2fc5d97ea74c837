// rf_chunk.cuh -- what the two product kernels of the chunk operators share
// (rf_chunk_mma.cu, rf_chunk_few.cu): a launch's parameters, where a raw
// chunk's rows lie in shared memory, the decoders of quantized blocks to fp16
// pairs, the activations, bounded waits and copies.
//
// Rows of any length by tensor copies.  A tensor map's rows have to be
// multiples of 16 bytes apart; rows of rb bytes are not, but P = 16 /
// gcd(rb, 16) of them together are.  The map's rows are such super-rows, and a
// chunk of 64 matrix rows is P boxes, one for each position j in the
// super-row, whose first byte j * rb + c * (chunk bytes) is rounded down to 16;
// a thread skips the remainder.  Rows behind the last whole super-row (fewer
// than 16 of a tensor) are copied by their threads.
#pragma once

#include <cuda_bf16.h>

#include "rf_chunk.h"
#include "rf_half.cuh"
#include "rf_tcgen05.cuh"

namespace rf {
namespace chunk {

constexpr int kM = 128;              // matrix rows per item (MMA M)

__host__ __device__ constexpr int block_size(int fmt) { return fmt == RF_Q4_0 ? 18 : (fmt == RF_Q8_0 ? 34 : (fmt == RF_MXFP4 ? 17 : 144)); }

// Box bytes: the chunk's, with what rounding its first byte down takes, as an
// odd number of 16-byte units (see Block::load); with 16 matrix rows to a
// super-row an even one, which keeps the boxes 128 bytes aligned.
__host__ __device__ constexpr int box_bytes(int fmt, int P)
{
    const int n = chunk_bytes(fmt) + (fmt != RF_Q4_K && P > 1 ? 16 : 0);
    return P < 16 && n / 16 % 2 == 0 ? n + 16 : n;
}

struct Params {
    CUtensorMap map[2];
    const uint8_t *W[2];
    int64_t rb, row0, group_rows, total_rows;
    const uint8_t *img;
    const float *inv;
    ChunkPlan *plan;
    const ChunkTile *tiles;
    int32_t P, logP;          // matrix rows per super-row
    int32_t bw;               // box bytes: chunk bytes, 16 more when P > 1
    int32_t copies;           // 0: every row is behind the last super-row
    int32_t slots, raws;      // stages of activations and raw chunks in shared memory,
    uint32_t slot, raw_at;    // bytes of a slice of such a stage, and where the chunks begin
    int32_t rows, nst, nch, nb, nrt, gated;   // rows of Y; slices, chunks, blocks of a row; row tiles
    int32_t act, dtype;
    float alpha, limit;
    const float *bias[2];
    const void *residual;
    int64_t ldr, ldy;
    void *Y;
    float *sums;              // with several parts: [part][projection][row of the call][rows]
    float *held;              // 16-bit calls' sums between segments: [CTA][operand row][kM]
    int32_t segment, held_rows;   // slices of a segment, operand rows of a CTA's share
    int32_t parts, part_chunks, n_row;
    int32_t withhold;         // test hook: the first stage of the first item is never copied
    long long limit_cycles;   // of a wait
};

// Row of a half of the tile for each of its 64 threads (tensor-memory lanes):
// neighbours take rows at the same position of successive super-rows, which
// lie box_bytes apart (and store to columns P apart).
__device__ __forceinline__ int lane_row(int e, int logP) { return ((e & ((64 >> logP) - 1)) << logP) + (e >> (6 - logP)); }

// ------------------------------------------------------------------ decoding
// One block of 32 weights from any byte of shared memory: its scale's bits and
// its quant words.  4-byte loads, shifted to the block's first byte (and over
// the scale); a Q8_0 block's nine words are fewer 8-byte loads and a word's
// shift (2048 rows through 4096 x 11008: 212 against 216 us; with four quant
// words it is the other way, 573 against 588 us for a Q4_0 routed FFN).
template <int FMT>
struct Block {
    static constexpr int NS = FMT == RF_MXFP4 ? 1 : 2, NW = FMT == RF_Q8_0 ? 8 : 4;   // scale bytes, quant words
    static constexpr int ND = (7 + NS + 4 * NW) / 8;
    uint32_t q[NW], s;
    __device__ __forceinline__ void load(const uint8_t *row, int at)
    {
        const uint32_t off = smem_addr(row) + (uint32_t)at, sh = 8u * (off & 3u);
        uint32_t x[NW + 1];
        if constexpr (NW == 8) {
            uint32_t y[2 * ND];
            const uint2 *src = reinterpret_cast<const uint2 *>(row + at - (off & 7u));
#pragma unroll
            for (int i = 0; i < ND; ++i) {
                const uint2 v = src[i];
                y[2 * i] = v.x, y[2 * i + 1] = v.y;
            }
#pragma unroll
            for (int i = 0; i < NW + 1; ++i) x[i] = (off & 4u) != 0 ? y[i + 1] : y[i];
        } else {
            const uint32_t *src = reinterpret_cast<const uint32_t *>(row + at - (off & 3u));
#pragma unroll
            for (int i = 0; i < NW + 1; ++i) x[i] = src[i];
        }
        s = (x[0] >> sh) & (NS == 1 ? 0xFFu : 0xFFFFu);
#pragma unroll
        for (int i = 0; i < NW; ++i) q[i] = __funnelshift_rc(x[i], x[i + 1], sh + 8 * NS);
    }
};

__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}

// How low terms are kept.  kOne: none.  kPlain: as they are (16-bit
// activations: their products join the high ones' sums; a weight is then off
// by 2^-25 at most).  kScaled: times 2^11 (fp32: 22 bits of the weight).
enum Low { kOne, kPlain, kScaled };

// fp32 weights as a pair of fp16 values and the pair of what they leave.
template <int L>
__device__ __forceinline__ void two_terms(float w0, float w1, uint32_t &hi, uint32_t &lo)
{
    const __half2 h = __floats2half2_rn(w0, w1);
    hi = h2_bits(h);
    if constexpr (L != kOne) {
        const float2 f = __half22float2(h);
        const float m = L == kScaled ? 2048.f : 1.f;
        lo = h2_bits(__floats2half2_rn((w0 - f.x) * m, (w1 - f.y) * m));
    }
}
// The same for products n * d of small integers (fp16 pairs that number(j)
// gives) and an fp16 scale, in fp16: hi rounds the product, and what it leaves
// has at most 11 bits and is a multiple of d's last place, hence of fp16's
// least number, so that one fused multiply-add gives it exactly.
template <int L>
__device__ __forceinline__ void product(uint32_t n, uint32_t dd, uint32_t &hi, uint32_t &lo)
{
    hi = hmul2(n, dd);
    if constexpr (L != kOne) lo = hfma2(n, dd, hi ^ 0x80008000u);
    if constexpr (L == kScaled) lo = hmul2(lo, 0x68006800u);
}
template <int L, class F>
__device__ __forceinline__ void products(uint32_t d, F number, uint32_t (&hi)[16], uint32_t (&lo)[16])
{
#pragma unroll
    for (int j = 0; j < 16; ++j) product<L>(number(j), d * 0x00010001u, hi[j], lo[j]);
}

// Q4_0, d and its four quant words: pair 4 m + s holds nibbles s and s + 4 of
// word m.  0x6400 | n is the fp16 value 1024 + n (and 0x6400 | 16 n is 1024 +
// 16 n), so n - 8 is exact; one multiply by d rounds the weight once.
__device__ __forceinline__ uint32_t q4_0_pair(uint32_t q, int s)
{
    const uint32_t t = (s & 2) ? q >> 8 : q;
    return (s & 1) ? hfma2((t & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD480D480u)   // x / 16 - 72
                   : hsub2((t & 0x000F000Fu) | 0x64006400u, 0x64086408u);
}
template <int L>
__device__ __forceinline__ void q4_0_block(uint32_t d, const uint32_t (&q)[4], uint32_t (&hi)[16], uint32_t (&lo)[16])
{
    products<L>(d, [&](int j) { return q4_0_pair(q[j >> 2], j & 3); }, hi, lo);
}
// Q8_0: with the sign bit flipped, 0x6400 | u is 1024 + q + 128.
__device__ __forceinline__ uint32_t q8_0_pair(uint32_t q, int s)
{
    return hsub2(prmt(q ^ 0x80808080u, 0x64646464u, s ? 0x7362u : 0x5140u), 0x64806480u);
}
template <int L>
__device__ __forceinline__ void q8_0_block(uint32_t d, const uint32_t (&q)[8], uint32_t (&hi)[16], uint32_t (&lo)[16])
{
    products<L>(d, [&](int j) { return q8_0_pair(q[j >> 1], j & 1); }, hi, lo);
}
// Four bytes of two E2M1 codes each as four fp16 pairs (low nibble, high).
__device__ __forceinline__ void e2m1x8(uint32_t q, uint32_t (&h)[4])
{
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(q));
}
// MXFP4: pair j holds byte j's two codes, scaled by 2^(E - 127): exact whenever
// the product is representable.  Where that factor is none of fp16's normal
// numbers (for any lane of the warp: e8m0_far, `any`) it is split in two (one
// rounding).
__device__ __forceinline__ uint32_t e8m0_place(uint32_t E) { return E - 113u; }
__device__ __forceinline__ bool e8m0_far(uint32_t largest_place) { return __any_sync(0xffffffffu, largest_place >= 30u); }
__device__ __forceinline__ uint32_t e8m0_factor(uint32_t E) { return E * 0x04000400u - 112u * 0x04000400u; }
__device__ __forceinline__ void e8m0_factors(uint32_t E, uint32_t &s1, uint32_t &s2)
{
    const int k = (int)E - 127;
    s2 = 0x3C003C00u;
    if (E == 255u) s1 = 0x7E007E00u;   // NaN
    else if (k > 15) s1 = 0x78007800u, s2 = pow2_h(min(k - 15, 15)) * 0x00010001u;
    else if (k < -24) s1 = 0x0C000C00u, s2 = k + 12 >= -24 ? pow2_h(k + 12) * 0x00010001u : 0u;
    else s1 = pow2_h(k) * 0x00010001u;
}
__device__ __forceinline__ void mxfp4_block(uint32_t E, const uint32_t (&q)[4], bool any, uint32_t (&hi)[16])
{
    const uint32_t s = e8m0_factor(E);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        uint32_t h[4];
        e2m1x8(q[m], h);
#pragma unroll
        for (int e = 0; e < 4; ++e) hi[4 * m + e] = hmul2(h[e], s);
    }
    if (any) {   // (again: the vote's answer is not waited for)
        uint32_t s1, s2;
        e8m0_factors(E, s1, s2);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            uint32_t h[4];
            e2m1x8(q[m], h);
#pragma unroll
            for (int e = 0; e < 4; ++e) hi[4 * m + e] = hmul2(hmul2(h[e], s1), s2);
        }
    }
}
// Half T (0: low nibbles, 1: high) of slice Q of a Q4_K super-block at `s`
// (16-byte aligned): sub-block 2 Q + T, d * sc * q - dmin * m by one fused
// multiply-add in fp32 (its products are exact).
struct Q4K {
    float ds, dm;
    uint32_t q[8];
    int T;
    __device__ __forceinline__ void load(const uint8_t *s, int Q, int half)
    {
        T = half;
        const uint4 h = *reinterpret_cast<const uint4 *>(s);
        const uint4 qa = *reinterpret_cast<const uint4 *>(s + 16 + 32 * Q), qb = *reinterpret_cast<const uint4 *>(s + 32 + 32 * Q);
        const float d = __half2float(__ushort_as_half((unsigned short)(h.x & 0xFFFFu)));
        const float dmin = __half2float(__ushort_as_half((unsigned short)(h.x >> 16)));
        const int j = 2 * Q + T;
        uint32_t sc, m;
        if (j < 4) {
            sc = (h.y >> (8 * j)) & 63u;
            m = (h.z >> (8 * j)) & 63u;
        } else {
            const uint32_t b = (h.w >> (8 * (j - 4))) & 0xFFu;
            sc = (b & 15u) | (((h.y >> (8 * (j - 4) + 6)) & 3u) << 4);
            m = (b >> 4) | (((h.z >> (8 * (j - 4) + 6)) & 3u) << 4);
        }
        ds = d * (float)sc, dm = dmin * (float)m;
        q[0] = qa.x, q[1] = qa.y, q[2] = qa.z, q[3] = qa.w, q[4] = qb.x, q[5] = qb.y, q[6] = qb.z, q[7] = qb.w;
    }
    // Word k's two pairs.
    template <int L>
    __device__ __forceinline__ void pairs(int k, uint32_t &h0, uint32_t &l0, uint32_t &h1, uint32_t &l1) const
    {
        const uint32_t v = (q[k] >> (4 * T)) & 0x0F0F0F0Fu;
        float f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            f[e] = fmaf(ds, __uint_as_float(prmt(v, 0x4B000000u, 0x7440u + e)) - 8388608.f, -dm);
        two_terms<L>(f[0], f[1], h0, l0);
        two_terms<L>(f[2], f[3], h1, l1);
    }
};
template <int L>
__device__ __forceinline__ void q4k_block(const uint8_t *s, int Q, int T, uint32_t (&hi)[16], uint32_t (&lo)[16])
{
    Q4K b;
    b.load(s, Q, T);
#pragma unroll
    for (int k = 0; k < 8; ++k) b.pairs<L>(k, hi[2 * k], lo[2 * k], hi[2 * k + 1], lo[2 * k + 1]);
}

template <int FMT, int L>
__device__ __forceinline__ void block_pairs(const Block<FMT> &b, bool any, uint32_t (&hi)[16], uint32_t (&lo)[16])
{
    if constexpr (FMT == RF_Q4_0) q4_0_block<L>(b.s, b.q, hi, lo);
    else if constexpr (FMT == RF_Q8_0) q8_0_block<L>(b.s, b.q, hi, lo);
    else mxfp4_block(b.s, b.q, any, hi);
}

// ---------------------------------------------------------------- activations
// (A quotient by reciprocal, 2 ulp: without the exact division's slow path the
// lanes' values are computed side by side.  1 + exp overflows to 0, the limit.)
__device__ __forceinline__ float sigmoid_times(float z, float arg) { return __fdividef(z, 1.f + expf(-arg)); }
__device__ __forceinline__ float clamped_of(float g, float u, float alpha, float limit)
{
    g = g > limit ? limit : g;   // (NaN stays)
    u = u > limit ? limit : (u < -limit ? -limit : u);
    return sigmoid_times(g, alpha * g) * (u + 1.f);
}

template <int DT> struct Out;
template <> struct Out<RF_F32> {
    using T = float;
    static __device__ __forceinline__ float get(T v) { return v; }
    static __device__ __forceinline__ T put(float v) { return v; }
};
template <> struct Out<RF_F16> {
    using T = __half;
    static __device__ __forceinline__ float get(T v) { return __half2float(v); }
    static __device__ __forceinline__ T put(float v) { return __float2half_rn(v); }
};
template <> struct Out<RF_BF16> {
    using T = __nv_bfloat16;
    static __device__ __forceinline__ float get(T v) { return __bfloat162float(v); }
    static __device__ __forceinline__ T put(float v) { return __float2bfloat16_rn(v); }
};

// What follows the product, for one element: act(y, u) + residual, stored (y
// and u with their biases).
__device__ __forceinline__ void finish_one(const Params &p, int64_t row, int col, float y, float u)
{
    if (p.act == RF_ACT_SILU) y = sigmoid_times(y, y);
    else if (p.act == RF_ACT_GELU) y = 0.5f * y * (1.f + erff(y * 0.70710678118654752f));
    else if (p.act == RF_ACT_SWIGLU) y = sigmoid_times(y, y) * u;
    else if (p.act == RF_ACT_SWIGLU_CLAMPED) y = clamped_of(y, u, p.alpha, p.limit);
    const int64_t from = row * p.ldr + col, to = row * p.ldy + col;
    if (p.dtype == RF_F32) {
        if (p.residual) y += static_cast<const float *>(p.residual)[from];
        static_cast<float *>(p.Y)[to] = y;
    } else if (p.dtype == RF_F16) {
        if (p.residual) y += Out<RF_F16>::get(static_cast<const __half *>(p.residual)[from]);
        static_cast<__half *>(p.Y)[to] = Out<RF_F16>::put(y);
    } else {
        if (p.residual) y += Out<RF_BF16>::get(static_cast<const __nv_bfloat16 *>(p.residual)[from]);
        static_cast<__nv_bfloat16 *>(p.Y)[to] = Out<RF_BF16>::put(y);
    }
}

// Barriers and copies by shared-memory address: the roles' loops are chains of
// a few instructions, and a generic pointer's conversion would be among them.
__device__ __forceinline__ void bar_arrive(uint32_t bar)
{
    asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0];\n\t}" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(bar), "r"(bytes)
                 : "memory");
}
// Whether phase `parity` has completed: at once (test), within the hardware's
// own time (try), or within `ns` nanoseconds, the thread set aside meanwhile.
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool bar_try_ns(uint32_t bar, uint32_t parity, uint32_t ns)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(bar), "r"(parity), "r"(ns) : "memory");
    return ok != 0;
}
__device__ __forceinline__ void copy_bulk(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
                     "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
                 : "memory");
}
// A copy that was issued lands whatever else failed: wait for it (bounded,
// ignoring the status word), so that none is under way when the CTA exits.
__device__ __forceinline__ void bar_drain(uint32_t bar, uint32_t parity)
{
    const unsigned long long t0 = globaltimer_ns();
    while (!bar_try_ns(bar, parity, 20000u) && globaltimer_ns() - t0 < kWaitLimitNs) {
    }
}

}  // namespace chunk

// Products of the tiles of few tokens (rf_chunk_few.cu).
rf_status launch_chunk_few(const ChunkShape &sh, const chunk::Params &p, cudaStream_t s);

}  // namespace rf
