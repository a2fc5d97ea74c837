// rf_chunk_mma.cu -- quantized matrices times chunks of tokens on the
// fifth-generation tensor cores, one matrix or a stack of them with ragged
// groups of rows, and what follows the product in its epilogue.
//
//     Y[r] = residual[r] + act(W_g x_r + b_g, U_g x_r + b'_g)
//
// A pre-pass (rf_chunk.cu) has listed the token tiles (up to T rows of one
// group) and written each tile's activations as fp16 operand images.
// chunk_kernel: persistent CTAs draw items, a token tile times 128 matrix rows
// (with a gated activation 64 rows of W and the same 64 of U, so that both
// projections of a neuron meet in one warp).  Per CTA:
//   warp 0       copies raw weight bytes, a chunk of 128 rows at a time, with
//                2-D tensor copies;
//   warp 1       copies the operand slices of the token tile (1-D bulk);
//   warp 2       issues the products;
//   warp 3       draws the items;
//   decoders     three groups of four warps: each takes every third 64-input
//                slice, a thread its row, turns the raw bytes into fp16 pairs
//                and stores them to tensor memory, from where tcgen05.mma reads
//                the weights: they cost no shared-memory bandwidth, which is
//                what bounds tiles whose operands both lie there;
//   epilogue     four warps read the sums out of tensor memory, while the
//                others are at the next item.
//
// Rows of any length by tensor copies.  A tensor map's rows have to be
// multiples of 16 bytes apart; rows of rb bytes are not, but P = 16 /
// gcd(rb, 16) of them together are.  The map's rows are such super-rows, and a
// chunk of 64 matrix rows is P boxes, one for each position j in the
// super-row, whose first byte j * rb + c * (chunk bytes) is rounded down to 16;
// a thread skips the remainder.  Rows behind the last whole super-row (fewer
// than 16 of a tensor) are read by their threads directly.
//
// Order of the inputs.  A product does not care in which order its inputs are
// summed, so a slice's inputs are in the order in which the decoder finds them
// cheapest (slice_order in rf_chunk.cu): for MXFP4 the two nibbles of a byte,
// for Q4_0 nibbles four apart.
//
// Precision: see rf.h.  Two fp16 terms of an activation are two rows of the
// operand (8 high, 8 low) with sums of their own; the low terms are scaled by
// 2^11.  Low terms of weights multiply the high terms of activations into a
// third sum (the product of two low terms is below 2^-22 of the result).
//
// Every wait is bounded; after a failure every role stops, copies and products
// already issued are waited for, and tensor memory is freed.
#include <algorithm>
#include <cstring>
#include <mutex>

#include <cuda_bf16.h>

#include "rf_chunk.h"
#include "rf_half.cuh"
#include "rf_tcgen05.cuh"

namespace rf {
namespace {

__device__ int g_chunk_status = 0;   // bounded waits that gave up

constexpr int kM = 128;              // matrix rows per item (MMA M)
constexpr int kGroups = 3;           // decoder groups of four warps
constexpr int kDec0 = 4, kEpi0 = kDec0 + 4 * kGroups;
constexpr int kThreads = 32 * (kEpi0 + 4);
// fp32 calls hold 64 sums a thread in the epilogue, whose warpgroup takes
// registers from that of the copies and the issue (96 a thread at launch:
// 40 + 152 + 3 * 96 = 5 * 96).
constexpr int kRegsRoles = 40, kRegsSums = 152;
constexpr int kItems = 4;            // items drawn ahead
constexpr int kItemUsers = 3 + 4 * kGroups + 4;

// Raw chunk: BPC blocks (of BE weights, BS bytes) of each row.
template <int FMT> struct Raw;
template <> struct Raw<RF_Q4_0> { static constexpr int BS = 18, BE = 32, BPC = 8; };
template <> struct Raw<RF_Q8_0> { static constexpr int BS = 34, BE = 32, BPC = 8; };
template <> struct Raw<RF_MXFP4> { static constexpr int BS = 17, BE = 32, BPC = 16; };
template <> struct Raw<RF_Q4_K> { static constexpr int BS = 144, BE = 256, BPC = 1; };

// NT: operand rows per token tile; XT, WT: fp16 terms per activation, weight.
// A stage is KS slices of weights (tensor memory) and activations (shared
// memory): two where a slice's products are short, so that the issuing warp's
// chain of wait, issue and commit is paid half as often.
template <int FMT, int NT, int XT, int WT>
struct Cfg {
    static constexpr int CB = Raw<FMT>::BPC * Raw<FMT>::BS;            // chunk bytes per row
    static constexpr int QPC = Raw<FMT>::BPC * Raw<FMT>::BE / kSliceK; // slices per chunk
    static constexpr int BW = CB + (FMT == RF_Q4_K ? 0 : 16);          // box bytes at most
    static constexpr int T = NT / XT;                                  // tokens
    static constexpr int KS = NT == 128 && WT == 1 ? 2 : 1;
    static constexpr int S = 4;                                        // stages
    static constexpr int BT = NT * kSliceK * 2;                        // activation bytes per slice
    static constexpr int RAW = kM * BW;
    static constexpr int R = RAW > 32768 ? 2 : 4;                      // raw chunks in flight
    // Columns of one item's sums: one region of NT, or (two terms of both) T
    // of high products and T of the others.  With two terms of weights alone,
    // a second region for the low ones.
    static constexpr int ACC = WT == 2 && XT == 1 ? 2 * NT : NT;
    static constexpr int NBUF = 2 * ACC <= 256 ? 2 : 1;
    static constexpr int ACOL = 256;                                   // first column of the weights
    static constexpr int ASLICE = 32 * WT, ASTAGE = KS * ASLICE;
    // Sums of fp32 calls leave tensor memory every FLUSH slices: the tensor cores truncate each addition (about 1e-8 of the
    // sum, always towards zero), rounded additions in registers do not drift.
    static constexpr int FLUSH = XT == 2 ? 4 : 1 << 30;                // slices
    static constexpr size_t SMEM = (size_t)S * KS * BT + (size_t)R * RAW + 16;
    static_assert(ACC * NBUF <= 256 && S * ASTAGE <= 256, "tensor memory");
    static_assert(QPC % KS == 0 && FLUSH % KS == 0, "a stage lies in one chunk and between two flushes");
    static_assert(T % 16 == 0, "the epilogue takes 16 tokens at a time");
    static_assert(kGroups <= S, "groups wait within one phase of a stage");
    static_assert(SMEM <= 231000, "shared memory");
};

struct Item {
    int32_t group, row0, cnt, gran, rt, stop, pad[2];
};

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
    int32_t rows, nst, nch, nb, nrt, gated;   // rows of Y; slices, chunks, blocks of a row; row tiles
    int32_t act, dtype;
    float alpha, limit;
    const float *bias[2];
    const void *residual;
    int64_t ldr, ldy;
    void *Y;
    int32_t withhold;         // test hook: CTA 0 never copies this slice's activations
    unsigned long long limit_ns;
};

__host__ __device__ constexpr uint32_t idesc_n(int n)
{
    return (1u << 4) | (0u << 7) | (0u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kM >> 4) << 24);
}

// ------------------------------------------------------------------ decoding
// A slice's bytes as words from its first byte; word<B>, byte<B>, half<B> at
// byte B.
template <int SBYTES>
struct Win {
    static constexpr int NO = (SBYTES + 3) / 4;
    uint32_t w[NO];
    template <int B> __device__ __forceinline__ uint32_t word() const
    {
        if constexpr (B % 4 == 0) return w[B / 4];
        else return __funnelshift_r(w[B / 4], w[B / 4 + 1], 8 * (B % 4));
    }
    template <int B> __device__ __forceinline__ uint32_t byte() const { return (w[B / 4] >> (8 * (B % 4))) & 0xFFu; }
    template <int B> __device__ __forceinline__ uint32_t half() const
    {
        static_assert(B % 2 == 0, "fp16 scale at an odd byte");
        return (w[B / 4] >> (8 * (B % 4))) & 0xFFFFu;
    }
    // From shared memory at any byte: 8-byte loads (rows are multiples of 16
    // bytes apart, so 32 lanes' 4-byte loads would hit 8 banks four times),
    // then a word's and a byte's shift.
    __device__ __forceinline__ void load(const uint8_t *raw, uint32_t off)
    {
        constexpr int ND = (NO + 3) / 2;
        uint32_t x[2 * ND];
        const uint2 *s = reinterpret_cast<const uint2 *>(raw + (off & ~7u));
#pragma unroll
        for (int i = 0; i < ND; ++i) {
            const uint2 v = s[i];
            x[2 * i] = v.x;
            x[2 * i + 1] = v.y;
        }
        const bool odd = (off & 4u) != 0;
        const uint32_t sh = 8u * (off & 3u);
#pragma unroll
        for (int i = 0; i < NO + 1; ++i) x[i] = odd ? x[i + 1] : x[i];
#pragma unroll
        for (int i = 0; i < NO; ++i) w[i] = __funnelshift_r(x[i], x[i + 1], sh);
    }
    // From global memory, `n` bytes of a row (the rest read as 0): aligned
    // words, none that holds no byte of them.
    __device__ __forceinline__ void load_global(const uint8_t *a, int n)
    {
        const uintptr_t ua = reinterpret_cast<uintptr_t>(a);
        const uint32_t *a4 = reinterpret_cast<const uint32_t *>(ua & ~(uintptr_t)3);
        const uint32_t sh = 8u * (uint32_t)(ua & 3);
        const int end = (int)(ua & 3) + n;
        uint32_t x[NO + 1];
#pragma unroll
        for (int i = 0; i < NO + 1; ++i) {
            const int rem = end - 4 * i;
            const uint32_t v = rem > 0 ? __ldg(a4 + i) : 0u;
            x[i] = rem >= 4 ? v : v & ((1u << (8 * (rem > 0 ? rem : 0))) - 1u);
        }
#pragma unroll
        for (int i = 0; i < NO; ++i) w[i] = __funnelshift_r(x[i], x[i + 1], sh);
    }
};

// fp32 weights as a pair of fp16 values and the pair of what they leave,
// scaled by 2^11.
__device__ __forceinline__ void two_terms(float w0, float w1, uint32_t &hi, uint32_t &lo)
{
    const __half2 h = __floats2half2_rn(w0, w1);
    const float2 f = __half22float2(h);
    hi = h2_bits(h);
    lo = h2_bits(__floats2half2_rn((w0 - f.x) * 2048.f, (w1 - f.y) * 2048.f));
}

__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}

// Q4_0, d and its four quant words: pair s of word m holds nibbles s and s + 4.
// 0x6400 | n is the fp16 value 1024 + n (and 0x6400 | 16 n is 1024 + 16 n), so
// n - 8 is exact; one multiply by d rounds the weight once.
template <int WT>
__device__ __forceinline__ void q4_0_block(uint32_t d, const uint32_t (&q)[4], uint32_t (&hi)[16], uint32_t (&lo)[16])
{
    const uint32_t dd = d | (d << 16);
    const float df = __half2float(__ushort_as_half((unsigned short)d));
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const uint32_t v[2] = {q[m], q[m] >> 8};
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const uint32_t t = v[s >> 1];
            if constexpr (WT == 1) {
                const uint32_t n = (s & 1) ? hfma2((t & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD480D480u)   // x / 16 - 72
                                           : hsub2((t & 0x000F000Fu) | 0x64006400u, 0x64086408u);
                hi[4 * m + s] = hmul2(n, dd);
            } else {
                const uint32_t u = (t >> (4 * (s & 1))) & 0x000F000Fu;
                const float a = __uint_as_float(0x4B000000u | (u & 15u)) - 8388616.f;   // 2^23 + n - (2^23 + 8)
                const float b = __uint_as_float(0x4B000000u | (u >> 16)) - 8388616.f;
                two_terms(df * a, df * b, hi[4 * m + s], lo[4 * m + s]);
            }
        }
    }
}
// Q8_0: with the sign bit flipped, 0x6400 | u is 1024 + q + 128.
template <int WT>
__device__ __forceinline__ void q8_0_block(uint32_t d, const uint32_t (&q)[8], uint32_t (&hi)[16], uint32_t (&lo)[16])
{
    const uint32_t dd = d | (d << 16);
    const float df = __half2float(__ushort_as_half((unsigned short)d));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t v = q[j] ^ 0x80808080u;
        if constexpr (WT == 1) {
            hi[2 * j] = hmul2(hsub2(prmt(v, 0x64646464u, 0x5140u), 0x64806480u), dd);
            hi[2 * j + 1] = hmul2(hsub2(prmt(v, 0x64646464u, 0x7362u), 0x64806480u), dd);
        } else {
            float f[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                f[e] = df * (__uint_as_float(prmt(v, 0x4B000000u, 0x7440u + e)) - 8388736.f);   // 2^23 + 128 + q
            two_terms(f[0], f[1], hi[2 * j], lo[2 * j]);
            two_terms(f[2], f[3], hi[2 * j + 1], lo[2 * j + 1]);
        }
    }
}
// MXFP4: pair j holds byte j's two codes, scaled by 2^(E - 127): exact whenever
// the product is representable, in two steps outside fp16's exponents (one
// rounding).
__device__ __forceinline__ void mxfp4_block(uint32_t E, const uint32_t (&q)[4], uint32_t (&hi)[16])
{
    const int k = (int)E - 127;
    uint32_t s1, s2 = 0u;
    if (E == 255u) s1 = 0x7E00u;                       // NaN scale
    else if (k >= -14 && k <= 15) s1 = (uint32_t)(k + 15) << 10;
    else if (k > 15) s1 = 0x7800u, s2 = pow2_h(min(k - 15, 15));
    else if (k >= -24) s1 = pow2_h(k);
    else s1 = 0x0C00u, s2 = k + 12 >= -24 ? pow2_h(k + 12) : 0u;
    const uint32_t ss = s1 | (s1 << 16);
#pragma unroll
    for (int j = 0; j < 16; ++j) hi[j] = hmul2(e2m1x2_h2(q[j >> 2] >> (8 * (j & 3))), ss);
    if (E != 255u && (k < -24 || k > 15)) {
        const uint32_t s22 = s2 | (s2 << 16);
#pragma unroll
        for (int j = 0; j < 16; ++j) hi[j] = hmul2(hi[j], s22);
    }
}
// Half T (0: low nibbles, 1: high) of slice Q of a Q4_K super-block at `s`
// (16-byte aligned): sub-block 2 Q + T, d * sc * q - dmin * m by one fused
// multiply-add in fp32 (its products are exact).
template <int WT>
__device__ __forceinline__ void q4k_block(const uint8_t *s, int Q, int T, uint32_t (&hi)[16], uint32_t (&lo)[16])
{
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
    const float ds = d * (float)sc, dm = dmin * (float)m;
    const uint32_t qw[8] = {qa.x, qa.y, qa.z, qa.w, qb.x, qb.y, qb.z, qb.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t v = (qw[k] >> (4 * T)) & 0x0F0F0F0Fu;
        float f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            f[e] = fmaf(ds, __uint_as_float(prmt(v, 0x4B000000u, 0x7440u + e)) - 8388608.f, -dm);
        if constexpr (WT == 1) {
            hi[2 * k] = h2_bits(__floats2half2_rn(f[0], f[1]));
            hi[2 * k + 1] = h2_bits(__floats2half2_rn(f[2], f[3]));
        } else {
            two_terms(f[0], f[1], hi[2 * k], lo[2 * k]);
            two_terms(f[2], f[3], hi[2 * k + 1], lo[2 * k + 1]);
        }
    }
}

template <int FMT, int WT, int BLK, class W>
__device__ __forceinline__ void win_block(const W &win, uint32_t (&hi)[16], uint32_t (&lo)[16])
{
    constexpr int O = BLK * Raw<FMT>::BS;
    if constexpr (FMT == RF_Q4_0) {
        const uint32_t q[4] = {win.template word<O + 2>(), win.template word<O + 6>(), win.template word<O + 10>(),
                               win.template word<O + 14>()};
        q4_0_block<WT>(win.template half<O>(), q, hi, lo);
    } else if constexpr (FMT == RF_Q8_0) {
        const uint32_t q[8] = {win.template word<O + 2>(),  win.template word<O + 6>(),  win.template word<O + 10>(),
                               win.template word<O + 14>(), win.template word<O + 18>(), win.template word<O + 22>(),
                               win.template word<O + 26>(), win.template word<O + 30>()};
        q8_0_block<WT>(win.template half<O>(), q, hi, lo);
    } else {
        const uint32_t q[4] = {win.template word<O + 1>(), win.template word<O + 5>(), win.template word<O + 9>(),
                               win.template word<O + 13>()};
        mxfp4_block(win.template byte<O>(), q, hi);
    }
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

// Sixteen tokens' sums z of this lane's matrix row, as rows r0.. of Y (the
// first n of them): bias, activation, residual, stores.  Gated: lanes 16 apart
// hold the gate and the up projection of a neuron; of two tokens, lanes below
// 16 finish the first, the others the second.
template <int DT>
__device__ __forceinline__ void finish(const Params &p, float (&z)[16], const float (&inv)[16], float bias, int64_t r0, int n,
                                       int col, bool in, int half)
{
    using O = Out<DT>;
    using T = typename O::T;
#pragma unroll
    for (int u = 0; u < 16; ++u) z[u] = fmaf(z[u], inv[u], bias);
    T *y = static_cast<T *>(p.Y) + r0 * p.ldy + col;
    const T *res = static_cast<const T *>(p.residual) + r0 * p.ldr + col;
    if (p.gated) {
        float o[8], add[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) add[u] = 0.f;
        if (p.residual) {
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (in && 2 * u + half < n) add[u] = O::get(res[(2 * u + half) * p.ldr]);
        }
        float other[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) other[u] = __shfl_xor_sync(0xffffffffu, half ? z[2 * u] : z[2 * u + 1], 16);
        if (p.act == RF_ACT_SWIGLU) {
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const float g = half ? other[u] : z[2 * u], up = half ? z[2 * u + 1] : other[u];
                o[u] = sigmoid_times(g, g) * up;
            }
        } else {
#pragma unroll
            for (int u = 0; u < 8; ++u)
                o[u] = clamped_of(half ? other[u] : z[2 * u], half ? z[2 * u + 1] : other[u], p.alpha, p.limit);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (in && 2 * u + half < n) y[(2 * u + half) * p.ldy] = O::put(o[u] + add[u]);
    } else {
        float add[16];
#pragma unroll
        for (int u = 0; u < 16; ++u) add[u] = 0.f;
        if (p.residual) {
#pragma unroll
            for (int u = 0; u < 16; ++u)
                if (in && u < n) add[u] = O::get(res[u * p.ldr]);
        }
        if (p.act == RF_ACT_SILU) {
#pragma unroll
            for (int u = 0; u < 16; ++u) z[u] = sigmoid_times(z[u], z[u]);
        } else if (p.act == RF_ACT_GELU) {
#pragma unroll
            for (int u = 0; u < 16; ++u) z[u] = 0.5f * z[u] * (1.f + erff(z[u] * 0.70710678118654752f));
        }
#pragma unroll
        for (int u = 0; u < 16; ++u)
            if (in && u < n) y[u * p.ldy] = O::put(z[u] + add[u]);
    }
}
__device__ __forceinline__ void finish_typed(const Params &p, float (&z)[16], const float (&inv)[16], float bias, int64_t r0,
                                             int n, int col, bool in, int half)
{
    if (p.dtype == RF_F32) finish<RF_F32>(p, z, inv, bias, r0, n, col, in, half);
    else if (p.dtype == RF_F16) finish<RF_F16>(p, z, inv, bias, r0, n, col, in, half);
    else finish<RF_BF16>(p, z, inv, bias, r0, n, col, in, half);
}
__device__ __forceinline__ void load_inv(const float *inv, float (&f)[16])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 v = __ldg(reinterpret_cast<const float4 *>(inv) + i);
        f[4 * i] = v.x, f[4 * i + 1] = v.y, f[4 * i + 2] = v.z, f[4 * i + 3] = v.w;
    }
}

template <int FMT, int NT, int XT, int WT>
__global__ void __launch_bounds__(kThreads, 1) chunk_kernel(const __grid_constant__ Params p)
{
    using C = Cfg<FMT, NT, XT, WT>;
    constexpr int S = C::S, KS = C::KS, R = C::R, QPC = C::QPC, NBUF = C::NBUF, GT = kGranRows / XT;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *b_t = smem;                       // [S][KS slices]
    uint8_t *raw = b_t + S * KS * C::BT;       // [R][RAW], then 16 bytes that a last load may touch
    // bfull: a stage's activations have landed; full: so have they, and its
    // weights are decoded (an arrival per decoder warp and slice); done: its
    // products are through.
    __shared__ uint64_t full[S], bfull[S], done[S], rfull[R], rempty[R], accfull[NBUF], accempty[NBUF], ifull[kItems], iempty[kItems],
        drained;
    __shared__ Item items[kItems];
    __shared__ uint32_t s_tmem;
    __shared__ int s_stop;
    volatile int *stop = &s_stop;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) mbar_init(&full[i], 4 * KS), mbar_init(&bfull[i], 1), mbar_init(&done[i], 1);
        for (int i = 0; i < R; ++i) mbar_init(&rfull[i], 1), mbar_init(&rempty[i], 4 * kGroups);
        for (int i = 0; i < NBUF; ++i) mbar_init(&accfull[i], 1), mbar_init(&accempty[i], 4);
        for (int i = 0; i < kItems; ++i) mbar_init(&ifull[i], 1), mbar_init(&iempty[i], kItemUsers);
        mbar_init(&drained, 1);
        s_stop = 0;
        fence_barrier_init();
    }
    if (warp == 3) {
        tmem_alloc(&s_tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        if (mbar_try_wait(bar, parity)) return true;
        if (*stop) return false;
        if (mbar_wait_bounded(bar, parity, &g_chunk_status, p.limit_ns)) return true;
        *stop = 1;
        return false;
    };
    // A warp's waits; the next item, copied from its slot (one arrival a warp).
    auto waits = [&](uint64_t *bar, uint32_t parity) -> bool { return __all_sync(0xffffffffu, wait(bar, parity)); };
    auto take = [&](uint32_t it, Item &w) -> bool {
        const int slot = it % kItems;
        if (!waits(&ifull[slot], (it / kItems) & 1)) return false;
        const int32_t *src = reinterpret_cast<const int32_t *>(&items[slot]);
        w.group = __shfl_sync(0xffffffffu, src[0], 0), w.row0 = __shfl_sync(0xffffffffu, src[1], 0);
        w.cnt = __shfl_sync(0xffffffffu, src[2], 0), w.gran = __shfl_sync(0xffffffffu, src[3], 0);
        w.rt = __shfl_sync(0xffffffffu, src[4], 0), w.stop = __shfl_sync(0xffffffffu, src[5], 0);
        __syncwarp();
        if (lane == 0) mbar_arrive(&iempty[slot]);
        return w.stop == 0;
    };

    // (Registers are traded for good: the roles do not join again before the end.)
    if (warp < kDec0) {
    if constexpr (XT == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRoles));
    if (warp == 3) {
        if (lane == 0) {
            const int total = p.plan->n_tiles * p.nrt;   // at most 2^30
            for (uint32_t it = 0;; ++it) {
                const int slot = it % kItems;
                if (!wait(&iempty[slot], ((it / kItems) & 1) ^ 1)) break;
                Item &w = items[slot];
                const int index = atomicAdd(&p.plan->next, 1);
                w.stop = index >= total;
                if (!w.stop) {
                    const ChunkTile t = p.tiles[index / p.nrt];
                    w.group = t.group, w.row0 = t.row0, w.cnt = t.cnt, w.gran = t.gran;
                    w.rt = index % p.nrt;
                }
                const bool end = w.stop != 0;
                mbar_arrive(&ifull[slot]);
                if (end) break;
            }
        }
        __syncwarp();
    } else if (warp == 0) {
        // Raw rows: lane l copies box l of a chunk (half l / P, position l % P).
        const int half = lane >> p.logP, j = lane & (p.P - 1);
        const bool copies = half < 2 && p.copies;
        const uint32_t box = (uint32_t)((64 >> p.logP) * p.bw);
        const int xj = (int)((int64_t)j * p.rb);
        uint32_t rc = 0;
        Item w;
        for (uint32_t it = 0; take(it, w); ++it) {
            const int64_t first = p.row0 + (int64_t)w.group * p.group_rows +
                                  (p.gated ? (int64_t)w.rt * 64 : (int64_t)w.rt * 128 + 64 * half);
            const int y = (int)((first - j + p.P - 1) >> p.logP);   // first super-row with position j in the tile
            const CUtensorMap *map = &p.map[p.gated ? half & 1 : 0];
            bool ok = true;
            for (int c = 0; c < p.nch; ++c, ++rc) {
                const int r = rc % R;
                if (!(ok = waits(&rempty[r], ((rc / R) & 1) ^ 1))) break;
                if (lane == 0) {
                    if (p.copies) mbar_arrive_expect_tx(&rfull[r], (uint32_t)(kM * p.bw));
                    else mbar_arrive(&rfull[r]);
                }
                __syncwarp();
                if (copies)
                    tma_2d_g2s(raw + r * C::RAW + lane * box, map, ((xj + c * C::CB) & ~15) >> 1, y, &rfull[r]);
            }
            if (!ok) break;
        }
        // Every copy issued lands before the CTA can exit.
        if (lane == 0)
            for (uint32_t i = rc > R ? rc - R : 0; i < rc; ++i) mbar_drain(&rfull[i % R], (i / R) & 1);
        __syncwarp();
    } else if (warp == 1) {
        uint32_t n = 0;          // stages so far
        uint32_t skipped = 0xffffffffu;
        Item w;
        for (uint32_t it = 0; take(it, w); ++it) {
            bool ok = true;
            if (lane == 0) {
                const uint32_t bytes = (uint32_t)((w.cnt + GT - 1) / GT) * kGranBytes;   // of a slice
                const uint8_t *src = p.img + (int64_t)w.gran * p.nst * kGranBytes;
                for (int b = 0; b < p.nst; b += KS, ++n) {
                    const int st = n % S;
                    if (!(ok = wait(&done[st], ((n / S) & 1) ^ 1))) break;
                    if (blockIdx.x == 0 && n == (uint32_t)p.withhold) {
                        skipped = n;
                        continue;
                    }
                    const int slices = min(KS, p.nst - b);
                    mbar_arrive_expect_tx(&bfull[st], slices * bytes);
                    for (int i = 0; i < slices; ++i)
                        bulk_g2s(b_t + (st * KS + i) * C::BT, src + (int64_t)(b + i) * bytes, bytes, &bfull[st]);
                }
            }
            if (!__shfl_sync(0xffffffffu, (int)ok, 0)) break;
        }
        // Every copy issued lands before the CTA can exit.
        if (lane == 0)
            for (uint32_t i = n > S ? n - S : 0; i < n; ++i)
                if (i != skipped) mbar_drain(&bfull[i % S], (i / S) & 1);
        __syncwarp();
    } else if (warp == 2) {
        const uint64_t bd0 = smem_desc(smem_addr(b_t), 1024);
        const uint64_t bd1 = smem_desc(smem_addr(b_t), 2048);   // every other 8 rows: the high (or low) terms
        const bool leader = elect_one();
        uint32_t n = 0, seg = 0;   // stages, sums
        bool any = false, ok = true;
        Item w;
        for (uint32_t it = 0; ok && take(it, w); ++it) {
            const int grans = (w.cnt + GT - 1) / GT;
            const uint32_t id = WT == 2 && XT == 2 ? idesc_n((grans + 1) / 2 * 16) : idesc_n(kGranRows * grans);
            for (int b = 0; b < p.nst; ++n) {
                const bool fresh = b % C::FLUSH == 0;
                const uint32_t acc = tmem + (seg % NBUF) * C::ACC;
                if (fresh) {
                    if (!(ok = waits(&accempty[seg % NBUF], ((seg / NBUF) & 1) ^ 1))) break;
                }
                const int st = n % S;
                if (!(ok = waits(&full[st], (n / S) & 1))) break;
                tc_fence_after();
                any = true;
                if (leader) {
#pragma unroll
                    for (int i = 0; i < KS; ++i) {
                        if (i > 0 && b + i >= p.nst) break;
                        const uint32_t a = tmem + C::ACOL + (uint32_t)(st * C::ASTAGE + i * C::ASLICE);
                        const uint64_t slot = (uint64_t)(((st * KS + i) * C::BT) >> 4);
#pragma unroll
                        for (int k = 0; k < kSliceK / 16; ++k) {
                            const uint32_t add = !fresh || i > 0 || k > 0;
                            if constexpr (WT == 2 && XT == 2) {
                                tc_mma_ts(acc, a + 8 * k, bd1 + slot + 16 * k, id, add);
                                tc_mma_ts(acc + C::T, a + 8 * k, bd1 + slot + 64 + 16 * k, id, add);
                                tc_mma_ts(acc + C::T, a + 32 + 8 * k, bd1 + slot + 16 * k, id, 1u);
                            } else {
                                tc_mma_ts(acc, a + 8 * k, bd0 + slot + 16 * k, id, add);
                                if constexpr (WT == 2) tc_mma_ts(acc + NT, a + 32 + 8 * k, bd0 + slot + 16 * k, id, add);
                            }
                        }
                    }
                    tc_commit(&done[st]);
                }
                b += KS;
                if (b >= p.nst || b % C::FLUSH == 0) {
                    if (leader) tc_commit(&accfull[seg % NBUF]);
                    ++seg;
                }
            }
        }
        // Every issued product completes before tensor memory is freed.
        if (any) {
            if (leader) tc_commit(&drained);
            mbar_drain(&drained, 0);
        }
        __syncwarp();
    }
    } else if (warp < kEpi0) {
        // Decoders: lane's half of the tile (lanes 16 apart hold the same row
        // of both) and row in it.
        const int grp = (warp - kDec0) >> 2, w4 = warp & 3;
        const int half = lane >> 4, i = 16 * w4 + (lane & 15);
        const uint32_t a0 = tmem + C::ACOL + ((uint32_t)(32 * w4) << 16);
        const int64_t copied = p.copies ? p.total_rows & ~(int64_t)(p.P - 1) : 0;   // rows in whole super-rows
        const int nst = (p.nst + KS - 1) / KS * KS;   // with the slice that fills the last stage
        uint32_t n0 = 0, rc = 0;       // slices and chunks before this chunk
        int turn = 0;                  // n0 % kGroups
        bool ok = true;
        Item w;
        for (uint32_t it = 0; ok && take(it, w); ++it) {
            const int64_t first = p.row0 + (int64_t)w.group * p.group_rows +
                                  (p.gated ? (int64_t)w.rt * 64 : (int64_t)w.rt * 128 + 64 * half);
            const int64_t row = first + i;
            const int j = (int)(row & (p.P - 1));
            const int s = (int)((row >> p.logP) - ((first - j + p.P - 1) >> p.logP));
            const uint32_t at = (uint32_t)((half << p.logP) + j) * (uint32_t)((64 >> p.logP) * p.bw) + (uint32_t)(s * p.bw) +
                                ((uint32_t)(j * p.rb) & 15u);
            const bool tail = row >= copied && row < p.total_rows;
            const uint8_t *direct = p.W[p.gated ? half : 0] + (tail ? row : 0) * p.rb;
            for (int c = 0; ok && c < p.nch; ++c, ++rc) {
                const int r = rc % R, nq = min(QPC, nst - c * QPC);
                if (!(ok = waits(&rfull[r], (rc / R) & 1))) break;
                const uint8_t *src = raw + r * C::RAW;
                int q = grp - turn;
                if (q < 0) q += kGroups;
                for (; q < nq; q += kGroups) {
                    const uint32_t n = n0 + q;
                    const int st = n / KS % S;
                    if (!(ok = waits(&done[st], ((n / (KS * S)) & 1) ^ 1))) break;
                    const bool none = KS > 1 && c * QPC + q >= p.nst;   // (nothing of this slice is read)
                    tc_fence_after();
                    const uint32_t a = a0 + (uint32_t)(st * C::ASTAGE + n % KS * C::ASLICE);
                    uint32_t hi[16], lo[16];
                    if (none) {
                    } else if constexpr (FMT == RF_Q4_K) {
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            q4k_block<WT>(src + at, q, t, hi, lo);
                            tmem_st16(a + 16 * t, hi);
                            if constexpr (WT == 2) tmem_st16(a + 32 + 16 * t, lo);
                        }
                    } else {
                        constexpr int SBYTES = 2 * Raw<FMT>::BS;
                        Win<SBYTES> win;
                        const int b0 = 2 * (c * QPC + q);
                        if (tail) win.load_global(direct + (int64_t)b0 * Raw<FMT>::BS, min(2, p.nb - b0) * Raw<FMT>::BS);
                        else win.load(src, at + (uint32_t)(q * SBYTES));
                        win_block<FMT, WT, 0>(win, hi, lo);
                        tmem_st16(a, hi);
                        if constexpr (WT == 2) tmem_st16(a + 32, lo);
                        if (b0 + 1 < p.nb) {
                            win_block<FMT, WT, 1>(win, hi, lo);
                        } else {   // behind the last block: the next row's bytes
#pragma unroll
                            for (int k = 0; k < 16; ++k) hi[k] = lo[k] = 0u;
                        }
                        tmem_st16(a + 16, hi);
                        if constexpr (WT == 2) tmem_st16(a + 48, lo);
                    }
                    tmem_st_wait();
                    tc_fence_before();
                    if (!(ok = waits(&bfull[st], (n / (KS * S)) & 1))) break;
                    if (lane == 0) mbar_arrive(&full[st]);
                }
                if (!ok) break;
                __syncwarp();
                if (lane == 0) mbar_arrive(&rempty[r]);
                n0 += nq;
                turn = (turn + nq) % kGroups;
            }
        }
    } else {
        if constexpr (XT == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSums));
        // Epilogue: lane's row as the decoders have it.
        const int w4 = warp & 3, half = lane >> 4, i = 16 * w4 + (lane & 15);
        const uint32_t lanes = (uint32_t)(32 * w4) << 16;
        uint32_t seg = 0;
        Item w;
        for (uint32_t it = 0; take(it, w); ++it) {
            const int col = p.gated ? w.rt * 64 + i : w.rt * 128 + 64 * half + i;
            const bool in = col < p.rows;
            const float *bias = p.gated && half ? p.bias[1] : p.bias[0];
            const float b = bias && in ? bias[(int64_t)w.group * p.rows + col] : 0.f;
            const float *inv = p.inv + (int64_t)w.gran * GT;
            auto release = [&] {   // the sums are read: others may overwrite them
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&accempty[seg % NBUF]);
                ++seg;
            };
            if constexpr (XT == 1) {
                float next[16];
                load_inv(inv, next);
                if (!waits(&accfull[seg % NBUF], (seg / NBUF) & 1)) break;
                tc_fence_after();
                const uint32_t acc = tmem + lanes + (seg % NBUF) * C::ACC;
#pragma unroll 1
                for (int t0 = 0; t0 < w.cnt; t0 += 16) {
                    float z[16], f[16];
                    uint32_t v[16], l[16];
                    tmem_ld16(acc + t0, v);
                    if constexpr (WT == 2) tmem_ld16(acc + NT + t0, l);
#pragma unroll
                    for (int u = 0; u < 16; ++u) f[u] = next[u];
                    if (t0 + 16 < w.cnt) load_inv(inv + t0 + 16, next);
                    tmem_ld_wait();
#pragma unroll
                    for (int u = 0; u < 16; ++u)
                        z[u] = WT == 2 ? fmaf(__uint_as_float(l[u]), 1.f / 2048.f, __uint_as_float(v[u])) : __uint_as_float(v[u]);
                    if (t0 + 16 >= w.cnt) release();
                    finish_typed(p, z, f, b, (int64_t)w.row0 + t0, w.cnt - t0, col, in, half);
                }
            } else {
                // 64 tokens' sums in registers, over the item's flushes.
                float sum[C::T];
                bool ok = true;
#pragma unroll
                for (int u = 0; u < C::T; ++u) sum[u] = 0.f;
#pragma unroll 1
                for (int b0 = 0; b0 < p.nst; b0 += C::FLUSH) {
                    if (!(ok = waits(&accfull[seg % NBUF], (seg / NBUF) & 1))) break;
                    tc_fence_after();
                    const uint32_t acc = tmem + lanes + (seg % NBUF) * C::ACC;
#pragma unroll
                    for (int t0 = 0; t0 < C::T; t0 += 8) {
                        if (t0 < w.cnt) {
                            // 8 high and 8 low sums, side by side or in two regions.
                            uint32_t v[16];
                            if constexpr (WT == 1) tmem_ld16(acc + 2 * t0, v);
                            else tmem_ld8x2(acc + t0, acc + C::T + t0, v);
                            tmem_ld_wait();
#pragma unroll
                            for (int u = 0; u < 8; ++u)
                                sum[t0 + u] += fmaf(__uint_as_float(v[8 + u]), 1.f / 2048.f, __uint_as_float(v[u]));
                        }
                    }
                    release();
                }
                if (!ok) break;
#pragma unroll
                for (int t0 = 0; t0 < C::T; t0 += 16) {
                    if (t0 < w.cnt) {
                        float z[16], f[16];
                        load_inv(inv + t0, f);
#pragma unroll
                        for (int u = 0; u < 16; ++u) z[u] = sum[t0 + u];
                        finish<RF_F32>(p, z, f, b, (int64_t)w.row0 + t0, w.cnt - t0, col, in, half);
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 3) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int FMT, int NT, int XT, int WT>
rf_status launch(const Params &p, int grid, cudaStream_t s)
{
    using C = Cfg<FMT, NT, XT, WT>;
    static std::once_flag once[64];
    static bool ok[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return RF_ERR_CUDA;
    }
    std::call_once(once[dev & 63], [dev] {
        ok[dev & 63] = cudaFuncSetAttribute(chunk_kernel<FMT, NT, XT, WT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            (int)C::SMEM) == cudaSuccess;
        cudaGetLastError();
    });
    if (!ok[dev & 63]) return RF_ERR_CUDA;
    chunk_kernel<FMT, NT, XT, WT><<<grid, kThreads, C::SMEM, s>>>(p);
    return last_cuda_error();
}

template <int FMT>
rf_status launch_fmt(const ChunkShape &sh, const Params &p, int grid, cudaStream_t s)
{
    if constexpr (FMT != RF_MXFP4) {
        if (sh.wt == 2) return sh.xt == 2 ? launch<FMT, 128, 2, 2>(p, grid, s) : launch<FMT, 128, 1, 2>(p, grid, s);
    } else {
        if (sh.xt == 2) return launch<FMT, 128, 2, 1>(p, grid, s);
    }
    return sh.nt == 256 ? launch<FMT, 256, 1, 1>(p, grid, s) : launch<FMT, 128, 1, 1>(p, grid, s);
}

}  // namespace

rf_status read_and_clear_chunk_status()
{
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_chunk_status, sizeof(int)) != cudaSuccess) return RF_ERR_CUDA;
    if (v != 0) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(g_chunk_status, &zero, sizeof(int)) != cudaSuccess) return RF_ERR_CUDA;
    }
    return static_cast<rf_status>(v);
}

rf_status launch_chunk_mma(const ChunkGemm &g, cudaStream_t s)
{
    const ChunkShape &sh = g.sh;
    Params p;
    std::memset(&p, 0, sizeof(p));
    const int64_t be = block_elems_of(sh.fmt), bs = (int64_t)block_bytes_of(sh.fmt);
    p.rb = sh.in_dim / be * bs;
    int P = 16;
    while (P > 1 && p.rb * (P / 2) % 16 == 0) P /= 2;
    p.P = P;
    while ((1 << p.logP) < P) ++p.logP;
    const int cb = sh.fmt == RF_Q4_0 || sh.fmt == RF_Q4_K ? 144 : 272;
    p.bw = cb + (P > 1 ? 16 : 0);
    p.gated = g.up != nullptr;
    p.W[0] = g.W;
    p.W[1] = g.up;
    const int64_t super = g.total_rows / P;
    p.copies = super > 0;
    for (int i = 0; i < (p.gated ? 2 : 1) && p.copies; ++i)
        if (!encode_u16_map(&p.map[i], p.W[i], (uint64_t)(P * p.rb / 2), (uint64_t)super, (uint64_t)(P * p.rb),
                            (uint32_t)(p.bw / 2), (uint32_t)(64 / P)))
            return RF_ERR_CUDA;
    p.row0 = g.row0;
    p.group_rows = g.group_rows;
    p.total_rows = g.total_rows;
    p.plan = reinterpret_cast<ChunkPlan *>(g.ws);
    p.tiles = reinterpret_cast<const ChunkTile *>(g.ws + sh.at_tiles);
    p.inv = reinterpret_cast<const float *>(g.ws + sh.at_inv);
    p.img = g.ws + sh.at_img;
    p.rows = (int32_t)sh.rows;
    p.nst = sh.nst;
    p.nch = (int32_t)((p.rb + cb - 1) / cb);
    p.nb = (int32_t)(sh.in_dim / be);
    p.nrt = (int32_t)((sh.rows + (p.gated ? 63 : 127)) / (p.gated ? 64 : 128));
    p.act = g.epi.act;
    p.alpha = g.epi.alpha;
    p.limit = g.epi.limit;
    p.bias[0] = g.epi.bias;
    p.bias[1] = g.epi.up_bias;
    p.residual = g.epi.residual;
    p.ldr = g.epi.ld_residual;
    p.dtype = g.dtype;
    p.Y = g.Y;
    p.ldy = g.ldy;
    p.limit_ns = kWaitLimitNs;
    p.withhold = -1;
    if (const unsigned long long lim = take_wait_fault()) {
        p.limit_ns = lim;
        p.withhold = sh.nst > 1 ? 1 : 0;
    }
    const int grid = (int)std::min<int64_t>(num_sms(), sh.cap_tiles * p.nrt);
    switch (sh.fmt) {
    case RF_Q4_0: return launch_fmt<RF_Q4_0>(sh, p, grid, s);
    case RF_Q8_0: return launch_fmt<RF_Q8_0>(sh, p, grid, s);
    case RF_Q4_K: return launch_fmt<RF_Q4_K>(sh, p, grid, s);
    default: return launch_fmt<RF_MXFP4>(sh, p, grid, s);
    }
}

}  // namespace rf
