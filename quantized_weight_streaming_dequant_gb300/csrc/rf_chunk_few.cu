// rf_chunk_few.cu -- products of the chunk operators where a group has few
// tokens: the same items, images and results as rf_chunk_mma.cu's, for token
// tiles of up to 16 operand rows.
//
// There a decoded slice passes through tensor memory, with a barrier before and
// one behind it, and a tile of few tokens waits for those more than for its
// products.  Here a warp decodes 16 rows straight into the fragments of
// mma.sync.m16n8k16 and multiplies them itself: nothing stands between a
// weight's bytes and its product but registers.  A decoded weight is used for
// at most 16 tokens, so the tensor cores' rate matters less than the way there.
//
// A CTA (two per SM) draws items of 128 matrix rows (64 of W and 64 of U with a
// gated activation) of a token tile.  One warp copies raw chunks and the
// tile's operand slices; each of the other eight takes 8 rows of either half of
// the tile.  Lane (g, t), of eight by four, owns row g of both halves and
// slice t of every four: a slice's two blocks are the fragments' columns,
// in the order in which the decoder has them (the sum over inputs does not
// care), and the token g of a tile of eight has its inputs in the same order.
// So gate and up of a neuron end in one thread.
//
// Terms.  fp32 calls have two fp16 terms an activation.  With up to four tokens
// a tile's eight columns are four high and four low terms, so that one product
// does both; with up to eight they are products of their own.  Low terms of
// weights multiply either (Q8_0 and Q4_0: exact as they are, because n * d less
// its rounding is a multiple of fp16's least number; Q4_K: scaled by 2^11).
//
// Bound.  By 2048 weights (a warp's 16 rows x 128 inputs, MXFP4, one term) an
// SM takes about 75 cycles: 32 of the tensor cores (16 a product and SM
// quarter), 40 of integer instructions, 46 of memory; 16 warps an SM overlap
// them as far as their registers (96 a thread) let them.  The copies are a limit
// of their own: alone they run at 5.2 TB/s in the first case (87 of the experts
// have rows, 1.15 GB) and at 4.1 in the third, of 6.8 measured.  Measured, us a
// call on the GPU:
//                                                   here   through tensor memory
//   77 bf16 tokens, 128 experts of 2880 MXFP4        314   372   (copies alone: 224)
//   6 fp32 tokens, the same                           98   135   (copies alone:  79,
//                                                         with a slower pre-pass)
//   45 fp32 rows, 64 groups of 1408 x 2048 Q8_0       34    51   (copies alone:  28)
//   8 bf16 tokens, 2 x 11008 x 4096 Q4_0              28    41
// Steps (first case, us): 458 with all of a block decoded before its products
// and 8-byte loads; 412 with 4-byte loads, the item's end prefetched and one
// address for both rows; 370 with tiles of 8 operand rows; 348 with a chunk's
// scales looked at together; 317 with one stage for a raw chunk and its operand
// slices (one barrier a chunk instead of three).  At 370 it took 244 without
// the products.  Tried and not kept: several chains of sums for each kind of
// product (352 against 348); scales looked at beside the products, which are
// done again if need be (340 against 317: registers); tiles of 32 operand rows
// (see chunk_shape).
#include <algorithm>
#include <mutex>
#include <type_traits>

#include "rf_chunk.cuh"

namespace rf {
using namespace chunk;
namespace {

__device__ int g_few_status = 0;   // bounded waits that gave up

constexpr int kWarps = 8;          // that multiply; one more copies

// NT: operand rows per token tile, 8 (of two terms: four tokens, whose terms are
// columns of one product) or 16; XT, WT: fp16 terms per activation, weight.
template <int FMT, int NT, int XT, int WT>
struct Few {
    static constexpr int CB = chunk_bytes(FMT), QPC = chunk_weights(FMT) / kSliceK;
    static constexpr bool BOTH = NT == 8 && XT == 2;                     // a column of either term
    static constexpr int T = NT / XT, NJ = (T + 7) / 8;                  // tokens, and tiles of eight of them
    static constexpr int GB = NT * kSliceK * 2;                          // operand bytes of a slice
    // MXFP4: a four of slices are every other one of a chunk (see Weights).
    static constexpr bool SPREAD = FMT == RF_MXFP4;
    static constexpr int N = BOTH ? WT : XT + WT - 1;                    // kinds of products
    // Q4_K's low terms in fp32 calls are scaled; the others' are exact as they are.
    static constexpr int LOW = WT == 1 ? kOne : (XT == 2 && FMT == RF_Q4_K ? kScaled : kPlain);
    // Two CTAs share an SM's 228 KB, of which each leaves 1 KB to the system.
    static constexpr int SHARED = 115200;
    // A stage: a raw chunk and the tile's operand slices for it.
    static constexpr int RAW = kM * box_bytes(FMT, 8), OPS = QPC * GB, STAGE = RAW + OPS;
    static constexpr int S = SHARED / STAGE < 4 ? SHARED / STAGE : 4;
    static constexpr int SMEM = S * STAGE;
    static constexpr int FULL = 0, EMPTY = S, BARS = 2 * S;
    static_assert(S >= 2, "two stages");
    static_assert(QPC == (SPREAD ? 8 : 4), "fours of slices of a chunk");
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A block of 32 weights of a row, decoded four pairs at a time.  4-byte loads
// from any byte of shared memory: the rows of a warp's eight g are an odd
// number of 16-byte units apart, the slices of its four t 4 * (1 mod 4) bytes,
// so that its 32 lanes meet 32 banks.
template <int FMT, int L>
struct Weights {
    static constexpr int NS = FMT == RF_MXFP4 ? 1 : 2, NW = FMT == RF_Q8_0 ? 8 : 4;   // scale bytes, quant words
    uint32_t q[NW], s1, s2;
    // From byte sh / 8 of the word at `src`.
    __device__ __forceinline__ void load(const uint8_t *from, uint32_t sh)
    {
        const uint32_t *src = reinterpret_cast<const uint32_t *>(from);
        uint32_t x[NW + 1];
#pragma unroll
        for (int i = 0; i < NW + 1; ++i) x[i] = src[i];
        s1 = (x[0] >> sh) & (NS == 1 ? 0xFFu : 0xFFFFu);
#pragma unroll
        for (int i = 0; i < NW; ++i) q[i] = __funnelshift_rc(x[i], x[i + 1], sh + 8 * NS);
        if constexpr (FMT != RF_MXFP4) s1 *= 0x00010001u;
    }
    // MXFP4's factor (ANY: a warp's lane needs it split).
    template <bool ANY>
    __device__ __forceinline__ void scale()
    {
        const uint32_t E = s1;
        s1 = e8m0_factor(E);
        if constexpr (ANY) e8m0_factors(E, s1, s2);
    }
    // A block behind the row's last one.
    __device__ __forceinline__ void clear() { s1 = s2 = 0u; }
    template <bool ANY>
    __device__ __forceinline__ void pairs(int m, uint32_t (&hi)[4], uint32_t (&lo)[4]) const
    {
        if constexpr (FMT == RF_MXFP4) {
            e2m1x8(q[m], hi);
#pragma unroll
            for (int k = 0; k < 4; ++k) hi[k] = hmul2(hi[k], s1);
            if constexpr (ANY) {
#pragma unroll
                for (int k = 0; k < 4; ++k) hi[k] = hmul2(hi[k], s2);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if constexpr (FMT == RF_Q4_0) product<L>(q4_0_pair(q[m], k), s1, hi[k], lo[k]);
                else product<L>(q8_0_pair(q[2 * m + (k >> 1)], k & 1), s1, hi[k], lo[k]);
            }
        }
    }
};
template <int L>
struct Weights<RF_Q4_K, L> {
    Q4K b;
    __device__ __forceinline__ void clear() { b.ds = b.dm = 0.f; }
    template <bool ANY>
    __device__ __forceinline__ void pairs(int m, uint32_t (&hi)[4], uint32_t (&lo)[4]) const
    {
        b.template pairs<L>(2 * m, hi[0], lo[0], hi[1], lo[1]);
        b.template pairs<L>(2 * m + 1, hi[2], lo[2], hi[3], lo[3]);
    }
};

// LONG: sums of 16-bit calls leave the tensor cores' truncated additions with
// every raw chunk, as rows of several segments need it (see chunk_shape); the
// registers for both sums cost shorter rows 0 to 4 % (77 bf16 tokens through the
// experts 308 against 305 us, 150 fp16 tokens 435 against 422, 16 fp16 tokens
// through 22016 x 4096 Q8_0 50.6 against 48.7).
template <int FMT, int NT, int XT, int WT, bool LONG>
__global__ void __launch_bounds__(32 * (kWarps + 1), 2) few_kernel(const __grid_constant__ Params p)
{
    using C = Few<FMT, NT, XT, WT>;
    constexpr int NJ = C::NJ, QPC = C::QPC;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ uint64_t bars[C::BARS];
    __shared__ int s_stop;
    volatile int *stop = &s_stop;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::BARS; ++i) mbar_init(&bars[i], i >= C::EMPTY ? kWarps : 1);
        s_stop = 0;
        fence_barrier_init();
    }
    __syncthreads();
    const uint32_t bar0 = smem_addr(bars);
    auto bar = [&](int i) -> uint32_t { return bar0 + 8u * (uint32_t)i; };
    auto wait = [&](uint32_t at, uint32_t parity) -> bool {
        if (bar_try(at, parity)) return true;
        const long long t0 = clock64();
        while (!bar_try_ns(at, parity, 20000u))
            if (*stop || *reinterpret_cast<volatile int *>(&g_few_status) != 0 || clock64() - t0 > p.limit_cycles) {
                record_status(&g_few_status, RF_ERR_TIMEOUT);
                *stop = 1;
                return false;
            }
        return true;
    };
    auto waits = [&](uint32_t at, uint32_t parity) -> bool { return __all_sync(0xffffffffu, wait(at, parity)); };
    const int total = p.plan->n_tiles * p.nrt * p.parts;   // at most 2^30

    if (warp == kWarps) {
        // Lane l copies box l of a chunk (half l / P, position l % P), lane 0
        // the operand slices too.
        const int half = lane >> p.logP, j = lane & (p.P - 1);
        const bool copies = half < 2 && p.copies;
        const uint32_t dst = smem_addr(smem) + (uint32_t)lane * (uint32_t)((64 >> p.logP) * p.bw), dst_ops = smem_addr(smem) + C::RAW;
        const int xj = (int)((int64_t)j * p.rb);
        const CUtensorMap *map = &p.map[p.gated ? half & 1 : 0];
        uint32_t n = 0, r = 0, ph = 1;   // stages copied; place in the ring and phase
        uint32_t skipped = 0xffffffffu;
        bool ok = true;
        for (int index = blockIdx.x; ok && index < total; index += gridDim.x) {
            const int at = index / p.parts, part = index % p.parts;
            const ChunkTile w = p.tiles[at / p.nrt];
            const int rt = at % p.nrt;
            const int64_t first = p.row0 + (int64_t)w.group * p.group_rows +
                                  (p.gated ? (int64_t)rt * 64 : (int64_t)rt * 128 + 64 * half);
            const int y = (int)((first - j + p.P - 1) >> p.logP);   // first super-row with position j in the tile
            const uint8_t *src = p.img + ((int64_t)w.gran * p.nst + part * p.part_chunks * QPC) * C::GB;
            for (int c = part * p.part_chunks, end = min(p.nch, c + p.part_chunks); ok && c < end; ++c) {
                if (!(ok = waits(bar(C::EMPTY + r), ph))) break;
                const bool withhold = blockIdx.x == 0 && n == 0 && p.withhold;   // (CTA 0 has the first item)
                if (withhold) skipped = n;
                if (lane == 0) bar_expect(bar(C::FULL + r), (uint32_t)(C::OPS + (p.copies ? kM * p.bw : 0)));
                __syncwarp();
                if (!withhold) {
                    if (copies) copy_box(dst + r * C::STAGE, map, ((xj + c * C::CB) & ~15) >> 1, y, bar(C::FULL + r));
                    if (lane == 0) copy_bulk(dst_ops + r * C::STAGE, src, C::OPS, bar(C::FULL + r));
                }
                src += C::OPS;
                ++n;
                if (++r == C::S) r = 0, ph ^= 1u;
            }
        }
        // Every copy issued lands before the CTA can exit.
        if (lane == 0)
            for (uint32_t i = n > C::S ? n - C::S : 0; i < n; ++i)
                if (i != skipped) bar_drain(bar(C::FULL + i % C::S), (i / C::S) & 1);
        return;
    }

    const int g = lane >> 2, t = lane & 3, i = lane_row(8 * warp + g, p.logP);
    const int64_t copied = p.copies ? p.total_rows & ~(int64_t)(p.P - 1) : 0;   // rows in whole super-rows
    const int swz = ((g ^ (2 * t)) & 7) * 16;   // see prep_kernel
    uint32_t r = 0, ph = 0;
    ChunkTile next = {};
    if ((int)blockIdx.x < total) next = p.tiles[blockIdx.x / p.parts / p.nrt];
    for (int index = blockIdx.x; index < total; index += gridDim.x) {
        const int at = index / p.parts, part = index % p.parts;
        const ChunkTile w = next;
        const int rt = at % p.nrt;
        // The row of half 1 lies 64 rows of a box behind half 0's: P divides 64.
        int64_t row[2];
        bool tail[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            row[h] = p.row0 + (int64_t)w.group * p.group_rows + (p.gated ? (int64_t)rt * 64 : (int64_t)rt * 128 + 64 * h) + i;
            tail[h] = row[h] >= copied && row[h] < p.total_rows;
        }
        const int64_t first = row[0] - i;
        const int j = (int)(row[0] & (p.P - 1));
        const int s = (int)((row[0] >> p.logP) - ((first - j + p.P - 1) >> p.logP));
        const uint32_t half = (uint32_t)(64 * p.bw);
        const uint32_t start = (uint32_t)j * (uint32_t)((64 >> p.logP) * p.bw) + (uint32_t)(s * p.bw) + ((uint32_t)(j * p.rb) & 15u);
        // This lane's first block (Q4_K: super-block), and the word in which it begins.
        const uint32_t off = start + (FMT == RF_Q4_K ? 0 : t * (C::SPREAD ? 4 : 2) * block_size(FMT));
        const uint32_t mis = off & 3u, word = off - mis;
        const bool tails = __any_sync(0xffffffffu, tail[0] || tail[1]);
        // Sums of (row g of half h, token 8 q + 2 t + e): [..][q][2 h + e], for
        // each kind of product.  fp32: rounded additions move them to `sum` every
        // eight products, because the tensor cores truncate each of theirs, always
        // towards zero (with sixteen a routed FFN of 960 and 5408 inputs is 1.0e-6
        // from 64 bits, and no faster).
        float acc[C::N][NJ][4], sum[NJ][4];
        auto flush = [&] {
#pragma unroll
            for (int q = 0; q < NJ; ++q)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    // By terms of (weight, activation): high high, high low, low high.
                    float f[C::N];
#pragma unroll
                    for (int n = 0; n < C::N; ++n) f[n] = acc[n][q][k];
                    const float scaled = 1.f / 2048.f;
                    if constexpr (C::BOTH) {   // (the column says which of the activation's)
                        if constexpr (WT == 2) f[0] = C::LOW == kScaled ? fmaf(f[1], scaled, f[0]) : f[0] + f[1];
                    } else if constexpr (XT == 2) {
                        if constexpr (WT == 2) f[C::LOW == kScaled ? 1 : 0] += f[2];
                        f[0] = fmaf(f[1], scaled, f[0]);
                    } else if constexpr (WT == 2) {
                        f[0] += f[1];
                    }
                    sum[q][k] += f[0];
#pragma unroll
                    for (int n = 0; n < C::N; ++n) acc[n][q][k] = 0.f;
                }
        };
#pragma unroll
        for (int q = 0; q < NJ; ++q)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                sum[q][k] = 0.f;
#pragma unroll
                for (int n = 0; n < C::N; ++n) acc[n][q][k] = 0.f;
            }
        // What the end of the item needs, asked for early.
        float bias[2];
        int col[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            col[h] = p.gated ? rt * 64 + i : rt * 128 + 64 * h + i;
            const float *from = p.gated && h ? p.bias[1] : p.bias[0];
            bias[h] = from && p.parts == 1 && col[h] < p.rows ? from[(int64_t)w.group * p.rows + col[h]] : 0.f;
        }
        float inv[NJ][2];
#pragma unroll
        for (int q = 0; q < NJ; ++q)
#pragma unroll
            for (int e = 0; e < 2; ++e) inv[q][e] = __ldg(p.inv + (int64_t)w.gran * C::T + min(8 * q + 2 * t + e, w.cnt - 1));
        if (index + (int)gridDim.x < total) next = p.tiles[(index + (int)gridDim.x) / p.parts / p.nrt];
        for (int c = part * p.part_chunks, end = min(p.nch, c + p.part_chunks); c < end; ++c) {
            if (!waits(bar(C::FULL + r), ph)) return;
            uint8_t *src = smem + r * C::STAGE, *lane_src = src + word;
            const uint8_t *ops = src + C::RAW + t * C::GB + swz;
            if (tails) {
                // Rows that the boxes do not reach, copied to where they would
                // put them.
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (tail[h]) {
                        const uint8_t *from = p.W[p.gated ? h : 0] + row[h] * p.rb + (int64_t)c * C::CB;
                        const int n = (int)min((int64_t)C::CB, p.rb - (int64_t)c * C::CB);
#pragma unroll 1
                        for (int k = t; k < n; k += 4) src[start + h * half + k] = __ldg(from + k);
                    }
                __syncwarp();
            }
            // Whether a scale of the warp's blocks is none of fp16's normal numbers.
            bool any = false;
            if constexpr (FMT == RF_MXFP4) {
                uint32_t place = 0;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        place = max(place, e8m0_place(src[start + h * half + (4 * t + k) * block_size(FMT)]));
                any = e8m0_far(place);
            }
            const bool ragged = FMT != RF_Q4_K && 2 * (c + 1) * QPC > p.nb;
            // Four slices.
            auto four = [&](int q4, auto any_scale) {
                constexpr bool ANY = decltype(any_scale)::value;
                const uint8_t *x = ops + q4 * C::GB;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    Weights<FMT, C::LOW> wt[2];
                    if constexpr (FMT == RF_Q4_K) {
                        wt[0].b.load(lane_src, t, e), wt[1].b.load(lane_src + half, t, e);
                    } else {
                        const uint32_t at = mis + (2 * (C::SPREAD ? q4 / 4 : 0) + e) * block_size(FMT);
                        const uint8_t *from = lane_src + (at & ~3u);
                        wt[0].load(from, 8u * (at & 3u)), wt[1].load(from + half, 8u * (at & 3u));
                    }
                    if constexpr (FMT == RF_MXFP4) wt[0].template scale<ANY>(), wt[1].template scale<ANY>();
                    if (ragged) {
                        const int sl = C::SPREAD ? 2 * t + q4 / 4 : q4 + t;   // slice of the chunk
                        const bool dead = 2 * (c * QPC + sl) + e >= p.nb;     // the bytes are the next row's
                        if (dead) wt[0].clear(), wt[1].clear();
                    }
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        uint32_t hi[2][4], lo[2][4];
#pragma unroll
                        for (int h = 0; h < 2; ++h) wt[h].template pairs<ANY>(m, hi[h], lo[h]);
#pragma unroll
                        for (int q = 0; q < NJ; ++q) {
                            if (NJ > 1 && 8 * q >= w.cnt) break;
                            // (Of two terms the low ones' eight rows are behind the high ones'.)
                            const uint8_t *xm = x + q * 1024 + (4 * e + m) * 128;
                            const uint4 v = *reinterpret_cast<const uint4 *>(xm);
                            [[maybe_unused]] uint4 l = {};
                            if constexpr (XT == 2 && !C::BOTH) l = *reinterpret_cast<const uint4 *>(xm + 1024);
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const uint32_t b0 = k ? v.z : v.x, b1 = k ? v.w : v.y;
                                mma16816(acc[0][q], hi[0][2 * k], hi[1][2 * k], hi[0][2 * k + 1], hi[1][2 * k + 1], b0, b1);
                                if constexpr (XT == 2 && !C::BOTH)
                                    mma16816(acc[1][q], hi[0][2 * k], hi[1][2 * k], hi[0][2 * k + 1], hi[1][2 * k + 1],
                                             k ? l.z : l.x, k ? l.w : l.y);
                                if constexpr (WT == 2)
                                    mma16816(acc[C::N - 1][q], lo[0][2 * k], lo[1][2 * k], lo[0][2 * k + 1], lo[1][2 * k + 1], b0, b1);
                            }
                        }
                    }
                    if constexpr (XT == 2) flush();
                }
            };
            if (FMT == RF_MXFP4 && any) {
#pragma unroll 1
                for (int q4 = 0; q4 < QPC; q4 += 4) four(q4, std::true_type());
            } else {
#pragma unroll
                for (int q4 = 0; q4 < QPC; q4 += 4) four(q4, std::false_type());
            }
            if constexpr (LONG) flush();
            if (tails) fence_async_smem();   // the next copy follows these stores
            __syncwarp();
            if (lane == 0) bar_arrive(bar(C::EMPTY + r));
            if (++r == C::S) r = 0, ph ^= 1u;
        }
        if constexpr (XT == 1 && !LONG) flush();
        if constexpr (C::BOTH) {   // the low terms' columns are two lanes on
#pragma unroll
            for (int k = 0; k < 4; ++k) sum[0][k] = fmaf(__shfl_xor_sync(0xffffffffu, sum[0][k], 2), 1.f / 2048.f, sum[0][k]);
        }
        // What follows the product.
#pragma unroll
        for (int q = 0; q < NJ; ++q)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int tok = 8 * q + 2 * t + e;
                if (tok >= w.cnt) continue;   // (at most C::T)
                const int64_t y = w.row0 + tok;
                float z[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) z[h] = fmaf(sum[q][2 * h + e], inv[q][e], bias[h]);
                if (p.parts > 1) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (col[h] < p.rows)
                            p.sums[((int64_t)(part * (1 + p.gated) + (p.gated ? h : 0)) * p.n_row + y) * p.rows + col[h]] = z[h];
                } else if (p.gated) {
                    if (col[0] < p.rows) finish_one(p, y, col[0], z[0], z[1]);
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (col[h] < p.rows) finish_one(p, y, col[h], z[h], 0.f);
                }
            }
    }
}

template <int FMT, int NT, int XT, int WT, bool LONG>
rf_status launch(const Params &p, int grid, cudaStream_t s)
{
    using C = Few<FMT, NT, XT, WT>;
    static std::once_flag once[64];
    static bool ok[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return RF_ERR_CUDA;
    }
    std::call_once(once[dev & 63], [dev] {
        ok[dev & 63] = cudaFuncSetAttribute(few_kernel<FMT, NT, XT, WT, LONG>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) ==
                       cudaSuccess;
        cudaGetLastError();
    });
    if (!ok[dev & 63]) return RF_ERR_CUDA;
    few_kernel<FMT, NT, XT, WT, LONG><<<grid, 32 * (kWarps + 1), C::SMEM, s>>>(p);
    return last_cuda_error();
}

template <int FMT, int NT>
rf_status launch_terms(const ChunkShape &sh, const Params &p, int grid, cudaStream_t s)
{
    if (sh.xt == 2) return launch<FMT, NT, 2, FMT == RF_MXFP4 ? 1 : 2, false>(p, grid, s);
    if constexpr (FMT != RF_MXFP4)
        if (sh.wt == 2) return sh.segments ? launch<FMT, NT, 1, 2, true>(p, grid, s) : launch<FMT, NT, 1, 2, false>(p, grid, s);
    return sh.segments ? launch<FMT, NT, 1, 1, true>(p, grid, s) : launch<FMT, NT, 1, 1, false>(p, grid, s);
}
template <int FMT>
rf_status launch_fmt(const ChunkShape &sh, const Params &p, int grid, cudaStream_t s)
{
    return sh.nt > 8 ? launch_terms<FMT, 16>(sh, p, grid, s) : launch_terms<FMT, 8>(sh, p, grid, s);
}

}  // namespace

rf_status read_and_clear_few_status()
{
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_few_status, sizeof(int)) != cudaSuccess) return RF_ERR_CUDA;
    if (v != 0) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(g_few_status, &zero, sizeof(int)) != cudaSuccess) return RF_ERR_CUDA;
    }
    return static_cast<rf_status>(v);
}

rf_status launch_chunk_few(const ChunkShape &sh, const Params &p, cudaStream_t s)
{
    const int grid = (int)std::min<int64_t>(2 * num_sms(), sh.cap_tiles * p.nrt * p.parts);
    switch (sh.fmt) {
    case RF_Q4_0: return launch_fmt<RF_Q4_0>(sh, p, grid, s);
    case RF_Q8_0: return launch_fmt<RF_Q8_0>(sh, p, grid, s);
    case RF_Q4_K: return launch_fmt<RF_Q4_K>(sh, p, grid, s);
    default: return launch_fmt<RF_MXFP4>(sh, p, grid, s);
    }
}

}  // namespace rf
