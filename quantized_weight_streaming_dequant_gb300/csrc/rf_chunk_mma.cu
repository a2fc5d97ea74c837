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
//   decoders     four groups of four warps, each with a stage of its own (a
//                64-input slice) or half of one of two (two or four slices): a
//                thread takes its row, turns the raw bytes into fp16 pairs and
//                stores them to tensor memory, from where tcgen05.mma reads the
//                weights: they cost no shared-memory bandwidth, which is what
//                bounds tiles whose operands both lie there;
//   epilogue     four warps read the sums out of tensor memory, while the
//                others are at the next item.
//
// Order of the inputs.  A product does not care in which order its inputs are
// summed, so a slice's inputs are in the order in which the decoder finds them
// cheapest (slice_order in rf_chunk.cu): for MXFP4 the two nibbles of a byte,
// for Q4_0 nibbles four apart.
//
// Precision: see rf.h.  Two fp16 terms of an activation are two rows of the
// operand (8 high, 8 low) with sums of their own; the low terms are scaled by
// 2^11.  Low terms of weights multiply the high terms of activations (the
// product of two low terms is below 2^-22 of the result).
//
// Every wait is bounded; after a failure every role stops, copies and products
// already issued are waited for, and tensor memory is freed.
//
// Bound.  A slice of 128 x 64 weights costs its decoding (half-rate integer
// instructions of 16 warps: about 190 cycles for Q4_0 and MXFP4, twice that for
// two terms), its products (384 cycles at 192 rows) and its copies; the roles
// run side by side, but a stage passes from one to the next by barriers (100 to
// 200 cycles each), so that a slice takes 410 to 640 cycles where the longest of
// the three alone would take 200 to 450.  Measured (us a launch):
//   2048 bf16 rows, 2 x 11008 x 4096 Q4_0      258   1.43 PFLOP/s (0.75 of the
//                                                    measured cuBLAS rate)
//   2048 bf16 rows, 4096 x 11008 Q8_0          182   1.01 PFLOP/s
//   8192 bf16 rows, 128 experts of 2880 x 2880 MXFP4, gate, up and down:
//                                              666   0.61 PFLOP/s, 2.5 TB/s
//   5000 fp16 rows (two terms), 24 groups of 4000 x 2080 Q4_0:   142
// The first with products alone (no copies, no decoding): 180.  Items are drawn
// four ahead, so that a CTA's last four are fixed early: with few items an SM
// nothing is left to even out.  Neighbouring lanes of an epilogue hold rows P
// apart (lane_row): where rows are no multiples of 16 bytes (P = 8 for 2,880
// MXFP4 inputs) a warp's store of 32 values touches 16 to 32 sectors.
// Tried and not kept (the first case, us, against 268 at the time unless said
// otherwise): tiles of 256 rows, whose sums fit once, 308; activations in a ring
// of bytes instead of slots, 460 against 295; the issuing role in lane 0 by
// number, 388 against 300; an issuing loop that is not unrolled, 1027 against
// 840 in the third case; six stages of weights for tiles of 64 rows, three
// decoder groups, more raw chunks in flight, and fewer or larger stages of
// activations: nothing; dependent launches, 54 against 38 in a small call; waits
// that poll without the hardware's own pause, 10 to 20 % slower.
#include <algorithm>
#include <cstring>
#include <mutex>

#include "rf_chunk.cuh"

namespace rf {
using namespace chunk;
namespace {

__device__ int g_chunk_status = 0;   // bounded waits that gave up

constexpr int kDec0 = 4;             // first decoder warp; the epilogue's four follow the decoders
constexpr int kItems = 4;            // items drawn ahead
constexpr int kInFlight = 16;        // stages of activations in flight at most
constexpr int kRaws = 8;             // raw chunks in flight at most

// NT: operand rows per token tile at most; XT, WT: fp16 terms per activation, weight.
// A stage is KS slices of weights (tensor memory) and activations (shared
// memory): several where a slice's products are short, so that what a stage
// costs to hand over (the issuing warp's waits and commits, about 140 cycles,
// and the way to the decoders and back) is paid less often.  Four slices
// instead of two: 512 bf16 tokens through the experts below 592 against 681 us;
// two instead of one for two terms of both: 512 fp32 tokens through
// 2 x 11008 x 4096 Q4_0 281 against 287, but 5000 fp16 rows (one term of the
// activations) 162 against 153, and 192 bf16 rows no difference.
template <int FMT, int NT, int XT, int WT>
struct Cfg {
    static constexpr int CB = chunk_bytes(FMT);                        // chunk bytes per row
    static constexpr int QPC = chunk_weights(FMT) / kSliceK;           // slices per chunk
    static constexpr int BW = box_bytes(FMT, 8);                       // box bytes at most
    static constexpr int T = NT / XT;                                  // tokens
    static constexpr int KS = NT > 128 ? 1 : (WT == 1 ? 4 : XT);
    static constexpr int S = KS > 1 ? 2 : 4;                           // stages of weights
    static constexpr int G = 4, GPS = G / S;                           // decoder groups of four warps; those of a stage
    static constexpr int KD = KS / GPS;                                // slices of a stage that one of them decodes
    static constexpr int EPI0 = kDec0 + 4 * G, THREADS = 32 * (EPI0 + 4);
    static constexpr int USERS = 3 + 4 * G + 4;                        // warps that take an item
    // Registers a thread: what a launch gives every warp, and what the roles
    // trade among them (fp32 calls hold 64 sums a thread in the epilogue).
    static constexpr int REGS = 65536 / THREADS / 8 * 8, RROLES = 40, RDEC = REGS - 8;
    static constexpr int REPI = (G + 2) * REGS - RROLES - G * RDEC;
    static constexpr int BT = NT * kSliceK * 2;                        // activation bytes per slice at most
    static constexpr int RAW = kM * BW;
    static constexpr int LOW = WT == 1 ? 0 : (XT == 1 ? 1 : 2);        // Low
    // Columns of one item's sums (with two terms of both: T of high products,
    // T of the others).
    static constexpr int ACC = NT;
    static constexpr int ASLICE = 32 * WT, ASTAGE = KS * ASLICE;
    static constexpr int ACOL = 512 - S * ASTAGE;                      // first column of the weights
    static constexpr int NBUF = 2 * ACC <= ACOL ? 2 : 1;
    // Sums of fp32 calls leave tensor memory every FLUSH slices: the tensor
    // cores truncate each addition (about 1e-8 of the sum, always towards
    // zero), rounded additions in registers do not drift.  Q4_K's weights have
    // a mean, so that its sums grow over a row: sooner (1.3e-6 against 0.7e-6
    // from 64 bits in a routed FFN).
    // 16-bit calls' leave it at the end of the row, or of a segment of it (LONG).
    static constexpr int FLUSH = XT == 1 ? 1 << 30 : (FMT == RF_Q4_K ? 2 : 4);
    // Shared memory: stages of activations, raw chunks, and 16 bytes that a
    // last load may touch.  Activations come from L2 in about as long as eight
    // slices take; the weights come from memory and get the rest.
    static constexpr int SHARED = 230000;
    static constexpr size_t SMEM = SHARED + 16;
    static constexpr int LEAST = (NT > 128 ? 6 : 8) / KS;              // stages of activations at least
    // Barriers, by number.
    static constexpr int FULL = 0, ADONE = FULL + S, BFULL = ADONE + S, BDONE = BFULL + kInFlight, RFULL = BDONE + kInFlight,
                         REMPTY = RFULL + kRaws, ACCF = REMPTY + kRaws, ACCE = ACCF + NBUF, IFULL = ACCE + NBUF, IEMPTY = IFULL + kItems,
                         DRAIN = IEMPTY + kItems, BARS = DRAIN + 1;
    static_assert(ACC * NBUF <= ACOL, "tensor memory");
    static_assert(QPC % KS == 0 && FLUSH % KS == 0, "a stage lies in one chunk and between two flushes");
    static_assert(T % 16 == 0, "the epilogue takes 16 tokens at a time");
    static_assert(G % S == 0 && (S & (S - 1)) == 0 && KS % GPS == 0, "each group has a stage, or a share of one");
    static_assert(REPI <= 248 && REPI % 8 == 0 && RROLES < REGS, "registers");
    static_assert(LEAST * KS * BT + 2 * RAW <= SHARED && LEAST <= kInFlight, "the least stages and two chunks fit");
};

struct Item {
    int32_t group, row0, cnt, gran, rt, stop, part, first;   // first: the launch's first item
};

__host__ __device__ constexpr uint32_t idesc_n(int n)
{
    return (1u << 4) | (0u << 7) | (0u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kM >> 4) << 24);
}

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
// The same for a part of the row's inputs: the sums alone.
__device__ __forceinline__ void keep(const Params &p, const float (&z)[16], const float (&inv)[16], int part, int64_t r0, int n,
                                     int col, bool in, int half)
{
    float *y = p.sums + ((int64_t)(part * (1 + p.gated) + (p.gated ? half : 0)) * p.n_row + r0) * p.rows + col;
#pragma unroll
    for (int u = 0; u < 16; ++u)
        if (in && u < n) y[(int64_t)u * p.rows] = z[u] * inv[u];
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

__device__ __forceinline__ void bar_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// LONG: 16-bit rows of several segments.  A form of its own, because with the
// segment's length as a variable every row pays (2048 bf16 tokens through
// 2 x 11008 x 4096 274 against 272 us, 5000 fp16 rows of 24 groups 158 against
// 156, the routed FFN of 2048 tokens 749 against 743); segments cost long rows 0
// to 1 % (2048 bf16 tokens through 4096 x 32768 506 us either way, fp16 through
// 4096 x 11008 308 against 305).
template <int FMT, int NT, int XT, int WT, bool LONG>
__global__ void __launch_bounds__((Cfg<FMT, NT, XT, WT>::THREADS), 1) chunk_kernel(const __grid_constant__ Params p)
{
    using C = Cfg<FMT, NT, XT, WT>;
    constexpr int S = C::S, KS = C::KS, QPC = C::QPC, NBUF = C::NBUF, GT = kGranRows / XT;
    constexpr int G = C::G, kEpi0 = C::EPI0;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *raw = smem + p.raw_at;
    // FULL: a stage's weights are decoded (an arrival per decoder warp); BFULL: its activations have landed; ADONE, BDONE: its products
    // are through; RFULL, REMPTY: raw chunks; ACCF, ACCE: sums; IFULL, IEMPTY:
    // items.
    __shared__ uint64_t bars[C::BARS];
    __shared__ Item items[kItems];
    __shared__ uint32_t s_tmem;
    __shared__ int s_stop;
    volatile int *stop = &s_stop;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::BARS; ++i) {
            uint32_t n = 1;
            if (i < C::ADONE) n = 4 * C::GPS;
            else if (i >= C::REMPTY && i < C::ACCF) n = 4 * G;
            else if (i >= C::ACCE && i < C::IFULL) n = 4;
            else if (i >= C::IEMPTY && i < C::DRAIN) n = C::USERS;
            mbar_init(&bars[i], n);
        }
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
    const uint32_t bar0 = smem_addr(bars);
    auto bar = [&](int i) -> uint32_t { return bar0 + 8u * (uint32_t)i; };
    // Bounded by the SM's clock (reading the global timer takes as long as a
    // stage's products).  Short, because every role has a few of it in its
    // loop, and a role's instructions are fetched anew whenever the other
    // roles' have pushed them out.
    auto wait = [&](uint32_t at, uint32_t parity) -> bool {
        if (bar_try(at, parity)) return true;
        const long long t0 = clock64();
        while (!bar_try_ns(at, parity, 20000u))
            if (*stop || *reinterpret_cast<volatile int *>(&g_chunk_status) != 0 || clock64() - t0 > p.limit_cycles) {
                record_status(&g_chunk_status, RF_ERR_TIMEOUT);
                *stop = 1;
                return false;
            }
        return true;
    };
    // A warp's waits; the next item, copied from its slot (one arrival a warp).
    auto waits = [&](uint32_t at, uint32_t parity) -> bool { return __all_sync(0xffffffffu, wait(at, parity)); };
    auto take = [&](uint32_t it, Item &w) -> bool {
        const int slot = it % kItems;
        if (!waits(bar(C::IFULL + slot), (it / kItems) & 1)) return false;
        const int32_t *src = reinterpret_cast<const int32_t *>(&items[slot]);
        w.group = __shfl_sync(0xffffffffu, src[0], 0), w.row0 = __shfl_sync(0xffffffffu, src[1], 0);
        w.cnt = __shfl_sync(0xffffffffu, src[2], 0), w.gran = __shfl_sync(0xffffffffu, src[3], 0);
        w.rt = __shfl_sync(0xffffffffu, src[4], 0), w.stop = __shfl_sync(0xffffffffu, src[5], 0);
        w.part = __shfl_sync(0xffffffffu, src[6], 0);
        __syncwarp();
        if (lane == 0) bar_arrive(bar(C::IEMPTY + slot));
        return w.stop == 0;
    };

    // (Registers are traded for good: the roles do not join again before the end.)
    if (warp < kDec0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::RROLES));
    if (warp == 3) {
        if (lane == 0) {
            const int total = p.plan->n_tiles * p.nrt * p.parts;   // at most 2^30
            for (uint32_t it = 0;; ++it) {
                const int slot = it % kItems;
                if (!wait(bar(C::IEMPTY + slot), ((it / kItems) & 1) ^ 1)) break;
                Item &w = items[slot];
                const int index = atomicAdd(&p.plan->next, 1);
                w.stop = index >= total;
                if (!w.stop) {
                    const int at = index / p.parts;
                    const ChunkTile t = p.tiles[at / p.nrt];
                    w.group = t.group, w.row0 = t.row0, w.cnt = t.cnt, w.gran = t.gran;
                    w.rt = at % p.nrt;
                    w.part = index % p.parts;
                    w.first = index == 0;
                }
                const bool end = w.stop != 0;
                bar_arrive(bar(C::IFULL + slot));
                if (end) break;
            }
        }
        __syncwarp();
    } else if (warp == 0) {
        // Raw rows: lane l copies box l of a chunk (half l / P, position l % P).
        const int half = lane >> p.logP, j = lane & (p.P - 1);
        const bool copies = half < 2 && p.copies;
        const uint32_t dst = smem_addr(raw) + (uint32_t)lane * (uint32_t)((64 >> p.logP) * p.bw);
        const int xj = (int)((int64_t)j * p.rb);
        const CUtensorMap *map = &p.map[p.gated ? half & 1 : 0];
        uint32_t rc = 0, r = 0, ph = 1;
        Item w;
        for (uint32_t it = 0; take(it, w); ++it) {
            const int64_t first = p.row0 + (int64_t)w.group * p.group_rows +
                                  (p.gated ? (int64_t)w.rt * 64 : (int64_t)w.rt * 128 + 64 * half);
            const int y = (int)((first - j + p.P - 1) >> p.logP);   // first super-row with position j in the tile
            bool ok = true;
            for (int c = w.part * p.part_chunks, end = min(p.nch, c + p.part_chunks); c < end; ++c) {
                if (!(ok = waits(bar(C::REMPTY + r), ph))) break;
                if (lane == 0) {
                    if (p.copies) bar_expect(bar(C::RFULL + r), (uint32_t)(kM * p.bw));
                    else bar_arrive(bar(C::RFULL + r));
                }
                __syncwarp();
                if (copies) copy_box(dst + r * C::RAW, map, ((xj + c * C::CB) & ~15) >> 1, y, bar(C::RFULL + r));
                ++rc;
                if (++r == (uint32_t)p.raws) r = 0, ph ^= 1u;
            }
            if (!ok) break;
        }
        // Every copy issued lands before the CTA can exit.
        if (lane == 0) {
            const uint32_t raws = (uint32_t)p.raws;
            for (uint32_t i = rc > raws ? rc - raws : 0; i < rc; ++i) bar_drain(bar(C::RFULL + i % raws), (i / raws) & 1);
        }
        __syncwarp();
    } else if (warp == 1) {
        // Activations, a stage at a time.
        if (lane == 0) {
            const uint32_t ring = smem_addr(smem);
            uint32_t n = 0, ib = 0, ph = 1;   // stages copied; place in the ring and phase
            uint32_t skipped = 0xffffffffu;
            bool ok = true;
            for (uint32_t it = 0; ok; ++it) {
                const int slot = it % kItems;
                if (!wait(bar(C::IFULL + slot), (it / kItems) & 1)) break;
                const int grans = (items[slot].cnt + GT - 1) / GT, gran = items[slot].gran, end = items[slot].stop;
                const int from = items[slot].part * p.part_chunks * QPC, nsl = min(p.nst - from, p.part_chunks * QPC);
                const bool withhold = p.withhold && items[slot].first;
                bar_arrive(bar(C::IEMPTY + slot));
                if (end) break;
                const uint32_t slice = (uint32_t)grans * kGranBytes;
                const uint8_t *src = p.img + (int64_t)gran * p.nst * kGranBytes + (int64_t)from * slice;
                for (int b = 0; b < nsl; b += KS, ++n) {
                    if (!(ok = wait(bar(C::BDONE + ib), ph))) break;
                    if (withhold && b == 0) {
                        skipped = n;
                    } else {
                        const int slices = KS > 1 ? min(KS, nsl - b) : 1;
                        bar_expect(bar(C::BFULL + ib), slices * slice);
                        for (int i = 0; i < slices; ++i)
                            copy_bulk(ring + (ib * KS + i) * p.slot, src + i * slice, slice, bar(C::BFULL + ib));
                    }
                    src += KS * slice;
                    if (++ib == (uint32_t)p.slots) ib = 0, ph ^= 1u;
                }
            }
            // Every copy issued lands before the CTA can exit.
            const uint32_t slots = (uint32_t)p.slots;
            for (uint32_t i = n > slots ? n - slots : 0; i < n; ++i)
                if (i != skipped) bar_drain(bar(C::BFULL + i % slots), (i / slots) & 1);
        }
        __syncwarp();
    } else if (warp == 2) {
        // Products, the whole role in one elected thread (a warp that waits
        // as one and elects per stage is as fast, but then how often the
        // election runs is the compiler's choice; lane 0 by its number keeps
        // the operands out of uniform registers: 388 against 300 us for 2048
        // tokens through 2 x 11008 x 4096 Q4_0).
        if (elect_one()) {
            const uint64_t bd0 = smem_desc(smem_addr(smem), 1024);
            const uint64_t bd1 = smem_desc(smem_addr(smem), 2048);   // every other 8 rows: the high (or low) terms
            uint32_t sa = 0, pa = 0;           // stage of weights and its phase
            uint32_t ib = 0, pb = 0;           // stage of activations and its phase
            uint32_t seg = 0;                  // sums
            bool any = false, ok = true, ready = false;
            for (uint32_t it = 0; ok; ++it) {
                const int slot = it % kItems;
                if (!wait(bar(C::IFULL + slot), (it / kItems) & 1)) break;
                const int grans = (items[slot].cnt + GT - 1) / GT, end = items[slot].stop;
                const int nsl = min(p.nst - items[slot].part * p.part_chunks * QPC, p.part_chunks * QPC);
                bar_arrive(bar(C::IEMPTY + slot));
                if (end) break;
                const uint32_t id = WT == 2 && XT == 2 ? idesc_n((grans + 1) / 2 * 16) : idesc_n(kGranRows * grans);
                const int flush = LONG ? p.segment : C::FLUSH;
                for (int b = 0; b < nsl;) {
                    const bool fresh = (b & (flush - 1)) == 0;
                    const uint32_t acc = tmem + (seg % NBUF) * C::ACC;
                    if (fresh) {
                        if (!(ok = wait(bar(C::ACCE + seg % NBUF), ((seg / NBUF) & 1) ^ 1))) break;
                    }
                    if (!ready && !(ok = wait(bar(C::BFULL + ib), pb) && wait(bar(C::FULL + sa), pa))) break;
                    const uint32_t a_done = bar(C::ADONE + sa), b_done = bar(C::BDONE + ib);
                    const uint32_t a0 = tmem + C::ACOL + sa * C::ASTAGE, at = (ib * KS * p.slot) >> 4;
                    const int slices = KS > 1 ? min(KS, nsl - b) : 1;
                    // The next stage's barriers are read (about 130 cycles
                    // each) beside this one's products.
                    if (++sa == S) sa = 0, pa ^= 1u;
                    if (++ib == (uint32_t)p.slots) ib = 0, pb ^= 1u;
                    const bool b_next = bar_test(bar(C::BFULL + ib), pb), f_next = bar_test(bar(C::FULL + sa), pa);
                    tc_fence_after();
                    any = true;
#pragma unroll 1
                    for (int i = 0; i < KS; ++i) {
                        if (i > 0 && i >= slices) break;
                        const uint32_t a = a0 + (uint32_t)(i * C::ASLICE);
                        const uint64_t at_i = at + i * (p.slot >> 4);
#pragma unroll
                        for (int k = 0; k < kSliceK / 16; ++k) {
                            const uint32_t add = !fresh || i > 0 || k > 0;
                            if constexpr (WT == 2 && XT == 2) {
                                tc_mma_ts(acc, a + 8 * k, bd1 + at_i + 16 * k, id, add);
                                tc_mma_ts(acc + C::T, a + 8 * k, bd1 + at_i + 64 + 16 * k, id, add);
                                tc_mma_ts(acc + C::T, a + 32 + 8 * k, bd1 + at_i + 16 * k, id, 1u);
                            } else {
                                tc_mma_ts(acc, a + 8 * k, bd0 + at_i + 16 * k, id, add);
                                if constexpr (WT == 2) tc_mma_ts(acc, a + 32 + 8 * k, bd0 + at_i + 16 * k, id, 1u);
                            }
                        }
                    }
                    bar_commit(a_done);
                    bar_commit(b_done);
                    ready = b_next && f_next;
                    b += KS;
                    if (b >= nsl || (b & (flush - 1)) == 0) {
                        bar_commit(bar(C::ACCF + seg % NBUF));
                        ++seg;
                    }
                }
            }
            // Every issued product completes before tensor memory is freed.
            if (any) {
                bar_commit(bar(C::DRAIN));
                bar_drain(bar(C::DRAIN), 0);
            }
        }
        __syncwarp();
    }
    } else if (warp < kEpi0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::RDEC));
        // Decoders: lane's half of the tile (lanes 16 apart hold the same row
        // of both) and row in it.
        const int grp = (warp - kDec0) >> 2, w4 = warp & 3;
        const int half = lane >> 4, i = lane_row(16 * w4 + (lane & 15), p.logP);
        const uint32_t a0 = tmem + C::ACOL + ((uint32_t)(32 * w4) << 16);
        const int64_t copied = p.copies ? p.total_rows & ~(int64_t)(p.P - 1) : 0;   // rows in whole super-rows
        const int stage = grp / C::GPS, s0 = grp % C::GPS * C::KD;   // the group's stage, and its first slice there
        const uint32_t a = a0 + (uint32_t)(stage * C::ASTAGE + s0 * C::ASLICE);
        uint32_t m = 0;                // stages before this chunk
        uint32_t r = 0, ph = 0;        // raw chunk and its phase
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
            for (int c = w.part * p.part_chunks, end = min(p.nch, c + p.part_chunks); ok && c < end; ++c) {
                const int nq = min(QPC, p.nst - c * QPC), ns = (nq + KS - 1) / KS;   // its slices and stages
                if (!(ok = waits(bar(C::RFULL + r), ph))) break;
                uint8_t *src = raw + r * C::RAW + at;
                if (tail) {
                    // A row that the boxes do not reach, copied to where they
                    // would put it (by every group, each for itself).
                    const uint8_t *g = p.W[p.gated ? half : 0] + row * p.rb + (int64_t)c * C::CB;
                    const int n = (int)min((int64_t)C::CB, p.rb - (int64_t)c * C::CB);
#pragma unroll 1
                    for (int k = 0; k < n; ++k) src[k] = __ldg(g + k);
                }
                for (int q = (stage - (int)m) & (S - 1); q < ns; q += S) {
                    uint32_t hi[16], lo[16];
                    bool open = false;   // the stage is known to be free
                    bool any = false;    // a scale far from 1 in the stage
                    if constexpr (FMT == RF_MXFP4) {
                        uint32_t place = 0;
#pragma unroll
                        for (int k = 0; k < 2 * C::KD; ++k)
                            place = max(place, e8m0_place(src[(2 * (KS * q + s0) + k) * block_size(FMT)]));
                        any = e8m0_far(place);
                    }
                    auto opened = [&]() -> bool {
                        if (!open) {
                            if (!waits(bar(C::ADONE + stage), (((m + (uint32_t)q) / S) & 1) ^ 1)) return false;
                            tc_fence_after();
                            open = true;
                        }
                        return true;
                    };
                    auto store = [&](int at_col) -> bool {
                        if (!opened()) return false;
                        tmem_st16(a + at_col, hi);
                        if constexpr (WT == 2) tmem_st16(a + 32 + at_col, lo);
                        return true;
                    };
#pragma unroll 1
                    for (int e = 0; e < C::KD; ++e) {
                        const int sl = q * KS + s0 + e;   // slice of the chunk
                        if ((C::GPS > 1 || e > 0) && sl >= nq) break;
                        if constexpr (FMT == RF_Q4_K) {
                            q4k_block<C::LOW>(src, sl, 0, hi, lo);
                            if (!(ok = store(C::ASLICE * e))) break;
                            q4k_block<C::LOW>(src, sl, 1, hi, lo);
                            store(C::ASLICE * e + 16);
                        } else {
                            constexpr int BS = block_size(FMT);
                            Block<FMT> blk[2];
#pragma unroll
                            for (int t = 0; t < 2; ++t) blk[t].load(src, (2 * sl + t) * BS);
                            block_pairs<FMT, C::LOW>(blk[0], any, hi, lo);
                            if (!(ok = store(C::ASLICE * e))) break;
                            block_pairs<FMT, C::LOW>(blk[1], any, hi, lo);
                            if (2 * (c * QPC + sl) + 1 >= p.nb) {   // behind the last block: the next row's bytes
#pragma unroll
                                for (int k = 0; k < 16; ++k) hi[k] = lo[k] = 0u;
                            }
                            store(C::ASLICE * e + 16);
                        }
                    }
                    if (C::GPS > 1 && ok) ok = opened();   // (a share without slices)
                    if (!ok) break;
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) bar_arrive(bar(C::FULL + stage));
                }
                if (!ok) break;
                if (tail) fence_async_smem();   // the next copy follows these stores
                __syncwarp();
                if (lane == 0) bar_arrive(bar(C::REMPTY + r));
                if (++r == (uint32_t)p.raws) r = 0, ph ^= 1u;
                m += ns;
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REPI));
        // Epilogue: lane's row as the decoders have it.
        const int w4 = warp & 3, half = lane >> 4, i = lane_row(16 * w4 + (lane & 15), p.logP);
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
                if (lane == 0) bar_arrive(bar(C::ACCE + seg % NBUF));
                ++seg;
            };
            const int nsl = min(p.nst - w.part * p.part_chunks * QPC, p.part_chunks * QPC);
            if constexpr (XT == 1) {
                bool ok = true;
#pragma unroll 1
                for (int b0 = 0; b0 < (LONG ? nsl : 1); b0 += LONG ? p.segment : 1) {
                    // Sums so far, this thread's own: of a row that has several segments.
                    [[maybe_unused]] float *held = LONG ? p.held + ((int64_t)blockIdx.x * p.held_rows * kM + 32 * w4 + lane) : nullptr;
                    const bool last = !LONG || b0 + p.segment >= nsl;
                    float next[16];
                    load_inv(inv, next);
                    if (!(ok = waits(bar(C::ACCF + seg % NBUF), (seg / NBUF) & 1))) break;
                    tc_fence_after();
                    const uint32_t acc = tmem + lanes + (seg % NBUF) * C::ACC;
#pragma unroll 1
                    for (int t0 = 0; t0 < w.cnt; t0 += 16) {
                        float z[16], f[16];
                        uint32_t v[16];
                        tmem_ld16(acc + t0, v);
#pragma unroll
                        for (int u = 0; u < 16; ++u) f[u] = next[u];
                        if (t0 + 16 < w.cnt) load_inv(inv + t0 + 16, next);
                        tmem_ld_wait();
#pragma unroll
                        for (int u = 0; u < 16; ++u) z[u] = __uint_as_float(v[u]);
                        if (t0 + 16 >= w.cnt) release();
                        if (LONG && b0 > 0) {
#pragma unroll
                            for (int u = 0; u < 16; ++u) z[u] += held[(t0 + u) * kM];
                        }
                        if (!last) {
#pragma unroll
                            for (int u = 0; u < 16; ++u) held[(t0 + u) * kM] = z[u];
                        } else if (p.parts > 1) {
                            keep(p, z, f, w.part, (int64_t)w.row0 + t0, w.cnt - t0, col, in, half);
                        } else {
                            finish_typed(p, z, f, b, (int64_t)w.row0 + t0, w.cnt - t0, col, in, half);
                        }
                    }
                }
                if (!ok) break;
            } else {
                // 64 tokens' sums in registers, over the item's flushes.
                float sum[C::T];
                bool ok = true;
#pragma unroll
                for (int u = 0; u < C::T; ++u) sum[u] = 0.f;
#pragma unroll 1
                for (int b0 = 0; b0 < nsl; b0 += C::FLUSH) {
                    if (!(ok = waits(bar(C::ACCF + seg % NBUF), (seg / NBUF) & 1))) break;
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
                        if (p.parts > 1) keep(p, z, f, w.part, (int64_t)w.row0 + t0, w.cnt - t0, col, in, half);
                        else finish<RF_F32>(p, z, f, b, (int64_t)w.row0 + t0, w.cnt - t0, col, in, half);
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

// The parts' sums of each row, added in order of the parts, and what follows
// the product.  blockIdx.y: kJoinRows rows of a token tile.
constexpr int kJoinRows = 4;
__global__ void __launch_bounds__(128) join_parts_kernel(const __grid_constant__ Params p, int pieces)
{
    const int at = (int)blockIdx.y / pieces, t0 = (int)blockIdx.y % pieces * kJoinRows;
    if (at >= p.plan->n_tiles) return;
    const ChunkTile tile = p.tiles[at];
    const int col = (int)blockIdx.x * 128 + (int)threadIdx.x, n = min(tile.cnt - t0, kJoinRows);
    if (col >= p.rows || n <= 0) return;
    const int64_t step = (int64_t)p.n_row * p.rows;   // from one projection to the next
    const float b0 = p.bias[0] ? p.bias[0][(int64_t)tile.group * p.rows + col] : 0.f;
    const float b1 = p.bias[1] ? p.bias[1][(int64_t)tile.group * p.rows + col] : 0.f;
    const float *s = p.sums + (int64_t)(tile.row0 + t0) * p.rows + col;
    float z[kJoinRows], u[kJoinRows];
#pragma unroll
    for (int t = 0; t < kJoinRows; ++t) z[t] = u[t] = 0.f;
    const int64_t part = (1 + p.gated) * step;
    for (int i = 0; i < p.parts; i += 4, s += 4 * part) {   // (four parts' loads at a time)
        float v[4][kJoinRows], w[4][kJoinRows];
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int t = 0; t < kJoinRows; ++t) {
                const bool there = i + k < p.parts && t < n;
                v[k][t] = there ? s[k * part + (int64_t)t * p.rows] : 0.f;
                w[k][t] = there && p.gated ? s[k * part + step + (int64_t)t * p.rows] : 0.f;
            }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int t = 0; t < kJoinRows; ++t) z[t] += v[k][t], u[t] += w[k][t];
    }
#pragma unroll
    for (int t = 0; t < kJoinRows; ++t) {
        if (t >= n) break;
        finish_one(p, tile.row0 + t0 + t, col, z[t] + b0, u[t] + b1);
    }
}

template <int FMT, int NT, int XT, int WT, bool LONG>
rf_status launch(Params &p, int grid, cudaStream_t s)
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
        ok[dev & 63] = cudaFuncSetAttribute(chunk_kernel<FMT, NT, XT, WT, LONG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            (int)C::SMEM) == cudaSuccess;
        cudaGetLastError();
    });
    if (!ok[dev & 63]) return RF_ERR_CUDA;
    const int stage = C::KS * (int)p.slot;
    p.raws = std::min(kRaws, (C::SHARED - C::LEAST * stage) / C::RAW);
    p.slots = std::min(kInFlight, (C::SHARED - p.raws * C::RAW) / stage);
    p.raw_at = (uint32_t)(p.slots * stage);
    chunk_kernel<FMT, NT, XT, WT, LONG><<<grid, C::THREADS, C::SMEM, s>>>(p);
    return last_cuda_error();
}

// One fp16 term an activation: rows of several segments, or of one.
template <int FMT, int NT, int WT>
rf_status launch_one(const ChunkShape &sh, Params &p, int grid, cudaStream_t s)
{
    return sh.segments ? launch<FMT, NT, 1, WT, true>(p, grid, s) : launch<FMT, NT, 1, WT, false>(p, grid, s);
}
template <int FMT>
rf_status launch_fmt(const ChunkShape &sh, Params &p, int grid, cudaStream_t s)
{
    constexpr int WT = FMT == RF_MXFP4 ? 1 : 2;
    if (sh.xt == 2) return launch<FMT, 128, 2, WT, false>(p, grid, s);
    if constexpr (WT == 2)
        if (sh.wt == 2) return launch_one<FMT, 128, 2>(sh, p, grid, s);
    return sh.nt > 128 ? launch_one<FMT, 192, 1>(sh, p, grid, s) : launch_one<FMT, 128, 1>(sh, p, grid, s);
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
    const int cb = chunk_bytes(sh.fmt);
    p.bw = box_bytes(sh.fmt, P);
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
    p.limit_cycles = 2 * (long long)kWaitLimitNs;   // (at most 2.07 GHz)
    p.withhold = 0;
    if (const unsigned long long lim = take_wait_fault()) {
        p.limit_cycles = 2 * (long long)lim;
        p.withhold = 1;
    }
    p.slot = (uint32_t)sh.nt * kSliceK * 2;
    p.parts = sh.parts;
    p.part_chunks = sh.part_chunks;
    p.n_row = (int32_t)sh.n_row;
    p.sums = reinterpret_cast<float *>(g.ws + sh.at_sums);
    p.held = reinterpret_cast<float *>(g.ws + sh.at_held);
    p.segment = sh.segment;
    p.held_rows = sh.segments ? sh.nt : 0;
    const int grid = (int)std::min<int64_t>(num_sms(), sh.cap_tiles * p.nrt * p.parts);
    rf_status st;
    if (sh.few) st = launch_chunk_few(sh, p, s);
    else switch (sh.fmt) {
    case RF_Q4_0: st = launch_fmt<RF_Q4_0>(sh, p, grid, s); break;
    case RF_Q8_0: st = launch_fmt<RF_Q8_0>(sh, p, grid, s); break;
    case RF_Q4_K: st = launch_fmt<RF_Q4_K>(sh, p, grid, s); break;
    default: st = launch_fmt<RF_MXFP4>(sh, p, grid, s); break;
    }
    if (st != RF_OK || p.parts == 1) return st;
    const int pieces = (sh.tile_tokens() + kJoinRows - 1) / kJoinRows;
    join_parts_kernel<<<dim3((unsigned)((p.rows + 127) / 128), (unsigned)(sh.cap_tiles * pieces)), 128, 0, s>>>(p, pieces);
    return last_cuda_error();
}

}  // namespace rf
