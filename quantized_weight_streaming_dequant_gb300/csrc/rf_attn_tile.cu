// rf_attn_tile.cu -- attention of long chunks on the fifth-generation tensor
// cores (same mathematics as rf_attn.cu).
//
// Three launches:
//   plan   one CTA lists the query tiles (heaviest first: later positions see
//          more) and lays the sequences' 128-position tiles out end to end.
//   stage  rewrites what the products read into the operand layouts, once per
//          call instead of once per query tile: codes of K and V as fp16
//          tiles (V transposed), queries as one or two fp16 terms per element
//          scaled by a power of two per row, and the blocks' units.  It moves
//          3 bytes per code (and 2 to 4 per query element), which 128-row
//          tiles read back many times.
//   tiles  persistent CTAs draw items: two tiles of 128 query rows (tokens x
//          heads of one K/V head; one tile above head_dim 128, whose S and O
//          fill tensor memory) and part of their positions.  A CTA walks the
//          visible ones, 128 at a time:
//              S = Q K^T (tcgen05.mma from shared memory, fp32 in tensor
//              memory) -> weights by one thread per row (no shuffles) -> P in
//              fp16 over S's own columns -> O += P V (P from tensor memory).
//          One thread issues the products of the two tiles alternately, so
//          that one tile's exponentials run under the other's products; O
//          stays in tensor memory and is rescaled only when a row's maximum
//          has grown by more than w_lazy (the weights' exponent range allows
//          it; the factor cancels).
// Bound: the tensor pipe for long rows: 4 * 128 * 128 * head_dim flops per
// step and tile (twice that for fp32, whose queries and weights are two fp16
// terms), against 16,384 exponentials.
// Measured (plan / stage / tiles / join, us): 8192-token bf16 prompt, 32 / 8
// heads of 128: 5 / 36 / 386 / - (1.42 PFLOP/s in the tiles, 0.73 of the
// measured bf16 rate); fp32, 511 tokens against 32,768 positions: 5 / 48 /
// 361 / 21 (1.51 PFLOP/s with both terms); fp16, ragged prompts of 8193 tokens
// in all under a window of 128, 64 / 8 heads of 64: 5 / 31 / 85 / -.  The same
// tiles without the softmax's work take 322, 308 and 46 us, so the products
// bound the long ones: a step's operands (Q and K for S, V for O, and the
// copies) are 256 KB of shared-memory traffic for 2,048 tensor cycles, which
// is all that 128 bytes a cycle allow (a pair of CTAs that share B would halve
// half of it).  Tried and not kept: two threads per row (16 softmax warps,
// 462 us for the prompt's call against 454), handing over the first half of P
// early (465 against 466), products issued by one lane from per-thread
// registers (576 against 454; fp32 chunk 1,343 against 620: operands in
// uniform registers let one warp keep the pipe busy), maxima applied at once
// beyond 2^1.5 instead of 2^7 for 16-bit types (486 against 466).
//
// Every wait is bounded; after a failure every role stops, copies and
// products already issued are waited for, and tensor memory is freed.
#include <algorithm>
#include <cfloat>
#include <climits>
#include <mutex>

#include "rf_attn.h"
#include "rf_tcgen05.cuh"

namespace rf {
namespace {

__device__ int g_tile_status = 0;    // bounded waits that gave up
// Positions or pages that do not exist: a word of its own, since waits end
// early while theirs is set.
__device__ int g_tile_invalid = 0;

constexpr int kTile = 128;          // query rows, and positions, per tile
constexpr int kSoftWarps = 8;       // four per tile: a thread per row
constexpr int kMainThreads = 32 * (kSoftWarps + 4);   // ... and a warpgroup of which two warps issue products and copies
// Registers: 168 a thread at launch; the last warpgroup gives up what the
// softmax warpgroups take (2 * 232 + 40 = 3 * 168), so that a thread holds
// its row's 128 scores.
constexpr int kRegsSoftmax = 232, kRegsOther = 40;
constexpr int kFlush = 16;          // position tiles that fp32 sums stay in tensor memory
constexpr int kPadParts = 8;        // CTAs that zero the rows of no sequence

// What the plan kernel leaves for the others.
struct TilePlan {
    int32_t n_q, n_kv;              // query tiles, position tiles
    int32_t next;                   // work items drawn
    int32_t pad;
};
// Two query tiles of a sequence: tokens [tok, end) at most, the first at
// position pos; position tiles [t_lo, t_hi[x]) of the kvn staged at kv0 are
// seen by tile x, staged tile 0 starting at position 128 * kvf.
struct __align__(16) QTile {
    int32_t seq, tok, end, kv0, kvf, t_lo, t_hi[2];
    int64_t pos, pad;
};

// head_dim rounded up (DP) is walked in SUB pieces of DW elements, each an
// operand image of its own: 64, 128 or two times 128.
template <int DP> struct Dims {
    static constexpr int SUB = DP > 128 ? 2 : 1, DW = DP / SUB;
    static constexpr int NT = DP > 128 ? 1 : 2;   // query tiles per item (tensor memory holds S and O of each)
    static constexpr int IMG = kTile * DW * 2;    // bytes of an image
};

struct TileParams {
    AttnParams a;
    int hpt, head_tiles, tqt;       // heads per tile, tiles per K/V head, tokens per 128-row tile
    int nt;                         // query tiles per item: 2, or 1 for head_dim above 128
    int cap_q, cap_kv;              // capacities of the lists below
    int cap_seq;                    // position tiles of one sequence, at most: its share of cap_kv
    TilePlan *plan;
    QTile *q_tiles;                 // [cap_q]
    int32_t *kv_base;               // [n_seq]: first position tile of a sequence
    int32_t *kv_first;              // [n_seq]: its position / 128 (window)
    uint8_t *q_img;                 // [cap_q][kv head][head tile][tile][NS][128 x DP] fp16
    float *q_unit;                  // [cap_q][kv head][head tile][2][128]
    uint8_t *k_img, *v_img;         // [kv head][cap_kv][128 x DP] fp16
    float *units;                   // [kv head][cap_kv][12]: 2^ek, ev, 2^-ev of four blocks
    float4 *sums;                   // fp32: [CTA][2][DP / 4][128] sums taken out of tensor memory
    int split_tiles;                // position tiles per part
    float qk_abs;                   // |scale| * log2(e); its sign is in the queries
    bool negate;
    unsigned long long limit;
};

// ---------------------------------------------------------------------- plan
// Exclusive prefix sum over the CTA's 1024 threads.
__device__ __forceinline__ int64_t scan1024(int64_t v, int64_t *part, int64_t *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) part[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int64_t y = part[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t z = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) y += z;
        }
        part[lane] = y;
    }
    __syncthreads();
    const int64_t base = warp ? part[warp - 1] : 0;
    *total = part[31];
    __syncthreads();
    return base + x - v;
}

__global__ void __launch_bounds__(1024) tile_plan_kernel(const __grid_constant__ TileParams p)
{
    __shared__ int64_t part[32];
    __shared__ int64_t s_at[1024], s_past[1024];    // of each sequence of a round: first query tile, ...
    __shared__ int s_t0[1024], s_nq[1024], s_kv0[1024], s_kvn[1024], s_kvf[1024];
    pdl_launch_dependents();
    pdl_wait();
    const rf_kv_batch &b = p.a.b;
    const int ctt = p.nt * p.tqt, tid = (int)threadIdx.x;
    int64_t kv_at = 0, q_at = 0;
    for (int s0 = 0; s0 < b.n_seq; s0 += 1024) {
        const int s = s0 + tid;
        int64_t nt = 0, first = 0, past = 0;
        int nq = 0, t0 = 0;
        if (s < b.n_seq) {
            t0 = max(b.q_start[s], 0);
            nq = max(0, min(b.q_start[s + 1], b.n_tok) - t0);
            past = (int64_t)b.past[s] + (t0 - b.q_start[s]);
            const int64_t last = past + nq - 1;
            if (nq > 0 && last >= 0) {
                const int64_t lo = p.a.window > 0 ? max((int64_t)0, past - p.a.window + 1) : 0;
                first = lo / kTile;
                // A sequence that is longer than max_len (or its table) keeps to
                // its share: the staged tiles of the others are not its own.
                const int64_t tiles = last / kTile + 1;
                if (tiles > p.cap_seq) record_status(&g_tile_invalid, RF_ERR_INVALID_ARG);
                nt = max((int64_t)0, min(tiles, (int64_t)p.cap_seq) - first);
            }
            if (past < 0 && nq > 0) record_status(&g_tile_invalid, RF_ERR_INVALID_ARG);
        }
        int64_t total_kv, total_q;
        const int64_t kv0 = kv_at + scan1024(nt, part, &total_kv);
        const int64_t at = q_at + scan1024((nq + ctt - 1) / ctt, part, &total_q);
        // past the capacity (only where q_start decreases): not staged
        const int64_t kvn = max((int64_t)0, min(nt, (int64_t)p.cap_kv - kv0));
        if (kvn < nt) record_status(&g_tile_invalid, RF_ERR_INVALID_ARG);
        if (s < b.n_seq) {
            p.kv_base[s] = (int)min(kv0, (int64_t)p.cap_kv);
            p.kv_first[s] = (int)first;
        }
        s_at[tid] = at, s_past[tid] = past, s_t0[tid] = t0, s_nq[tid] = nq;
        s_kv0[tid] = (int)min(kv0, (int64_t)p.cap_kv), s_kvn[tid] = (int)kvn, s_kvf[tid] = (int)first;
        __syncthreads();
        // The round's query tiles; later positions first: they see more.
        for (int64_t i = q_at + tid; i < min(q_at + total_q, (int64_t)p.cap_q); i += 1024) {
            int lo = 0, hi = 1024;                   // the last sequence that starts at i or before
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_at[mid] <= i) lo = mid;
                else hi = mid;
            }
            const int tiles = (s_nq[lo] + ctt - 1) / ctt, off = (tiles - 1 - (int)(i - s_at[lo])) * ctt;
            QTile q;
            q.seq = s0 + lo;
            q.tok = s_t0[lo] + off;
            q.end = s_t0[lo] + s_nq[lo];
            q.kv0 = s_kv0[lo];
            q.kvf = s_kvf[lo];
            q.pos = s_past[lo] + off;
            q.pad = 0;
            q.t_lo = p.a.window > 0 ? max(0, (int)(max((int64_t)0, q.pos - p.a.window + 1) / kTile) - q.kvf) : 0;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int toks = x < p.nt ? min(p.tqt, q.end - (q.tok + x * p.tqt)) : 0;
                const int64_t last = q.pos + x * p.tqt + toks - 1;
                q.t_hi[x] = toks > 0 && last >= 0 ? (int)min((int64_t)s_kvn[lo], last / kTile + 1 - q.kvf) : 0;
            }
            p.q_tiles[i] = q;
        }
        __syncthreads();
        kv_at += total_kv;
        q_at += total_q;
    }
    if (tid == 0) *p.plan = TilePlan{(int)min(q_at, (int64_t)p.cap_q), (int)min(kv_at, (int64_t)p.cap_kv), 0, 0};
}

// --------------------------------------------------------------------- stage
// One position tile of one K/V head by 256 threads.
template <int DP>
__device__ __forceinline__ void stage_kv(const TileParams &p, int tile, int head)
{
    __shared__ int64_t s_blk[4];   // cache block of each 32 positions, or -1
    const rf_kv_cache &c = p.a.c;
    const int D = c.head_dim, tid = threadIdx.x;
    // the sequence: the last one whose first tile is not after this one
    if (tid < 4) {
        int lo = 0, hi = p.a.b.n_seq;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.kv_base[mid] <= tile) lo = mid;
            else hi = mid;
        }
        const int64_t pos = (int64_t)(p.kv_first[lo] + tile - p.kv_base[lo]) * kTile + 32 * tid;
        const int end = min(p.a.b.q_start[lo + 1], p.a.b.n_tok);
        const int64_t len = (int64_t)p.a.b.past[lo] + end - p.a.b.q_start[lo];
        int64_t blk = -1;
        if (pos < len) {
            const int page = page_of(p.a.b, c, lo, pos);
            const int per = c.page_size / kKvBlock;
            if (page >= 0) blk = ((int64_t)page * c.n_kv_heads + head) * per + (pos / kKvBlock) % per;
            else record_status(&g_tile_invalid, RF_ERR_INVALID_ARG);
        }
        s_blk[tid] = blk;
        // a block that does not exist has unit 0 and exponent -inf: weight 0
        const uint32_t ek = blk >= 0 ? c.k_scale[blk] : 0u, ev = blk >= 0 ? c.v_scale[blk] : 0u;
        float *u = p.units + ((int64_t)head * p.cap_kv + tile) * 12;
        const float nan = __uint_as_float(0x7fc00000u);
        u[tid] = blk >= 0 ? scale_value(ek) : 0.f;
        u[4 + tid] = blk < 0 ? -INFINITY : ev == 255u ? nan : (float)((int)ev - 127);
        u[8 + tid] = blk < 0 ? 0.f : ev == 255u ? nan : scale_value(254u - ev);
    }
    __syncthreads();
    constexpr int DW = Dims<DP>::DW;
    const int64_t img = ((int64_t)head * p.cap_kv + tile) * (kTile * DP * 2);
    // K: 16-byte unit (row n, elements 8k..) of a piece at (n/8) * 16 DW + k * 128 + (n%8) * 16.
    uint8_t *ki = p.k_img + img;
    // A thread turns 16 elements (the load-store pipe, not memory, bounds this
    // kernel: wide reads, and stores that fill whole lines).
    for (int w = tid; w < kTile * DP / 16; w += 256) {
        const int piece = w / (kTile * DW / 16), v16 = w % (kTile * DW / 16);
        const int n = (v16 >> 3) / (DW / 16) * 8 + (v16 & 7), k = (v16 >> 3) % (DW / 16);   // elements 16 k.. of the piece
        uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
        const int64_t blk = s_blk[n >> 5];
        if (blk >= 0 && piece * DW + 16 * k < D) {
            uint4 v = *reinterpret_cast<const uint4 *>(c.k + (blk * kKvBlock + (n & 31)) * D + piece * DW + 16 * k);
            v.x ^= 0x80808080u, v.y ^= 0x80808080u, v.z ^= 0x80808080u, v.w ^= 0x80808080u;
            lo = make_uint4(codes_lo(v.x), codes_hi(v.x), codes_lo(v.y), codes_hi(v.y));
            hi = make_uint4(codes_lo(v.z), codes_hi(v.z), codes_lo(v.w), codes_hi(v.w));
        }
        uint8_t *dst = ki + piece * Dims<DP>::IMG + (n / 8) * (16 * DW) + k * 256 + (n % 8) * 16;
        *reinterpret_cast<uint4 *>(dst) = lo;
        *reinterpret_cast<uint4 *>(dst + 128) = hi;
    }
    // V transposed: unit (row d, positions 8t..) at (d/8) * 2048 + t * 128 + (d%8) * 16;
    // a thread turns 8 positions x 4 elements.
    uint8_t *vi = p.v_img + img;
    for (int w = tid; w < kTile * DP / 32; w += 256) {
        const int d = 4 * (w % (DP / 4)), t = w / (DP / 4);
        uint32_t v[8];
        const int64_t blk = s_blk[t >> 2];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = blk >= 0 && d < D
                       ? *reinterpret_cast<const uint32_t *>(c.v + (blk * kKvBlock + (8 * t + i) % 32) * D + d) ^ 0x80808080u
                       : 0x80808080u;
        uint32_t o[2][8];                            // two elements (16 bytes each) to a sector
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const uint32_t a = prmt(v[i], v[i + 1], 0x5140u), b = prmt(v[i], v[i + 1], 0x7362u);
            const uint32_t x[4] = {codes_lo(a), codes_hi(a), codes_lo(b), codes_hi(b)};
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e >> 1][4 * (e & 1) + i / 2] = x[e];
        }
        uint8_t *dst = vi + (d / 8) * 2048 + t * 128 + (d % 8) * 16;
        store_sector(dst, o[0]);
        store_sector(dst + 32, o[1]);
    }
}

// Two 128-row query tiles by 256 threads: a quarter- or half-warp per row
// (DP / 8 lanes of eight elements).
template <typename T, int DP>
__device__ __forceinline__ void stage_q(const TileParams &p, int qt, int head, int ht)
{
    constexpr int NS = sizeof(T) == 4 ? 2 : 1, LPR = DP / 8, RPW = 32 / LPR, NT = Dims<DP>::NT, DW = Dims<DP>::DW;
    const AttnParams &a = p.a;
    const QTile q = p.q_tiles[qt];
    const int end = q.end, D = a.c.head_dim;
    const int h0 = head * a.group + ht * p.hpt, nh = min(p.hpt, a.group - ht * p.hpt);
    const int64_t at = ((int64_t)qt * a.c.n_kv_heads + head) * p.head_tiles + ht;
    uint8_t *img = p.q_img + at * (NT * NS * kTile * DP * 2);
    float *unit = p.q_unit + at * (2 * kTile);
    const int lane = threadIdx.x & 31, k = lane % LPR;
    for (int r = (int)(threadIdx.x >> 5) * RPW + lane / LPR; r < NT * kTile; r += 8 * RPW) {
        const int x = r / kTile, n = r % kTile, ti = n / p.hpt, hi = n % p.hpt;
        const int tok = q.tok + x * p.tqt + ti;
        const bool ok = ti < p.tqt && hi < nh && tok < end;
        float f[8] = {};
        if (ok && 8 * k < D) {
            const T *src = static_cast<const T *>(a.q) + (int64_t)tok * a.q_lt + (int64_t)(h0 + hi) * a.q_lh + 8 * k;
            load8<T>(src, a.q_vec8, a.q_vec, f);
        }
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[i]));
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        float factor;
        const float up = row_power(amax, p.qk_abs, &factor) * (p.negate ? -1.f : 1.f);
        if (k == 0) unit[r] = factor;
        uint4 hi4, lo4;
        uint32_t *ph = reinterpret_cast<uint32_t *>(&hi4), *pl = reinterpret_cast<uint32_t *>(&lo4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float u = f[2 * i] * up, v = f[2 * i + 1] * up;
            ph[i] = pack_h2(u, v);
            const float2 h = unpack_h2(ph[i]);
            pl[i] = pack_h2(u - h.x, v - h.y);
        }
        uint8_t *dst = img + x * (NS * kTile * DP * 2) + k / (DW / 8) * Dims<DP>::IMG + (n / 8) * (16 * DW) + k % (DW / 8) * 128 + (n % 8) * 16;
        *reinterpret_cast<uint4 *>(dst) = hi4;
        if constexpr (NS == 2) *reinterpret_cast<uint4 *>(dst + kTile * DP * 2) = lo4;
    }
}

// Rows of tokens before the first sequence and past the last (a padded
// batch) read as zeros.
template <typename T>
__device__ __forceinline__ void zero_padding(const AttnParams &p, int part)
{
    const int head = max(0, min(p.b.q_start[0], p.b.n_tok)), tail = max(head, min(p.b.q_start[p.b.n_seq], p.b.n_tok));
    const int per = p.n_heads * (p.c.head_dim / 4), n_pad = head + p.b.n_tok - tail;
    const float zero[4] = {};
    for (int64_t w = part * 256 + (int)threadIdx.x; w < (int64_t)n_pad * per; w += kPadParts * 256) {
        const int j = (int)(w / per), h = (int)(w % per) / (p.c.head_dim / 4), d = 4 * ((int)(w % per) % (p.c.head_dim / 4));
        const int64_t t = j < head ? j : tail + (j - head);
        store4<T>(static_cast<T *>(p.out) + t * p.o_lt + (int64_t)h * p.o_lh + d, p.o_vec, zero);
    }
}

// grid: position tiles x K/V heads, query tiles x K/V heads x head tiles,
// then kPadParts CTAs for the rows of no sequence.
template <typename T, int DP>
__global__ void __launch_bounds__(256) tile_stage_kernel(const __grid_constant__ TileParams p)
{
    pdl_launch_dependents();
    pdl_wait();
    int u = (int)blockIdx.x;
    const int heads = p.a.c.n_kv_heads;
    if (u < p.cap_kv * heads) {
        const int tile = u / heads;
        if (tile < p.plan->n_kv) stage_kv<DP>(p, tile, u % heads);
        return;
    }
    u -= p.cap_kv * heads;
    const int ht = u % p.head_tiles;
    u /= p.head_tiles;
    const int qt = u / heads;
    if (qt >= p.cap_q) {
        zero_padding<T>(p.a, (int)(gridDim.x - 1 - blockIdx.x));
        return;
    }
    if (qt < p.plan->n_q) stage_q<T, DP>(p, qt, u % heads, ht);
}

// --------------------------------------------------------------------- tiles
// Slots of the ring, each an image of a piece of K or V; the queries take as
// many bytes as 2 NS of them.
template <int DP, int NS> __host__ __device__ constexpr int ring_slots() { return DP >= 128 ? 7 - 2 * NS : 14 - 4 * NS; }
template <int DP, int NS> __host__ __device__ constexpr size_t tile_smem()
{
    return (size_t)Dims<DP>::IMG * (2 * NS + ring_slots<DP, NS>());
}

__host__ __device__ constexpr uint32_t tile_idesc(int n)
{
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);
}

// Two fp32 values per instruction.
__device__ __forceinline__ uint64_t f2(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void f2_split(uint64_t v, float &a, float &b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// sums = sums * pend (or 0 at first) + O, or with `back` the result into O.
template <int DP>
__device__ __forceinline__ void flush(uint32_t to, float4 *sums, float pend, bool more, bool back = false)
{
#pragma unroll 1
    for (int d = 0; d < DP; d += 16) {
        uint32_t o[16];
        float4 v[4] = {};
        tmem_ld16(to + d, o);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (more) v[k] = sums[(d / 4 + k) * kTile];
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[k].x = fmaf(v[k].x, pend, __uint_as_float(o[4 * k]));
            v[k].y = fmaf(v[k].y, pend, __uint_as_float(o[4 * k + 1]));
            v[k].z = fmaf(v[k].z, pend, __uint_as_float(o[4 * k + 2]));
            v[k].w = fmaf(v[k].w, pend, __uint_as_float(o[4 * k + 3]));
            if (!back) sums[(d / 4 + k) * kTile] = v[k];
            o[4 * k] = __float_as_uint(v[k].x), o[4 * k + 1] = __float_as_uint(v[k].y);
            o[4 * k + 2] = __float_as_uint(v[k].z), o[4 * k + 3] = __float_as_uint(v[k].w);
        }
        if (back) tmem_st16(to + d, o);
    }
    if (back) tmem_st_wait();
}

// One work item: two query tiles of one head tile against one part of their
// positions.
struct Item {
    int64_t q_at;                   // index of the query images
    int64_t pos;                    // position of tile 0's first token
    int64_t base;                   // first position of the first tile walked
    int32_t n[2];                   // position tiles walked by each query tile
    int32_t kv;                     // index of the first staged one
    int32_t tok, end, head, ht, part;
    int32_t index;                  // of the item
    int32_t stop;
};

// A persistent CTA: the copy warp draws items (heaviest first) and runs ahead
// into the next one, whose first products start under the last one's output.
template <typename T, int DP>
__global__ void __launch_bounds__(kMainThreads, 1) attn_tile_kernel(const __grid_constant__ TileParams p)
{
    constexpr int NS = sizeof(T) == 4 ? 2 : 1;
    constexpr int R = ring_slots<DP, NS>();
    constexpr int SLOT = Dims<DP>::IMG, SUB = Dims<DP>::SUB, DW = Dims<DP>::DW, NT = Dims<DP>::NT;
    static_assert(NT * SUB == 2, "the queries of an item take 2 NS slots");
    constexpr int kItems = 4;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t *q_s = smem;                          // [NT][NS][SUB][SLOT]
    uint8_t *ring = smem + 2 * NS * SLOT;         // [R][SLOT]: the pieces of K0, V0, K1, V1, ...
    __shared__ uint64_t full[R], empty[R], qfull[1], qempty[1], sfull[2], pready[2], pvdone[2], drained[1];
    __shared__ uint64_t ifull[kItems], iempty[kItems];
    __shared__ Item items[kItems];
    __shared__ uint32_t s_tmem;
    __shared__ int s_stop;
    volatile int *stop = &s_stop;

    const AttnParams &a = p.a;
    // A value taken from one lane is known to be the same in all, so that the
    // products' operands live in uniform registers.
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < R; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        mbar_init(qfull, 1);
        mbar_init(qempty, 1);
        for (int x = 0; x < 2; ++x) {
            mbar_init(&sfull[x], 1);
            mbar_init(&pready[x], 4);
            mbar_init(&pvdone[x], 1);
        }
        mbar_init(drained, 1);
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&ifull[i], 1);
            mbar_init(&iempty[i], kSoftWarps + 1);
        }
        s_stop = 0;
        fence_barrier_init();
    }
    if (warp == kSoftWarps) {
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
        if (mbar_wait_bounded(bar, parity, &g_tile_status, p.limit)) return true;
        *stop = 1;
        return false;
    };
    pdl_launch_dependents();
    pdl_wait();

    // (Registers are traded in each branch for good: the roles do not join
    // again before the end.)
    if (warp >= kSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == kSoftWarps + 1) {
        // Items and copies: both query tiles, then K and V of each position
        // tile.
        if (lane == 0) {
            const int total = p.plan->n_q * a.c.n_kv_heads * p.head_tiles * a.splits;
            uint32_t iq = 0, ikv = 0;              // items with copies, ring slots used
            bool ok = true;
            for (uint32_t it = 0; ok; ++it) {
                const int slot = it % kItems;
                if (!wait(&iempty[slot], ((it / kItems) & 1) ^ 1)) break;
                Item &w = items[slot];
                const int index = atomicAdd(&p.plan->next, 1);
                w.stop = index >= total;
                if (w.stop) {
                    mbar_arrive(&ifull[slot]);
                    break;
                }
                int u = index;
                w.index = index;
                w.part = u % a.splits;
                u /= a.splits;
                w.ht = u % p.head_tiles;
                u /= p.head_tiles;
                w.head = u % a.c.n_kv_heads;
                const int qt = u / a.c.n_kv_heads;
                const QTile q = p.q_tiles[qt];
                w.q_at = ((int64_t)qt * a.c.n_kv_heads + w.head) * p.head_tiles + w.ht;
                w.pos = q.pos, w.tok = q.tok, w.end = q.end;
                const int from = q.t_lo + w.part * p.split_tiles;
                int n[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) w.n[x] = n[x] = max(0, min(q.t_hi[x], from + p.split_tiles) - from);
                w.kv = q.kv0 + from;
                w.base = (int64_t)(q.kvf + from) * kTile;
                const int64_t q_at = w.q_at, img = ((int64_t)w.head * p.cap_kv + w.kv) * (SUB * SLOT);
                mbar_arrive(&ifull[slot]);
                const int nmax = max(n[0], n[1]);
                if (nmax == 0) continue;
                if (!wait(qempty, (iq & 1) ^ 1)) break;
                ++iq;
                mbar_arrive_expect_tx(qfull, 2 * NS * SLOT);
                const uint8_t *src = p.q_img + q_at * (2 * NS * SLOT);
#pragma unroll
                for (int i = 0; i < 2 * NS; ++i) bulk_g2s(q_s + i * SLOT, src + i * SLOT, SLOT, qfull);
                for (int i = 0; i < 2 * SUB * nmax; ++i) {
                    const int s = ikv % R, kv = i % (2 * SUB), sub = kv % SUB;
                    if (!(ok = wait(&empty[s], ((ikv / R) & 1) ^ 1))) break;
                    mbar_arrive_expect_tx(&full[s], SLOT);
                    bulk_g2s(ring + s * SLOT, (kv >= SUB ? p.v_img : p.k_img) + img + ((int64_t)(i / (2 * SUB)) * SUB + sub) * SLOT, SLOT, &full[s]);
                    ++ikv;
                }
            }
            // Every copy issued lands before the CTA can exit.
            if (iq > 0) mbar_drain(qfull, (iq - 1) & 1);
            for (uint32_t i = ikv > R ? ikv - R : 0; i < ikv; ++i) mbar_drain(&full[i % R], (i / R) & 1);
        }
        __syncwarp();
    } else if (warp == kSoftWarps) {
        // Products.  Tile x: S at columns 128 x, P over it (the weights of
        // block b in S's columns 32 b: 16 columns of fp16 pairs a term), O at
        // 256 + DP x.  All in one thread's order, which is what lets a tile's
        // next scores follow its values over the same columns.  The warp runs
        // as one; `leader` is the thread that issues.
        const uint64_t qd = smem_desc(smem_addr(q_s), 16 * DW), kd = smem_desc(smem_addr(ring), 16 * DW);
        const uint64_t vd = smem_desc(smem_addr(ring), 2048);
        const bool leader = elect_one();
        bool ok = true, any = false;
        uint32_t iq = 0, steps[2] = {0, 0};
        int rs = 0;                                // ring slot of the next piece, and its phase
        uint32_t rph = 0;
        auto waits = [&](uint64_t *bar, uint32_t parity) -> bool { return __all_sync(0xffffffffu, wait(bar, parity)); };
        auto commit = [&](uint64_t *bar) {
            if (leader) tc_commit(bar);
        };
        auto next = [&] {
            if (++rs == R) rs = 0, rph ^= 1u;
        };
        // Scores of tile x from piece `sub` of K in `slot`; the last piece
        // hands S over.
        auto scores = [&](int x, int slot, int sub) {
            tc_fence_after();
            const uint64_t q0 = qd + (uint64_t)(((x * NS * SUB + sub) * SLOT) >> 4), k0 = kd + (uint64_t)((slot * SLOT) >> 4);
            if (leader) {
#pragma unroll 1
                for (int t = NS - 1; t >= 0; --t)
#pragma unroll
                    for (int k = 0; k < DW / 16; ++k)
                        tc_mma(tmem + 128 * x, q0 + ((t * SUB * SLOT + k * 256) >> 4), k0 + 16 * k, tile_idesc(kTile),
                               !(sub == 0 && t == NS - 1 && k == 0));
                if (sub == SUB - 1) tc_commit(&sfull[x]);
            }
        };
        auto values = [&](int x, int slot, int sub, bool add) {
            tc_fence_after();
            const uint64_t v0 = vd + (uint64_t)((slot * SLOT) >> 4);
            if (leader) {
#pragma unroll 1
                for (int t = NS - 1; t >= 0; --t)
#pragma unroll
                    for (int k = 0; k < kTile / 16; ++k)
                        tc_mma_ts(tmem + 256 + DP * x + DW * sub, tmem + 128 * x + 32 * (k >> 1) + 16 * t + 8 * (k & 1), v0 + 16 * k,
                                  tile_idesc(DW), add || !(t == NS - 1 && k == 0));
                if (sub == SUB - 1) tc_commit(&pvdone[x]);
            }
        };
        for (uint32_t it = 0; ok; ++it) {
            const int slot = it % kItems;
            if (!waits(&ifull[slot], (it / kItems) & 1)) break;
            const int n0 = __shfl_sync(0xffffffffu, items[slot].n[0], 0), n1 = __shfl_sync(0xffffffffu, items[slot].n[1], 0);
            const int end = __shfl_sync(0xffffffffu, items[slot].stop, 0);
            __syncwarp();
            if (leader) mbar_arrive(&iempty[slot]);
            if (end) break;
            const int nmax = max(n0, n1);
            if (nmax == 0) continue;
            if (!waits(qfull, iq & 1)) break;
            ++iq;
#pragma unroll
            for (int sub = 0; sub < SUB; ++sub) {
                if (!(ok = ok && waits(&full[rs], rph))) break;
                any = true;
                if (n0 > 0) scores(0, rs, sub);
                if (n1 > 0) scores(1, rs, sub);
                commit(&empty[rs]);
                next();
            }
            if (!ok) break;
            if (nmax == 1) commit(qempty);
            for (int j = 0; ok && j < nmax; ++j) {
                const bool more = j + 1 < nmax, add = NS == 2 ? j % kFlush != 0 : j > 0;
                if constexpr (SUB == 1) {
                    // Two tiles in turn: each one's values, then its next scores.
                    const int vs = rs;
                    if (!(ok = waits(&full[vs], rph))) break;
                    next();
                    const int ns = rs;
                    if (more && !(ok = waits(&full[ns], rph))) break;
                    if (j < n0) {
                        if (!(ok = waits(&pready[0], steps[0] & 1))) break;
                        ++steps[0];
                        values(0, vs, 0, add);
                        if (j + 1 < n0) scores(0, ns, 0);
                    }
                    if (j < n1) {
                        if (!(ok = waits(&pready[1], steps[1] & 1))) break;
                        ++steps[1];
                        values(1, vs, 0, add);
                    }
                    commit(&empty[vs]);
                    if (j + 1 < n1) scores(1, ns, 0);
                    if (more) {
                        commit(&empty[ns]);
                        next();
                    }
                } else {
                    if (!(ok = waits(&pready[0], steps[0] & 1))) break;
                    ++steps[0];
#pragma unroll
                    for (int i = 0; i < 2 * SUB; ++i) {
                        if (i >= SUB && !more) break;
                        if (!(ok = waits(&full[rs], rph))) break;
                        if (i < SUB) values(0, rs, i, add);
                        else scores(0, rs, i - SUB);
                        commit(&empty[rs]);
                        next();
                    }
                }
                if (ok && j + 2 == nmax) commit(qempty);
            }
        }
        // Every issued product completes before tensor memory is freed.
        if (any) {
            commit(drained);
            mbar_drain(drained, 0);
        }
        __syncwarp();
    }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        // Softmax: thread i of group x owns row i of tile x (tensor-memory
        // lane i).
        const int x = warp >> 2, i = (warp & 3) * 32 + lane;
        const int ti = i / p.hpt, hi = i % p.hpt;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + 128 * x, to = tmem + lanes + 256 + DP * x;
        uint32_t step = 0;                         // steps of this tile
        bool ok = true;
        for (uint32_t it = 0; ok; ++it) {
            const int slot = it % kItems;
            ok = __all_sync(0xffffffffu, wait(&ifull[slot], (it / kItems) & 1));
            if (!ok) break;
            const Item &w = items[slot];           // given back after the output
            if (w.stop) break;
            const int nx = w.n[x];
            const bool row_ok = x < NT && ti < p.tqt && hi < min(p.hpt, a.group - w.ht * p.hpt) && w.tok + x * p.tqt + ti < w.end;
            // The visible positions [first, top] of the row, counted from the
            // first tile's first.
            const int top = row_ok ? (int)(w.pos - w.base) + x * p.tqt + ti : INT_MIN / 2;
            const int first = a.window > 0 ? (int)max((int64_t)top - a.window + 1, (int64_t)INT_MIN / 2) : INT_MIN / 2;
            const float bq = p.q_unit[w.q_at * (2 * kTile) + x * kTile + i];
            float m = -INFINITY, l = 0.f;
            // [position tile][2^ek, ev, 2^-ev][block]
            const float4 *units = reinterpret_cast<const float4 *>(p.units + ((int64_t)w.head * p.cap_kv + w.kv) * 12);
            // fp32: the tensor core truncates its sums, which drifts by about
            // 1e-8 per step; so O is added to sums in memory every kFlush
            // tiles.  pend: growth of m since the last time.
            auto sums = [&] { return p.sums + ((int64_t)w.index * 2 + x) * (DP / 4) * kTile + i; };
            float pend = 1.f;
            float4 ku, ev, iv;
            if (nx > 0) ku = units[0], ev = units[1], iv = units[2];
            for (int j = 0; j < nx; ++j, ++step) {
                float bk[4] = {bq * ku.x, bq * ku.y, bq * ku.z, bq * ku.w};
                float es[4] = {ev.x, ev.y, ev.z, ev.w}, is[4] = {iv.x, iv.y, iv.z, iv.w};
                units += 3;
                if (j + 1 < nx) ku = units[0], ev = units[1], iv = units[2];
#pragma unroll
                for (int b = 0; b < 4; ++b) bk[b] = bk[b] == 0.f ? FLT_MIN : bk[b];   // -inf scores stay -inf
                ok = __all_sync(0xffffffffu, wait(&sfull[x], step & 1));
                if (!ok) break;
                tc_fence_after();
                // Hidden scores become -inf, and the units of a block without a
                // visible one do not count.
                const int at = kTile * j;
                const bool edge = __any_sync(0xffffffffu, row_ok && (top < at + kTile - 1 || first > at));
                uint32_t seen[4];
                if (edge) {
                    const int c_hi = top + 1 - at, c_lo = first - at;
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const int hi_b = min(32, max(0, c_hi - 32 * b)), lo_b = min(32, max(0, c_lo - 32 * b));
                        seen[b] = (uint32_t)(((1ull << hi_b) - 1) & ~((1ull << lo_b) - 1));
                        if (seen[b] == 0u) bk[b] = 1.f, es[b] = 0.f, is[b] = 0.f;
                    }
                }
                auto hide = [&](uint32_t (&v)[32], uint32_t see) {
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (!(see >> k & 1u)) v[k] = 0xff800000u;
                };
                auto most = [&](const uint32_t (&t)[32]) {
                    float v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v[e] = fmaxf(__uint_as_float(t[e]), __uint_as_float(t[4 + e]));
#pragma unroll
                        for (int k = 8; k < 32; k += 8)
                            v[e] = fmaxf(fmaxf(v[e], __uint_as_float(t[k + e])), __uint_as_float(t[k + 4 + e]));
                    }
                    return fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
                };
                // 16-bit types hold the row's scores between the maximum and
                // the weights; fp32's second terms leave no registers for
                // that, so its scores are read twice.
                constexpr bool kHold = NS == 1;
                uint32_t s[kHold ? 4 : 2][32];
                float mn = m;
                if constexpr (kHold) {
#pragma unroll
                    for (int b = 0; b < 4; ++b) tmem_ld32(ts + 32 * b, s[b]);
                    tmem_ld_wait();
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        if (edge) hide(s[b], seen[b]);
                        mn = fmaxf(mn, fmaf(most(s[b]), bk[b], es[b]));
                    }
                } else {
#pragma unroll
                    for (int b = 0; b < 4; b += 2) {
                        tmem_ld32(ts + 32 * b, s[0]);
                        tmem_ld32(ts + 32 * b + 32, s[1]);
                        tmem_ld_wait();
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            if (edge) hide(s[c], seen[b + c]);
                            mn = fmaxf(mn, fmaf(most(s[c]), bk[b + c], es[b + c]));
                        }
                    }
                }
                if (NS == 2 && j > 0 && j % kFlush == 0) {
                    ok = __all_sync(0xffffffffu, wait(&pvdone[x], (step - 1) & 1));
                    if (!ok) break;
                    tc_fence_after();
                    flush<DP>(to, sums(), pend, j > kFlush);
                    pend = 1.f;
                }
                if (__any_sync(0xffffffffu, mn > m + w_lazy<NS == 2>())) {
                    const float alpha = exp2_fast(m - (mn == -INFINITY ? 0.f : mn));
                    m = mn;
                    l *= alpha;
                    pend *= alpha;
                    if (NS == 2 ? j % kFlush != 0 : j > 0) {
                        ok = __all_sync(0xffffffffu, wait(&pvdone[x], (step - 1) & 1));
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int d = 0; d < DP; d += 16) {
                            uint32_t o[16];
                            tmem_ld16(to + d, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                            tmem_st16(to + d, o);
                        }
                        tmem_st_wait();
                    }
                }
                const float mu = (m == -INFINITY ? 0.f : m) - w_shift<NS == 2>();
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    uint32_t (&t)[32] = s[kHold ? b : b & 1];
                    if constexpr (!kHold) {
                        if (b % 2 == 0) {
                            tmem_ld32(ts + 32 * b, s[0]);
                            tmem_ld32(ts + 32 * b + 32, s[1]);
                            tmem_ld_wait();
                        }
                        if (edge) hide(t, seen[b]);
                    }
                    const uint64_t k2 = f2(bk[b], bk[b]), off = f2(es[b] - mu, es[b] - mu);
                    uint64_t sum[2] = {0, 0};
                    uint32_t ph[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        float u, v;
                        f2_split(f2_fma(f2(__uint_as_float(t[2 * k]), __uint_as_float(t[2 * k + 1])), k2, off), u, v);
                        u = exp2_fast(u);
                        v = exp2_fast(v);
                        sum[k & 1] = f2_add(sum[k & 1], f2(u, v));
                        ph[k] = pack_h2(u, v);
                        if constexpr (NS == 2) t[2 * k] = __float_as_uint(u), t[2 * k + 1] = __float_as_uint(v);
                    }
                    tmem_st16(ts + 32 * b, ph);
                    if constexpr (NS == 2) {
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const float2 h = unpack_h2(ph[k]);
                            ph[k] = pack_h2(__uint_as_float(t[2 * k]) - h.x, __uint_as_float(t[2 * k + 1]) - h.y);
                        }
                        tmem_st16(ts + 32 * b + 16, ph);
                    }
                    float u, v;
                    f2_split(f2_add(sum[0], sum[1]), u, v);
                    l = fmaf(u + v, is[b], l);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&pready[x]);
            }
            if (ok && nx > 0) ok = __all_sync(0xffffffffu, wait(&pvdone[x], (step - 1) & 1));
            if (!ok) break;
            tc_fence_after();
            const int tok = w.tok + x * p.tqt + ti, h = w.head * a.group + w.ht * p.hpt + hi, D = a.c.head_dim;
            const bool none = m == -INFINITY && l == 0.f;   // (NaN scores are seen, and raise no maximum)
            if (NS == 2 && nx > kFlush) flush<DP>(to, sums(), pend, true, true);
            float inv = 0.f;
            const int64_t prow = ((int64_t)tok * a.n_heads + h) * a.splits + w.part;
            if (a.splits > 1) {
                if (row_ok) a.part_ml[prow] = make_float2(m, l);
                inv = 1.f;
            } else if (!none) {
                if (a.sinks && row_ok) l += exp2_fast(fmaf(a.sinks[h], kLog2e, w_shift<NS == 2>() - m));
                inv = 1.f / l;
            }
#pragma unroll 1
            for (int c = 0; c < DP; c += 32) {
                uint32_t o[32];
                if (nx > 0) {
                    tmem_ld32(to + c, o);
                    tmem_ld_wait();
                }
                if (!row_ok) continue;
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = none ? 0u : __float_as_uint(__uint_as_float(o[k]) * inv);
                // A thread writes whole 32-byte sectors of its row where they
                // are aligned: narrower stores of rows that lie apart cost a
                // windowed prompt 27 of 143 us.
                if (a.splits > 1) {
                    float *dst = a.part_o + prow * D + c;
#pragma unroll
                    for (int k = 0; k < 32; k += 8)
                        if (c + k < D && !none) {
                            const uint32_t v[8] = {o[k], o[k + 1], o[k + 2], o[k + 3], o[k + 4], o[k + 5], o[k + 6], o[k + 7]};
                            store_sector(dst + k, v);
                        }
                    continue;
                }
                T *dst = static_cast<T *>(a.out) + (int64_t)tok * a.o_lt + (int64_t)h * a.o_lh + c;
                if (a.o_sector) {
                    constexpr int E = 32 / sizeof(T);
#pragma unroll
                    for (int k = 0; k < 32; k += E) {
                        if (c + k >= D) continue;
                        uint32_t v[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            if constexpr (sizeof(T) == 4) v[e] = o[k + e];
                            else v[e] = pack2<T>(__uint_as_float(o[k + 2 * e]), __uint_as_float(o[k + 2 * e + 1]));
                        }
                        store_sector(dst + k, v);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 32; k += 4)
                        if (c + k < D) {
                            const float v[4] = {__uint_as_float(o[k]), __uint_as_float(o[k + 1]), __uint_as_float(o[k + 2]), __uint_as_float(o[k + 3])};
                            store4<T>(dst + k, a.o_vec, v);
                        }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&iempty[slot]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kSoftWarps) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------ host side
struct Layout {
    int64_t cap_q, cap_kv, cap_seq;
    int splits, split_tiles;
    size_t plan, q_tiles, kv_base, kv_first, q_img, q_unit, k_img, v_img, units, sums, part_o, part_ml, total;
};

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

void tile_shape(const AttnParams &p, TileParams *t)
{
    t->hpt = std::min(p.group, kTile);
    t->head_tiles = (p.group + t->hpt - 1) / t->hpt;
    t->tqt = kTile / t->hpt;
    t->nt = p.c.head_dim > 128 ? 1 : 2;
}

Layout layout(const AttnParams &p, const TileParams &t, int dtype, int64_t max_len)
{
    Layout L = {};
    const int ns = dtype == RF_F32 ? 2 : 1, dp = p.c.head_dim > 128 ? 256 : p.c.head_dim > 64 ? 128 : 64;
    const int64_t ctt = t.nt * t.tqt;
    L.cap_q = p.b.n_tok / ctt + std::min<int64_t>(p.b.n_seq, p.b.n_tok);
    // No sequence's position tiles exceed max_len's; with a window, all of
    // them together do not exceed the windows' and the new tokens', however
    // long the sequences are (positions are below 2^31).
    auto tiles_of = [](int64_t len) { return std::min<int64_t>((len + kTile - 1) / kTile, 1 << 24); };
    L.cap_seq = tiles_of(max_len);
    L.cap_kv = p.b.n_seq * L.cap_seq;
    if (p.window > 0) {
        const int64_t windows = (p.b.n_seq * std::min(p.window, max_len) + p.b.n_tok) / kTile + 3LL * p.b.n_seq;
        if (windows < L.cap_kv) {
            L.cap_kv = windows;
            L.cap_seq = tiles_of((int64_t)p.b.table_width * p.c.page_size);
        }
    }
    const int64_t kvh = p.c.n_kv_heads;
    // Parts of the position tiles: the number for which the items' rounds over
    // the SMs take the least time, in steps of one position tile (about 2 us,
    // twice that for fp32): a round is its part's tiles and about two more to
    // start and to write, and parts cost their write and read in the join.
    const int64_t ctas = std::max<int64_t>(1, std::min<int64_t>(L.cap_q, (p.b.n_tok + ctt - 1) / ctt) * kvh * t.head_tiles);
    int64_t seen = (max_len + kTile - 1) / kTile;
    if (p.window > 0) seen = std::min<int64_t>(seen, (p.window + ctt) / kTile + 2);
    const double join = (double)p.b.n_tok * p.n_heads * p.c.head_dim * 8 / (6.0e6 * 2.0 * ns);
    double best = 0;
    for (int64_t s = 1; s <= std::min<int64_t>(64, std::max<int64_t>(1, seen / 4)); ++s) {
        const int64_t per = (seen + s - 1) / s, rounds = (ctas * s + num_sms() - 1) / num_sms();
        const double cost = (double)rounds * (per + 2) + (s > 1 ? s * join + 3 : 0);
        if (s == 1 || cost < best) {
            best = cost;
            L.split_tiles = (int)per;
        }
    }
    L.splits = (int)((seen + L.split_tiles - 1) / L.split_tiles);
    size_t at = 0;
    auto take = [&at](size_t n) {
        const size_t here = at;
        at += up256(n);
        return here;
    };
    const size_t slot = (size_t)kTile * dp * 2;
    L.plan = take(sizeof(TilePlan));
    L.q_tiles = take(L.cap_q * sizeof(QTile));
    L.kv_base = take(p.b.n_seq * sizeof(int32_t));
    L.kv_first = take(p.b.n_seq * sizeof(int32_t));
    L.q_img = take(L.cap_q * kvh * t.head_tiles * t.nt * ns * slot);
    L.q_unit = take(L.cap_q * kvh * t.head_tiles * 2 * kTile * sizeof(float));
    L.k_img = take(L.cap_kv * kvh * slot);
    L.v_img = take(L.cap_kv * kvh * slot);
    L.units = take(L.cap_kv * kvh * 12 * sizeof(float));
    if (ns == 2 && L.split_tiles > kFlush)
        L.sums = take(L.cap_q * kvh * t.head_tiles * L.splits * 2 * (dp / 4) * kTile * sizeof(float4));
    if (L.splits > 1) {
        const size_t rows = (size_t)p.b.n_tok * p.n_heads * L.splits;
        L.part_o = take(rows * p.c.head_dim * sizeof(float));
        L.part_ml = take(rows * sizeof(float2));
    }
    L.total = at;
    return L;
}

template <typename T, int DP>
rf_status launch_tiles(const TileParams &t, cudaStream_t s, bool chain)
{
    constexpr int NS = sizeof(T) == 4 ? 2 : 1;
    static_assert(tile_smem<DP, NS>() + 3072 <= 232448, "tiles exceed the 227 KB of shared memory");
    static std::once_flag once[64];
    static bool okd[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return RF_ERR_CUDA;
    }
    std::call_once(once[dev & 63], [dev] {
        okd[dev & 63] = cudaFuncSetAttribute(attn_tile_kernel<T, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)tile_smem<DP, NS>()) == cudaSuccess;
        cudaGetLastError();
    });
    if (!okd[dev & 63]) return RF_ERR_CUDA;
    const AttnParams &a = t.a;
    const int64_t kvh = a.c.n_kv_heads, ctas = (int64_t)t.cap_q * kvh * t.head_tiles;
    const int64_t stage = (int64_t)t.cap_kv * kvh + ctas + kPadParts;
    // (CTAs draw items until they get one past the last: that count is an int too)
    if (stage > 0x7fffffffLL || ctas * a.splits > 0x7fffffffLL - 65536) return RF_ERR_TOO_LARGE;
    if (const rf_status st = launch_kernel(tile_plan_kernel, dim3(1), dim3(1024), 0, s, chain, t)) return st;
    if (const rf_status st = launch_kernel(tile_stage_kernel<T, DP>, dim3((unsigned)stage), dim3(256), 0, s, true, t))
        return st;
    return launch_kernel(attn_tile_kernel<T, DP>, dim3((unsigned)std::min<int64_t>(ctas * a.splits, num_sms())), dim3(kMainThreads),
                         tile_smem<DP, NS>(), s, true, t);
}

}  // namespace

bool attn_tile_takes(const AttnParams &p, int64_t max_len)
{
    // Rows (tokens x heads of a group) per sequence and the work in all.
    // Measured in us, rows kernel / tiles, one sequence, bf16, four heads of
    // 128 to a K/V head, against 30,000 positions: 64 rows 58 / 67, 128 rows
    // 108 / 71, 256 rows 201 / 85; against 1,000: 64 rows 16 / 24, 256 rows
    // 21 / 32; 16 sequences against 8,000: 64 rows 235 / 247, 128 rows 397 /
    // 250 (fp32: 324 / 326, 572 / 342).  Tiles pay from about 96 rows, once
    // the work outweighs two more launches and the staging.
    const int64_t per_seq = tokens_per_seq(p), rows = per_seq * p.group;
    const int64_t seen = p.window > 0 ? std::min(max_len, p.window + per_seq) : max_len;
    return rows >= 96 && (double)rows * seen * p.b.n_seq >= 5e5;
}

size_t attn_tile_workspace(const AttnParams &p, int dtype, int64_t max_len)
{
    TileParams t;
    tile_shape(p, &t);
    return layout(p, t, dtype, max_len).total;
}

void attn_tile_plan(const AttnParams &p, int dtype, int64_t max_len, rf_attention_plan *out)
{
    TileParams t;
    tile_shape(p, &t);
    const Layout L = layout(p, t, dtype, max_len);
    out->tiles = 1, out->parts = L.splits, out->part_positions = (int64_t)L.split_tiles * kTile;
    out->item_tokens = t.nt * t.tqt, out->head_tiles = t.head_tiles;
}

rf_status launch_attn_tile(AttnParams p, int dtype, int64_t max_len, void *workspace, cudaStream_t s, bool chain)
{
    TileParams t;
    tile_shape(p, &t);
    const Layout L = layout(p, t, dtype, max_len);
    if (L.cap_q > 0x3fffffffLL || L.cap_kv > 0x3fffffffLL || (L.splits > 1 && !attn_join_takes(p))) return RF_ERR_TOO_LARGE;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.splits = L.splits;
    p.part_o = reinterpret_cast<float *>(ws + L.part_o);
    p.part_ml = reinterpret_cast<float2 *>(ws + L.part_ml);
    t.a = p;
    t.cap_q = (int)L.cap_q, t.cap_kv = (int)L.cap_kv, t.cap_seq = (int)L.cap_seq;
    t.plan = reinterpret_cast<TilePlan *>(ws + L.plan);
    t.q_tiles = reinterpret_cast<QTile *>(ws + L.q_tiles);
    t.kv_base = reinterpret_cast<int32_t *>(ws + L.kv_base);
    t.kv_first = reinterpret_cast<int32_t *>(ws + L.kv_first);
    t.q_img = ws + L.q_img;
    t.q_unit = reinterpret_cast<float *>(ws + L.q_unit);
    t.k_img = ws + L.k_img, t.v_img = ws + L.v_img;
    t.units = reinterpret_cast<float *>(ws + L.units);
    t.sums = reinterpret_cast<float4 *>(ws + L.sums);
    t.split_tiles = L.split_tiles;
    t.qk_abs = p.qk_scale < 0.f ? -p.qk_scale : p.qk_scale;
    t.negate = p.qk_scale < 0.f;
    t.limit = kWaitLimitNs;
    const int D = p.c.head_dim;
    rf_status st = with_dtype(dtype, [&](auto v) {
        using T = decltype(v);
        if (D > 128) return launch_tiles<T, 256>(t, s, chain);
        return D > 64 ? launch_tiles<T, 128>(t, s, chain) : launch_tiles<T, 64>(t, s, chain);
    });
    if (st != RF_OK) return st;
    return p.splits > 1 ? launch_attn_join(p, dtype, s) : RF_OK;
}

rf_status read_and_clear_attn_tile_status()
{
    int v[2] = {0, 0};
    const int zero = 0;
    if (cudaMemcpyFromSymbol(&v[0], g_tile_status, sizeof(int)) != cudaSuccess ||
        cudaMemcpyFromSymbol(&v[1], g_tile_invalid, sizeof(int)) != cudaSuccess)
        return RF_ERR_CUDA;
    if ((v[0] != 0 && cudaMemcpyToSymbol(g_tile_status, &zero, sizeof(int)) != cudaSuccess) ||
        (v[1] != 0 && cudaMemcpyToSymbol(g_tile_invalid, &zero, sizeof(int)) != cudaSuccess))
        return RF_ERR_CUDA;
    return static_cast<rf_status>(v[0] != 0 ? v[0] : v[1]);
}

}  // namespace rf
