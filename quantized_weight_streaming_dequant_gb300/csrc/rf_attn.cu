// rf_attn.cu -- attention over the paged cache of 8-bit codes: the entry
// point, the kernel for single tokens and short chunks, and the join of
// split rows.
//
// Mathematics.  A block of 32 positions has one unit 2^ek for its keys and
// one unit 2^ev for its values, so with codes k', v'
//     x_j = scale*log2(e) * 2^ek * (q . k'_j) + ev,   w_j = 2^(x_j - m),
//     out = sum_j w_j v'_j / sum_j w_j 2^-ev,
// m the running maximum of x.  Putting the value unit into the exponent
// makes both products run on bare codes, which are exact in fp16, and costs
// nothing: x is one multiply-add per score either way, and the sum one
// multiply-add instead of an addition.
//
// attn_rows_kernel.  Bound: the cache's bytes (one read of K and V), so the
// work per byte has to stay below the memory's pace.  Scores are computed
// transposed, S^T = K Q^T: positions fill the 16 rows of mma.m16n8k16 and
// the (few) query rows its 8 columns, so no tensor work is spent on rows
// that a group of up to eight heads does not have, and a K or V fragment is
// converted once for all of them.  Fragment orders are free along the
// contracted dimension and along head_dim, so each lane converts runs of 16
// bytes as they lie in memory: no transposition of V, and P^T comes from S^T
// by movmatrix.  tcgen05 would need its 64-row minimum and a trip through
// tensor memory for eight rows.  Each warp streams its own blocks through a
// private ring of cp.async copies (no CTA barrier in the loop); warps and
// CTAs are joined at the end.
// Measured: fp32, one token against 131,072 positions of 8 heads of 128 (four
// query heads each): 48 us (5.6 TB/s, 0.82 of the measured copy rate) and 7
// for the join; bf16, 48 ragged sequences of up to 16,001 positions, 8 heads
// of 64 (eight each): 78 us (5.1 TB/s) and 8.  Neither memory nor issue is
// full (0.82 and 0.75 of the copy rate, 50 and 65 % of the issue slots): the
// registers of queries and O leave 8 and 16 warps an SM, too few to hide the
// chains that turn codes into fp16 (five instructions for four codes, and two
// more to pair V's) and into weights.  Tried and not kept: equal shares of all blocks
// over one wave of CTAs (62 and 104 us against 54 and 88 for the calls: SMs
// differ in speed, and the shares' state costs registers), three CTAs an SM
// for head_dim 128 (66 against 54: spills), two and six waves of parts
// instead of four (106 and 95 against 86), keys as fp16 subnormals, which
// saves them the subtraction (86 against 87 before empty parts left early).
#include <algorithm>
#include <climits>
#include <cmath>
#include <mutex>

#include "rf_attn.h"

namespace rf {
namespace {

__device__ int g_attn_status = 0;   // positions or pages that do not exist

constexpr int kWarps = 4;

__device__ __forceinline__ uint32_t mov_trans(uint32_t v)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait_group()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Byte offset of a 16-byte run in a 32-position tile.  Where a row is 64, 128
// or 256 bytes (SWZ), runs are permuted so that the eight lanes of a
// shared-memory phase hit all banks: K reads rows g, g+1 x four runs, V rows
// 2c x two neighbouring runs.
template <bool SWZ> __device__ __forceinline__ int k_off(int row, int run, int D)
{
    const int o = row * D + run * 16;
    return SWZ && D > 64 ? o ^ ((row & 1) << 6) : o;
}
template <bool SWZ> __device__ __forceinline__ int v_off(int row, int byte, int D)
{
    const int o = row * D + byte;
    return SWZ ? o ^ (((row >> 1) & 3) << 5) : o;
}

template <int DP> __host__ __device__ constexpr int ring_stages() { return DP == 256 ? 2 : 3; }
template <int DP> size_t rows_smem(int D)
{
    return (size_t)kWarps * ring_stages<DP>() * 64 * D + 256;
}

struct RowTiling {
    int hpt, head_tiles, tq;   // heads per tile, tiles per K/V head, tokens per tile
};

// DP: head_dim rounded up to 64, 128 or 256.  NR: query rows / 8.  SPLIT:
// queries and weights as two fp16 terms (fp32 activations).
template <typename T, int DP, int NR, bool SPLIT, bool SWZ>
__global__ void __launch_bounds__(32 * kWarps, DP == 256 ? 1 : DP == 128 ? 2 : NR == 1 ? 4 : 2)
    attn_rows_kernel(const __grid_constant__ AttnParams p, const RowTiling tl)
{
    constexpr int ST = ring_stages<DP>();
    constexpr int NS = SPLIT ? 2 : 1;
    constexpr int KS = DP / 16;                 // k-steps of Q K^T
    constexpr int MT = DP / 16;                 // 16-row tiles of O^T
    constexpr int VB = DP == 64 ? 8 : 16;       // bytes of V per lane, position and run
    constexpr int ROWS = 8 * NR;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_meta[kWarps][ST];
    __shared__ float s_m[kWarps][ROWS], s_l[kWarps][ROWS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int D = SWZ ? DP : p.c.head_dim;

    // This CTA: token tile that starts at t, K/V head and its head tile, part.
    int u = (int)blockIdx.x;
    const int part = u % p.splits;
    u /= p.splits;
    const int ht = u % tl.head_tiles;
    u /= tl.head_tiles;
    const int kvh = u % p.c.n_kv_heads, t = u / p.c.n_kv_heads;
    pdl_launch_dependents();
    pdl_wait();
    const int seq = find_seq_warp(p.b.q_start, p.b.n_seq, t);
    int n_here = 1;
    int64_t pos0 = -1;
    if (seq >= 0) {
        const int first = p.b.q_start[seq];
        if ((t - first) % tl.tq != 0) return;
        n_here = min(tl.tq, min(p.b.q_start[seq + 1], p.b.n_tok) - t);
        pos0 = (int64_t)p.b.past[seq] + (t - first);
        if (pos0 < 0 && threadIdx.x == 0) record_status(&g_attn_status, RF_ERR_INVALID_ARG);
    }
    const int h0 = kvh * p.group + ht * tl.hpt, nh = min(tl.hpt, p.group - ht * tl.hpt);

    // Blocks of 32 positions that some row sees, and this part of them.
    const int64_t pos_last = pos0 + n_here - 1;
    int64_t lo = 0;
    if (p.window > 0) lo = max((int64_t)0, pos0 - p.window + 1);
    int b_lo = (int)(lo / kKvBlock), b_hi = seq >= 0 && pos_last >= 0 ? (int)(pos_last / kKvBlock) + 1 : 0;
    // (positions past the table have no page, however many there are)
    const int b_cap = (int)min((int64_t)INT_MAX, (int64_t)p.b.table_width * (p.c.page_size / kKvBlock));
    if (b_hi > b_cap) {
        if (threadIdx.x == 0) record_status(&g_attn_status, RF_ERR_INVALID_ARG);
        b_hi = b_cap;
    }
    {
        const int64_t from = b_lo + (int64_t)part * p.split_blocks;
        const int to = part == p.splits - 1 ? b_hi : (int)min((int64_t)b_hi, from + p.split_blocks);
        b_lo = (int)min(from, (int64_t)b_hi);
        b_hi = to;
    }

    // A part past the end of its sequence sees nothing.
    if (p.splits > 1 && b_hi <= b_lo) {
        const int row = (int)threadIdx.x, ti = row / tl.hpt, hi = row % tl.hpt;
        if (row < ROWS && ti < n_here && hi < nh)
            p.part_ml[((int64_t)(t + ti) * p.n_heads + h0 + hi) * p.splits + part] = make_float2(-INFINITY, 0.f);
        return;
    }

    // Ring of this warp: stage s holds K then V of one block.  The first
    // copies go out before the queries are read.
    const int stage_bytes = 64 * D;
    uint8_t *ring = smem + (size_t)warp * ST * stage_bytes;
    const int n_it = b_hi - b_lo > warp ? (b_hi - b_lo - warp + kWarps - 1) / kWarps : 0;
    const int per_page = p.c.page_size / kKvBlock;
    int64_t pg_block = -1;    // lane i: block index in the cache of iteration (it & ~31) + i
    int pg_meta = 0;          // its scale bytes, bit 16: valid
    auto issue = [&](int it) {
        if ((it & 31) == 0) {
            const int blk = b_lo + warp + kWarps * (it + lane);
            pg_block = -1;
            pg_meta = 0;
            if (it + lane < n_it) {
                const int page = page_of(p.b, p.c, seq, (int64_t)blk * kKvBlock);
                if (page >= 0) {
                    pg_block = ((int64_t)page * p.c.n_kv_heads + kvh) * per_page + blk % per_page;
                    pg_meta = (int)p.c.k_scale[pg_block] | (int)p.c.v_scale[pg_block] << 8 | 1 << 16;
                } else {
                    record_status(&g_attn_status, RF_ERR_INVALID_ARG);
                }
            }
        }
        const int64_t blk = __shfl_sync(0xffffffffu, pg_block, it & 31);
        const int st = it % ST;
        if (lane == (it & 31)) s_meta[warp][st] = pg_meta;
        if (blk >= 0) {
            uint8_t *kd = ring + st * stage_bytes, *vd = kd + 32 * D;
            const int8_t *ks = p.c.k + blk * kKvBlock * D, *vs = p.c.v + blk * kKvBlock * D;
#pragma unroll
            for (int i = 0; i < DP / 16; ++i) {
                const int w = i * 32 + lane;          // 16-byte run of the block
                if (SWZ || w < 2 * D) {
                    const int row = SWZ ? w / (DP / 16) : 0, run = SWZ ? w % (DP / 16) : w;
                    cp_async16(kd + (SWZ ? k_off<SWZ>(row, run, DP) : 16 * w), ks + 16 * w);
                    cp_async16(vd + (SWZ ? v_off<SWZ>(row, 16 * run, DP) : 16 * w), vs + 16 * w);
                }
            }
        }
    };
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) {
        if (i < n_it) issue(i);
        cp_async_commit();
    }

    // Query fragments (columns of S^T): lane (g, c) holds row 8r + g, elements
    // 64s + 16c .. + 15 of each 64-run s, scaled by a power of two that
    // brings the row's maximum to [512, 1024).
    uint32_t qf[NR][KS][NS][2];
    float qs[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const int row = 8 * r + g, ti = row / tl.hpt, hi = row % tl.hpt;
        const bool ok = ti < n_here && hi < nh;
        const T *src = static_cast<const T *>(p.q) + (int64_t)(t + ti) * p.q_lt + (int64_t)(h0 + hi) * p.q_lh;
        float f[DP / 4];
        float amax = 0.f;
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
            const int at = 64 * (k >> 2) + 16 * c + 4 * (k & 3);
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            if (ok && at < D) load4<T>(src + at, p.q_vec, v);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                f[4 * k + m] = v[m];
                amax = fmaxf(amax, fabsf(v[m]));
            }
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const float up = row_power(amax, p.qk_scale, &qs[r]);
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float a = f[4 * k + 2 * e] * up, b = f[4 * k + 2 * e + 1] * up;
                qf[r][k][0][e] = pack_h2(a, b);
                if constexpr (SPLIT) {
                    const float2 h = unpack_h2(qf[r][k][0][e]);
                    qf[r][k][1][e] = pack_h2(a - h.x, b - h.y);
                }
            }
    }
    // Rows 8r + 2c + e as S^T holds them: score factor and newest position.
    float bq[NR][2];
    int64_t top[NR][2];
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            bq[r][e] = __shfl_sync(0xffffffffu, qs[r], (2 * c + e) * 4);
            const int row = 8 * r + 2 * c + e;
            top[r][e] = row / tl.hpt < n_here ? pos0 + row / tl.hpt : -1;
        }

    float o[NR][MT][4];
    float m[NR][2], l[NR][2];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[r][i][e] = 0.f;
        m[r][0] = m[r][1] = -INFINITY;
        l[r][0] = l[r][1] = 0.f;
    }

    for (int it = 0; it < n_it; ++it) {
        __syncwarp();                                 // the stage written next was read by all
        if (it + ST - 1 < n_it) issue(it + ST - 1);
        cp_async_commit();
        cp_async_wait_group<ST - 1>();
        __syncwarp();
        const int st = it % ST;
        const int meta = s_meta[warp][st];
        if (!(meta >> 16)) continue;                  // no such page: nothing seen
        const uint8_t *kt = ring + st * stage_bytes, *vt = kt + 32 * D;
        const int64_t p_lo = (int64_t)(b_lo + warp + kWarps * it) * kKvBlock;

        // S^T, two tiles of 16 positions.
        float s[2][NR][4];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[mt][r][e] = 0.f;
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int k = 0; k < KS / 4; ++k) {
                const int row = 16 * mt + g;
                uint4 a = *reinterpret_cast<const uint4 *>(kt + k_off<SWZ>(row, 4 * k + c, D));
                uint4 b = *reinterpret_cast<const uint4 *>(kt + k_off<SWZ>(row + 8, 4 * k + c, D));
                const uint32_t wa[4] = {a.x ^ 0x80808080u, a.y ^ 0x80808080u, a.z ^ 0x80808080u, a.w ^ 0x80808080u};
                const uint32_t wb[4] = {b.x ^ 0x80808080u, b.y ^ 0x80808080u, b.z ^ 0x80808080u, b.w ^ 0x80808080u};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t a0 = codes_lo(wa[j]), a1 = codes_lo(wb[j]), a2 = codes_hi(wa[j]), a3 = codes_hi(wb[j]);
#pragma unroll
                    for (int r = 0; r < NR; ++r)
#pragma unroll
                        for (int n = NS - 1; n >= 0; --n)
                            mma_16816(s[mt][r], a0, a1, a2, a3, qf[r][4 * k + j][n][0], qf[r][4 * k + j][n][1]);
                }
            }

        // Scores to weights.
        const uint32_t Ek = meta & 255, Ev = (meta >> 8) & 255;
        const float ku = scale_value(Ek);
        const float ev = Ev == 255u ? __uint_as_float(0x7fc00000u) : (float)((int)Ev - 127);
        const float iv = scale_value(Ev == 255u ? 255u : 254u - Ev);   // 2^-ev
        const bool edge = p_lo + kKvBlock - 1 > pos0 || (p.window > 0 && p_lo <= pos_last - p.window);
        float w[2][NR][4];
        bool grew = false;
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float bk = bq[r][e] * ku;
                float best = -INFINITY;
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        float x = fmaf(s[mt][r][2 * y + e], bk, ev);
                        if (edge) {
                            const int64_t at = p_lo + 16 * mt + 8 * y + g;
                            if (at > top[r][e] || (p.window > 0 && at <= top[r][e] - p.window)) x = -INFINITY;
                        }
                        w[mt][r][2 * y + e] = x;
                        best = fmaxf(best, x);
                    }
                grew |= best > m[r][e] + w_lazy<SPLIT>();
            }
        // The maximum that the weights go by is raised only when some lane
        // has outgrown it by w_lazy (the weights' range allows that much),
        // so most blocks need one vote and no exchange between lanes.
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mn = m[r][e];
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt) mn = fmaxf(mn, fmaxf(w[mt][r][e], w[mt][r][2 + e]));
                    mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, 4));
                    mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, 8));
                    mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, 16));
                    const float alpha = exp2_fast(m[r][e] - (mn == -INFINITY ? 0.f : mn));
                    m[r][e] = mn;
                    l[r][e] *= alpha;
#pragma unroll
                    for (int i = 0; i < MT; ++i) o[r][i][e] *= alpha, o[r][i][2 + e] *= alpha;
                }
        }
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float mu = (m[r][e] == -INFINITY ? 0.f : m[r][e]) - w_shift<SPLIT>();
                float sum = 0.f;
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        float &x = w[mt][r][2 * y + e];
                        x = exp2_fast(x - mu);
                        sum += x;
                    }
                // the sum's unit; a lane that sees nothing of the block adds no NaN unit
                const bool none = edge && w[0][r][e] == 0.f && w[0][r][2 + e] == 0.f && w[1][r][e] == 0.f && w[1][r][2 + e] == 0.f;
                l[r][e] = none ? l[r][e] : fmaf(sum, iv, l[r][e]);
            }

        // O^T += V^T P^T.  The tensor core truncates its fp32 sums, so for
        // fp32 a block's product starts from zero and is added with rounding:
        // over thousands of blocks the truncations would drift (1e-5 relative
        // at 32,768 positions, which 16-bit outputs do not see).
        uint32_t pf[2][NR][NS][2];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const float a = w[mt][r][2 * y], b = w[mt][r][2 * y + 1];
                    const uint32_t hi = pack_h2(a, b);
                    pf[mt][r][0][y] = mov_trans(hi);
                    if constexpr (SPLIT) {
                        const float2 h = unpack_h2(hi);
                        pf[mt][r][1][y] = mov_trans(pack_h2(a - h.x, b - h.y));
                    }
                }
#pragma unroll
        for (int half = 0; half < (DP == 256 ? 2 : 1); ++half) {
            uint32_t v[2][4][VB / 4];                 // positions 2c, 2c+1, 2c+8, 2c+9 of each 16
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int row = 16 * mt + 2 * c + (y & 1) + 8 * (y >> 1);
                    const uint8_t *src = vt + v_off<SWZ>(row, 128 * half + VB * g, D);
                    if constexpr (VB == 16) {
                        const uint4 a = *reinterpret_cast<const uint4 *>(src);
                        v[mt][y][0] = a.x, v[mt][y][1] = a.y, v[mt][y][2] = a.z, v[mt][y][3] = a.w;
                    } else {
                        const uint2 a = *reinterpret_cast<const uint2 *>(src);
                        v[mt][y][0] = a.x, v[mt][y][1] = a.y;
                    }
                }
#pragma unroll
            for (int k = 0; k < VB / 4; ++k)
#pragma unroll
                for (int x = 0; x < 2; ++x) {         // bytes 2x, 2x+1 of the words: one 16-row tile
                    const int i = half * (MT / (DP == 256 ? 2 : 1)) + 2 * k + x;
                    float acc[NR][4] = {};
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt) {
                        const uint32_t sel = x ? 0x7362u : 0x5140u;
                        const uint32_t p0 = prmt(v[mt][0][k], v[mt][1][k], sel) ^ 0x80808080u;
                        const uint32_t p1 = prmt(v[mt][2][k], v[mt][3][k], sel) ^ 0x80808080u;
                        const uint32_t a0 = codes_lo(p0), a1 = codes_hi(p0), a2 = codes_lo(p1), a3 = codes_hi(p1);
#pragma unroll
                        for (int r = 0; r < NR; ++r)
#pragma unroll
                            for (int n = NS - 1; n >= 0; --n)
                                mma_16816(SPLIT ? acc[r] : o[r][i], a0, a1, a2, a3, pf[mt][r][n][0], pf[mt][r][n][1]);
                    }
                    if constexpr (SPLIT) {
#pragma unroll
                        for (int r = 0; r < NR; ++r)
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[r][i][e] += acc[r][e];
                    }
                }
        }
    }

    // Join the warps: maxima, sums and O^T through shared memory.
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[r][e] += __shfl_xor_sync(0xffffffffu, l[r][e], 4);
            l[r][e] += __shfl_xor_sync(0xffffffffu, l[r][e], 8);
            l[r][e] += __shfl_xor_sync(0xffffffffu, l[r][e], 16);
            if (g == 0) {
                s_m[warp][8 * r + 2 * c + e] = m[r][e];
                s_l[warp][8 * r + 2 * c + e] = l[r][e];
            }
        }
    __syncwarp();
    // [row][head_dim] floats, inside this warp's ring (ROWS * D * 4 <= its
    // bytes: 32 or 64 bytes a dimension of 128 or more).
    float *po = reinterpret_cast<float *>(ring);
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int d = DP == 64 ? 8 * g + 2 * i : 128 * (i / 8) + 16 * g + 2 * (i % 8);
            if (d < D) {
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    *reinterpret_cast<float2 *>(po + (8 * r + 2 * c + e) * D + d) = make_float2(o[r][i][e], o[r][i][2 + e]);
            }
        }
    __syncthreads();
    const int ring_floats = ST * stage_bytes / 4;
    const float *all = reinterpret_cast<const float *>(smem);
    for (int w = (int)threadIdx.x; w < ROWS * (D / 4); w += 32 * kWarps) {
        const int row = w / (D / 4), d = 4 * (w % (D / 4)), ti = row / tl.hpt, hi = row % tl.hpt;
        if (ti >= n_here || hi >= nh) continue;
        float M = -INFINITY;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) M = fmaxf(M, s_m[k][row]);
        float L = 0.f, a[4] = {0.f, 0.f, 0.f, 0.f};
        const float mu = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            const float f = exp2_fast(s_m[k][row] - mu);
            L = fmaf(f, s_l[k][row], L);
            const float4 v = *reinterpret_cast<const float4 *>(all + k * ring_floats + row * D + d);
            a[0] = fmaf(f, v.x, a[0]);
            a[1] = fmaf(f, v.y, a[1]);
            a[2] = fmaf(f, v.z, a[2]);
            a[3] = fmaf(f, v.w, a[3]);
        }
        const int64_t tok = t + ti;
        const int h = h0 + hi;
        if (p.splits > 1) {
            const int64_t at = (tok * p.n_heads + h) * p.splits + part;
            *reinterpret_cast<float4 *>(p.part_o + at * D + d) = make_float4(a[0], a[1], a[2], a[3]);
            if (d == 0) p.part_ml[at] = make_float2(M, L);
        } else {
            const bool none = M == -INFINITY && L == 0.f;   // (NaN scores are seen, and raise no maximum)
            if (p.sinks && !none) L += exp2_fast(fmaf(p.sinks[h], kLog2e, w_shift<SPLIT>() - mu));
            const float inv = none ? 0.f : 1.f / L;
#pragma unroll
            for (int e = 0; e < 4; ++e) a[e] *= inv;
            store4<T>(static_cast<T *>(p.out) + tok * p.o_lt + (int64_t)h * p.o_lh + d, p.o_vec, a);
        }
    }
}

// Joins the parts of a row in their order.  WPR: warps per (token, head) row:
// one where a row has few parts, eight (a CTA) where it has more, since a
// part is a dependent round trip to memory (38 parts of 32 rows: 24 us with
// one warp each, 5 with eight).
template <typename T, int WPR>
__global__ void __launch_bounds__(256) attn_join_kernel(const __grid_constant__ AttnParams p)
{
    __shared__ __align__(16) float s_o[WPR > 1 ? 8 : 1][256];
    __shared__ float s_l[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, D = p.c.head_dim;
    const int64_t row = WPR > 1 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 8 + warp;
    pdl_launch_dependents();
    pdl_wait();
    if (row >= (int64_t)p.b.n_tok * p.n_heads) return;
    const int64_t tok = row / p.n_heads;
    const int h = (int)(row % p.n_heads);
    const float2 *ml = p.part_ml + row * p.splits;
    float M = -INFINITY;
    bool any = false;                              // a part that saw something, were it only NaN scores
    // a token that belongs to no sequence may have no parts
    if (find_seq_warp(p.b.q_start, p.b.n_seq, (int)tok) >= 0)
        for (int k = lane; k < p.splits; k += 32) {
            const float2 v = ml[k];
            M = fmaxf(M, v.x);
            any |= !(v.x == -INFINITY && v.y == 0.f);
        }
    any = __any_sync(0xffffffffu, any);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float L = 0.f, a[2][4] = {};
    const float mu = M == -INFINITY ? 0.f : M;
    if (any) {
#pragma unroll 4
        for (int k = WPR > 1 ? warp : 0; k < p.splits; k += WPR) {
            const float2 v = ml[k];
            if (v.x == -INFINITY && v.y == 0.f) continue;      // an empty part wrote no sums
            const float f = exp2_fast(v.x - mu);
            L = fmaf(f, v.y, L);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int d = 128 * i + 4 * lane;
                if (d < D) {
                    const float4 x = *reinterpret_cast<const float4 *>(p.part_o + (row * p.splits + k) * D + d);
                    a[i][0] = fmaf(f, x.x, a[i][0]);
                    a[i][1] = fmaf(f, x.y, a[i][1]);
                    a[i][2] = fmaf(f, x.z, a[i][2]);
                    a[i][3] = fmaf(f, x.w, a[i][3]);
                }
            }
        }
    }
    if constexpr (WPR > 1) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            *reinterpret_cast<float4 *>(&s_o[warp][128 * i + 4 * lane]) = make_float4(a[i][0], a[i][1], a[i][2], a[i][3]);
        if (lane == 0) s_l[warp] = L;
        __syncthreads();
        if (warp > 0) return;
        L = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) L += s_l[k];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                a[i][e] = 0.f;
#pragma unroll
                for (int k = 0; k < 8; ++k) a[i][e] += s_o[k][128 * i + 4 * lane + e];
            }
    }
    if (p.sinks && any) L += exp2_fast(fmaf(p.sinks[h], kLog2e, w_shift<sizeof(T) == 4>() - mu));
    T *out = static_cast<T *>(p.out) + tok * p.o_lt + (int64_t)h * p.o_lh;
    const float inv = any ? 1.f / L : 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int d = 128 * i + 4 * lane;
        if (d < D) {
#pragma unroll
            for (int e = 0; e < 4; ++e) a[i][e] *= inv;
            store4<T>(out + d, p.o_vec, a[i]);
        }
    }
}

// NR and the tiling of the rows kernel.
int rows_tiling(const AttnParams &p, RowTiling *tl)
{
    // Eight rows hold one token of a group of up to eight heads; sixteen are
    // taken where they are filled (head_dim above 128 leaves no registers).
    const int64_t rows = (int64_t)p.group * tokens_per_seq(p);
    const int nr = rows > 8 && p.c.head_dim <= 128 ? 2 : 1;
    tl->hpt = std::min(p.group, 8 * nr);
    tl->head_tiles = (p.group + tl->hpt - 1) / tl->hpt;
    tl->tq = 8 * nr / tl->hpt;
    return nr;
}

// Blocks of 32 positions a tile of tq tokens may see.
int64_t visible_blocks(const AttnParams &p, int64_t max_len, int tq)
{
    const int64_t seen = p.window > 0 ? std::min(max_len, p.window + tq + kKvBlock) : max_len;
    return (seen + kKvBlock - 1) / kKvBlock;
}

void choose_splits(AttnParams *p, const RowTiling &tl, int64_t max_len)
{
    const int64_t blocks = visible_blocks(*p, max_len, tl.tq);
    const int64_t per_seq = tokens_per_seq(*p);
    const int64_t tiles = std::min<int64_t>(p->b.n_tok, (per_seq + tl.tq - 1) / tl.tq * p->b.n_seq) *
                          p->c.n_kv_heads * tl.head_tiles;
    const int occ = p->c.head_dim > 128 ? 1 : p->c.head_dim > 64 ? 2 : 4;
    // One sequence: its parts fill the SMs once.  Several: parts of equal
    // size, about four waves of them, so that long sequences do not leave
    // the others' SMs idle.  A part has a block for each warp at least.
    const int64_t want = (int64_t)num_sms() * occ * (p->b.n_seq > 1 ? 4 : 1);
    int64_t splits = std::max<int64_t>(1, want / tiles);
    splits = std::min<int64_t>(splits, std::max<int64_t>(1, blocks / kWarps));
    // Up to four blocks a warp, one part without a join is as fast on the GPU
    // (us with one part / with parts, 32 K/V heads of 128: 7.4 / 9.5 at 300
    // positions, 8.6 / 8.4 at 500, 11.7 / 11.1 at 1,000, 14.4 / 10.6 at
    // 2,000) and a launch less on the host.
    if (blocks <= 4 * kWarps) splits = 1;
    splits = std::min<int64_t>(splits, 128);
    p->split_blocks = (int)((blocks + splits - 1) / splits);
    p->splits = (int)((blocks + p->split_blocks - 1) / std::max(1, p->split_blocks));
    p->splits = std::max(1, p->splits);
}

template <typename T, int DP, int NR>
rf_status launch_rows_nr(const AttnParams &p, const RowTiling &tl, cudaStream_t s, bool chain)
{
    constexpr bool SPLIT = sizeof(T) == 4;
    const int64_t ctas = (int64_t)p.b.n_tok * p.c.n_kv_heads * tl.head_tiles * p.splits;
    if (ctas > 0x7fffffffLL) return RF_ERR_TOO_LARGE;
    const size_t smem = rows_smem<DP>(p.c.head_dim);
    auto go = [&](auto *kernel, bool *ok, std::once_flag *once) -> rf_status {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) {
            cudaGetLastError();
            return RF_ERR_CUDA;
        }
        std::call_once(once[dev & 63], [&] {
            ok[dev & 63] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                (int)rows_smem<DP>(DP)) == cudaSuccess;
            cudaGetLastError();
        });
        if (!ok[dev & 63]) return RF_ERR_CUDA;
        return launch_kernel(kernel, dim3((unsigned)ctas), dim3(32 * kWarps), smem, s, chain, p, tl);
    };
    if (p.c.head_dim == DP) {
        static bool ok[64];
        static std::once_flag once[64];
        return go(&attn_rows_kernel<T, DP, NR, SPLIT, true>, ok, once);
    }
    static bool ok[64];
    static std::once_flag once[64];
    return go(&attn_rows_kernel<T, DP, NR, SPLIT, false>, ok, once);
}

template <typename T>
rf_status launch_rows(const AttnParams &p, const RowTiling &tl, int nr, cudaStream_t s, bool chain)
{
    const int D = p.c.head_dim;
    if (D > 128) return launch_rows_nr<T, 256, 1>(p, tl, s, chain);
    if (D > 64)
        return nr == 2 ? launch_rows_nr<T, 128, 2>(p, tl, s, chain) : launch_rows_nr<T, 128, 1>(p, tl, s, chain);
    return nr == 2 ? launch_rows_nr<T, 64, 2>(p, tl, s, chain) : launch_rows_nr<T, 64, 1>(p, tl, s, chain);
}

size_t parts_bytes(const AttnParams &p)
{
    if (p.splits <= 1) return 0;
    const size_t rows = (size_t)p.b.n_tok * p.n_heads * p.splits;
    return rows * ((size_t)p.c.head_dim * sizeof(float) + sizeof(float2));
}

// The parameters that the arguments fix; max_len becomes the bound used.
rf_status plan(const rf_kv_cache *cache, const rf_kv_batch *batch, int dtype, int n_heads, int64_t window,
               int64_t *max_len, AttnParams *p)
{
    if (!dtype_ok(dtype)) return RF_ERR_UNSUPPORTED_FMT;
    if (const rf_status st = check_kv(cache, batch)) return st;
    if (n_heads < 1 || n_heads % cache->n_kv_heads != 0 || window < 0 || *max_len < 0) return RF_ERR_INVALID_ARG;
    if (n_heads > 4096) return RF_ERR_TOO_LARGE;
    const int64_t cap = (int64_t)batch->table_width * cache->page_size;
    if (*max_len == 0 || *max_len > cap) *max_len = cap;
    p->c = *cache, p->b = *batch;
    p->n_heads = n_heads, p->group = n_heads / cache->n_kv_heads;
    p->window = window <= INT_MAX ? window : 0;   // positions are below 2^31: it hides none
    return RF_OK;
}

}  // namespace

bool attn_join_takes(const AttnParams &p) { return (int64_t)p.b.n_tok * p.n_heads <= INT_MAX; }

rf_status launch_attn_join(const AttnParams &p, int dtype, cudaStream_t s)
{
    const int64_t rows = (int64_t)p.b.n_tok * p.n_heads;
    return with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        if (p.splits > 8) return launch_kernel(attn_join_kernel<T, 8>, dim3((unsigned)rows), dim3(256), 0, s, true, p);
        return launch_kernel(attn_join_kernel<T, 1>, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, s, true, p);
    });
}

rf_status read_and_clear_attn_status()
{
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_attn_status, sizeof(int)) != cudaSuccess) return RF_ERR_CUDA;
    if (v != 0) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(g_attn_status, &zero, sizeof(int)) != cudaSuccess) return RF_ERR_CUDA;
    }
    return static_cast<rf_status>(v);
}

}  // namespace rf

using namespace rf;

extern "C" {

size_t rf_attention_workspace_bytes(const rf_kv_cache *cache, const rf_kv_batch *batch, int dtype, int n_heads,
                                    int64_t window, int64_t max_len)
{
    AttnParams p = {};
    if (plan(cache, batch, dtype, n_heads, window, &max_len, &p) != RF_OK || batch->n_tok == 0) return 0;
    if (attn_tile_takes(p, max_len)) return attn_tile_workspace(p, dtype, max_len);
    RowTiling tl;
    rows_tiling(p, &tl);
    choose_splits(&p, tl, max_len);
    return parts_bytes(p);
}

rf_status rf_debug_attention_plan(const rf_kv_cache *cache, const rf_kv_batch *batch, int dtype, int n_heads,
                                  int64_t window, int64_t max_len, rf_attention_plan *out)
{
    AttnParams p = {};
    if (!out) return RF_ERR_INVALID_ARG;
    if (const rf_status st = plan(cache, batch, dtype, n_heads, window, &max_len, &p)) return st;
    *out = rf_attention_plan{};
    out->sms = num_sms();
    if (batch->n_tok == 0) return RF_OK;
    if (attn_tile_takes(p, max_len)) {
        attn_tile_plan(p, dtype, max_len, out);
        return RF_OK;
    }
    RowTiling tl;
    rows_tiling(p, &tl);
    choose_splits(&p, tl, max_len);
    out->parts = p.splits, out->part_positions = (int64_t)p.split_blocks * kKvBlock;
    out->item_tokens = tl.tq, out->head_tiles = tl.head_tiles;
    return RF_OK;
}

rf_status rf_attention(const rf_kv_cache *cache, const rf_kv_batch *batch, int dtype, const void *q,
                       int64_t q_ld_tok, int64_t q_ld_head, int n_heads, float scale, int64_t window,
                       const float *sinks, void *out, int64_t out_ld_tok, int64_t out_ld_head, int64_t max_len,
                       void *workspace, size_t workspace_bytes, unsigned flags, void *stream)
{
    AttnParams p = {};
    if (const rf_status st = plan(cache, batch, dtype, n_heads, window, &max_len, &p)) return st;
    const int D = cache->head_dim;
    if (!std::isfinite(scale) || (flags & ~RF_CHAIN) != 0) return RF_ERR_INVALID_ARG;
    if (batch->n_tok > 0 && (!q || !out || q_ld_tok < D || q_ld_head < D || out_ld_tok < D || out_ld_head < D))
        return RF_ERR_INVALID_ARG;
    const size_t b = (size_t)dtype_bytes(dtype);
    if (!aligned_to(q, b) || !aligned_to(out, b) || !aligned_to(sinks, 4) || !aligned_to(workspace, 256))
        return RF_ERR_MISALIGNED;
    if (batch->n_tok == 0) return RF_OK;
    p.q = q, p.out = out, p.sinks = sinks;
    p.q_lt = q_ld_tok, p.q_lh = q_ld_head, p.o_lt = out_ld_tok, p.o_lh = out_ld_head;
    p.qk_scale = (float)((double)scale * 1.4426950408889634);
    p.q_vec = aligned_to(q, 4 * b) && q_ld_tok % 4 == 0 && q_ld_head % 4 == 0;
    p.o_vec = aligned_to(out, 4 * b) && out_ld_tok % 4 == 0 && out_ld_head % 4 == 0;
    p.q_vec8 = aligned_to(q, 8 * b) && q_ld_tok % 8 == 0 && q_ld_head % 8 == 0;
    p.o_sector = aligned_to(out, 32) && (out_ld_tok * (int64_t)b) % 32 == 0 && (out_ld_head * (int64_t)b) % 32 == 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool chain = (flags & RF_CHAIN) != 0;
    if (attn_tile_takes(p, max_len)) {
        if (!workspace || workspace_bytes < attn_tile_workspace(p, dtype, max_len)) return RF_ERR_INVALID_ARG;
        return launch_attn_tile(p, dtype, max_len, workspace, s, chain);
    }
    RowTiling tl;
    const int nr = rows_tiling(p, &tl);
    choose_splits(&p, tl, max_len);
    const size_t need = parts_bytes(p);
    if (need > 0 && (!workspace || workspace_bytes < need)) return RF_ERR_INVALID_ARG;
    if (p.splits > 1 && !attn_join_takes(p)) return RF_ERR_TOO_LARGE;
    if (need > 0) {
        p.part_o = static_cast<float *>(workspace);
        p.part_ml = reinterpret_cast<float2 *>(p.part_o + (size_t)p.b.n_tok * p.n_heads * p.splits * D);
    }
    rf_status st = with_dtype(dtype, [&](auto t) { return launch_rows<decltype(t)>(p, tl, nr, s, chain); });
    if (st != RF_OK || p.splits == 1) return st;
    return launch_attn_join(p, dtype, s);
}

}  // extern "C"
