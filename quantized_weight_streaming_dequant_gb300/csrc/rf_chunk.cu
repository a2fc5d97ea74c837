// rf_chunk.cu -- entry points of the chunk operators and the kernels around
// their products (rf_chunk_mma.cu, rf_chunk_few.cu): the token tiles and operand
// images before them, the sum over a token's experts after them.
//
// prep_kernel, one launch:
//   * its last CTA lists the token tiles: up to T rows of one group each.
//   * the others write the images.  A granule is 16 operand rows (16 tokens,
//     or 8 tokens of two terms; half of that for tiles of 8 operand rows) of a
//     group of GT tokens; granule q of group g is granule offsets[g] / GT + g +
//     q of the images: no two groups meet, and no scan over the groups is
//     needed to find a place.  A CTA takes eight rows of a granule, or a share
//     of their slices: a warp finds its row's largest value, hence a power of
//     two, then rounds the row to fp16; the eight rows' units of 16 bytes meet
//     in shared memory in the layout of the products' operand (K-major core
//     matrices, 2 KB a granule and slice) and leave as whole lines.
// It reads X once from memory (the second pass over a row finds it in L2 or
// closer) and writes 2 bytes an element (4 with two terms).  Bound: latency of
// its chain offsets - row - scale - row - lines, and with long rows the loads in
// flight: 2048 x 11008 bf16 in 25 us (3.6 TB/s, in and out), 2002 x 11008 fp32
// in 31 us, 8192 x 2880 fp32 in 31 us.  Units written by the threads that
// loaded them, eight rows a warp: 33, 48 and 49 us.  A few rows: 5 us.
//
// join_kernel adds a token's experts: 94 MB in and 12 MB out in 17 us (6.2
// TB/s), bound by memory.
#include <cuda_bf16.h>

#include <algorithm>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "rf_chunk.h"
#include "rf_device.cuh"
#include "rf_half.cuh"

namespace rf {
namespace {

__device__ int g_chunk_invalid = 0;   // offsets or order entries out of range

constexpr int kPrepThreads = 256;
constexpr int kPrepRows = 8;         // tokens per CTA of the pre-pass
constexpr int64_t kMaxPieces = 1LL << 30;
constexpr int64_t kMaxSums = 16LL << 20;   // floats of parts' sums at most
constexpr int64_t kMaxParts = 16;

template <int DT> struct Elem;
template <> struct Elem<RF_F32> { using T = float; };
template <> struct Elem<RF_F16> { using T = __half; };
template <> struct Elem<RF_BF16> { using T = __nv_bfloat16; };

__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// Four consecutive elements (vec: aligned to them all).
__device__ __forceinline__ void load4(const float *x, bool vec, float (&f)[4])
{
    if (vec) {
        const float4 v = *reinterpret_cast<const float4 *>(x);
        f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = x[e];
    }
}
template <class T>
__device__ __forceinline__ void load4(const T *x, bool vec, float (&f)[4])
{
    T t[4];
    if (vec) *reinterpret_cast<uint2 *>(t) = *reinterpret_cast<const uint2 *>(x);
    else {
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] = x[e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = to_f32(t[e]);
}

// N consecutive elements' bits (vec: aligned to them all, or to 16 bytes).
template <class T, int N> struct Some { uint32_t w[N * sizeof(T) / 4]; };
template <class T, int N>
__device__ __forceinline__ void load(const T *x, bool vec, Some<T, N> &v)
{
    constexpr int W = N * sizeof(T) / 4;
    static_assert(W == 2 || W == 4, "8 or 16 bytes");
    if (vec) {
        if constexpr (W == 4) {
            const uint4 q = *reinterpret_cast<const uint4 *>(x);
            v.w[0] = q.x, v.w[1] = q.y, v.w[2] = q.z, v.w[3] = q.w;
        } else {
            const uint2 q = *reinterpret_cast<const uint2 *>(x);
            v.w[0] = q.x, v.w[1] = q.y;
        }
    } else {
        T t[N];
#pragma unroll
        for (int e = 0; e < N; ++e) t[e] = x[e];
        memcpy(v.w, t, sizeof(t));
    }
}
template <class T, int N>
__device__ __forceinline__ float element(const Some<T, N> &v, int e)
{
    if constexpr (sizeof(T) == 4) return __uint_as_float(v.w[e]);
    else if constexpr (std::is_same<T, __half>::value) return __half2float(__ushort_as_half((unsigned short)(v.w[e / 2] >> (e & 1) * 16)));
    else return __uint_as_float(e & 1 ? v.w[e / 2] & 0xFFFF0000u : v.w[e / 2] << 16);
}
// The larger magnitudes of m and of all words (of halfword pairs: of either),
// as bits; and the largest of those as a value.
template <class T, int N>
__device__ __forceinline__ uint32_t larger(uint32_t m, const Some<T, N> &v)
{
#pragma unroll
    for (uint32_t w : v.w) {
        if constexpr (sizeof(T) == 4) m = max(m, w & 0x7FFFFFFFu);
        else m = __vmaxu2(m, w & 0x7FFF7FFFu);
    }
    return m;
}
template <class T>
__device__ __forceinline__ float largest(uint32_t m)
{
    if constexpr (sizeof(T) == 4) return __uint_as_float(m);
    const uint32_t h = max(m & 0xFFFFu, m >> 16);
    if constexpr (std::is_same<T, __half>::value) return __half2float(__ushort_as_half((unsigned short)h));
    return __uint_as_float(h << 16);
}

struct PrepParams {
    const void *X;
    int64_t ldx, n_x;
    const int32_t *offsets;   // NULL: one group of all rows
    const int32_t *order;
    int32_t per, n_row, n_group;
    int32_t in_dim, nst, order8;   // order8: which inputs a 16-byte unit holds
    int32_t gran_tokens, tile_tokens, cap_tiles, cap_gran, parts, by_row, vec, few, spread;
    ChunkPlan *plan;
    ChunkTile *tiles;
    float *inv;               // by place in the granules
    uint8_t *img;
};

// Rows [a, b) of group g; none when its offsets are not in order.
__device__ __forceinline__ bool group_rows(const PrepParams &p, int g, int &a, int &b)
{
    a = p.offsets ? p.offsets[g] : 0;
    b = p.offsets ? p.offsets[g + 1] : p.n_row;
    const bool ok = a >= 0 && b >= a && b <= p.n_row;
    if (!ok) a = b = 0;
    return ok;
}

// Exclusive prefix sum over the CTA, and the total.
__device__ __forceinline__ int scan_block(int v, int *part, int *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) part[warp] = x;
    __syncthreads();
    int base = 0, sum = 0;
    for (int w = 0; w < kPrepThreads / 32; ++w) {
        if (w < warp) base += part[w];
        sum += part[w];
    }
    __syncthreads();
    *total = sum;
    return base + x - v;
}

__device__ void list_tiles(const PrepParams &p)
{
    const int GT = p.gran_tokens;
    __shared__ int part[kPrepThreads / 32];
    int next = 0;
    for (int g0 = 0; g0 < p.n_group; g0 += kPrepThreads) {
        const int g = g0 + (int)threadIdx.x;
        int a = 0, b = 0;
        if (g < p.n_group && !group_rows(p, g, a, b)) record_status(&g_chunk_invalid, RF_ERR_INVALID_ARG);
        const int n = (b - a + p.tile_tokens - 1) / p.tile_tokens;
        int total;
        const int at = next + scan_block(n, part, &total);
        for (int t = 0; t < n && at + t < p.cap_tiles; ++t) {
            ChunkTile w;
            w.group = g;
            w.row0 = a + t * p.tile_tokens;
            w.cnt = min(p.tile_tokens, b - w.row0);
            w.gran = a / GT + g + t * (p.tile_tokens / GT);
            p.tiles[at + t] = w;
        }
        next += total;
    }
    if (threadIdx.x == 0) {
        p.plan->n_tiles = min(next, p.cap_tiles);   // (more only when groups overlap)
        p.plan->next = 0;
    }
}

// Which inputs the 16-byte units of a 32-input block hold, as the decoders
// of rf_chunk_mma.cu order a block's weights: unit u is made of a =
// inputs 4u.. and b = 16 + 4u.. (kOrderPairs, kOrderSpread), or 8u.. and
// 8u + 4.. (kOrderPlain).
constexpr int kOrderPlain = 0, kOrderPairs = 1, kOrderSpread = 2;
__device__ __forceinline__ void slice_order(int order, const float (&a)[4], const float (&b)[4], float (&f)[8])
{
    if (order == kOrderPairs) {          // MXFP4: the two nibbles of a byte
        f[0] = a[0], f[1] = b[0], f[2] = a[1], f[3] = b[1], f[4] = a[2], f[5] = b[2], f[6] = a[3], f[7] = b[3];
    } else if (order == kOrderSpread) {  // Q4_0: nibbles four apart in a word
        f[0] = a[0], f[1] = a[2], f[2] = b[0], f[3] = b[2], f[4] = a[1], f[5] = a[3], f[6] = b[1], f[7] = b[3];
    } else {
        f[0] = a[0], f[1] = a[1], f[2] = a[2], f[3] = a[3], f[4] = b[0], f[5] = b[1], f[6] = b[2], f[7] = b[3];
    }
}

// FOURS: fours of slices of a row in flight.
template <int DT, int XT, int FOURS>
__global__ void __launch_bounds__(kPrepThreads) prep_kernel(const __grid_constant__ PrepParams p)
{
    using T = typename Elem<DT>::T;
    const int GT = p.gran_tokens, H = max(1, GT / kPrepRows);   // tokens of a granule, CTAs that share it
    if (blockIdx.x == gridDim.x - 1) {
        list_tiles(p);
        return;
    }
    // A CTA's place: a share of a granule; or a row, if it is the first of one
    // (rows fewer than the granules that there might be).
    const int part = blockIdx.x % p.parts, place_of = blockIdx.x / p.parts;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // The first group that has the place: more than one only when offsets
    // decrease, and then what one CTA writes is still one group's.
    __shared__ int s_group, s_row, s_cnt, s_n, s_at, s_gran, s_sub;
    if (tid == 0) s_group = INT32_MAX;
    __syncthreads();
    int mine = INT32_MAX, row = 0, a = 0, b = 0, q = 0;
    for (int g = tid; g < p.n_group && mine == INT32_MAX; g += kPrepThreads) {
        if (!group_rows(p, g, a, b)) continue;
        if (p.by_row) {
            row = place_of;
            q = (row - a) / GT;
            if (row < a || row >= b || (row - a) % min(GT, kPrepRows) != 0) continue;
        } else {
            q = place_of / H - (a / GT + g);
            if (q < 0 || q >= (b - a + GT - 1) / GT) continue;
            row = a + q * GT + place_of % H * kPrepRows;
        }
        mine = g;
    }
    if (mine != INT32_MAX) atomicMin(&s_group, mine);
    __syncthreads();
    if (s_group == INT32_MAX) return;
    if (mine == s_group) {
        const int tt = p.tile_tokens / GT;   // granules per whole tile
        s_gran = a / GT + mine + q;
        s_row = row;
        s_cnt = min(min(kPrepRows, GT), b - row);
        s_at = s_gran - q + q / tt * tt;     // the tile's first granule
        s_n = min(tt, (b - a - q / tt * p.tile_tokens + GT - 1) / GT);
        s_sub = (row - a) % GT / kPrepRows;
    }
    __syncthreads();
    const int gran = s_gran, sub = s_sub;
    // A warp takes a row: its largest value, hence its scale, then its inputs.
    static_assert(kPrepRows == kPrepThreads / 32, "a warp per row");
    int64_t src = -1;
    if (warp < s_cnt) {
        const int row = s_row + warp;
        src = p.order ? p.order[row] / p.per : row;
        if (p.order && (p.order[row] < 0 || src >= p.n_x)) {
            src = -1;
            if (lane == 0) record_status(&g_chunk_invalid, RF_ERR_INVALID_ARG);
        }
    }
    const T *x = static_cast<const T *>(p.X) + (src >= 0 ? src * p.ldx : 0);
    // (fp16 values are operands as they are.)
    float m = 0.f;
    if (!std::is_same<T, __half>::value && src >= 0) {
        constexpr int E = 16 / sizeof(T);
        uint32_t bits = 0;
        // (Eight loads at a time, the last ones too: a loop's remainder would
        // wait for each.)
        for (int k = E * lane; k < p.in_dim; k += 8 * 32 * E) {
            Some<T, E> v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = {};
                if (k + i * 32 * E < p.in_dim) load(x + k + i * 32 * E, p.vec, v[i]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) bits = larger(bits, v[i]);
        }
        m = largest<T>(bits);
        if (!(m < INFINITY)) {   // what is not finite does not count
            m = 0.f;
            for (int k = lane; k < p.in_dim; k += 32) {
                const float f = fabsf((float)x[k]);
                if (f < INFINITY) m = fmaxf(m, f);
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    // The largest value to [2^14, 2^15), by a factor within fp32's normal
    // numbers (so is its inverse).
    const int exponent = (int)(__float_as_uint(m) >> 23) - 127;
    const int k2 = m == 0.f ? 0 : max(-126, min(126, 14 - exponent));
    const float scale = __uint_as_float((uint32_t)(k2 + 127) << 23);
    if (part == 0 && lane == 0 && warp < GT)
        p.inv[(int64_t)gran * GT + sub * kPrepRows + warp] = __uint_as_float((uint32_t)(127 - k2) << 23);

    // Four slices of a row are two loads of four elements a lane.  The unit of
    // a lane is made of its own elements and its neighbour's `with` lanes on
    // (slice_order): the lower one's from the first load, the other's from the
    // second.  In shared memory the eight rows' units of a slice meet, each
    // turned by its place for the banks, and leave as whole lines.
    __shared__ uint4 tile[FOURS * 4 * XT][64];
    const int with = p.order8 == kOrderPlain ? 1 : 4;
    const bool upper = (lane & with) != 0;
    const int place = lane & 7, u = p.order8 == kOrderPlain ? place >> 1 : place & 3;
    const int block = (lane >> 3) + (upper ? 4 : 0), c = 4 * (block & 1) + u;   // of the four slices, and the unit in its slice
    const int bytes = GT * XT * kSliceK * 2, fours = (p.nst + 3) / 4;
    uint8_t *out = p.img + ((int64_t)s_at * p.nst + (gran - s_at)) * bytes + sub * 1024;
    const int64_t step = (int64_t)s_n * bytes;
    for (int q0 = part; q0 < fours; q0 += p.parts * FOURS) {
        Some<T, 4> v[FOURS][2];
#pragma unroll
        for (int i = 0; i < FOURS; ++i)
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int k = 256 * (q0 + i * p.parts) + 128 * n + 4 * lane;
                v[i][n] = {};
                if (src >= 0 && k < p.in_dim) load(x + k, p.vec, v[i][n]);
            }
#pragma unroll
        for (int i = 0; i < FOURS; ++i) {
            Some<T, 4> other;
#pragma unroll
            for (int w = 0; w < (int)sizeof(T); ++w)
                other.w[w] = __shfl_xor_sync(0xffffffffu, upper ? v[i][0].w[w] : v[i][1].w[w], with);
            float a[4], b[4], f[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                a[e] = upper ? element(other, e) : element(v[i][0], e);
                b[e] = upper ? element(v[i][1], e) : element(other, e);
            }
            slice_order(p.order8, a, b, f);
            uint32_t h[4], l[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float f0 = f[2 * e] * scale, f1 = f[2 * e + 1] * scale;
                const __half2 g = __floats2half2_rn(f0, f1);
                h[e] = h2_bits(g);
                if constexpr (XT == 2) {
                    const float2 w = __half22float2(g);
                    l[e] = h2_bits(__floats2half2_rn(fabsf(w.x) < INFINITY ? (f0 - w.x) * 2048.f : 0.f,
                                                     fabsf(w.y) < INFINITY ? (f1 - w.y) * 2048.f : 0.f));
                }
            }
            const int sl = 4 * i + (block >> 1);
            tile[sl * XT][8 * c + (warp ^ c)] = make_uint4(h[0], h[1], h[2], h[3]);
            if constexpr (XT == 2) tile[sl * XT + 1][8 * c + (warp ^ c)] = make_uint4(l[0], l[1], l[2], l[3]);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < FOURS * XT; ++i) {
            const int n = i * kPrepThreads + tid, of = n >> 6, sl = of / XT, term = of % XT, cc = (n >> 3) & 7, r = n & 7;
            const int s = 4 * (q0 + sl / 4 * p.parts) + (sl & 3);
            if (s >= p.nst || r >= GT) continue;
            // Few tokens' kernel reads a row's units of four slices at once (of
            // MXFP4, every other one of eight): they lie one after the other,
            // each slice's turned in its 128 bytes, for the banks.
            const int at = p.spread ? (s & ~7) | (s & 1) << 2 | (s >> 1 & 3) : s;
            const int turn = p.few ? 2 * (at & 3) : 0;
            // (The low terms' rows follow the high ones'.)
            uint8_t *to = out + at * step + cc * 128 + (GT < kPrepRows ? ((term * GT + r) ^ turn) * 16 : term * 1024 + (r ^ turn) * 16);
            *reinterpret_cast<uint4 *>(to) = tile[of][8 * cc + (r ^ cc)];
        }
        __syncthreads();
    }
}

// y_t = residual_t + sum_k w_tk d[place_tk], in selection order; four columns a
// thread.
struct JoinParams {
    const float *d, *w;
    const int32_t *place;
    const void *residual;
    void *Y;
    int64_t ldr, ldy, n_tok, n, ldd;
    int32_t top_k, nb, vec;
};
template <int DT>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ JoinParams p)
{
    using T = typename Elem<DT>::T;
    const int64_t t = blockIdx.x / p.nb;
    const int64_t c = 4 * ((int64_t)(blockIdx.x % p.nb) * 256 + threadIdx.x);
    if (c >= p.n) return;   // (a multiple of 32)
    float y[4] = {0.f, 0.f, 0.f, 0.f};
    for (int k0 = 0; k0 < p.top_k; k0 += 4) {   // (four experts' loads at a time)
        float4 v[4];
        float w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t at = t * p.top_k + k0 + k;
            const bool there = k0 + k < p.top_k;
            w[k] = there ? p.w[at] : 0.f;
            v[k] = there ? *reinterpret_cast<const float4 *>(p.d + (int64_t)p.place[at] * p.ldd + c) : float4{};
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k0 + k >= p.top_k) break;
            y[0] = fmaf(w[k], v[k].x, y[0]), y[1] = fmaf(w[k], v[k].y, y[1]);
            y[2] = fmaf(w[k], v[k].z, y[2]), y[3] = fmaf(w[k], v[k].w, y[3]);
        }
    }
    if (p.residual) {
        float f[4];
        load4(static_cast<const T *>(p.residual) + t * p.ldr + c, p.vec, f);
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] += f[e];
    }
    T o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if constexpr (DT == RF_F32) o[e] = y[e];
        else if constexpr (DT == RF_F16) o[e] = __float2half_rn(y[e]);
        else o[e] = __float2bfloat16_rn(y[e]);
    }
    T *out = static_cast<T *>(p.Y) + t * p.ldy + c;
    if (p.vec) {
        if constexpr (DT == RF_F32) *reinterpret_cast<float4 *>(out) = *reinterpret_cast<float4 *>(o);
        else *reinterpret_cast<uint2 *>(out) = *reinterpret_cast<uint2 *>(o);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) out[e] = o[e];
    }
}

bool fmt_has_chunks(int fmt) { return fmt == RF_Q4_0 || fmt == RF_Q8_0 || fmt == RF_MXFP4 || fmt == RF_Q4_K; }
bool dtype_ok(int d) { return d == RF_F32 || d == RF_F16 || d == RF_BF16; }
// X's and Y's types of a product's dtype (X's, with RF_Y_F32 or without).
int x_dtype(int d) { return d & ~RF_Y_F32; }
int y_dtype(int d) { return (d & RF_Y_F32) != 0 ? RF_F32 : d; }
int dtype_size(int d) { return d == RF_F32 ? 4 : 2; }
size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

// Parts of the rows' inputs.  With fewer items than fill the SMs evenly, an
// item's inputs are shared out, and a second launch adds the parts' sums:
// worth it while it saves a tenth of the SMs' rounds after what that launch,
// the sums' traffic and the items' starts cost.  In SM cycles, as measured: a
// slice's by what bounds it, 4,000 an item (2,500 where two CTAs share the SM),
// 3,500 a launch, 1,500 bytes of sums a cycle.  9 fp32 tokens through
// 2 x 11008 x 4096 Q4_0: 46 us, in one part 60; 8 tokens 36, in one part 43; 77
// through 4099 x 4096 Q4_K 40, in one 60.  An estimate, fitted to such calls
// through one matrix: it takes a round for one CTA an SM also where two share
// it, and the tiles of groups for what the rows of a group on average need.
// (The last part's warps adding the sums in the product's launch instead of a
// second one: 60 us against 55 in the first case, they read them one latency
// after another.)
void choose_parts(ChunkShape &sh, bool gated)
{
    const int64_t tiles = sh.n_group == 1 ? (sh.n_row + sh.tile_tokens() - 1) / sh.tile_tokens()
                                          : std::min(sh.cap_tiles, std::max(sh.n_row / sh.tile_tokens(), std::min(sh.n_group, sh.n_row)));
    const int64_t items = tiles * ((sh.rows + (gated ? 63 : 127)) / (gated ? 64 : 128)), sms = num_sms();
    const int64_t per = chunk_weights(sh.fmt) / kSliceK, nch = (sh.nst + per - 1) / per;
    const int64_t slice = sh.few ? std::max<int64_t>(sh.wt == 2 ? 500 : 375, 128 * (sh.nt == 8 ? sh.wt : (sh.xt + sh.wt - 1) * (sh.tile_tokens() / 8)))
                          : sh.wt == 2 ? (sh.fmt == RF_Q4_K ? 1400 : 1000) : (sh.nt > 128 ? 640 : 420);
    auto cost = [&](int64_t parts) {
        const int64_t slices = std::min<int64_t>((nch + parts - 1) / parts * per, sh.nst);
        const int64_t sums = parts > 1 ? 3500 + parts * (1 + gated) * sh.n_row * sh.rows * 8 / 1500 : 0;
        return (items * parts + sms - 1) / sms * (slice * slices + (sh.few ? 2500 : 4000)) + sums;
    };
    int64_t best = 1;
    if (items < 4 * sms)
        for (int64_t parts = 2; parts <= std::min<int64_t>(nch, kMaxParts); ++parts)
            if (10 * cost(parts) < 9 * cost(1) && cost(parts) < cost(best) &&
                parts * (1 + gated) * sh.n_row * sh.rows <= kMaxSums)
                best = parts;
    sh.part_chunks = (int)((nch + best - 1) / best);
    sh.parts = (int)((nch + sh.part_chunks - 1) / sh.part_chunks);
}

// Slices after which a 16-bit call's sums leave the tensor cores for a rounded
// addition.  The tensor cores truncate theirs, always towards zero, so that a
// sum of one sign drifts with its length: 2^20 inputs in one go end 6.9e-3 low
// (fourteen times half a step of fp16), 16,384 1.2e-4, 4,096 3e-5.  bf16 outputs
// do not see 1.2e-4; what is rounded more finely leaves sooner.
constexpr int kSegment = 64, kSegmentBf16 = 256;

// The operands of a product of n_row rows shared by n_group groups.  Tiles of
// 192 operand rows where the groups fill them (a weight slice is decoded once
// per tile), of 128 where they do not; both let tensor memory hold two items'
// sums, so that an epilogue runs beside the next item's products.  (Tiles of 160
// rows, which fill the last round of 2048 tokens through 4096 x 11008 better,
// take 214 us against 182.)  Tiles of up to 16 operand rows multiply from
// registers (rf_chunk_few.cu), us against the way through tensor memory: 8 bf16
// tokens through 2 x 11008 x 4096 Q4_0 28 against 41, 16 32 against 41; 4 fp32
// tokens 32 against 45, 8 35 against 46; 77 bf16 tokens through 128 MXFP4
// experts of 2880 314 against 372, 128 396 against 422, 128 fp32 tokens 471
// against 484.  Two terms of weights for 16 rows are the exceptions (fp16 tokens:
// Q4_0 45 against 43, Q4_K 79 against 61), and groups well below 16 rows that
// come in tiles of 16 (256 bf16 tokens through the experts 511 against 482).
// Two such tiles instead of one of 32 rows: 32 bf16 tokens 47 against 43, 32 fp16
// 63 against 47, 16 fp32 60 against 46.
ChunkShape chunk_shape(int fmt, int dtype, int64_t n_group, int64_t rows, int64_t in_dim, int64_t n_row, bool gated)
{
    ChunkShape sh;
    sh.fmt = fmt;
    sh.xt = x_dtype(dtype) == RF_F32 ? 2 : 1;
    // bf16 outputs: a weight's rounding to fp16 is an eighth of half a step.  2048
    // tokens through 2 x 11008 x 4096 Q4_0 end 1.68e-3 from 64 bits (their own
    // rounding: 1.66e-3) in 274 us; two terms take 472.  Of an fp32 output it
    // would be most of the error.
    sh.wt = dtype != RF_BF16 && fmt != RF_MXFP4 ? 2 : 1;
    sh.n_row = n_row, sh.n_group = n_group, sh.rows = rows, sh.in_dim = in_dim;
    sh.nst = (int)((in_dim + kSliceK - 1) / kSliceK);
    // Operand rows of a group: twice the average, so that most groups have one tile.
    const int64_t each = n_group == 1 ? sh.xt * n_row : 2 * sh.xt * ((n_row + n_group - 1) / n_group);
    sh.nt = each <= 8 ? 8 : each <= 16 ? 16 : each <= 32 ? 32 : each <= 64 ? 64 : sh.wt == 1 && sh.xt == 1 && each > 256 ? 192 : 128;
    sh.few = sh.nt <= 16;
    const int per = chunk_weights(fmt) / kSliceK;
    if (sh.few) sh.nst = (sh.nst + per - 1) / per * per;
    const int64_t T = sh.tile_tokens(), GT = sh.gran_tokens();
    sh.cap_tiles = std::min<int64_t>(n_row, n_row / T + n_group);
    sh.cap_gran = n_row / GT + n_group;
    choose_parts(sh, gated);
    sh.segment = dtype == RF_BF16 ? kSegmentBf16 : kSegment;
    sh.segments = sh.xt == 1 && std::min(sh.nst, sh.part_chunks * per) > sh.segment;
    // Every region's size grows with the rows, whatever tile they take (images
    // of whole chunks as few rows have them, tiles as of four tokens).
    const int64_t nch = (sh.nst + per - 1) / per;
    size_t at = sizeof(ChunkPlan);
    sh.at_tiles = at, at = up256(at + (size_t)(n_row / 4 + n_group) * sizeof(ChunkTile));
    sh.at_inv = at, at = up256(at + (size_t)sh.cap_gran * GT * sizeof(float));
    sh.at_img = at, at = up256(at + (size_t)sh.cap_gran * nch * per * sh.gran_bytes());
    // Parts are for calls of few items, hence of fewer rows than n_part; all of
    // them take segments that whole rows of a call may take.
    const int64_t nrt = (rows + (gated ? 63 : 127)) / (gated ? 64 : 128), few_items = 4 * num_sms();
    const int64_t n_part = nrt > 0 && nrt < few_items ? std::min(n_row, T * (few_items / nrt + 1)) : 0;
    const int64_t sums = std::min(kMaxSums, std::min(nch, kMaxParts) * (1 + gated) * n_part * rows);
    const bool held = sh.xt == 1 && !sh.few && sh.nst > sh.segment;
    sh.upto = up256(at + (size_t)sums * sizeof(float)) + (held ? up256((size_t)num_sms() * sh.nt * 128 * sizeof(float)) : 0);
    sh.at_sums = at;
    if (sh.parts > 1) at = up256(at + (size_t)sh.parts * (1 + gated) * n_row * rows * sizeof(float));
    sh.at_held = at;
    if (sh.segments && !sh.few) at = up256(at + (size_t)num_sms() * sh.nt * 128 * sizeof(float));
    sh.bytes = at;
    return sh;
}

// Sizes that a product takes, for the entry points and the workspace.
rf_status check_sizes(int fmt, int dtype, int64_t n_group, int64_t rows, int64_t in_dim, int64_t n_row)
{
    if (!fmt_has_chunks(fmt) || !dtype_ok(x_dtype(dtype))) return RF_ERR_UNSUPPORTED_FMT;
    if (n_group < 1 || rows < 0 || n_row < 0 || in_dim <= 0 || in_dim % block_elems_of(fmt) != 0) return RF_ERR_INVALID_ARG;
    if (in_dim > (1 << 20) || rows > 0x7fffffffLL || n_group > 65536 || n_row > kMaxPieces) return RF_ERR_TOO_LARGE;
    for (const bool gated : {false, true}) {
        const ChunkShape sh = chunk_shape(fmt, dtype, n_group, rows, in_dim, n_row, gated);
        if (sh.cap_gran > kMaxPieces || sh.cap_tiles * ((rows + 63) / 64) > kMaxPieces) return RF_ERR_TOO_LARGE;
    }
    return RF_OK;
}

bool gated_act(int act) { return act == RF_ACT_SWIGLU || act == RF_ACT_SWIGLU_CLAMPED; }

rf_status check_epilogue(const rf_epilogue &e, const void *up, int64_t rows)
{
    if (e.act < RF_ACT_NONE || e.act > RF_ACT_SWIGLU_CLAMPED || e.reserved != 0) return RF_ERR_INVALID_ARG;
    if (gated_act(e.act) != (up != nullptr) || (e.up_bias && !up)) return RF_ERR_INVALID_ARG;
    if (e.act == RF_ACT_SWIGLU_CLAMPED && (!(e.alpha > -INFINITY && e.alpha < INFINITY) || !(e.limit > 0.f)))
        return RF_ERR_INVALID_ARG;
    if (e.residual && e.ld_residual < rows) return RF_ERR_INVALID_ARG;
    return RF_OK;
}
bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

struct Source {
    int dtype;
    const void *X;
    int64_t ldx, n_x;
    const int32_t *offsets, *order;
    int per;
};

template <int DT, int XT>
rf_status launch_prep_t(const PrepParams &p, int64_t blocks, cudaStream_t s)
{
    if ((p.nst + 3) / 4 <= p.parts) prep_kernel<DT, XT, 1><<<(unsigned)(blocks + 1), kPrepThreads, 0, s>>>(p);
    else prep_kernel<DT, XT, 4><<<(unsigned)(blocks + 1), kPrepThreads, 0, s>>>(p);
    return last_cuda_error();
}

// The token tiles and the images of one product's rows.
rf_status launch_prep(const ChunkShape &sh, const Source &x, uint8_t *ws, cudaStream_t s)
{
    PrepParams p;
    p.X = x.X, p.ldx = x.ldx, p.n_x = x.n_x;
    p.offsets = x.offsets, p.order = x.order, p.per = x.per;
    p.n_row = (int32_t)sh.n_row, p.n_group = (int32_t)sh.n_group;
    p.in_dim = (int32_t)sh.in_dim, p.nst = sh.nst;
    p.order8 = sh.fmt == RF_MXFP4 ? kOrderPairs : (sh.fmt == RF_Q4_0 ? kOrderSpread : kOrderPlain);
    p.gran_tokens = sh.gran_tokens();
    p.tile_tokens = sh.tile_tokens();
    p.few = sh.few;
    p.spread = sh.few && sh.fmt == RF_MXFP4;
    p.cap_tiles = (int32_t)sh.cap_tiles, p.cap_gran = (int32_t)sh.cap_gran;
    const int size = dtype_size(x.dtype);
    p.vec = aligned(x.X, 16) && (x.ldx * size) % 16 == 0;
    p.plan = reinterpret_cast<ChunkPlan *>(ws);
    p.tiles = reinterpret_cast<ChunkTile *>(ws + sh.at_tiles);
    p.inv = reinterpret_cast<float *>(ws + sh.at_inv);
    p.img = ws + sh.at_img;
    // Rows' slices are shared out among CTAs while there are few rows (each
    // finds its rows' maxima again).
    const int64_t share = std::max(1, sh.gran_tokens() / kPrepRows);
    const int64_t busy = std::min<int64_t>(sh.cap_gran * share, sh.n_row);   // CTAs with rows, at most
    p.parts = (int32_t)std::max<int64_t>(1, std::min<int64_t>((sh.nst + 3) / 4, 4 * num_sms() / std::max<int64_t>(1, busy)));
    p.by_row = sh.n_row < sh.cap_gran * share;
    const int64_t blocks = busy * p.parts;
    if (blocks > 0x7ffffffeLL) return RF_ERR_TOO_LARGE;
    if (x.dtype == RF_F32)
        return sh.xt == 2 ? launch_prep_t<RF_F32, 2>(p, blocks, s) : launch_prep_t<RF_F32, 1>(p, blocks, s);
    return x.dtype == RF_F16 ? launch_prep_t<RF_F16, 1>(p, blocks, s) : launch_prep_t<RF_BF16, 1>(p, blocks, s);
}

// Prepared and multiplied.  `total_rows`: rows of the weight tensors.
rf_status run_product(const ChunkShape &sh, const Source &x, const void *W, const void *up, int64_t row0, int64_t group_rows,
                      int64_t total_rows, const rf_epilogue &epi, int dtype, void *Y, int64_t ldy, void *ws, cudaStream_t s)
{
    rf_status st = launch_prep(sh, x, static_cast<uint8_t *>(ws), s);
    if (st != RF_OK) return st;
    ChunkGemm g;
    g.sh = sh;
    g.W = static_cast<const uint8_t *>(W);
    g.up = static_cast<const uint8_t *>(up);
    g.row0 = row0, g.group_rows = group_rows, g.total_rows = total_rows;
    g.epi = epi;
    g.dtype = dtype;
    g.Y = Y, g.ldy = ldy;
    g.ws = static_cast<uint8_t *>(ws);
    return launch_chunk_mma(g, s);
}

rf_status check_workspace(const void *ws, size_t have, size_t need)
{
    if (need == 0) return RF_OK;
    if (!ws || have < need) return RF_ERR_INVALID_ARG;
    return aligned(ws, 256) ? RF_OK : RF_ERR_MISALIGNED;
}

const rf_epilogue kNoEpilogue = {nullptr, nullptr, nullptr, 0, RF_ACT_NONE, 0.f, 0.f, 0};

// The routed FFN's workspace.
struct MoeLayout {
    ChunkShape up, down;
    size_t at_idx, at_w, at_offsets, at_order, at_place, at_route, at_product, at_h, bytes;
    int64_t ldd;   // row stride of the experts' outputs
};
MoeLayout moe_layout(int fmt, int n_expert, int top_k, int64_t n_ff, int64_t n_embd, int dtype, int64_t n_tok, bool upto = false)
{
    MoeLayout m;
    const int64_t n_row = n_tok * top_k;
    m.up = chunk_shape(fmt, dtype, n_expert, n_ff, n_embd, n_row, true);
    // fp16 calls take h as two fp16 terms: rounded once it put outputs 12 % further
    // from 64 bits (2.32e-4 against 2.08e-4, their own rounding; in some calls 50 %)
    // in 227 instead of 267 us (500 tokens, top-4 of 32 MXFP4 experts of 2880).  In
    // bf16 calls that rounding is an eighth of half a step (1.664e-3 against
    // 1.661e-3), and two terms would cost 913 us instead of 745 (2048 tokens
    // through 128 such experts).
    m.down = chunk_shape(fmt, dtype == RF_F16 ? RF_F32 : dtype, n_expert, n_embd, n_ff, n_row, false);
    m.ldd = n_embd;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t here = at;
        at = up256(at + n);
        return here;
    };
    m.at_idx = take(4 * n_row), m.at_w = take(4 * n_row), m.at_offsets = take(4 * ((size_t)n_expert + 1));
    m.at_order = take(4 * n_row), m.at_place = take(4 * n_row);
    m.at_route = take(route_workspace(n_tok, n_expert, top_k));
    // (upto: for this call and every one of fewer tokens.)
    m.at_product = take(upto ? std::max(m.up.upto, m.down.upto) : std::max(m.up.bytes, m.down.bytes));   // the second product prepares after the first has run
    m.at_h = take(4 * (size_t)n_row * std::max(n_ff, n_embd)); // h, read before the experts' outputs are written
    m.bytes = at;
    return m;
}

rf_status check_route(int dtype, const void *logits, int64_t ld, int64_t n_tok, int n_expert, int top_k)
{
    if (!dtype_ok(dtype)) return RF_ERR_UNSUPPORTED_FMT;
    if (n_expert < 1 || n_expert > 1024 || top_k < 1 || top_k > 8 || top_k > n_expert || n_tok < 0 || ld < n_expert ||
        (!logits && n_tok > 0))
        return RF_ERR_INVALID_ARG;
    if (!aligned(logits, dtype_size(dtype))) return RF_ERR_MISALIGNED;
    if (n_tok > kMaxPieces / top_k) return RF_ERR_TOO_LARGE;
    return RF_OK;
}

}  // namespace

rf_status read_and_clear_chunk_invalid()
{
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_chunk_invalid, sizeof(int)) != cudaSuccess) return RF_ERR_CUDA;
    if (v != 0) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(g_chunk_invalid, &zero, sizeof(int)) != cudaSuccess) return RF_ERR_CUDA;
    }
    return static_cast<rf_status>(v);
}

}  // namespace rf

using namespace rf;

extern "C" {

size_t rf_gemm_grouped_workspace_bytes(int fmt, int n_group, int64_t rows, int64_t in_dim, int dtype, int64_t n_row)
{
    if (check_sizes(fmt, dtype, n_group, rows, in_dim, n_row) != RF_OK || rows == 0 || n_row == 0) return 0;
    return std::max(chunk_shape(fmt, dtype, n_group, rows, in_dim, n_row, false).upto,
                    chunk_shape(fmt, dtype, n_group, rows, in_dim, n_row, true).upto);
}

size_t rf_gemm_fused_workspace_bytes(int fmt, int64_t rows, int64_t in_dim, int dtype, int64_t n_tok)
{
    return rf_gemm_grouped_workspace_bytes(fmt, 1, rows, in_dim, dtype, n_tok);
}

rf_status rf_gemm_fused(int fmt, const void *W, const void *up, int64_t row_start, int64_t row_end, int64_t in_dim, int dtype,
                        int64_t n_tok, const void *X, int64_t ldx, const rf_epilogue *epi, void *Y, int64_t ldy,
                        void *workspace, size_t workspace_bytes, void *stream)
{
    const rf_epilogue e = epi ? *epi : kNoEpilogue;
    const int64_t rows = row_end - row_start;
    if (row_start < 0 || row_end < row_start) return RF_ERR_INVALID_ARG;
    rf_status st = check_sizes(fmt, dtype, 1, rows, in_dim, n_tok);
    if (st != RF_OK) return st;
    if (!W || (n_tok > 0 && rows > 0 && (!X || !Y)) || ldx < in_dim || ldy < rows) return RF_ERR_INVALID_ARG;
    if ((st = check_epilogue(e, up, rows)) != RF_OK) return st;
    const int size = dtype_size(x_dtype(dtype)), size_y = dtype_size(y_dtype(dtype));
    if (!aligned(W, 16) || !aligned(up, 16) || !aligned(X, size) || !aligned(Y, size_y) || !aligned(e.residual, size_y) ||
        !aligned(e.bias, 4) || !aligned(e.up_bias, 4))
        return RF_ERR_MISALIGNED;
    if (rows == 0 || n_tok == 0) return RF_OK;
    const ChunkShape sh = chunk_shape(fmt, dtype, 1, rows, in_dim, n_tok, up != nullptr);
    if ((st = check_workspace(workspace, workspace_bytes, sh.bytes)) != RF_OK) return st;
    const Source x = {x_dtype(dtype), X, ldx, n_tok, nullptr, nullptr, 1};
    return run_product(sh, x, W, up, row_start, rows, row_end, e, y_dtype(dtype), Y, ldy, workspace, static_cast<cudaStream_t>(stream));
}

rf_status rf_gemm_grouped(int fmt, const void *W, const void *up, int n_group, int64_t rows, int64_t in_dim, int dtype,
                          const void *X, int64_t ldx, int64_t n_x, const int32_t *offsets, const int32_t *order, int per,
                          int64_t n_row, const rf_epilogue *epi, void *Y, int64_t ldy, void *workspace,
                          size_t workspace_bytes, void *stream)
{
    const rf_epilogue e = epi ? *epi : kNoEpilogue;
    rf_status st = check_sizes(fmt, dtype, n_group, rows, in_dim, n_row);
    if (st != RF_OK) return st;
    if (!W || !offsets || (n_row > 0 && rows > 0 && !Y) || (n_x > 0 && !X) || n_x < 0 || ldx < in_dim || ldy < rows || per < 1 ||
        (!order && n_x < n_row))
        return RF_ERR_INVALID_ARG;
    if ((st = check_epilogue(e, up, rows)) != RF_OK) return st;
    const int size = dtype_size(x_dtype(dtype)), size_y = dtype_size(y_dtype(dtype));
    if (!aligned(W, 16) || !aligned(up, 16) || !aligned(X, size) || !aligned(Y, size_y) || !aligned(e.residual, size_y) ||
        !aligned(e.bias, 4) || !aligned(e.up_bias, 4) || !aligned(offsets, 4) || !aligned(order, 4))
        return RF_ERR_MISALIGNED;
    if (rows == 0 || n_row == 0) return RF_OK;
    const ChunkShape sh = chunk_shape(fmt, dtype, n_group, rows, in_dim, n_row, up != nullptr);
    if ((st = check_workspace(workspace, workspace_bytes, sh.bytes)) != RF_OK) return st;
    const Source x = {x_dtype(dtype), X, ldx, n_x, offsets, order, per};
    return run_product(sh, x, W, up, 0, rows, (int64_t)n_group * rows, e, y_dtype(dtype), Y, ldy, workspace,
                       static_cast<cudaStream_t>(stream));
}

size_t rf_moe_route_tokens_workspace_bytes(int64_t n_tok, int n_expert, int top_k)
{
    if (n_tok <= 0 || n_expert < 1 || n_expert > 1024 || top_k < 1 || top_k > 8 || top_k > n_expert ||
        n_tok > kMaxPieces / top_k)
        return 0;
    return route_workspace(n_tok, n_expert, top_k);
}

rf_status rf_moe_route_tokens(int dtype, const void *logits, int64_t ld, int64_t n_tok, int n_expert, int top_k, int32_t *idx,
                              float *w, int32_t *offsets, int32_t *order, int32_t *place, void *workspace,
                              size_t workspace_bytes, void *stream)
{
    rf_status st = check_route(dtype, logits, ld, n_tok, n_expert, top_k);
    if (st != RF_OK) return st;
    if (!offsets || (n_tok > 0 && (!idx || !w || !order || !place))) return RF_ERR_INVALID_ARG;
    if (!aligned(idx, 4) || !aligned(w, 4) || !aligned(offsets, 4) || !aligned(order, 4) || !aligned(place, 4))
        return RF_ERR_MISALIGNED;
    if ((st = check_workspace(workspace, workspace_bytes, n_tok > 0 ? route_workspace(n_tok, n_expert, top_k) : 0)) != RF_OK)
        return st;
    return launch_route_tokens(dtype, logits, ld, n_tok, n_expert, top_k, idx, w, offsets, order, place, workspace,
                               static_cast<cudaStream_t>(stream));
}

size_t rf_moe_tokens_workspace_bytes(int fmt, int n_expert, int top_k, int64_t n_ff, int64_t n_embd, int dtype, int64_t n_tok)
{
    if (n_tok <= 0 || n_expert < 1 || n_expert > 1024 || top_k < 1 || top_k > 8 || top_k > n_expert ||
        n_tok > kMaxPieces / top_k || n_ff <= 0 || n_embd <= 0 || !dtype_ok(dtype))
        return 0;
    if (check_sizes(fmt, dtype, n_expert, n_ff, n_embd, n_tok * top_k) != RF_OK ||
        check_sizes(fmt, dtype, n_expert, n_embd, n_ff, n_tok * top_k) != RF_OK)
        return 0;
    return moe_layout(fmt, n_expert, top_k, n_ff, n_embd, dtype, n_tok, true).bytes;
}

rf_status rf_moe_ffn_tokens(int fmt, int dtype, int logits_dtype, const void *logits, int64_t ld_logits, int n_expert,
                            int top_k, int64_t n_tok, const void *gate, const void *up, const void *down,
                            const float *gate_bias, const float *up_bias, const float *down_bias, int act, float alpha,
                            float limit, int64_t n_ff, int64_t n_embd, const void *X, int64_t ldx, const void *residual,
                            int64_t ld_residual, void *Y, int64_t ldy, void *workspace, size_t workspace_bytes, void *stream)
{
    rf_status st = check_route(logits_dtype, logits, ld_logits, n_tok, n_expert, top_k);
    if (st != RF_OK) return st;
    if (n_ff <= 0 || n_embd <= 0) return RF_ERR_INVALID_ARG;
    if (!dtype_ok(dtype)) return RF_ERR_UNSUPPORTED_FMT;
    if ((st = check_sizes(fmt, dtype, n_expert, n_ff, n_embd, n_tok * top_k)) != RF_OK ||
        (st = check_sizes(fmt, dtype, n_expert, n_embd, n_ff, n_tok * top_k)) != RF_OK)
        return st;
    if (!gate || !up || !down || (n_tok > 0 && (!X || !Y)) || ldx < n_embd || ldy < n_embd ||
        (residual && ld_residual < n_embd) || !gated_act(act))
        return RF_ERR_INVALID_ARG;
    const rf_epilogue first = {gate_bias, up_bias, nullptr, 0, act, alpha, limit, 0};
    if ((st = check_epilogue(first, up, n_ff)) != RF_OK) return st;
    const int size = dtype_size(dtype);
    if (!aligned(gate, 16) || !aligned(up, 16) || !aligned(down, 16) || !aligned(X, size) || !aligned(Y, size) ||
        !aligned(residual, size) || !aligned(gate_bias, 4) || !aligned(up_bias, 4) || !aligned(down_bias, 4))
        return RF_ERR_MISALIGNED;
    if (n_tok == 0) return RF_OK;
    const int64_t nb = (n_embd / 4 + 255) / 256;
    if (n_tok * nb > 0x7fffffffLL) return RF_ERR_TOO_LARGE;
    const MoeLayout m = moe_layout(fmt, n_expert, top_k, n_ff, n_embd, dtype, n_tok);
    if ((st = check_workspace(workspace, workspace_bytes, m.bytes)) != RF_OK) return st;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int32_t *idx = reinterpret_cast<int32_t *>(ws + m.at_idx), *offsets = reinterpret_cast<int32_t *>(ws + m.at_offsets);
    int32_t *order = reinterpret_cast<int32_t *>(ws + m.at_order), *place = reinterpret_cast<int32_t *>(ws + m.at_place);
    float *w = reinterpret_cast<float *>(ws + m.at_w), *h = reinterpret_cast<float *>(ws + m.at_h);
    st = launch_route_tokens(logits_dtype, logits, ld_logits, n_tok, n_expert, top_k, idx, w, offsets, order, place,
                             ws + m.at_route, s);
    if (st != RF_OK) return st;
    const int64_t n_row = n_tok * top_k;
    const Source x = {dtype, X, ldx, n_tok, offsets, order, top_k};
    st = run_product(m.up, x, gate, up, 0, n_ff, n_expert * n_ff, first, RF_F32, h, n_ff, ws + m.at_product, s);
    if (st != RF_OK) return st;
    const Source hs = {RF_F32, h, n_ff, n_row, offsets, nullptr, 1};
    rf_epilogue second = kNoEpilogue;
    second.bias = down_bias;
    st = run_product(m.down, hs, down, nullptr, 0, n_embd, n_expert * n_embd, second, RF_F32, h, m.ldd, ws + m.at_product, s);
    if (st != RF_OK) return st;
    JoinParams j;
    j.d = h, j.w = w, j.place = place;
    j.residual = residual, j.Y = Y;
    j.ldr = ld_residual, j.ldy = ldy, j.n_tok = n_tok, j.n = n_embd, j.ldd = m.ldd;
    j.top_k = top_k, j.nb = (int32_t)nb;
    j.vec = aligned(Y, 4 * size) && ldy % 4 == 0 && (!residual || (aligned(residual, 4 * size) && ld_residual % 4 == 0));
    const unsigned grid = (unsigned)(n_tok * nb);
    if (dtype == RF_F32) join_kernel<RF_F32><<<grid, 256, 0, s>>>(j);
    else if (dtype == RF_F16) join_kernel<RF_F16><<<grid, 256, 0, s>>>(j);
    else join_kernel<RF_BF16><<<grid, 256, 0, s>>>(j);
    return last_cuda_error();
}

}  // extern "C"
