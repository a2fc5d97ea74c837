// rf_kv.cu -- the paged KV cache of 8-bit codes: appending keys and values
// with the position rotation applied on the way (and rotating the queries in
// the same launch), and reading values back.
//
// One power-of-two scale per 32 tokens of a head.  A power of two makes every
// held value exact in fp32 (and in fp16 products of the attention kernels),
// and lets a block grow its scale by re-rounding held codes (a right shift to
// nearest even) without the original values.  Each of the 31 later tokens may
// make it grow, by 80 doublings in all; a re-rounding errs by at most half its
// new unit and units at least double, so the errors of a value, its first
// rounding among them, sum to less than one unit of the last scale.
//
// The rotation rounds each product and the sum on its own, so that the codes
// do not depend on how a compiler contracts them.
//
// Bound: HBM bytes for a prompt (q, k, v read once, codes and rotated q
// written once); for one token the chain launch - position - page - load -
// reduce - store.  A CTA owns the K or the V block of one head, with at most
// 32 values per thread (16 up to head_dim 128) in registers between the
// maximum and the rounding: the chain of dependent reads is long, so many
// small CTAs per SM hide it better than fewer with more values a thread.
// Other CTAs of the same grid rotate the queries.
// Measured: 8192 tokens of 32 query and 8 K/V heads of 128, fp32: 61 us
// (5.8 TB/s of the 356 MB it cannot do without, 0.86 of the measured copy
// rate); one token of 64 and 8 heads of 64: 5 us.  Reading back 8237 tokens
// of 8 heads of 128: 15 us (5.6 TB/s).
#include <algorithm>

#include "rf_kv.cuh"

namespace rf {
namespace {

__device__ int g_kv_status = 0;   // positions or pages that do not exist (read by rf_device_status)

constexpr int kAppendThreads = 256;
constexpr int kReadTokens = 8;    // tokens per CTA of the read kernel, at most
constexpr int kQHeads = 4;        // query heads per CTA of the rotation part

struct AppendParams {
    rf_kv_cache c;
    rf_kv_batch b;
    const void *k, *v, *q;
    void *q_out;
    int64_t k_lt, k_lh, v_lt, v_lh, q_lt, q_lh, qo_lt, qo_lh;
    const float *cos_tab, *sin_tab;
    int64_t n_pos;
    int n_heads, rot, style, chunk;
    unsigned parts;          // CTAs per chunk
    bool k_vec, v_vec, q_vec, qo_vec;
};

// Unit u of a head: two runs of four elements, at a and b.  In the rotated
// part the runs hold the pairs' members (half style: b = a + rot/2; pairs
// style: both are neighbouring pairs); beyond it they are neighbours.
struct Unit {
    int a, b, i;     // i: the first of the four rotation pairs, or -1
};
__device__ __forceinline__ Unit unit_at(int u, int rot, int style)
{
    if (8 * u >= rot || style == RF_ROPE_PAIRS) return Unit{8 * u, 8 * u + 4, 8 * u < rot ? 4 * u : -1};
    return Unit{4 * u, rot / 2 + 4 * u, 4 * u};
}

__device__ __forceinline__ void rotate_unit(float (&x)[4], float (&y)[4], const Unit &un, int style,
                                            const float *__restrict__ ct, const float *__restrict__ st)
{
    if (un.i < 0) return;
    const float4 c4 = __ldg(reinterpret_cast<const float4 *>(ct + un.i));
    const float4 s4 = __ldg(reinterpret_cast<const float4 *>(st + un.i));
    const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
    auto turn = [](float &a, float &b, float cc, float ss) {
        const float na = __fsub_rn(__fmul_rn(a, cc), __fmul_rn(b, ss));
        b = __fadd_rn(__fmul_rn(b, cc), __fmul_rn(a, ss));
        a = na;
    };
    if (style == RF_ROPE_HALF) {
#pragma unroll
        for (int m = 0; m < 4; ++m) turn(x[m], y[m], c[m], s[m]);
    } else {
        turn(x[0], x[1], c[0], s[0]);
        turn(x[2], x[3], c[1], s[1]);
        turn(y[0], y[1], c[2], s[2]);
        turn(y[2], y[3], c[3], s[3]);
    }
}

// The smallest scale byte whose unit keeps amax within 127 codes:
// amax = m 2^e with 1 <= m < 2 needs 2^(e-6) if m <= 127/64, else 2^(e-5).
// A NaN or infinite amax, or one above the range, gives kScaleNan.
__device__ __forceinline__ int scale_for(uint32_t amax_bits)
{
    const int E = (int)(amax_bits >> 23) - 6 + ((amax_bits & 0x7fffffu) > 0x7e0000u ? 1 : 0);
    return E > kScaleMax ? kScaleNan : E < kScaleMin ? kScaleMin : E;
}

// One block of one head, K or V, by the CTA.  UPT: units per thread.
template <typename T, int UPT>
__device__ __forceinline__ void append_block(const AppendParams &p, int half, int head, int t0, int n,
                                             int page, int64_t pos, uint32_t *s_max)
{
    const int tid = (int)threadIdx.x;
    // Unit tid % upr of tokens tid / upr, + per, + 2 per, ... (threads that
    // are left over idle).
    const int D = p.c.head_dim, upr = D / 8, per = kAppendThreads / upr;
    const int j0 = tid / upr, j1 = j0 < per ? n : 0;
    const int in_page = (int)(pos & (p.c.page_size - 1));
    const int r = in_page & (kKvBlock - 1);            // tokens of the block held before
    const T *src = static_cast<const T *>(half ? p.v : p.k) + head * (half ? p.v_lh : p.k_lh);
    const int64_t lt = half ? p.v_lt : p.k_lt;
    const bool vec = half ? p.v_vec : p.k_vec;
    const int rot = half ? 0 : p.rot;
    const int64_t ph = (int64_t)page * p.c.n_kv_heads + head;
    int8_t *codes = (half ? p.c.v : p.c.k) + (ph * p.c.page_size + (in_page - r)) * D;
    uint8_t *scale = (half ? p.c.v_scale : p.c.k_scale) + ph * (p.c.page_size / kKvBlock) + in_page / kKvBlock;
    const int E_old = r > 0 ? *scale : 0;

    const Unit un = unit_at(tid - j0 * upr, rot, p.style);
    float x[UPT][4], y[UPT][4];
    uint32_t amax = 0;
#pragma unroll
    for (int k = 0; k < UPT; ++k) {
        const int j = j0 + k * per;                    // token of the call's part of the block
        if (j < j1) {
            const T *row = src + (int64_t)(t0 + j) * lt;
            load4<T>(row + un.a, vec, x[k]);
            load4<T>(row + un.b, vec, y[k]);
            if (rot) {
                const int64_t at = (pos + j) * (rot / 2);
                rotate_unit(x[k], y[k], un, p.style, p.cos_tab + at, p.sin_tab + at);
            }
            // Magnitudes as bits: a NaN is above infinity, so no value hides one.
#pragma unroll
            for (int m = 0; m < 4; ++m)
                amax = max(amax, max(__float_as_uint(x[k][m]) & 0x7fffffffu, __float_as_uint(y[k][m]) & 0x7fffffffu));
        }
    }
    amax = __reduce_max_sync(0xffffffffu, amax);
    if ((tid & 31) == 0) s_max[tid >> 5] = amax;
    __syncthreads();
    amax = __reduce_max_sync(0xffffffffu, s_max[tid & 7]);
    int E = scale_for(amax);
    if (r > 0) E = max(E, E_old);                      // kScaleNan stays
    if (E != kScaleNan) {
        const float inv = __uint_as_float((uint32_t)(254 - E) << 23);   // 2^(127-E)
        auto code = [inv](float v) { return (uint32_t)__float2int_rn(v * inv) & 0xffu; };
        auto word = [&](const float (&f)[4]) {
            return code(f[0]) | code(f[1]) << 8 | code(f[2]) << 16 | code(f[3]) << 24;
        };
#pragma unroll
        for (int k = 0; k < UPT; ++k) {
            const int j = j0 + k * per;
            if (j < j1) {
                int8_t *row = codes + (int64_t)(r + j) * D;
                *reinterpret_cast<uint32_t *>(row + un.a) = word(x[k]);
                *reinterpret_cast<uint32_t *>(row + un.b) = word(y[k]);
            }
        }
        if (r > 0 && E > E_old) {
            // Held codes in the larger unit; |code| <= 128 and the factor is
            // 2^-1 at most, so the product is exact before rint.
            const float f = E_old == 0 || E - E_old > 100 ? 0.f : __uint_as_float((uint32_t)(127 + E_old - E) << 23);
            for (int w = tid; w < r * D / 4; w += kAppendThreads) {
                const uint32_t old = reinterpret_cast<const uint32_t *>(codes)[w];
                uint32_t now = 0;
#pragma unroll
                for (int m = 0; m < 4; ++m)
                    now |= ((uint32_t)__float2int_rn((float)(int8_t)(old >> (8 * m)) * f) & 0xffu) << (8 * m);
                reinterpret_cast<uint32_t *>(codes)[w] = now;
            }
        }
    }
    if (tid == 0) *scale = (uint8_t)E;
    __syncthreads();                                   // s_max is used again
}

// grid: chunks of p.chunk tokens x (K and V of each head, then groups of
// kQHeads query heads), the heads of a chunk next to one another: they share
// its rows and tables, and the light K and V CTAs run beside the queries'.  The K/V part of a chunk handles the blocks whose
// first token of this call lies in the chunk (a block starts at a position
// that is a multiple of 32, or at its sequence's first token of the call).
template <typename T, int UPT>
__global__ void __launch_bounds__(kAppendThreads, UPT <= 2 ? 6 : 3) append_kernel(const __grid_constant__ AppendParams p)
{
    __shared__ uint32_t s_max[8];
    __shared__ int s_pos[32], s_n[32], s_page[32];
    const int tid = threadIdx.x;
    const int part = (int)(blockIdx.x % p.parts);
    const int t_lo = (int)(blockIdx.x / p.parts) * p.chunk, t_n = min(p.chunk, p.b.n_tok - t_lo);
    const bool kv_part = part < 2 * p.c.n_kv_heads;
    pdl_launch_dependents();
    pdl_wait();
    // One thread per token of the chunk: its position, whether it has one,
    // and (K/V part) whether it opens a block and how many tokens follow.
    if (tid < t_n) {
        const int t = t_lo + tid;
        const int s = last_start(p.b.q_start, p.b.n_seq, t);
        const int first = p.b.q_start[s], next = p.b.q_start[s + 1], past = p.b.past[s];   // in flight together
        int n = 0, page = -1;
        int64_t pos = -1;
        if (first <= t && t < next) {
            pos = (int64_t)past + t - first;
            if (kv_part) {
                if (t == first || (pos & (kKvBlock - 1)) == 0) {
                    const int end = min(next, p.b.n_tok);
                    n = min(kKvBlock - (int)(pos & (kKvBlock - 1)), end - t);
                    page = page_of(p.b, p.c, s, pos);
                    const bool turns = p.rot == 0 || pos + n <= p.n_pos;
                    // a block that runs past the rotation's tables keeps the tokens inside
                    if (!turns) n = max(0, (int)(p.n_pos - pos));
                    if (page < 0 || !turns) record_status(&g_kv_status, RF_ERR_INVALID_ARG);
                    if (page < 0) n = 0;
                }
            } else if (pos < 0 || pos > 0x7fffffffLL || (p.rot != 0 && pos >= p.n_pos)) {
                pos = -1;
                record_status(&g_kv_status, RF_ERR_INVALID_ARG);
            }
        }
        s_pos[tid] = (int)pos;   // below 2^31 where there is something to do
        s_n[tid] = n;
        s_page[tid] = page;
    }
    __syncthreads();
    if (kv_part) {
        for (int j = 0; j < t_n; ++j)
            if (s_n[j] > 0)
                append_block<T, UPT>(p, part & 1, part >> 1, t_lo + j, s_n[j], s_page[j], s_pos[j], s_max);
    } else {
        const int h0 = (part - 2 * p.c.n_kv_heads) * kQHeads;
        const int nh = min(kQHeads, p.n_heads - h0), upr = p.c.head_dim / 8;
        const int upt = nh * upr, per = kAppendThreads / upt;    // units per token (128 at most), tokens per pass
        const int j0 = tid / upt, v = tid - j0 * upt, h = h0 + v / upr;
        if (j0 >= per) return;
        const Unit un = unit_at(v % upr, p.rot, p.style);
        const T *src = static_cast<const T *>(p.q) + (int64_t)t_lo * p.q_lt + h * p.q_lh;
        T *dst = static_cast<T *>(p.q_out) + (int64_t)t_lo * p.qo_lt + h * p.qo_lh;
#pragma unroll 4
        for (int j = j0; j < t_n; j += per) {
            if (s_pos[j] < 0) continue;
            float x[4], y[4];
            load4<T>(src + j * p.q_lt + un.a, p.q_vec, x);
            load4<T>(src + j * p.q_lt + un.b, p.q_vec, y);
            if (p.rot) {
                const int64_t at = (int64_t)s_pos[j] * (p.rot / 2);
                rotate_unit(x, y, un, p.style, p.cos_tab + at, p.sin_tab + at);
            }
            store4<T>(dst + j * p.qo_lt + un.a, p.qo_vec, x);
            store4<T>(dst + j * p.qo_lt + un.b, p.qo_vec, y);
        }
    }
}

// Values at the batch's positions; a CTA per p.chunk tokens (at most eight).
// A thread turns eight codes of a head into 32 bytes, neighbouring threads
// neighbouring ones, for all tokens of the chunk at once.
__global__ void __launch_bounds__(256) read_kernel(const __grid_constant__ rf_kv_cache c,
                                                   const __grid_constant__ rf_kv_batch b, int chunk,
                                                   float *__restrict__ k_out, float *__restrict__ v_out,
                                                   bool sectors)
{
    __shared__ int s_page[kReadTokens], s_off[kReadTokens];
    const int t_lo = (int)blockIdx.x * chunk, t_n = min(chunk, b.n_tok - t_lo);
    pdl_launch_dependents();
    pdl_wait();
    if ((int)threadIdx.x < t_n) {
        const int t = t_lo + (int)threadIdx.x;
        const int s = find_seq(b.q_start, b.n_seq, t);
        int page = -1, off = 0;
        if (s >= 0) {
            const int64_t pos = (int64_t)b.past[s] + (t - b.q_start[s]);
            page = page_of(b, c, s, pos);
            if (page < 0) record_status(&g_kv_status, RF_ERR_INVALID_ARG);
            off = (int)(pos & (c.page_size - 1));
        }
        s_page[threadIdx.x] = page;
        s_off[threadIdx.x] = off;
    }
    __syncthreads();
    const int cpr = c.head_dim / 8, per = c.n_kv_heads * cpr;    // runs of eight codes per token
    for (int u = (int)threadIdx.x; u < 2 * per; u += 256) {
        const int side = u >= per, w = u - side * per, h = w / cpr, i = w - h * cpr;
        const int8_t *codes = (side ? c.v : c.k) + 8 * i;
        const uint8_t *scales = side ? c.v_scale : c.k_scale;
        float *out = (side ? v_out : k_out) + (int64_t)t_lo * per * 8 + 8 * w;
        uint2 code[kReadTokens];
        float unit[kReadTokens];
#pragma unroll
        for (int j = 0; j < kReadTokens; ++j) {
            code[j] = make_uint2(0u, 0u);
            unit[j] = 0.f;
            if (j < t_n && s_page[j] >= 0) {
                const int64_t ph = (int64_t)s_page[j] * c.n_kv_heads + h;
                code[j] = *reinterpret_cast<const uint2 *>(codes + (ph * c.page_size + s_off[j]) * c.head_dim);
                unit[j] = scale_value(scales[ph * (c.page_size / kKvBlock) + s_off[j] / kKvBlock]);
            }
        }
#pragma unroll
        for (int j = 0; j < kReadTokens; ++j) {
            if (j >= t_n) break;
            uint32_t v[8];
#pragma unroll
            for (int m = 0; m < 8; ++m)
                v[m] = __float_as_uint((float)(int8_t)((m < 4 ? code[j].x : code[j].y) >> (8 * (m & 3))) * unit[j]);
            float *dst = out + (int64_t)j * per * 8;
            if (sectors) {
                store_sector(dst, v);
            } else {
#pragma unroll
                for (int m = 0; m < 8; m += 4)
                    *reinterpret_cast<uint4 *>(dst + m) = make_uint4(v[m], v[m + 1], v[m + 2], v[m + 3]);
            }
        }
    }
}

}  // namespace

rf_status check_kv(const rf_kv_cache *c, const rf_kv_batch *b)
{
    if (!c || !b || !c->k || !c->v || !c->k_scale || !c->v_scale || !b->page_table || !b->past || !b->q_start)
        return RF_ERR_INVALID_ARG;
    if (c->n_pages < 1 || c->n_pages > 0x7fffffffLL || c->n_kv_heads < 1 || c->n_kv_heads > 1024 ||
        c->head_dim < 16 || c->head_dim > 256 || c->head_dim % 16 != 0 || c->reserved != 0)
        return RF_ERR_INVALID_ARG;
    if (c->page_size != 32 && c->page_size != 64 && c->page_size != 128 && c->page_size != 256)
        return RF_ERR_INVALID_ARG;
    if (b->n_seq < 1 || b->n_seq > 65536 || b->n_tok < 0 || b->table_width < 1 ||
        b->table_stride < b->table_width || b->reserved != 0)
        return RF_ERR_INVALID_ARG;
    if (!aligned_to(c->k, 16) || !aligned_to(c->v, 16) || !aligned_to(b->page_table, 4) ||
        !aligned_to(b->past, 4) || !aligned_to(b->q_start, 4))
        return RF_ERR_MISALIGNED;
    if (c->n_pages * c->n_kv_heads * c->page_size > (1LL << 40)) return RF_ERR_TOO_LARGE;
    return RF_OK;
}

rf_status read_and_clear_kv_status()
{
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_kv_status, sizeof(int)) != cudaSuccess) return RF_ERR_CUDA;
    if (v != 0) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(g_kv_status, &zero, sizeof(int)) != cudaSuccess) return RF_ERR_CUDA;
    }
    return static_cast<rf_status>(v);
}

}  // namespace rf

using namespace rf;

extern "C" {

rf_status rf_kv_append(const rf_kv_cache *cache, const rf_kv_batch *batch, int dtype, const void *k,
                       int64_t k_ld_tok, int64_t k_ld_head, const void *v, int64_t v_ld_tok,
                       int64_t v_ld_head, const void *q, int64_t q_ld_tok, int64_t q_ld_head,
                       void *q_out, int64_t q_out_ld_tok, int64_t q_out_ld_head, int n_heads,
                       const float *cos_tab, const float *sin_tab, int64_t n_pos, int rot, int style,
                       unsigned flags, void *stream)
{
    if (!dtype_ok(dtype)) return RF_ERR_UNSUPPORTED_FMT;
    if (const rf_status st = check_kv(cache, batch)) return st;
    const int D = cache->head_dim;
    if (rot < 0 || rot > D || rot % 8 != 0 || (rot > 0 && (!cos_tab || !sin_tab || n_pos < 1)) ||
        (style != RF_ROPE_HALF && style != RF_ROPE_PAIRS) || (flags & ~RF_CHAIN) != 0)
        return RF_ERR_INVALID_ARG;
    if (batch->n_tok > 0 &&
        (!k || !v || k_ld_tok < D || k_ld_head < D || v_ld_tok < D || v_ld_head < D))
        return RF_ERR_INVALID_ARG;
    if (q && (!q_out || n_heads < 1 || q_ld_tok < D || q_ld_head < D || q_out_ld_tok < D || q_out_ld_head < D))
        return RF_ERR_INVALID_ARG;
    const int b = dtype_bytes(dtype);
    for (const void *ptr : {k, v, q, (const void *)q_out})
        if (!aligned_to(ptr, (size_t)b)) return RF_ERR_MISALIGNED;
    if (rot > 0 && (!aligned_to(cos_tab, 16) || !aligned_to(sin_tab, 16))) return RF_ERR_MISALIGNED;
    if (q && n_heads > 4096) return RF_ERR_TOO_LARGE;
    if (batch->n_tok == 0) return RF_OK;
    AppendParams p;
    p.c = *cache, p.b = *batch;
    p.k = k, p.v = v, p.q = q, p.q_out = q_out;
    p.k_lt = k_ld_tok, p.k_lh = k_ld_head, p.v_lt = v_ld_tok, p.v_lh = v_ld_head;
    p.q_lt = q_ld_tok, p.q_lh = q_ld_head, p.qo_lt = q_out_ld_tok, p.qo_lh = q_out_ld_head;
    p.cos_tab = cos_tab, p.sin_tab = sin_tab, p.n_pos = n_pos;
    p.n_heads = q ? n_heads : 0, p.rot = rot, p.style = style;
    auto vec = [b](const void *ptr, int64_t lt, int64_t lh) {
        return aligned_to(ptr, (size_t)(4 * b)) && lt % 4 == 0 && lh % 4 == 0;
    };
    p.k_vec = vec(k, k_ld_tok, k_ld_head);
    p.v_vec = vec(v, v_ld_tok, v_ld_head);
    p.q_vec = q && vec(q, q_ld_tok, q_ld_head);
    p.qo_vec = q && vec(q_out, q_out_ld_tok, q_out_ld_head);
    // A chunk per token spreads a decode batch over CTAs; prompts open one
    // block in 32 tokens, so a chunk of 32 holds about one.
    p.chunk = (int64_t)batch->n_tok >= 16LL * batch->n_seq ? 32 : 1;
    const int q_groups = q ? (n_heads + kQHeads - 1) / kQHeads : 0;
    p.parts = (unsigned)(2 * cache->n_kv_heads + q_groups);
    const int64_t ctas = (((int64_t)batch->n_tok + p.chunk - 1) / p.chunk) * p.parts;
    if (ctas > 0x7fffffffLL) return RF_ERR_TOO_LARGE;
    const dim3 grid((unsigned)ctas);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool chain = (flags & RF_CHAIN) != 0;
    return with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        if (D <= 64) return launch_kernel(append_kernel<T, 1>, grid, dim3(kAppendThreads), 0, s, chain, p);
        if (D <= 128) return launch_kernel(append_kernel<T, 2>, grid, dim3(kAppendThreads), 0, s, chain, p);
        return launch_kernel(append_kernel<T, 4>, grid, dim3(kAppendThreads), 0, s, chain, p);
    });
}

rf_status rf_kv_read(const rf_kv_cache *cache, const rf_kv_batch *batch, float *k_out, float *v_out,
                     unsigned flags, void *stream)
{
    if (const rf_status st = check_kv(cache, batch)) return st;
    if ((batch->n_tok > 0 && (!k_out || !v_out)) || (flags & ~RF_CHAIN) != 0) return RF_ERR_INVALID_ARG;
    if (!aligned_to(k_out, 16) || !aligned_to(v_out, 16)) return RF_ERR_MISALIGNED;
    if (batch->n_tok == 0) return RF_OK;
    // Few tokens: one per CTA; many: eight share the lookup.
    const int chunk = batch->n_tok > 8 * num_sms() ? kReadTokens : 1;
    return launch_kernel(read_kernel, dim3((unsigned)(((int64_t)batch->n_tok + chunk - 1) / chunk)), dim3(256), 0,
                         static_cast<cudaStream_t>(stream), (flags & RF_CHAIN) != 0, *cache, *batch, chunk,
                         k_out, v_out, aligned_to(k_out, 32) && aligned_to(v_out, 32));
}

}  // extern "C"
