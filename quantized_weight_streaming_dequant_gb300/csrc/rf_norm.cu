// rf_norm.cu -- norms before and after a block fused with its gate, its
// residual scale and the residual sum.
//
// t = x (or its norm times post_weight), r = residual + scale * gate * t,
// y = r * rsqrt(mean r^2 + eps) * weight.  Every element is read once and
// written once: a row stays in the registers of one CTA between its (at most
// two) sums of squares, which are fp32 trees in a fixed order.
//
// Bound: HBM bytes for many rows; for one row the chain launch - load -
// reduce (- reduce) - store.  So a thread holds one 16-byte chunk when rows
// are fewer than the SMs (the most lanes on the row, the shortest chain) and
// up to four when there are many (fewer threads per row, so that several
// rows share an SM and hide one another's reductions).
// Measured: 8192 rows of 4096 fp32 with all parts 80 us (6.7 TB/s, 0.99 of
// the measured copy rate); one row of 4096 3.8 us, 77 rows of 2880 bf16
// 4.6 us (launch to end; a copy of that size takes about 2.5).
#include <algorithm>

#include "rf_kv.cuh"

namespace rf {
namespace {

constexpr int kMaxNorm = 32768;   // elements per row: 1024 threads x 32 registers

struct NormParams {
    const void *x, *residual;
    void *residual_out, *y;
    const float *post_weight, *gate, *weight;
    int64_t ldx, ldr, ldro, ldy, ld_gate;
    int n;
    float inv_n, eps, scale;
};

// Sum over the CTA in a fixed order, for every thread.  Each use of `part`
// (32 floats) is its own, so one barrier is enough.
__device__ __forceinline__ float block_sum(float v, float *part)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (blockDim.x == 32) return v;
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = (threadIdx.x & 31) < (blockDim.x >> 5) ? part[threadIdx.x & 31] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// E elements from p: one wide access (E > 1: p is aligned to it) or E = 1.
template <typename T, int E>
__device__ __forceinline__ void load_chunk(const T *p, float (&f)[E])
{
    if constexpr (E == 1) {
        f[0] = to_f32<T>(p[0]);
    } else {
        union { uint4 u; T t[16 / sizeof(T)]; } a;
        a.u = *reinterpret_cast<const uint4 *>(p);
#pragma unroll
        for (int i = 0; i < E; ++i) f[i] = to_f32<T>(a.t[i]);
    }
}
template <typename T, int E>
__device__ __forceinline__ void store_chunk(T *p, const float (&f)[E])
{
    if constexpr (E == 1) {
        p[0] = from_f32<T>(f[0]);
    } else {
        union { uint4 u; T t[16 / sizeof(T)]; } a;
#pragma unroll
        for (int i = 0; i < E; ++i) a.t[i] = from_f32<T>(f[i]);
        *reinterpret_cast<uint4 *>(p) = a.u;
    }
}
template <int E>
__device__ __forceinline__ void load_weights(const float *p, float (&f)[E])
{
    if constexpr (E == 1) {
        f[0] = *p;
    } else {
#pragma unroll
        for (int i = 0; i < E; i += 4) {
            const float4 a = *reinterpret_cast<const float4 *>(p + i);
            f[i] = a.x, f[i + 1] = a.y, f[i + 2] = a.z, f[i + 3] = a.w;
        }
    }
}

// One row per CTA; thread i owns chunks i, i + blockDim.x, ... (C of them at
// most), each of E elements.
template <typename T, int E, int C>
__global__ void __launch_bounds__(1024) norm_kernel(const __grid_constant__ NormParams p)
{
    __shared__ float part[2][32];
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(p.x);
    const T *res = static_cast<const T *>(p.residual);
    const int base = (int)threadIdx.x * E, step = (int)blockDim.x * E;
    float v[C][E], r[C][E];
    pdl_launch_dependents();
    pdl_wait();
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int i = base + c * step;
#pragma unroll
        for (int e = 0; e < E; ++e) v[c][e] = r[c][e] = 0.f;
        if (i < p.n) {
            if (x) load_chunk<T, E>(x + row * p.ldx + i, v[c]);
            if (res) load_chunk<T, E>(res + row * p.ldr + i, r[c]);
        }
    }
    float by = p.scale;
    if (x && p.post_weight) {
        float s = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int e = 0; e < E; ++e) s = fmaf(v[c][e], v[c][e], s);
        s = block_sum(s, part[0]);
        const float inv = rsqrtf(fmaf(s, p.inv_n, p.eps));
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = base + c * step;
            if (i < p.n) {
                float w[E];
                load_weights<E>(p.post_weight + i, w);
#pragma unroll
                for (int e = 0; e < E; ++e) v[c][e] *= inv * w[e];
            }
        }
    }
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int i = base + c * step;
        if (i < p.n) {
            if (x && p.gate) {
                float g[E];
                load_weights<E>(p.gate + row * p.ld_gate + i, g);
#pragma unroll
                for (int e = 0; e < E; ++e) v[c][e] *= g[e];
            }
#pragma unroll
            for (int e = 0; e < E; ++e) {
                r[c][e] = fmaf(by, v[c][e], r[c][e]);
                s = fmaf(r[c][e], r[c][e], s);
            }
            if (p.residual_out)
                store_chunk<T, E>(static_cast<T *>(p.residual_out) + row * p.ldro + i, r[c]);
        }
    }
    if (!p.y) return;
    s = block_sum(s, part[1]);
    const float inv = rsqrtf(fmaf(s, p.inv_n, p.eps));
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int i = base + c * step;
        if (i < p.n) {
            float w[E];
#pragma unroll
            for (int e = 0; e < E; ++e) w[e] = 1.f;
            if (p.weight) load_weights<E>(p.weight + i, w);
#pragma unroll
            for (int e = 0; e < E; ++e) w[e] *= r[c][e] * inv;
            store_chunk<T, E>(static_cast<T *>(p.y) + row * p.ldy + i, w);
        }
    }
}

template <typename T, int E>
rf_status launch_norm(const NormParams &p, int64_t n_tok, cudaStream_t s, bool chain)
{
    const int chunks = (p.n + E - 1) / E;
    constexpr int kMost = 32 / E;                     // chunks per thread: 32 registers
    // Few rows: one chunk per thread; many: four (sixteen elements at most).
    int want = n_tok <= num_sms() ? 1 : E == 1 ? 8 : E == 4 ? 4 : 2;
    want = std::max(want, (chunks + 1023) / 1024);
    int c = 1;
    while (c < want) c *= 2;
    if (c > kMost) return RF_ERR_TOO_LARGE;
    const int threads = std::max(32, ((chunks + c - 1) / c + 31) / 32 * 32);
    const dim3 grid((unsigned)n_tok), block((unsigned)threads);
    switch (c) {
    case 1: return launch_kernel(norm_kernel<T, E, 1>, grid, block, 0, s, chain, p);
    case 2: return launch_kernel(norm_kernel<T, E, 2>, grid, block, 0, s, chain, p);
    case 4: return launch_kernel(norm_kernel<T, E, 4>, grid, block, 0, s, chain, p);
    case 8:
        if constexpr (kMost >= 8) return launch_kernel(norm_kernel<T, E, 8>, grid, block, 0, s, chain, p);
        break;
    case 16:
        if constexpr (kMost >= 16) return launch_kernel(norm_kernel<T, E, 16>, grid, block, 0, s, chain, p);
        break;
    case 32:
        if constexpr (kMost >= 32) return launch_kernel(norm_kernel<T, E, 32>, grid, block, 0, s, chain, p);
        break;
    }
    return RF_ERR_TOO_LARGE;
}

}  // namespace
}  // namespace rf

using namespace rf;

extern "C" rf_status rf_norm_residual(int dtype, int64_t n_tok, int64_t n, const void *x,
                                      int64_t ldx, const float *post_weight, const float *gate,
                                      int64_t ld_gate, float scale, const void *residual,
                                      int64_t ld_residual, void *residual_out,
                                      int64_t ld_residual_out, const float *weight, void *y,
                                      int64_t ldy, float eps, unsigned flags, void *stream)
{
    if (!dtype_ok(dtype)) return RF_ERR_UNSUPPORTED_FMT;
    if (n < 1 || n_tok < 0 || (n_tok > 0 && ((!x && !residual) || (!residual_out && !y))) ||
        !(eps >= 0.f) || scale != scale || (flags & ~RF_CHAIN) != 0)
        return RF_ERR_INVALID_ARG;
    if ((x && ldx < n) || (residual && ld_residual < n) || (residual_out && ld_residual_out < n) ||
        (y && ldy < n) || (gate && ld_gate != 0 && ld_gate < n))
        return RF_ERR_INVALID_ARG;
    const size_t b = (size_t)dtype_bytes(dtype);
    for (const void *p : {x, residual, (const void *)residual_out, (const void *)y})
        if (!aligned_to(p, b)) return RF_ERR_MISALIGNED;
    for (const float *p : {post_weight, gate, weight})
        if (!aligned_to(p, 4)) return RF_ERR_MISALIGNED;
    if (n > kMaxNorm || n_tok > 0x7fffffffLL) return RF_ERR_TOO_LARGE;
    if (n_tok == 0) return RF_OK;
    NormParams p;
    p.x = x, p.residual = residual, p.residual_out = residual_out, p.y = y;
    p.post_weight = post_weight, p.gate = gate, p.weight = weight;
    p.ldx = ldx, p.ldr = ld_residual, p.ldro = ld_residual_out, p.ldy = ldy, p.ld_gate = ld_gate;
    p.n = (int)n;
    p.inv_n = 1.f / (float)n;
    p.eps = eps, p.scale = x ? scale : 0.f;
    // Wide accesses need every row of every operand on a 16-byte boundary.
    bool vec = n % (int64_t)(16 / b) == 0;
    auto rows = [&](const void *q, int64_t ld, size_t eb) {
        if (q && (!aligned_to(q, 16) || (ld * (int64_t)eb) % 16 != 0)) vec = false;
    };
    rows(x, ldx, b);
    rows(residual, ld_residual, b);
    rows(residual_out, ld_residual_out, b);
    rows(y, ldy, b);
    rows(post_weight, 0, 4);
    rows(weight, 0, 4);
    rows(gate, ld_gate, 4);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool chain = (flags & RF_CHAIN) != 0;
    return with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        return vec ? launch_norm<T, (int)(16 / sizeof(T))>(p, n_tok, s, chain)
                   : launch_norm<T, 1>(p, n_tok, s, chain);
    });
}
