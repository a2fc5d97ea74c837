// rf_kv.cuh -- what the kernels around the KV cache share: activation types,
// the batch's token lookup, and the launch helper with a programmatic
// dependency.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "rf.h"
#include "rf_device.cuh"
#include "rf_internal.h"

namespace rf {

constexpr int kKvBlock = 32;      // tokens that share a scale byte
constexpr int kScaleMin = 87;     // 2^-40: the smallest unit written
constexpr int kScaleMax = 167;    // 2^40: the largest
constexpr int kScaleNan = 255;

// ------------------------------------------------------------ activation types
template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v)
{
    return __bfloat162float(v);
}
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v)
{
    return __float2bfloat16_rn(v);
}

// Four consecutive elements.  vec: the address is aligned to all four.
template <typename T>
__device__ __forceinline__ void load4(const T *p, bool vec, float (&f)[4])
{
    if (vec) {
        if constexpr (sizeof(T) == 4) {
            const float4 a = *reinterpret_cast<const float4 *>(p);
            f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
        } else {
            union { uint2 u; T t[4]; } a;
            a.u = *reinterpret_cast<const uint2 *>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = to_f32<T>(a.t[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = to_f32<T>(p[i]);
    }
}
// Eight; vec8: the address is aligned to all of them (16 or 32 bytes).
template <typename T>
__device__ __forceinline__ void load8(const T *p, bool vec8, bool vec4, float (&f)[8])
{
    if (vec8) {
        if constexpr (sizeof(T) == 4) {
            asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7])
                         : "l"(p)
                         : "memory");
        } else {
            union { uint4 u; T t[8]; } a;
            a.u = *reinterpret_cast<const uint4 *>(p);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = to_f32<T>(a.t[i]);
        }
    } else {
        float u[4], v[4];
        load4<T>(p, vec4, u);
        load4<T>(p + 4, vec4, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = u[i], f[4 + i] = v[i];
    }
}
template <typename T>
__device__ __forceinline__ void store4(T *p, bool vec, const float (&f)[4])
{
    if (vec) {
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
        } else {
            union { uint2 u; T t[4]; } a;
#pragma unroll
            for (int i = 0; i < 4; ++i) a.t[i] = from_f32<T>(f[i]);
            *reinterpret_cast<uint2 *>(p) = a.u;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = from_f32<T>(f[i]);
    }
}

// 32 bytes in one store (a whole memory sector); p is aligned to them.
__device__ __forceinline__ void store_sector(void *p, const uint32_t (&w)[8])
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}
// Two elements as T, packed.
template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b)
{
    union { T t[2]; uint32_t u; } v;
    v.t[0] = from_f32<T>(a), v.t[1] = from_f32<T>(b);
    return v.u;
}

// ------------------------------------------------------------------- codes
// Codes 0, 1 / 2, 3 of a word, their sign bits flipped, as an fp16 pair:
// 0x6400 | u is 1024 + code + 128, so subtracting 1152 is exact.
__device__ __forceinline__ uint32_t codes_sub(uint32_t a)
{
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(0x64806480u));
    return r;
}
__device__ __forceinline__ uint32_t codes_lo(uint32_t w) { return codes_sub(prmt(w, 0x64646464u, 0x5140u)); }
__device__ __forceinline__ uint32_t codes_hi(uint32_t w) { return codes_sub(prmt(w, 0x64646464u, 0x7362u)); }

__device__ __forceinline__ uint32_t pack_h2(float a, float b)
{
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 unpack_h2(uint32_t v)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&v));
}
__device__ __forceinline__ float exp2_fast(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// ------------------------------------------------------------------- batch
// The last sequence s with q_start[s] <= t, or 0 if there is none.
__device__ __forceinline__ int last_start(const int32_t *q_start, int n_seq, int t)
{
    int lo = 0, hi = n_seq;   // q_start[lo] <= t or lo == 0; q_start[hi] > t or hi == n_seq
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (q_start[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

// The sequence that owns token t, or -1.  Reads only q_start[0 .. n_seq].
__device__ __forceinline__ int find_seq(const int32_t *q_start, int n_seq, int t)
{
    const int lo = last_start(q_start, n_seq, t);
    return q_start[lo] <= t && t < q_start[lo + 1] ? lo : -1;
}

// find_seq by a converged warp, in fewer round trips to memory: sequence t
// is tried first (a decode batch has one token each), then 32 entries at a
// time are compared.
__device__ __forceinline__ int find_seq_warp(const int32_t *q_start, int n_seq, int t)
{
    if (t < n_seq && q_start[t] == t && q_start[t + 1] == t + 1) return t;
    const int lane = threadIdx.x & 31;
    int lo = 0, n = n_seq;                 // q_start[lo .. lo + n] brackets t, if anything does
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int at = lo + lane * step;
        const bool below = lane * step < n && (lane == 0 || q_start[at] <= t);
        const int k = 31 - __clz(__ballot_sync(0xffffffffu, below));   // the last one not after t
        n = min(step, n - k * step);
        lo += k * step;
    }
    return q_start[lo] <= t && t < q_start[lo + 1] ? lo : -1;
}

// The page of position `pos` of sequence s, or -1 if it has none (positions
// from 2^31 on have none: kernels hold them in 32 bits).
__device__ __forceinline__ int page_of(const rf_kv_batch &b, const rf_kv_cache &c, int s, int64_t pos)
{
    const int64_t i = pos >> (31 - __clz(c.page_size));   // a power of two
    if (pos < 0 || pos > 0x7fffffffLL || i >= b.table_width) return -1;
    const int page = b.page_table[(int64_t)s * b.table_stride + i];
    return page >= 0 && page < c.n_pages ? page : -1;
}

// 2^(E-127) of a scale byte: E = 0 is the subnormal 2^-127, 255 is NaN.
__device__ __forceinline__ float scale_value(uint32_t E)
{
    return __uint_as_float(E == 255u ? 0x7fc00000u : E == 0u ? 0x00400000u : E << 23);
}

// Attention: what a query row is multiplied by, a power of two that brings
// its maximum (amax) to [512, 1024), and the factor of its scores that takes
// it back, times `scale`.  A row that holds an infinity has NaN for a factor:
// its scores are all infinite or NaN, and where all of them are minus
// infinity it would pass for one that sees nothing.
__device__ __forceinline__ float row_power(float amax, float scale, float *unit)
{
    const uint32_t bits = __float_as_uint(amax);
    const int ex = min(max(263 - (int)(bits >> 23), 1), 253);
    *unit = bits == 0x7f800000u ? __uint_as_float(0x7fc00000u) : scale * __uint_as_float((uint32_t)(254 - ex) << 23);
    return __uint_as_float((uint32_t)ex << 23);
}

// ---------------------------------------------------------------- host side
inline bool dtype_ok(int dtype) { return dtype == RF_F32 || dtype == RF_F16 || dtype == RF_BF16; }
inline int dtype_bytes(int dtype) { return dtype == RF_F32 ? 4 : 2; }
inline bool aligned_to(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// RF_OK if the fields of a cache and a batch are in range.
rf_status check_kv(const rf_kv_cache *c, const rf_kv_batch *b);

// Calls f with a value of the C++ type of `dtype`.
template <typename F>
rf_status with_dtype(int dtype, F &&f)
{
    switch (dtype) {
    case RF_F32: return f(float());
    case RF_F16: return f(__half());
    default: return f(__nv_bfloat16());
    }
}

// Launches kernel(args...); chain: with a programmatic dependency on the
// previous kernel of the stream.
template <typename... P, typename... A>
rf_status launch_kernel(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                        bool chain, A &&...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = chain ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
    cudaGetLastError();
    return e == cudaSuccess ? RF_OK : RF_ERR_CUDA;
}

}  // namespace rf
