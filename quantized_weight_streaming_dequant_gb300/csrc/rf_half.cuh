// rf_half.cuh -- fp16 pairs in 32-bit registers: what the decoders of the
// tensor-core kernels build weights from.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

namespace rf {

__device__ __forceinline__ uint32_t h2_bits(__half2 h)
{
    return (uint32_t)__half_as_ushort(__low2half(h)) | ((uint32_t)__half_as_ushort(__high2half(h)) << 16);
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// fp16 bits of 2^k: normal for k >= -14, subnormal down to 2^-24, 0 below,
// infinity above 2^15.
__device__ __forceinline__ uint32_t pow2_h(int k)
{
    if (k > 15) return 0x7C00u;
    if (k >= -14) return (uint32_t)(k + 15) << 10;
    if (k >= -24) return 1u << (k + 24);
    return 0u;
}
// Two E2M1 codes (the low 8 bits of `lo8`: low nibble, high nibble) as an
// fp16 pair (low half, high half), exactly.
__device__ __forceinline__ uint32_t e2m1x2_h2(uint32_t lo8)
{
    uint32_t r;
    asm("{\n\t.reg .b8 t;\n\tcvt.u8.u32 t, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}"
        : "=r"(r)
        : "r"(lo8));
    return r;
}

}  // namespace rf
