// bf16 and e4m3 conversions shared by the kernels that write pages.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

namespace sk {

// A power-of-two scale with a normal reciprocal: multiplying by 1 / scale rounds like dividing.
inline bool exact_reciprocal(float sc)
{
    int e = 0;
    const float m = frexpf(sc, &e);
    const float r = 1.f / sc;
    return m == 0.5f && r * sc == 1.f && std::isnormal(r) && std::isnormal(sc);
}

// Two floats divided by `scale` -> two e4m3fn codes (low byte from a), nearest even, saturated.  With
// RECIP the caller guarantees scale = 2^k and inv = 2^-k exactly, so x * inv is the correctly rounded
// x / scale (both round the same real number).
template <bool RECIP>
__device__ __forceinline__ uint32_t quant_e4m3x2(float a, float b, float scale, float inv)
{
    const float lo = RECIP ? a * inv : __fdiv_rn(a, scale);
    const float hi = RECIP ? b * inv : __fdiv_rn(b, scale);
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ void unpack_bf16x8(const uint4 v, float *f)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack_bf16x8(const float *f)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace sk
