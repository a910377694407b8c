// Small device helpers of the chunk-attention and attention-weight kernels: packed arithmetic, conversions,
// register reallocation, the products with A in tensor memory, and the tensor map of the pages.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "sk_internal.cuh"
#include "sk_sm100.cuh"

namespace sk {

// 2^x on the special-function unit, flushing subnormal results to zero; 2^-inf = 0.
__device__ __forceinline__ float ex2_ftz(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float fmax3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 ffma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

__device__ __forceinline__ float2 fadd2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// Two floats to a packed pair (lo in the low half), round to nearest even.
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// The e4m3 pair in the low 16 bits as a packed f16 pair (exact).
__device__ __forceinline__ uint32_t f16x2_of_e4m3(uint32_t v)
{
    uint32_t r;
    const uint16_t h = (uint16_t)(v & 0xFFFFu);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(h));
    return r;
}

// One row of Q spread over a warp (lane l: elements 4 l .. 4 l + 3, bf16) as two e4m3 terms of q * 2^e = hi + lo,
// with the row's largest |q| * 2^e in [128, 256).  A bf16 element of at least 2^-9 of that is hi + lo exactly.
__device__ __forceinline__ void split_q_row(uint2 raw, uint32_t &hi, uint32_t &lo, int &e)
{
    float q[4] = {__uint_as_float(raw.x << 16), __uint_as_float(raw.x & 0xFFFF0000u), __uint_as_float(raw.y << 16),
                  __uint_as_float(raw.y & 0xFFFF0000u)};
    float amax = fmaxf(fmaxf(fabsf(q[0]), fabsf(q[1])), fmaxf(fabsf(q[2]), fabsf(q[3])));
    for (int o = 16; o > 0; o >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    e = 0;
    if (amax > 0.f && amax < CUDART_INF_F) {
        int ex;
        frexpf(amax, &ex);                       // amax in [2^(ex-1), 2^ex)
        e = 8 - ex;
        e = e > 100 ? 100 : (e < -100 ? -100 : e);
    }
    hi = lo = 0;
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
        const float x0 = ldexpf(q[k], e), x1 = ldexpf(q[k + 1], e);
        uint16_t hc, lc;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hc) : "f"(x1), "f"(x0));
        const uint32_t hf = f16x2_of_e4m3(hc);
        float h0, h1;
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
            : "=f"(h0), "=f"(h1)
            : "r"(hf));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lc) : "f"(x1 - h1), "f"(x0 - h0));
        hi |= (uint32_t)hc << (8 * k);
        lo |= (uint32_t)lc << (8 * k);
    }
}

// mbar_wait_bounded with a test before the first suspending wait: a wait for what is complete costs less.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, const volatile int *abort, long long limit)
{
    return sm100::mbar_test_wait(bar, parity) || sm100::mbar_wait_bounded(bar, parity, abort, limit);
}

// Gives registers of this warpgroup back / takes them, all its warps together.
template <int N>
__device__ __forceinline__ void reg_dec()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <int N>
__device__ __forceinline__ void reg_inc()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

template <int N>
__device__ __forceinline__ void tmem_st32_u(uint32_t taddr, const uint32_t *v)
{
    float f[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        f[i] = __uint_as_float(v[i]);
    sm100::tmem_st32<N>(taddr, f);
}

// D (TMEM) (+)= A (TMEM, one row per lane, packed along the columns) x B (shared memory); called by a converged
// warp, issued by its elected lane.
__device__ __forceinline__ void mma_f16_ts_warp(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                                uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// Tensor map of Q rows [tokens][heads][256 bytes] (bf16, or e4m3 hi and lo codes): a box is 128 bytes of `heads` heads
// of `toks` tokens and lands as consecutive 128-byte-swizzled rows.
cudaError_t encode_q_map(CUtensorMap *map, const void *q, long long num_tokens, int H_q, bool fp8, int heads, int toks);

// Tensor map of the pages [blocks][heads][16 tokens][K | V] as 4-D: (128 bytes of a row, token within an 8-token
// group, 128-byte chunk of the row, 8-token group across all pages).  A box is `chunks` chunks of one page of one
// head and lands group by group, chunk by chunk, as 8 x 128 B swizzle atoms.
cudaError_t encode_page_map(CUtensorMap *map, const void *pages, long long num_blocks, int H_kv, bool fp8, int chunks);

}  // namespace sk
