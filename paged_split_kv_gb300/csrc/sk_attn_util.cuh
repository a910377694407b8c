// Small device helpers of the chunk-attention and attention-weight kernels: packed arithmetic, conversions,
// register reallocation, the products with A in tensor memory, and the tensor map of the pages.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "sk_cache_ops.cuh"
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

__device__ __forceinline__ float2 fmul2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
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

// Half a warp's row of Q (8 bf16 elements a lane) as two e4m3 terms of q * 2^e = hi + lo, the row's largest |q| * 2^e in
// [128, 256); returns e.  A bf16 element of at least 2^-9 of the largest is hi + lo exactly.
__device__ __forceinline__ int split_q_half_row(uint4 raw, uint2 &hi, uint2 &lo)
{
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    float q[8], amax = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        q[2 * k] = __uint_as_float(w[k] << 16);
        q[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
        amax = fmax3(amax, fabsf(q[2 * k]), fabsf(q[2 * k + 1]));
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    // amax in [2^(ex - 127), 2^(ex - 126)); none for a row of zeros, and for infinities, which saturate
    const int ex = __float_as_int(amax) >> 23;
    const int e = amax == 0.f || ex == 255 ? 0 : max(-100, min(100, 134 - ex));
    const float by = __int_as_float((127 + e) << 23);
    uint32_t h[4], l[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float x0 = q[2 * k] * by, x1 = q[2 * k + 1] * by;
        uint16_t hc, lc;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hc) : "f"(x1), "f"(x0));
        float h0, h1;
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
            : "=f"(h0), "=f"(h1)
            : "r"(f16x2_of_e4m3(hc)));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lc) : "f"(x1 - h1), "f"(x0 - h0));
        h[k] = hc;
        l[k] = lc;
    }
    hi = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
    lo = make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
    return e;
}

// Waits for the phase with the given parity like mbar_wait_bounded, in few instructions (every role waits in many places,
// and their code shares the instruction cache): a test, then suspended waits.  One that ends later than the limit allows
// has failed, whether the phase is over by then or not, so that a short limit expires although try_wait suspends.  (Tests
// in the loop instead cost 3 %, waits with a hint of 10 ms 2 %: 24 prompts 173 and 168 us against 165.)
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, const volatile int *abort, long long limit)
{
    if (sm100::mbar_test_wait(bar, parity))
        return true;
    const long long t0 = clock64();
    uint32_t ok;
    bool late;
    do {
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        late = clock64() - t0 > limit;
    } while (!ok && !late && !(abort != nullptr && *abort));
    return ok && !late;
}

// The same in fewer instructions, for kernels whose code fills the instruction cache: the clock in 32 bits, so limits up to
// the default of 4e9 cycles; no test before the first wait.
__device__ __forceinline__ bool wait_short(uint32_t bar, uint32_t parity, const volatile int *abort, uint32_t limit)
{
    const uint32_t t0 = (uint32_t)clock();
    uint32_t ok;
    bool late;
    do {
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        late = (uint32_t)clock() - t0 > limit;
    } while (!ok && !late && !(abort != nullptr && *abort));
    return ok && !late;
}

// Transposes a 4 x 4 matrix of 16-byte units held by a quad of lanes: lane b ends with unit b of every lane.
__device__ __forceinline__ void quad_transpose(uint4 (&w)[4], int lane)
{
#pragma unroll
    for (int m = 1; m <= 2; m <<= 1) {
        const bool up = (lane & m) != 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k & m)
                continue;
            uint4 &a = w[k], &b = w[k | m];
            uint4 send = up ? a : b;
            send.x = __shfl_xor_sync(0xffffffffu, send.x, m);
            send.y = __shfl_xor_sync(0xffffffffu, send.y, m);
            send.z = __shfl_xor_sync(0xffffffffu, send.z, m);
            send.w = __shfl_xor_sync(0xffffffffu, send.w, m);
            if (up)
                a = send;
            else
                b = send;
        }
    }
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

// Four products D (TMEM) (+)= A x B in one block: one lane is elected for all, and the descriptors (or A's tensor
// memory address) advance by constants.  Called by a converged warp.
#define SK_MMA4(A_OP, A_TYPE)                                                                                    \
    "{\n\t.reg .pred p, t, e;\n\t.reg ." A_TYPE " a1, a2, a3;\n\t.reg .b64 b1, b2, b3;\n\t"                              \
    "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"                                                               \
    "add.s" A_OP " a1, %1, %5;\n\tadd.s" A_OP " a2, %1, %5 + %5;\n\tadd.s" A_OP " a3, %1, %5 + %5 + %5;\n\t"         \
    "add.s64 b1, %2, %6;\n\tadd.s64 b2, %2, %6 + %6;\n\tadd.s64 b3, %2, %6 + %6 + %6;\n\t"                           \
    "elect.sync _|e, 0xffffffff;\n\t"

template <int kStepA, int kStepB>
__device__ __forceinline__ void mma4_f16_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate)
{
    asm volatile(SK_MMA4("64", "b64")
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n\t}" ::"r"(d_tmem),
                 "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "n"(kStepA), "n"(kStepB)
                 : "memory");
}

template <int kStepA, int kStepB>
__device__ __forceinline__ void mma4_f8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate)
{
    asm volatile(SK_MMA4("64", "b64")
                 "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, t;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a2, b2, %3, t;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a3, b3, %3, t;\n\t}" ::"r"(d_tmem),
                 "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "n"(kStepA), "n"(kStepB)
                 : "memory");
}

// A in tensor memory, one row per lane, packed along the columns.
template <int kStepA, int kStepB>
__device__ __forceinline__ void mma4_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate)
{
    asm volatile(SK_MMA4("32", "b32")
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t;\n\t}" ::"r"(d_tmem),
                 "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "n"(kStepA), "n"(kStepB)
                 : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// The run of a CTA: the batch's total cost, sequence s costing cost(s), is cut into `count` equal runs, and [lo, hi) is
// that of `index`.  With `tail` > 0 as many short runs follow, which share the last 16th of the cost between them (nothing
// when the runs are shorter than `least`).  Finds the sequence that lo lies in and the cost before it.  `part` and `found`
// are shared memory (kThreads / 32 and 2 words of 64 bits); every thread of the block calls it, and all get the same
// answer.
struct Run {
    long long lo, hi, before;
    int s;
};

template <int kThreads, typename Cost>
__device__ __forceinline__ Run find_run(int bs, int index, int count, int tail, long long least, long long *part,
                                        long long *found, Cost cost)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (bs + kThreads - 1) / kThreads;
    const int s0 = min(bs, tid * per), s1 = min(bs, s0 + per);
    long long mine = 0;
#pragma unroll 1
    for (int s = s0; s < s1; ++s)
        mine += cost(s);
    long long incl = mine;                           // inclusive prefix within the warp
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, incl, o);
        incl += lane >= o ? u : 0;
    }
    if (lane == 31)
        part[warp] = incl;
    __syncthreads();
    long long total = 0, before = incl - mine;
#pragma unroll 1
    for (int w = 0; w < kThreads / 32; ++w) {
        const long long u = part[w];
        before += w < warp ? u : 0;
        total += u;
    }
    __syncthreads();                                 // the caller may use the memory for something else
    Run r;
    // a little more than total / count (a 64-bit division takes thousands of cycles in all threads)
    auto share = [](long long cost, int runs) {
        return (long long)((float)cost / (float)runs * (1.f + 0x1p-20f)) + 1;
    };
    const long long first = tail > 0 && total >= least * count ? total - total / 16 : total;
    const long long each = share(first, count), after = share(total - first, max(tail, 1));
    auto bound = [&](int i) {
        return i <= count ? min(first, each * i) : min(total, first + after * (i - count));
    };
    r.lo = bound(index);
    r.hi = bound(index + 1);
    if (mine > 0 && r.lo >= before && r.lo < before + mine) {
        int s = s0;
#pragma unroll 1
        for (; s < s1 - 1; ++s) {
            const long long size = cost(s);
            if (r.lo < before + size)
                break;
            before += size;
        }
        found[0] = before;
        found[1] = s;
    }
    __syncthreads();
    r.before = r.lo < r.hi ? found[0] : 0;
    r.s = r.lo < r.hi ? (int)found[1] : bs;
    return r;
}

// A run has two slots for its parts of what several runs share: 0 for one that does not start it, 1 for one that does.
// The slots of the parts of what ends in `index`'s slot 0, the last one first: the first slots of the runs before, back to
// the run with a part that starts it.  Called by a warp; returns how many.
template <typename Used>
__device__ __forceinline__ int shared_slots(int index, Used used, int *slots)
{
    const int lane = threadIdx.x & 31;
    int n = 0;
    for (int r0 = index; r0 >= 0; r0 -= 32) {
        const int r = r0 - lane;
        const bool first = r >= 0 && r < index && used(2 * r + 1);
        const uint32_t starts = __ballot_sync(0xffffffffu, first);
        const int stop = starts ? __ffs(starts) - 1 : 31;
        const bool has = r >= 0 && lane <= stop && (first || used(2 * r));
        const uint32_t all = __ballot_sync(0xffffffffu, has);
        if (has)
            slots[n + __popc(all & ((1u << lane) - 1u))] = 2 * r + (first ? 1 : 0);
        n += __popc(all);
        if (starts)
            break;
    }
    return n;
}

// Registers per thread that a kernel is launched with; -1 where the query fails.
template <typename Kernel>
int kernel_registers(Kernel kernel)
{
    cudaFuncAttributes a{};
    if (cudaFuncGetAttributes(&a, kernel) == cudaSuccess)
        return a.numRegs;
    cudaGetLastError();
    return -1;
}

// Q as two e4m3 terms for e4m3 pages: row (t, hq) becomes 128 hi codes, then 128 lo codes at codes + 256 * row, and
// 2^-e in the float array behind them.
cudaError_t launch_split_q(const uint16_t *q, long long rows, void *codes, cudaStream_t stream);

// Tensor map of Q rows [tokens][heads][256 bytes] (bf16, or e4m3 hi and lo codes): a box is 128 bytes of `heads` heads
// of `toks` tokens and lands as consecutive 128-byte-swizzled rows.
cudaError_t encode_q_map(CUtensorMap *map, const void *q, long long num_tokens, int H_q, bool fp8, int heads, int toks);

// Tensor map of the pages [blocks][heads][16 tokens][K | V] as 4-D: (128 bytes of a row, token within an 8-token
// group, 128-byte chunk of the row, 8-token group across all pages).  A box is `chunks` chunks of one page of one
// head and lands group by group, chunk by chunk, as 8 x 128 B swizzle atoms.
cudaError_t encode_page_map(CUtensorMap *map, const void *pages, long long num_blocks, int H_kv, bool fp8, int chunks);

}  // namespace sk
