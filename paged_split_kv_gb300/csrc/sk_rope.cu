// Rotary positions with the KV write: one pass over this step's q, k and v.
//
// A pair (a, b) of a head's first rot_dim elements -- (2i, 2i + 1) interleaved, (i, i + rot_dim / 2)
// in halves -- turns by pos * freqs[i]:
//     a' = f (a cos - b sin),  b' = f (b cos + a sin)
// with f the attention factor of a long-context scaling.  Elements past rot_dim pass through.  q goes to
// q_out; k, turned, and v go to the page row of the token's slot (the row layout and the e4m3 rounding of
// sk_reshape_and_cache, except that k is rounded once, from its turned fp32 value).
//
// Angles: a frequency is held as a 64-bit fixed-point fraction of a revolution per position, so
// pos * F modulo 2^64 is the exact fractional revolution of the rounded frequency at any position, and
// only its top 32 bits are converted to a float for sincospif.  (An fp32 product pos * w loses 2^-24 of
// the angle itself, 0.06 rad at position 10^6.)
//
// Bound by HBM (by latency for a decode step): each q, k and v element is read and written once.  A CTA
// takes a token at a time; half a warp holds one 256-byte row, 16 bytes a lane, so the turned partner of
// the half layout is another lane's register (one shuffle each) and the lane's cosines and sines are the
// same for all of the token's heads.  The rows' loads go out before the angles are computed.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "sk_cache_ops.cuh"
#include "sk_quant.cuh"

namespace sk {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsAtOnce = kThreads / 16;       // rows one pass of the CTA covers
constexpr int kPasses = 3;                       // rows in flight per thread

struct RopeArgs {
    const uint16_t *q, *k, *v;
    long long q_stride, k_stride, v_stride;      // elements between tokens
    const int64_t *pos, *slots;
    const double *freqs;
    uint16_t *q_out;
    void *pages;
    float *acc;
    int32_t *pos_pages;
    int *status;
    long long num_slots;
    int num_tokens, hq, hkv, rot;
    float factor, k_scale, v_scale;
};

template <bool FP8, bool RECIP, bool INTER>
__global__ void __launch_bounds__(kThreads) rope_cache_kernel(const RopeArgs a)
{
    __shared__ float2 turn[2][kHeadDim / 2];     // (cos, sin) of the token's angles, two tokens deep
    wait_prior_grid();
    const int tid = threadIdx.x;
    const int lane = tid & 31, sub = lane & 15, grp = tid >> 4;
    const int half = a.rot >> 1;
    const int d0 = sub * 8;                      // this lane's first dimension
    const bool turns = d0 < a.rot;
    const int rows = a.hq + 2 * a.hkv;

    uint64_t step = 0;                           // revolutions per position of frequency `tid`, times 2^64
    if (tid < half) {
        double rev = __ldg(a.freqs + tid) * 0.15915494309189533577;
        rev -= floor(rev);
        step = (uint64_t)(rev * 18446744073709551616.0);
    }
    int buf = 0;
    for (int t = blockIdx.x; t < a.num_tokens; t += gridDim.x, buf ^= 1) {
        const long long pos = __ldg(a.pos + t);
        const long long slot = __ldg(a.slots + t);
        const bool bad = slot >= a.num_slots;
        const bool stored = slot >= 0 && !bad;
        if (bad && tid == 0)
            atomicOr(a.status, SK_DEV_BAD_BLOCK);
        const long long blk = stored ? slot / kPage : 0;
        const int off = (int)(stored ? slot - blk * kPage : 0);
        for (int r0 = 0; r0 < rows; r0 += kRowsAtOnce * kPasses) {
            uint4 x[kPasses];
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                const int r = r0 + i * kRowsAtOnce + grp;
                const uint16_t *src = nullptr;
                if (r < a.hq)
                    src = a.q + t * a.q_stride + (long long)r * kHeadDim;
                else if (r < rows && stored)
                    src = r < a.hq + a.hkv ? a.k + t * a.k_stride + (long long)(r - a.hq) * kHeadDim
                                           : a.v + t * a.v_stride + (long long)(r - a.hq - a.hkv) * kHeadDim;
                x[i] = src != nullptr ? *reinterpret_cast<const uint4 *>(src + d0) : make_uint4(0u, 0u, 0u, 0u);
            }
            if (r0 == 0) {
                if (tid < half) {
                    const uint64_t phase = (uint64_t)pos * step;
                    float s, c;
                    sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &s, &c);
                    turn[buf][tid] = make_float2(c * a.factor, s * a.factor);
                }
                __syncthreads();
            }
            // this lane's cosines and sines: 4 pairs interleaved, 8 in halves
            float2 cs[INTER ? 4 : 8];
            if (turns) {
                const int f0 = INTER ? d0 / 2 : (d0 < half ? d0 : d0 - half);
#pragma unroll
                for (int i = 0; i < (INTER ? 4 : 8); ++i)
                    cs[i] = turn[buf][f0 + i];
            } else {
#pragma unroll
                for (int i = 0; i < (INTER ? 4 : 8); ++i)
                    cs[i] = make_float2(1.f, 0.f);
            }
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                if (r0 + i * kRowsAtOnce >= rows)
                    break;                       // uniform in the CTA
                const int r = r0 + i * kRowsAtOnce + grp;
                const bool is_v = r >= a.hq + a.hkv;
                float y[8];
                unpack_bf16x8(x[i], y);
                float z[8];
                if constexpr (INTER) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        z[2 * e] = y[2 * e] * cs[e].x - y[2 * e + 1] * cs[e].y;
                        z[2 * e + 1] = y[2 * e + 1] * cs[e].x + y[2 * e] * cs[e].y;
                    }
                } else {
                    // the partner dimensions are rot/2 away: rot/16 lanes up or down in the same row
                    const bool low = d0 < half;
                    const int partner = (lane & 16) | ((turns ? (low ? sub + half / 8 : sub - half / 8) : sub) & 15);
                    uint4 o;
                    o.x = __shfl_sync(0xffffffffu, x[i].x, partner);
                    o.y = __shfl_sync(0xffffffffu, x[i].y, partner);
                    o.z = __shfl_sync(0xffffffffu, x[i].z, partner);
                    o.w = __shfl_sync(0xffffffffu, x[i].w, partner);
                    float w[8];
                    unpack_bf16x8(o, w);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        z[e] = y[e] * cs[e].x + (low ? -w[e] : w[e]) * cs[e].y;
                }
                if (is_v || !turns) {            // untouched elements keep their bits (0 * inf would not)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        z[e] = y[e];
                }
                if (r < a.hq) {
                    *reinterpret_cast<uint4 *>(a.q_out + ((long long)t * a.hq + r) * kHeadDim + d0) = pack_bf16x8(z);
                } else if (r < rows && stored) {
                    const int h = r - a.hq - (is_v ? a.hkv : 0);
                    const long long row = (blk * a.hkv + h) * kPage + off;
                    const int col = (is_v ? kHeadDim : 0) + d0;
                    if constexpr (FP8) {
                        const float sc = is_v ? a.v_scale : a.k_scale;
                        const float inv = RECIP ? 1.f / sc : 0.f;       // exact for a power of two
                        uint2 c;
                        c.x = quant_e4m3x2<RECIP>(z[0], z[1], sc, inv) | quant_e4m3x2<RECIP>(z[2], z[3], sc, inv) << 16;
                        c.y = quant_e4m3x2<RECIP>(z[4], z[5], sc, inv) | quant_e4m3x2<RECIP>(z[6], z[7], sc, inv) << 16;
                        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.pages) + row * (2 * kHeadDim) + col) = c;
                    } else {
                        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.pages) + row * (2 * kHeadDim) + col) =
                            is_v ? x[i] : pack_bf16x8(z);
                    }
                    if (!is_v && sub == 0) {
                        if (a.acc != nullptr)
                            a.acc[row] = 0.f;
                        if (a.pos_pages != nullptr)
                            a.pos_pages[row] = (int32_t)pos;
                    }
                }
            }
        }
        // the other buffer is free again: every thread has passed this token's barrier, so all have
        // read the token before
    }
}

}  // namespace

cudaError_t launch_rope_cache(const uint16_t *q, const uint16_t *k, const uint16_t *v, long long q_stride,
                              long long k_stride, long long v_stride, const int64_t *pos, const double *freqs,
                              const int64_t *slots, int num_tokens, int hq, int hkv, int rot, int interleaved,
                              float factor, uint16_t *q_out, void *pages, int kv_dtype, float k_scale, float v_scale,
                              long long num_blocks, float *acc, int32_t *pos_pages, int *status, int num_sms,
                              cudaStream_t stream)
{
    RopeArgs a{q, k, v, q_stride, k_stride, v_stride, pos, slots, freqs, q_out, pages, acc, pos_pages, status,
               num_blocks * kPage, num_tokens, hq, hkv, rot, factor, k_scale, v_scale};
    const int cap = num_sms * 8;                 // 8 CTAs of 256 threads per SM
    const dim3 grid((unsigned)(num_tokens < cap ? num_tokens : cap));
    const bool fp8 = kv_dtype == SK_KV_FP8_E4M3;
    const bool recip = fp8 && exact_reciprocal(k_scale) && exact_reciprocal(v_scale);
    auto kernel = interleaved ? (!fp8 ? rope_cache_kernel<false, false, true>
                                 : recip ? rope_cache_kernel<true, true, true> : rope_cache_kernel<true, false, true>)
                              : (!fp8 ? rope_cache_kernel<false, false, false>
                                 : recip ? rope_cache_kernel<true, true, false> : rope_cache_kernel<true, false, false>);
    return launch_pdl(kernel, grid, dim3(kThreads), 0, stream, a);
}

}  // namespace sk
