// Rotary positions with several axes (time, height and width of image and video patches) with the KV write: one pass over
// this step's q, k and v.
//
// A pair (a, b) of a head's first rot_dim elements -- (2i, 2i + 1) interleaved, (i, i + rot_dim / 2) in halves -- turns by
// angle = positions[axes[i]][t] * freqs[i]:
//     a' = f (a cos - b sin),  b' = f (b cos + a sin)
// Everything else is as for the write with one axis (sk_rope.cu): its angles (64-bit fractions of a revolution, exact at any
// position), its roundings, the page rows, the eviction state.
//
// Bound by HBM (by latency for a decode step): each q, k and v element is read and written once.  A warp takes 16 rows of a
// token by itself, eight lanes a row, and a lane holds 16 bytes of the row's first and 16 of its second half of the
// turned elements (the pass-through elements after them likewise): a pair is always in one lane, no lane needs another's
// row, and no warp waits for another.  The rows come asynchronously into shared memory of the warp, a piece ahead; each
// lane takes two of the token's 64 angles, exchanged there too.  Warps stay for several pieces, so that the frequencies,
// whose fractions take FP64, are converted once.
//
// Measured, 8191 tokens of 32 query and 8 KV heads: 33.3 us to bf16 pages (201 MB, 6.0 TB/s), 32.2 us to e4m3 pages
// (185 MB, 5.7 TB/s); the rows of a token shared out among a CTA, with barriers and lanes that exchange partners, took 44.5
// and 38.3.  Pieces of 24 rows 33.6 and 36.3, of 32 35.4 and 54.3, of 12 with three CTAs of an SM 34.3 and 40.9, of 8 32.6
// and 44.4.  64 tokens: 2.8 us, of which an empty launch is about 2; with CTAs of eight warps there too, on fewer SMs, 3.6.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "sk_cache_ops.cuh"
#include "sk_quant.cuh"

namespace sk {
namespace {

constexpr int kThreads = 256;                    // at most; a warp where there is less than one for each SM
constexpr int kPasses = 4;                       // a pass is four rows of a warp
constexpr int kPieceRows = 4 * kPasses;          // rows of a token that a warp takes at once
constexpr int kStages = 2;                       // pieces of a warp in shared memory: this one and the next
constexpr int kPieceBytes = kPieceRows * kHeadDim * 2;
constexpr int kWarpBytes = kStages * kPieceBytes + kHeadDim / 2 * 8;     // and (cos, sin) of its token's angles
constexpr int kCtas = 2;                         // CTAs of an SM

struct AxesArgs {
    const uint16_t *q, *k, *v;
    long long q_stride, k_stride, v_stride;      // elements between tokens
    const int64_t *pos, *slots;
    long long pos_stride;                        // elements between axes
    const uint8_t *axes;
    const double *freqs;
    uint16_t *q_out;
    void *pages;
    float *acc;
    int32_t *pos_pages;
    int *status;
    long long num_slots;
    int num_axes, num_tokens, hq, hkv, rot, pieces;      // pieces of a token
    float factor, k_scale, v_scale;
};

// One product and one fused product and sum each, in the order of the write with one axis, so that text has its bits.
__device__ __forceinline__ void turn_pair(float &a, float &b, float2 cs)
{
    const float x = a;
    a = __fmaf_rn(x, cs.x, -__fmul_rn(b, cs.y));
    b = __fmaf_rn(b, cs.x, __fmul_rn(x, cs.y));
}

template <bool FP8, bool RECIP, bool INTER>
__global__ void __launch_bounds__(kThreads, kCtas) rope_axes_kernel(const AxesArgs a)
{
    extern __shared__ __align__(16) uint8_t smem[];
    wait_prior_grid();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = lane & 7, sub = lane >> 3;
    const int half = a.rot >> 1, rows = a.hq + 2 * a.hkv;
    uint8_t *ring = smem + warp * kWarpBytes;
    float2 *turn = reinterpret_cast<float2 *>(ring + kStages * kPieceBytes);
    // This lane's two units of eight elements: of the two halves of what turns, or two of those behind it.
    const bool low = part < half / 8;
    const int d0 = 8 * (low ? part : a.rot / 8 + 2 * (part - half / 8)), d1 = low ? d0 + half : d0 + 8;
    const bool turned = low;                     // of both units
    // The warp's pieces, every `stride`-th, by token and piece of it (with divisions of 64 bits e4m3 pages took 34.1 us).
    const int stride = gridDim.x * (blockDim.x >> 5), first = blockIdx.x * (blockDim.x >> 5) + warp;
    const int step_t = stride / a.pieces, step_piece = stride - step_t * a.pieces;
    struct Item {
        int t, piece;
    };
    auto after = [&](Item i) {
        i.t += step_t;
        i.piece += step_piece;
        if (i.piece >= a.pieces) {
            i.piece -= a.pieces;
            ++i.t;
        }
        return i;
    };
    // Copies of a piece's rows into stage `st`; always a group, of nothing past the end.
    auto fetch = [&](Item at, int st) {
        if (at.t < a.num_tokens) {
            const int t = at.t, r0 = at.piece * kPieceRows + sub;
            const uint32_t dst = (uint32_t)__cvta_generic_to_shared(ring + st * kPieceBytes + sub * 256);
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                const int r = r0 + 4 * i;
                const uint16_t *src = r < a.hq           ? a.q + t * a.q_stride + (long long)r * kHeadDim
                                      : r < a.hq + a.hkv ? a.k + t * a.k_stride + (long long)(r - a.hq) * kHeadDim
                                                         : a.v + t * a.v_stride + (long long)(r - a.hq - a.hkv) * kHeadDim;
                if (r < rows) {
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + i * 1024 + d0 * 2), "l"(src + d0)
                                 : "memory");
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + i * 1024 + d1 * 2), "l"(src + d1)
                                 : "memory");
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    Item item{first / a.pieces, first % a.pieces};
    if (item.t >= a.num_tokens)
        return;
    fetch(item, 0);
    // Pairs `lane` and `32 + lane`: revolutions per position, times 2^64, and the positions that they go by.
    uint64_t step[2] = {0, 0};
    const int64_t *own_pos[2] = {a.pos, a.pos};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int pair = 32 * i + lane;
        if (pair < half) {
            double rev = __ldg(a.freqs + pair) * 0.15915494309189533577;
            rev -= floor(rev);
            step[i] = (uint64_t)(rev * 18446744073709551616.0);
            const int axis = __ldg(a.axes + pair);
            if (axis < a.num_axes) {
                own_pos[i] += axis * a.pos_stride;
            } else {                             // no such axis: the pair stays as it is
                step[i] = 0;
                atomicOr(a.status, SK_DEV_BAD_SEQ);
            }
        }
    }
    struct Place {
        long long pos, slot, turn[2];
    };
    auto place = [&](Item at) {
        const int t = min(at.t, a.num_tokens - 1);
        return Place{__ldg(a.pos + t), __ldg(a.slots + t), {__ldg(own_pos[0] + t), __ldg(own_pos[1] + t)}};
    };
    Place next = place(item);
    for (int st = 0; item.t < a.num_tokens; st ^= 1) {
        const int t = item.t, r0 = item.piece * kPieceRows + sub;
        const long long pos = next.pos, slot = next.slot, turn_pos0 = next.turn[0], turn_pos1 = next.turn[1];
        __syncwarp();                            // every lane is done with the stage that is filled now
        item = after(item);
        fetch(item, st ^ 1);
        next = place(item);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (32 * i + lane < half) {
                const uint64_t phase = (uint64_t)(i ? turn_pos1 : turn_pos0) * step[i];
                float s, c;
                sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &s, &c);
                turn[32 * i + lane] = make_float2(c * a.factor, s * a.factor);
            }
        }
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncwarp();
        // of this lane's pairs: eight in halves, four of each unit interleaved
        float2 cs[8];
        if (turned) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                cs[e] = turn[INTER ? (e < 4 ? d0 / 2 + e : d1 / 2 + e - 4) : d0 + e];
        }
        __syncwarp();
        const uint8_t *rows_at = ring + st * kPieceBytes + sub * 256;
        const bool bad = slot >= a.num_slots, stored = slot >= 0 && !bad;
        if (bad && lane == 0)
            atomicOr(a.status, SK_DEV_BAD_BLOCK);
        const long long blk = stored ? slot / kPage : 0;
        const int off = (int)(stored ? slot - blk * kPage : 0);
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int r = r0 + 4 * i;
            if (r >= rows)
                continue;
            const bool is_v = r >= a.hq + a.hkv;
            float y[8], w[8];
            const uint4 x0 = *reinterpret_cast<const uint4 *>(rows_at + i * 1024 + d0 * 2);
            const uint4 x1 = *reinterpret_cast<const uint4 *>(rows_at + i * 1024 + d1 * 2);
            unpack_bf16x8(x0, y);
            unpack_bf16x8(x1, w);
            if (turned && !is_v) {               // (elements that do not turn keep their bits)
                if constexpr (INTER) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        turn_pair(y[2 * e], y[2 * e + 1], cs[e]);
                        turn_pair(w[2 * e], w[2 * e + 1], cs[4 + e]);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        turn_pair(y[e], w[e], cs[e]);
                }
            }
            if (r < a.hq) {
                uint16_t *dst = a.q_out + ((long long)t * a.hq + r) * kHeadDim;
                *reinterpret_cast<uint4 *>(dst + d0) = pack_bf16x8(y);
                *reinterpret_cast<uint4 *>(dst + d1) = pack_bf16x8(w);
            } else if (stored) {
                const int h = r - a.hq - (is_v ? a.hkv : 0);
                const long long row = (blk * a.hkv + h) * kPage + off;
                const long long at = row * (2 * kHeadDim) + (is_v ? kHeadDim : 0);
                if constexpr (FP8) {
                    const float sc = is_v ? a.v_scale : a.k_scale;
                    const float inv = RECIP ? 1.f / sc : 0.f;       // exact for a power of two
                    auto codes = [&](const float *z) {
                        return make_uint2(
                            quant_e4m3x2<RECIP>(z[0], z[1], sc, inv) | quant_e4m3x2<RECIP>(z[2], z[3], sc, inv) << 16,
                            quant_e4m3x2<RECIP>(z[4], z[5], sc, inv) | quant_e4m3x2<RECIP>(z[6], z[7], sc, inv) << 16);
                    };
                    *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.pages) + at + d0) = codes(y);
                    *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.pages) + at + d1) = codes(w);
                } else {
                    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.pages) + at + d0) = is_v ? x0 : pack_bf16x8(y);
                    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.pages) + at + d1) = is_v ? x1 : pack_bf16x8(w);
                }
                if (!is_v && part == 0) {
                    if (a.acc != nullptr)
                        a.acc[row] = 0.f;
                    if (a.pos_pages != nullptr)
                        a.pos_pages[row] = (int32_t)pos;
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_rope_axes(const uint16_t *q, const uint16_t *k, const uint16_t *v, long long q_stride,
                             long long k_stride, long long v_stride, const int64_t *pos, long long pos_stride, int num_axes,
                             const double *freqs, const uint8_t *axes, const int64_t *slots, int num_tokens, int hq,
                             int hkv, int rot, int interleaved, float factor, uint16_t *q_out, void *pages, int kv_dtype,
                             float k_scale, float v_scale, long long num_blocks, float *acc, int32_t *pos_pages,
                             int *status, int num_sms, cudaStream_t stream)
{
    AxesArgs a{q, k, v, q_stride, k_stride, v_stride, pos, slots, pos_stride, axes, freqs, q_out, pages, acc, pos_pages,
               status, num_blocks * kPage, num_axes, num_tokens, hq, hkv, rot, (hq + 2 * hkv + kPieceRows - 1) / kPieceRows,
               factor, k_scale, v_scale};
    const long long items = (long long)num_tokens * a.pieces;
    int warps = kThreads / 32;
    while (warps > 1 && items < (long long)warps * num_sms)
        warps >>= 1;
    const long long ctas = (items + warps - 1) / warps, most = (long long)num_sms * kCtas;
    const dim3 grid((unsigned)(ctas < most ? ctas : most));
    const bool fp8 = kv_dtype == SK_KV_FP8_E4M3;
    const bool recip = fp8 && exact_reciprocal(k_scale) && exact_reciprocal(v_scale);
    auto pick = [&](auto inter) {
        constexpr bool I = decltype(inter)::value;
        return !fp8 ? rope_axes_kernel<false, false, I> : recip ? rope_axes_kernel<true, true, I>
                                                                : rope_axes_kernel<true, false, I>;
    };
    auto kernel = interleaved ? pick(std::true_type{}) : pick(std::false_type{});
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kThreads / 32 * kWarpBytes);
    return e != cudaSuccess ? e : launch_pdl(kernel, grid, dim3(32 * warps), (size_t)warps * kWarpBytes, stream, a);
}

}  // namespace sk
