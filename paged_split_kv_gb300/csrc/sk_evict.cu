// Eviction from the cache by gathered attention weight: which rows of a (sequence, KV head) stay, and
// the move of the rows that stay into the places of those that go.
//
// Select.  Row r < L of (s, h) ranks by (its position is among the last `recent`, its weight, the lower
// row); the first `budget` rows stay.  With the staying rows at or past row `budget` listed in ascending
// order, the m-th of them takes the place of the m-th row below `budget` that goes (equally many).  Rows
// below `budget` that stay are not touched, so a step that is n rows over its budget moves at most n rows
// a head instead of closing every gap, and no place is both read and written.
//
// The threshold is found by radix selection on a 32-bit key that orders like the weight (11, 11 and 10
// bits): histogram in shared memory, then the digit that holds the budget-th largest key.  One cluster of
// up to 16 CTAs serves a (sequence, head); each CTA keeps the keys of its contiguous share of the rows in
// shared memory, so weights and positions are read once, and the cluster's histograms and counts are
// summed through distributed shared memory.  Everything is counted, nothing depends on timing: ranks come
// from ballots and prefix sums.
//
// Move.  One warp (half a warp for e4m3 rows) copies a row of 2 * head_dim elements, 16 bytes a lane, its
// weight and its position; several rows are in flight per warp.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "sk_internal.cuh"

namespace sk {
namespace {

namespace cg = cooperative_groups;

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;

struct SelectArgs {
    const float *acc;
    const int32_t *pos;
    const int32_t *block_table;
    const int32_t *seq_lens;
    const int32_t *next_pos;
    int32_t *src, *dst, *counts, *new_lens;
    int *status;
    int bt_stride, num_blocks, hkv, budget, recent, cap, max_len, chunk;   // chunk: rows per CTA, a multiple of 32
};

struct SelectShared {
    uint32_t hist[3][kBins];
    uint32_t warp_sum[kSelWarps];
    uint32_t warp_a[kSelWarps], warp_b[kSelWarps];
    uint32_t found_digit, found_above;
    uint32_t ties, holes, tails;                 // this CTA's counts, read by the cluster
};

// Order-preserving key of a weight: larger weight, larger key; NaN like -inf; both zeros alike.
__device__ __forceinline__ uint32_t weight_key(float w)
{
    w = (w != w) ? -CUDART_INF_F : w + 0.f;
    const uint32_t u = __float_as_uint(w);
    return (u >> 31) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ uint32_t warp_sum_u32(uint32_t v) { return __reduce_add_sync(kFull, v); }

// Exclusive prefix over the CTA's warps of a per-warp count (the same in every lane); also the total.
__device__ __forceinline__ uint32_t warps_prefix(uint32_t v, uint32_t *buf, int warp, int lane, uint32_t *total)
{
    if (lane == 0)
        buf[warp] = v;
    __syncthreads();
    const uint32_t mine = buf[lane];             // kSelWarps == 32
    const uint32_t before = warp_sum_u32(lane < warp ? mine : 0u);
    *total = warp_sum_u32(mine);
    __syncthreads();
    return before;
}

__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(const SelectArgs a)
{
    extern __shared__ uint32_t keys[];           // [chunk]
    __shared__ SelectShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int csize = (int)cluster.num_blocks(), crank = (int)cluster.block_rank();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int pair = blockIdx.x / csize;
    const int s = pair / a.hkv, h = pair - s * a.hkv;
    wait_prior_grid();
    const int L = __ldg(a.seq_lens + s);
    const bool bad = L < 0 || L > a.max_len || (long long)L > (long long)a.bt_stride * kPage;
    const bool over = !bad && L > a.budget;
    if (crank == 0 && tid == 0) {
        if (bad)
            atomicOr(a.status, SK_DEV_BAD_SEQ);
        if (h == 0)
            a.new_lens[s] = over ? a.budget : L;
        if (!over)
            a.counts[pair] = 0;
    }
    if (!over)
        return;                                  // the whole cluster takes this branch

    const int lo = crank * a.chunk;
    const int n = max(0, min(a.chunk, L - lo));  // this CTA's rows [lo, lo + n)
    const int edge = __ldg(a.next_pos + s) - a.recent;
    for (int i = tid; i < 3 * kBins; i += kSelThreads)
        (&sh.hist[0][0])[i] = 0;
    __syncthreads();

    // ---- keys, and the first digit's histogram
    const int32_t *bt = a.block_table + (long long)s * a.bt_stride;
    auto count_digit = [&](uint32_t *hist, uint32_t digit, bool live) {
        // equal digits in the whole warp (rows never looked at, all zero) would serialise: one add
        const uint32_t active = __ballot_sync(kFull, live);
        if (active == 0)
            return;
        const uint32_t first = __shfl_sync(kFull, digit, __ffs(active) - 1);
        if (__all_sync(kFull, !live || digit == first)) {
            if (lane == 0)
                atomicAdd(hist + first, (uint32_t)__popc(active));
        } else if (live) {
            atomicAdd(hist + digit, 1u);
        }
    };
    for (int i0 = 0; i0 < n; i0 += kSelThreads) {
        const int i = i0 + tid;
        const bool live = i < n;
        uint32_t key = 0;
        if (live) {
            const int r = lo + i;
            const int blk = __ldg(bt + r / kPage);
            float w = -CUDART_INF_F;
            int pos = edge - 1;
            if (blk >= 0 && blk < a.num_blocks) {
                const long long at = ((long long)blk * a.hkv + h) * kPage + r % kPage;
                w = a.acc[at];
                pos = a.pos[at];
            } else {
                atomicOr(a.status, SK_DEV_BAD_BLOCK);
            }
            key = (a.recent > 0 && pos >= edge) ? 0xFFFFFFFFu : weight_key(w);
            keys[i] = key;
        }
        count_digit(sh.hist[0], key >> 21, live);
    }

    // ---- the budget-th largest key, digit by digit
    uint32_t prefix = 0, want = (uint32_t)a.budget;      // keys still to take among those with this prefix
    const int shift[3] = {21, 10, 0}, width[3] = {11, 11, 10};
#pragma unroll 1
    for (int d = 0; d < 3; ++d) {
        if (d > 0) {
            const uint32_t mask = d == 1 ? 0xFFE00000u : 0xFFFFFC00u;
            for (int i0 = 0; i0 < n; i0 += kSelThreads) {
                const int i = i0 + tid;
                const uint32_t key = i < n ? keys[i] : 0u;
                count_digit(sh.hist[d], (key >> shift[d]) & ((1u << width[d]) - 1u), i < n && (key & mask) == prefix);
            }
        }
        cluster.sync();                          // every CTA's histogram is complete
        // thread t holds bins 2 t and 2 t + 1, summed over the cluster; suffix sums from the top bin down
        uint32_t b0 = 0, b1 = 0;
        for (int c = 0; c < csize; ++c) {
            const uint2 v = *reinterpret_cast<const uint2 *>(cluster.map_shared_rank(&sh.hist[d][2 * tid], c));
            b0 += v.x;
            b1 += v.y;
        }
        uint32_t above = b0 + b1;                // inclusive suffix over the warp's higher lanes
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_down_sync(kFull, above, o);
            above += lane + o < 32 ? u : 0u;
        }
        if (lane == 0)
            sh.warp_sum[warp] = above;
        __syncthreads();
        const uint32_t higher = warp_sum_u32(lane > warp ? sh.warp_sum[lane] : 0u);
        above = above - b0 - b1 + higher;        // keys in bins above 2 t + 1
        if (above < want && above + b1 >= want) {
            sh.found_digit = 2 * tid + 1;
            sh.found_above = above;
        } else if (above + b1 < want && above + b1 + b0 >= want) {
            sh.found_digit = 2 * tid;
            sh.found_above = above + b1;
        }
        __syncthreads();
        prefix |= sh.found_digit << shift[d];
        want -= sh.found_above;
        __syncthreads();
    }
    // keys above `prefix` stay, and the first `want` rows whose key equals it

    // ---- a warp's rows are contiguous: [w0, w1) of this CTA's
    const int per_warp = (n + kSelWarps * 32 - 1) / (kSelWarps * 32) * 32;
    const int w0 = min(n, warp * per_warp), w1 = min(n, w0 + per_warp);
    uint32_t ties = 0;
    for (int i0 = w0; i0 < w1; i0 += 32) {
        const int i = i0 + lane;
        ties += __popc(__ballot_sync(kFull, i < w1 && keys[i] == prefix));
    }
    uint32_t cta_ties;
    uint32_t tie0 = warps_prefix(ties, sh.warp_sum, warp, lane, &cta_ties);
    if (tid == 0)
        sh.ties = cta_ties;
    cluster.sync();
    for (int c = 0; c < crank; ++c)
        tie0 += *cluster.map_shared_rank(&sh.ties, c);

    // the rows that go below the budget, and those that stay at or past it
    auto walk = [&](auto &&visit) {
        uint32_t tie = tie0;
        for (int i0 = w0; i0 < w1; i0 += 32) {
            const int i = i0 + lane;
            const uint32_t key = i < w1 ? keys[i] : 0u;
            const bool eq = i < w1 && key == prefix;
            const uint32_t eqs = __ballot_sync(kFull, eq);
            const uint32_t rank = tie + __popc(eqs & ((1u << lane) - 1u));
            tie += __popc(eqs);
            const bool stays = i < w1 && (key > prefix || (eq && rank < want));
            const int r = lo + i;
            visit(r, i < w1 && !stays && r < a.budget, stays && r >= a.budget);
        }
    };
    uint32_t holes = 0, tails = 0;
    walk([&](int, bool hole, bool tail) {
        holes += __popc(__ballot_sync(kFull, hole));
        tails += __popc(__ballot_sync(kFull, tail));
    });
    uint32_t cta_holes, cta_tails;
    uint32_t hole0 = warps_prefix(holes, sh.warp_a, warp, lane, &cta_holes);
    uint32_t tail0 = warps_prefix(tails, sh.warp_b, warp, lane, &cta_tails);
    if (tid == 0) {
        sh.holes = cta_holes;
        sh.tails = cta_tails;
    }
    cluster.sync();
    for (int c = 0; c < crank; ++c) {
        hole0 += *cluster.map_shared_rank(&sh.holes, c);
        tail0 += *cluster.map_shared_rank(&sh.tails, c);
    }
    if (crank == csize - 1 && tid == 0) {
        const uint32_t all = tail0 + cta_tails;  // warp 0's prefix is 0
        a.counts[pair] = (int32_t)all;
        if (all > (uint32_t)a.cap)
            atomicOr(a.status, SK_DEV_INTERNAL);
    }
    int32_t *src = a.src + (long long)pair * a.cap, *dst = a.dst + (long long)pair * a.cap;
    walk([&](int r, bool hole, bool tail) {
        const uint32_t hm = __ballot_sync(kFull, hole), tm = __ballot_sync(kFull, tail);
        const uint32_t below = (1u << lane) - 1u;
        if (hole && hole0 + __popc(hm & below) < (uint32_t)a.cap)
            dst[hole0 + __popc(hm & below)] = r;
        if (tail && tail0 + __popc(tm & below) < (uint32_t)a.cap)
            src[tail0 + __popc(tm & below)] = r;
        hole0 += __popc(hm);
        tail0 += __popc(tm);
    });
    cluster.sync();                              // no CTA leaves while another reads its counts
}

constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 4;                     // rows in flight per warp (bf16) or half warp (e4m3)

template <bool FP8>
__global__ void __launch_bounds__(kMoveThreads)
evict_move_kernel(const int32_t *__restrict__ src, const int32_t *__restrict__ dst,
                  const int32_t *__restrict__ counts, int cap, int ctas_per_pair,
                  const int32_t *__restrict__ block_table, int bt_stride, int num_blocks, int hkv, uint8_t *pages, float *acc, int32_t *pos, int *status)
{
    constexpr int kLanes = FP8 ? 16 : 32;        // lanes per row, 16 bytes each
    constexpr int kRowBytes = kLanes * 16;
    wait_prior_grid();
    const int pair = blockIdx.x / ctas_per_pair, part = blockIdx.x - pair * ctas_per_pair;
    const int s = pair / hkv, h = pair - s * hkv;
    int n = __ldg(counts + pair);
    if (n < 0 || n > cap) {
        if (threadIdx.x == 0 && part == 0)
            atomicOr(status, SK_DEV_BAD_SEQ);
        n = n < 0 ? 0 : cap;
    }
    const int sub = threadIdx.x % kLanes;
    const int unit = (part * kMoveThreads + threadIdx.x) / kLanes;
    const int units = ctas_per_pair * (kMoveThreads / kLanes);
    const int32_t *bt = block_table + (long long)s * bt_stride;
    const long long max_row = (long long)bt_stride * kPage;
    // the page row of logical row r, or -1
    auto place = [&](int r) -> long long {
        if (r < 0 || r >= max_row) {
            atomicOr(status, SK_DEV_BAD_SEQ);
            return -1;
        }
        const int blk = __ldg(bt + r / kPage);
        if (blk < 0 || blk >= num_blocks) {
            atomicOr(status, SK_DEV_BAD_BLOCK);
            return -1;
        }
        return ((long long)blk * hkv + h) * kPage + r % kPage;
    };
    for (int m0 = unit * kMoveRows; m0 < n; m0 += units * kMoveRows) {
        uint4 x[kMoveRows];
        long long to[kMoveRows];
        float w[kMoveRows];
        int32_t p[kMoveRows];
#pragma unroll
        for (int i = 0; i < kMoveRows; ++i) {
            to[i] = -1;
            if (m0 + i < n) {
                const long long from = place(__ldg(src + (long long)pair * cap + m0 + i));
                to[i] = place(__ldg(dst + (long long)pair * cap + m0 + i));
                if (from < 0)
                    to[i] = -1;
                if (to[i] >= 0) {
                    x[i] = *reinterpret_cast<const uint4 *>(pages + from * kRowBytes + sub * 16);
                    if (sub == 0) {
                        w[i] = acc[from];
                        p[i] = pos[from];
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kMoveRows; ++i) {
            if (to[i] < 0)
                continue;
            *reinterpret_cast<uint4 *>(pages + to[i] * kRowBytes + sub * 16) = x[i];
            if (sub == 0) {
                acc[to[i]] = w[i];
                pos[to[i]] = p[i];
            }
        }
    }
}

}  // namespace

cudaError_t launch_evict_select(const float *acc, const int32_t *pos, const int32_t *block_table, int bt_stride,
                                int num_blocks, const int32_t *seq_lens, const int32_t *next_pos, int bs, int hkv,
                                int budget, int recent, int max_len, int cap, int32_t *src, int32_t *dst,
                                int32_t *counts, int32_t *new_lens, int *status, cudaStream_t stream)
{
    // the smallest cluster whose CTAs hold their share of the keys in half an SM's shared memory, so that
    // two CTAs fit; 16 CTAs (a size that has to be allowed explicitly) with up to 192 KB each past that
    int c = 1;
    while (c < kEvictMaxCluster && (long long)c * (kEvictMaxChunk / 2) < max_len)
        c *= 2;
    SelectArgs a{acc, pos, block_table, seq_lens, next_pos, src, dst, counts, new_lens, status,
                 bt_stride, num_blocks, hkv, budget, recent, cap, max_len, 0};
    a.chunk = ((max_len + c - 1) / c + 31) / 32 * 32;
    const size_t smem = (size_t)a.chunk * 4;
    cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kEvictMaxChunk * 4);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)bs * (unsigned)hkv * (unsigned)c);
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)c;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, evict_select_kernel, a);
}

cudaError_t launch_evict_move(const int32_t *src, const int32_t *dst, const int32_t *counts, int cap, int bs, int hkv,
                              const int32_t *block_table, int bt_stride, int num_blocks, void *pages, int kv_dtype,
                              float *acc, int32_t *pos, int *status, int num_sms, cudaStream_t stream)
{
    const bool fp8 = kv_dtype == SK_KV_FP8_E4M3;
    const int pairs = bs * hkv;
    const int rows_per_cta = kMoveThreads / (fp8 ? 16 : 32) * kMoveRows;
    const int want = (cap + rows_per_cta - 1) / rows_per_cta;
    const int fill = (num_sms * 8 + pairs - 1) / pairs;          // 8 CTAs of 256 threads per SM over all pairs
    const int per_pair = want < fill ? want : fill;
    return launch_pdl(fp8 ? evict_move_kernel<true> : evict_move_kernel<false>,
                      dim3((unsigned)pairs * (unsigned)per_pair), dim3(kMoveThreads), 0, stream, src, dst, counts, cap,
                      per_pair, block_table, bt_stride, num_blocks, hkv, static_cast<uint8_t *>(pages),
                      acc, pos, status);
}

}  // namespace sk
