// Eviction from the cache by gathered attention weight: which rows of a (sequence, KV head) stay, and
// the move of the rows that stay into the places of those that go.
//
// Select.  Row r < L of (s, h) ranks by (its position is among the last `recent`, its weight, the lower
// row); the first `budget` rows stay.  With the staying rows at or past row `budget` listed in ascending
// order, the m-th of them takes the place of the m-th row below `budget` that goes (equally many).  Rows
// below `budget` that stay are not touched, so a step that is n rows over its budget moves at most n rows
// a head instead of closing every gap, and no place is both read and written.
//
// The threshold is found by radix selection on a 32-bit key that orders like the weight (11, 11 and 10 bits, fewer
// when a digit settles it): histogram in shared memory, then the digit that holds the budget-th largest key.  One
// cluster of up to 16 CTAs serves a (sequence, head); each CTA keeps the keys of its contiguous share of the rows in
// shared memory, so weights and positions are read once, four rows a load, and the cluster's histograms and counts
// are summed through distributed shared memory.  Two walks over the keys follow: one counts, per warp, the rows above
// the threshold and at it, below and past row `budget` (from these counts of all warps and CTAs follows how many ties
// each may take and where its lists start), one writes the lists.  Nothing depends on timing.
//
// Move.  One warp (half a warp for e4m3 rows) copies a row of 2 * head_dim elements, 16 bytes a lane, its
// weight and its position; several rows are in flight per warp.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <limits.h>
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
    int bt_stride, num_blocks, hkv, budget, recent, cap, max_len;
};

// Rows above the threshold and at it, below row `budget` (low) and from it on.
struct Counts {
    uint32_t above_low, ties_low, above_high, ties_high;
};

struct SelectShared {
    uint32_t hist[3][kBins];
    uint32_t warp_sum[kSelWarps];
    Counts warp[kSelWarps];
    Counts cta;                                  // read by the cluster
    uint32_t found_digit, found_above, found_count;
};

// Order-preserving key of a weight: larger weight, larger key; NaN like -inf; both zeros alike.
__device__ __forceinline__ uint32_t weight_key(float w)
{
    w = (w != w) ? -CUDART_INF_F : w + 0.f;
    const uint32_t u = __float_as_uint(w);
    return (u >> 31) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ uint32_t warp_sum_u32(uint32_t v) { return __reduce_add_sync(kFull, v); }

// Counts one digit of the warp's live keys.  Equal digits in the whole warp (rows never looked at, all zero) would
// serialise: one addition for all.
__device__ __forceinline__ void count_digit(uint32_t *hist, uint32_t digit, bool live)
{
    const uint32_t active = __ballot_sync(kFull, live);
    if (active == 0)
        return;
    const int first_lane = __ffs(active) - 1;
    const uint32_t first = __shfl_sync(kFull, digit, first_lane);
    if (__all_sync(kFull, !live || digit == first)) {
        if ((int)(threadIdx.x & 31) == first_lane)
            atomicAdd(hist + first, (uint32_t)__popc(active));
    } else if (live) {
        atomicAdd(hist + digit, 1u);
    }
}

__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(const SelectArgs a)
{
    extern __shared__ uint4 keys4[];             // four rows each
    __shared__ SelectShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int csize = (int)cluster.num_blocks(), crank = (int)cluster.block_rank();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int pair = blockIdx.x / csize;
    const int s = pair / a.hkv, h = pair - s * a.hkv;
    auto meet = [&]() {
        if (csize > 1)
            cluster.sync();
        else
            __syncthreads();
    };
#pragma unroll
    for (int d = 0; d < 3; ++d)
        reinterpret_cast<uint2 *>(sh.hist[d])[tid] = make_uint2(0u, 0u);
    wait_prior_grid();
    const int L = __ldg(a.seq_lens + s);
    const int edge = __ldg(a.next_pos + s) - a.recent;
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

    const int chunk = ((L + csize - 1) / csize + 127) / 128 * 128;
    const int lo = min(L, crank * chunk);
    const int n = min(chunk, L - lo);            // this CTA's rows [lo, lo + n)
    const int quads = (n + 3) / 4;
    __syncthreads();

    // ---- keys, and the first digit's histogram
    const int32_t *bt = a.block_table + (long long)s * a.bt_stride;
    constexpr int kAtOnce = 4;
    for (int i0 = 0; i0 < quads; i0 += kSelThreads * kAtOnce) {
        int blk[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int i = i0 + u * kSelThreads + tid;
            blk[u] = i < quads ? __ldg(bt + (lo + 4 * i) / kPage) : 0;
        }
        float4 w[kAtOnce];
        int4 p[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int i = i0 + u * kSelThreads + tid;
            w[u] = make_float4(-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F);
            p[u] = make_int4(INT_MIN, INT_MIN, INT_MIN, INT_MIN);
            if (i < quads) {
                if (blk[u] >= 0 && blk[u] < a.num_blocks) {
                    const long long at = ((long long)blk[u] * a.hkv + h) * kPage + (lo + 4 * i) % kPage;
                    w[u] = *reinterpret_cast<const float4 *>(a.acc + at);
                    if (a.recent > 0)
                        p[u] = *reinterpret_cast<const int4 *>(a.pos + at);
                } else {
                    atomicOr(a.status, SK_DEV_BAD_BLOCK);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int i = i0 + u * kSelThreads + tid;
            if (i0 + u * kSelThreads + warp * 32 >= quads)
                break;                           // uniform in the warp
            const bool rec = a.recent > 0;
            uint4 k;
            k.x = rec && p[u].x >= edge ? 0xFFFFFFFFu : weight_key(w[u].x);
            k.y = rec && p[u].y >= edge ? 0xFFFFFFFFu : weight_key(w[u].y);
            k.z = rec && p[u].z >= edge ? 0xFFFFFFFFu : weight_key(w[u].z);
            k.w = rec && p[u].w >= edge ? 0xFFFFFFFFu : weight_key(w[u].w);
            if (i < quads)
                keys4[i] = k;
            count_digit(sh.hist[0], k.x >> 21, 4 * i < n);
            count_digit(sh.hist[0], k.y >> 21, 4 * i + 1 < n);
            count_digit(sh.hist[0], k.z >> 21, 4 * i + 2 < n);
            count_digit(sh.hist[0], k.w >> 21, 4 * i + 3 < n);
        }
    }

    // ---- the budget-th largest key, digit by digit, until a digit's keys are all taken
    uint32_t prefix = 0, mask = 0, want = (uint32_t)a.budget;    // keys still to take among those with this prefix
    bool settled = false;
#pragma unroll
    for (int d = 0; d < 3; ++d) {
        constexpr int shift[3] = {21, 10, 0};
        if (settled)
            continue;
        if (d > 0) {
            for (int i0 = 0; i0 < quads; i0 += kSelThreads) {
                const int i = i0 + tid;
                const uint4 k = i < quads ? keys4[i] : make_uint4(0u, 0u, 0u, 0u);
                const uint32_t kk[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    count_digit(sh.hist[d], (kk[e] >> shift[d]) & (d == 1 ? 0x7FFu : 0x3FFu),
                                4 * i + e < n && (kk[e] & mask) == prefix);
            }
        }
        meet();                                  // every CTA's histogram is complete
        // thread t holds bins 2 t and 2 t + 1, summed over the cluster; suffix sums from the top bin down
        uint32_t b0 = 0, b1 = 0;
        if (csize > 1) {
#pragma unroll 4
            for (int c = 0; c < csize; ++c) {
                const uint2 v = *reinterpret_cast<const uint2 *>(cluster.map_shared_rank(&sh.hist[d][2 * tid], c));
                b0 += v.x;
                b1 += v.y;
            }
        } else {
            const uint2 v = *reinterpret_cast<const uint2 *>(&sh.hist[d][2 * tid]);
            b0 = v.x;
            b1 = v.y;
        }
        uint32_t above = b0 + b1;                // inclusive suffix over the warp's higher lanes
#pragma unroll
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
            sh.found_count = b1;
        } else if (above + b1 < want && above + b1 + b0 >= want) {
            sh.found_digit = 2 * tid;
            sh.found_above = above + b1;
            sh.found_count = b0;
        }
        __syncthreads();
        prefix |= sh.found_digit << shift[d];
        mask = d == 0 ? 0xFFE00000u : (d == 1 ? 0xFFFFFC00u : 0xFFFFFFFFu);
        want -= sh.found_above;
        settled = sh.found_count == want;
    }
    // rows with (key & mask) above `prefix` stay, and the first `want` rows that equal it

    // ---- first walk: a warp's rows are contiguous, [w0, w1) of this CTA's, 128 at a time
    const int per_warp = (n + kSelWarps * 128 - 1) / (kSelWarps * 128) * 128;
    const int w0 = min(n, warp * per_warp), w1 = min(n, w0 + per_warp);
    Counts mine = {0, 0, 0, 0};
    for (int i0 = w0; i0 < w1; i0 += 128) {
        const int i = i0 + 4 * lane;
        const uint4 k = i < w1 ? keys4[i / 4] : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t kk[4] = {k.x & mask, k.y & mask, k.z & mask, k.w & mask};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool live = i + e < w1, low = lo + i + e < a.budget;
            const uint32_t gt = live && kk[e] > prefix, eq = live && kk[e] == prefix;
            mine.above_low += low ? gt : 0u;
            mine.above_high += low ? 0u : gt;
            mine.ties_low += low ? eq : 0u;
            mine.ties_high += low ? 0u : eq;
        }
    }
    mine.above_low = warp_sum_u32(mine.above_low);
    mine.above_high = warp_sum_u32(mine.above_high);
    mine.ties_low = warp_sum_u32(mine.ties_low);
    mine.ties_high = warp_sum_u32(mine.ties_high);
    if (lane == 0)
        sh.warp[warp] = mine;
    __syncthreads();
    const Counts other = sh.warp[lane];          // kSelWarps == 32
    if (warp == 0) {
        const Counts all = {warp_sum_u32(other.above_low), warp_sum_u32(other.ties_low),
                            warp_sum_u32(other.above_high), warp_sum_u32(other.ties_high)};
        if (lane == 0)
            sh.cta = all;
    }
    meet();
    // ---- where this CTA's lists start: the CTAs before it, in row order
    uint32_t tie0 = 0, hole0 = 0, tail0 = 0;
    auto pass = [&](const Counts &c, int first_row, int rows) {
        // of `rows` rows from first_row on, ties are taken in order while the threshold has room
        const uint32_t low_rows = (uint32_t)max(0, min(rows, a.budget - first_row));
        const uint32_t room = want > tie0 ? want - tie0 : 0u;
        const uint32_t taken_low = min(room, c.ties_low), taken_high = min(room - taken_low, c.ties_high);
        hole0 += low_rows - c.above_low - taken_low;
        tail0 += c.above_high + taken_high;
        tie0 += c.ties_low + c.ties_high;
    };
    for (int c = 0; c < crank; ++c)
        pass(*cluster.map_shared_rank(&sh.cta, c), c * chunk, min(chunk, L - c * chunk));
    if (crank == csize - 1 && tid == 0) {
        const uint32_t before_tie = tie0, before_hole = hole0, before_tail = tail0;
        pass(sh.cta, lo, n);
        a.counts[pair] = (int32_t)tail0;
        if (tail0 > (uint32_t)a.cap)
            atomicOr(a.status, SK_DEV_INTERNAL);
        tie0 = before_tie;
        hole0 = before_hole;
        tail0 = before_tail;
    }
    if (csize > 1)
        cluster.barrier_arrive();                // this CTA has read the others' shared memory
    // and where this warp's do
    for (int w = 0; w < warp; ++w)
        pass(sh.warp[w], lo + min(n, w * per_warp), max(0, min(n, (w + 1) * per_warp) - min(n, w * per_warp)));

    // ---- second walk: the lists
    int32_t *src = a.src + (long long)pair * a.cap, *dst = a.dst + (long long)pair * a.cap;
    for (int i0 = w0; i0 < w1; i0 += 128) {
        const int i = i0 + 4 * lane;
        const uint4 k = i < w1 ? keys4[i / 4] : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t kk[4] = {k.x & mask, k.y & mask, k.z & mask, k.w & mask};
        uint32_t eqs = 0, stays = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            eqs |= (i + e < w1 && kk[e] == prefix) ? 1u << e : 0u;
            stays |= (i + e < w1 && kk[e] > prefix) ? 1u << e : 0u;
        }
        if (__any_sync(kFull, eqs != 0)) {
            uint32_t rank = __popc(eqs);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t u = __shfl_up_sync(kFull, rank, o);
                rank += lane >= o ? u : 0u;
            }
            const uint32_t total = __shfl_sync(kFull, rank, 31);
            rank += tie0 - __popc(eqs);
            tie0 += total;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (eqs >> e & 1u) {
                    stays |= rank < want ? 1u << e : 0u;
                    ++rank;
                }
            }
        }
        uint32_t holes = 0, tails = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool low = lo + i + e < a.budget, live = i + e < w1, st = stays >> e & 1u;
            holes |= live && low && !st ? 1u << e : 0u;
            tails |= live && !low && st ? 1u << e : 0u;
        }
        uint32_t both = __popc(holes) | __popc(tails) << 16;
        const uint32_t own = both;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(kFull, both, o);
            both += lane >= o ? u : 0u;
        }
        const uint32_t total = __shfl_sync(kFull, both, 31);
        both -= own;
        uint32_t hp = hole0 + (both & 0xFFFFu), tp = tail0 + (both >> 16);
        hole0 += total & 0xFFFFu;
        tail0 += total >> 16;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if ((holes >> e & 1u) && hp++ < (uint32_t)a.cap)
                dst[hp - 1] = lo + i + e;
            if ((tails >> e & 1u) && tp++ < (uint32_t)a.cap)
                src[tp - 1] = lo + i + e;
        }
    }
    if (csize > 1)
        cluster.barrier_wait();                  // no CTA leaves while another reads its counts
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
                                int32_t *counts, int32_t *new_lens, int *status, int num_sms, cudaStream_t stream)
{
    // The CTAs of a cluster hold all keys of the longest sequence in shared memory; with SMs to spare the cluster
    // grows to 8 CTAs (above that a cluster needs a whole GPC), as long as each has 4096 rows.
    const int pairs = bs * hkv;
    int c = (max_len + kEvictMaxChunk - 1) / kEvictMaxChunk;
    c = c < 1 ? 1 : c;
    int more = num_sms / pairs < (max_len + 4095) / 4096 ? num_sms / pairs : (max_len + 4095) / 4096;
    more = more < 8 ? more : 8;
    c = c > more ? c : more;
    SelectArgs a{acc, pos, block_table, seq_lens, next_pos, src, dst, counts, new_lens, status,
                 bt_stride, num_blocks, hkv, budget, recent, cap, max_len};
    const int chunk = ((max_len + c - 1) / c + 127) / 128 * 128;
    const size_t smem = (size_t)chunk * 4;
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
    cfg.numAttrs = c > 1 ? 2 : 1;
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
