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
// cluster of up to 16 CTAs serves a (sequence, head); each CTA keeps the keys of its contiguous share of the rows, the
// first 49152 in shared memory and 16384 more in registers, so weights and positions are read once, four rows a load, and the
// cluster's histograms and counts are summed through distributed shared memory.  Two walks over the keys follow: one
// counts, per warp, the rows above the threshold and at it, below and past row `budget` (from these counts of all warps
// and CTAs follows how many ties each may take and where its lists start), one writes the lists.  Nothing depends on
// timing.  Bound by instructions, a few per row and pass: four rows a lane throughout, with a path without masks for
// whole blocks of 128 rows (32 heads of up to 248k rows, 62k rows a CTA: load and first digit 18.5 us, second digit
// 8.5, walks 4 and 9, three exchanges 8).
//
// Move.  One warp (half a warp for e4m3 rows) copies a row of 2 * head_dim elements, 16 bytes a lane, its
// weight and its position; several rows are in flight per warp.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <math_constants.h>
#include <stdint.h>

#include "sk_cache_ops.cuh"

namespace sk {
namespace {

namespace cg = cooperative_groups;

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kAtOnce = 4;                       // row quads a thread loads at once
// Row quads of a CTA that are kept: the first in shared memory (192 KB, beside the histograms), the next in registers.
constexpr int kSharedQuads = 12 * kSelThreads, kKeptQuads = kSharedQuads + kAtOnce * kSelThreads;

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

// Counts one digit of the live ones among four keys a lane.  Equal digits in the whole warp (rows never looked at, all
// zero) would serialise: one addition for all.
__device__ __forceinline__ void count_digits(uint32_t *hist, const uint4 &digit, bool m0, bool m1, bool m2, bool m3)
{
    const uint32_t first = __shfl_sync(kFull, digit.x, 0);
    const bool same = digit.x == first && digit.y == first && digit.z == first && digit.w == first;
    if (__all_sync(kFull, same && m0 && m1 && m2 && m3)) {
        if ((threadIdx.x & 31) == 0)
            atomicAdd(hist + first, 128u);
        return;
    }
    if (m0)
        atomicAdd(hist + digit.x, 1u);
    if (m1)
        atomicAdd(hist + digit.y, 1u);
    if (m2)
        atomicAdd(hist + digit.z, 1u);
    if (m3)
        atomicAdd(hist + digit.w, 1u);
}

// Lane l holds the counts of the l-th of up to 32 consecutive parts of a row range.  Ties are taken in row order while
// the threshold has room for them: gives the number of ties before lane l's part, and the part's rows for either list.
struct Part {
    uint32_t ties_before, holes, tails;
};

__device__ __forceinline__ Part part_of(const Counts &c, int first_row, int rows, int budget, uint32_t want,
                                        uint32_t ties_before, int lane)
{
    const uint32_t ties = c.ties_low + c.ties_high;
    uint32_t incl = ties;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(kFull, incl, o);
        incl += lane >= o ? u : 0u;
    }
    Part p;
    p.ties_before = ties_before + incl - ties;
    const uint32_t room = want > p.ties_before ? want - p.ties_before : 0u;
    const uint32_t low = min(room, c.ties_low), high = min(room - low, c.ties_high);
    p.holes = (uint32_t)max(0, min(rows, budget - first_row)) - c.above_low - low;
    p.tails = c.above_high + high;
    return p;
}

// Waits until all but the last N groups of this thread's asynchronous copies are done.
template <int N>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(const SelectArgs a)
{
    extern __shared__ uint4 keys4[];             // four rows each, the first kSharedQuads of this CTA's
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
    for (int i = tid; i < 3 * kBins / 2; i += kSelThreads)
        reinterpret_cast<uint2 *>(sh.hist)[i] = make_uint2(0u, 0u);
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
    const int32_t *bt = a.block_table + (long long)s * a.bt_stride;
    __syncthreads();

    // the keys of row quad i, from its weights and positions; block_of is -1 past the rows, and for a bad block (reported)
    auto block_of = [&](int i) {
        const int blk = i < quads ? __ldg(bt + (lo + 4 * i) / kPage) : 0;
        if (blk < 0 || blk >= a.num_blocks)
            atomicOr(a.status, SK_DEV_BAD_BLOCK);
        return i < quads && blk < a.num_blocks ? blk : -1;
    };
    auto place_of = [&](int i, int blk) { return ((long long)blk * a.hkv + h) * kPage + (lo + 4 * i) % kPage; };
    const float4 no_weight = make_float4(-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F);
    const int4 no_pos = make_int4(INT_MIN, INT_MIN, INT_MIN, INT_MIN);
    auto weights = [&](int i, int blk) {
        return blk >= 0 ? *reinterpret_cast<const float4 *>(a.acc + place_of(i, blk)) : no_weight;
    };
    auto positions = [&](int i, int blk) {
        return blk >= 0 && a.recent > 0 ? *reinterpret_cast<const int4 *>(a.pos + place_of(i, blk)) : no_pos;
    };
    auto key_of = [&](float w, int pos) { return a.recent > 0 && pos >= edge ? 0xFFFFFFFFu : weight_key(w); };
    auto quad_key = [&](const float4 &w, const int4 &p) {
        return make_uint4(key_of(w.x, p.x), key_of(w.y, p.y), key_of(w.z, p.z), key_of(w.w, p.w));
    };
    auto quad_again = [&](int i) {               // computed again, past what is kept
        const int blk = block_of(i);
        return quad_key(weights(i, blk), positions(i, blk));
    };
    auto count_first = [&](int i, const uint4 &k) {
        count_digits(sh.hist[0], make_uint4(k.x >> 21, k.y >> 21, k.z >> 21, k.w >> 21), 4 * i < n, 4 * i + 1 < n,
                     4 * i + 2 < n, 4 * i + 3 < n);
    };

    // ---- keys, and the first digit's histogram.  The weights of all quads kept in shared memory are copied there at
    // once, asynchronously, and become keys in place; positions are loaded a round ahead (against loads four at a time: 68
    // us for 72 with a cold L2, 49 for 50 with a warm one).
    constexpr int kRounds = kSharedQuads / (kAtOnce * kSelThreads);
    static_assert(kRounds == 3, "the waits below");
    int blk[kRounds * kAtOnce];                  // -1 where this CTA has no rows (in short sequences, some have none at all)
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
#pragma unroll
        for (int u = r * kAtOnce; u < (r + 1) * kAtOnce; ++u)
            blk[u] = -1;
        if (r * kAtOnce * kSelThreads < quads) {     // uniform in the CTA
#pragma unroll
            for (int u = r * kAtOnce; u < (r + 1) * kAtOnce; ++u)
                blk[u] = block_of(u * kSelThreads + tid);
        }
    }
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        if (r * kAtOnce * kSelThreads >= quads)
            break;
#pragma unroll
        for (int u = r * kAtOnce; u < (r + 1) * kAtOnce; ++u) {
            const int i = u * kSelThreads + tid;
            if (blk[u] >= 0)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                 (uint32_t)__cvta_generic_to_shared(keys4 + i)),
                             "l"(a.acc + place_of(i, blk[u]))
                             : "memory");
            else if (i < quads)
                reinterpret_cast<float4 *>(keys4)[i] = no_weight;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    uint4 held[kAtOnce] = {};                    // this thread's quads kSharedQuads + u * kSelThreads + tid
    int4 p[2][kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u)
        p[0][u] = positions(u * kSelThreads + tid, blk[u]);
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        if (r * kAtOnce * kSelThreads >= quads)
            break;
        if (r + 1 < kRounds && (r + 1) * kAtOnce * kSelThreads < quads) {
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u)
                p[(r + 1) & 1][u] = positions(((r + 1) * kAtOnce + u) * kSelThreads + tid, blk[(r + 1) * kAtOnce + u]);
        }
        // with fewer rounds there are fewer groups behind this one
        if (r == 0 && 2 * kAtOnce * kSelThreads < quads)
            copies_wait<2>();
        else if (r <= 1 && (r + 1) * kAtOnce * kSelThreads < quads)
            copies_wait<1>();
        else
            copies_wait<0>();
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int i = (r * kAtOnce + u) * kSelThreads + tid;
            if (i - lane >= quads)
                break;                           // uniform in the warp
            uint4 k = make_uint4(0u, 0u, 0u, 0u);
            if (i < quads) {
                k = quad_key(reinterpret_cast<const float4 *>(keys4)[i], p[r & 1][u]);
                keys4[i] = k;
            }
            count_first(i, k);
        }
    }
    if (kSharedQuads + tid - lane < quads) {
        float4 w[kAtOnce];
        int4 q[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int i = kSharedQuads + u * kSelThreads + tid, b = block_of(i);
            w[u] = weights(i, b);
            q[u] = positions(i, b);
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int i = kSharedQuads + u * kSelThreads + tid;
            if (i - lane >= quads)
                break;
            held[u] = quad_key(w[u], q[u]);
            count_first(i, held[u]);
        }
#pragma unroll 1
        for (int i = kKeptQuads + tid; i - lane < quads; i += kSelThreads)
            count_first(i, quad_again(i));
    }

    // ---- the budget-th largest key, digit by digit, until a digit's keys are all taken
    uint32_t prefix = 0, mask = 0, want = (uint32_t)a.budget;    // keys still to take among those with this prefix
    int used = 0;                                // digits
#pragma unroll 1
    for (int d = 0; d < 3; ++d) {
        const int shift = d == 0 ? 21 : (d == 1 ? 10 : 0);
        if (d > 0) {
            const uint32_t digit = d == 1 ? 0x7FFu : 0x3FFu;
            auto count_quad = [&](int i, const uint4 &k) {
                const int left = n - 4 * i;
                const bool m0 = left > 0 && (k.x & mask) == prefix, m1 = left > 1 && (k.y & mask) == prefix;
                const bool m2 = left > 2 && (k.z & mask) == prefix, m3 = left > 3 && (k.w & mask) == prefix;
                if (!__any_sync(kFull, m0 || m1 || m2 || m3))
                    return;
                count_digits(sh.hist[d], make_uint4(k.x >> shift & digit, k.y >> shift & digit, k.z >> shift & digit,
                                                    k.w >> shift & digit), m0, m1, m2, m3);
            };
            const int in_shared = min(quads, kSharedQuads);
#pragma unroll 1
            for (int i = tid; i - lane < in_shared; i += kSelThreads)
                count_quad(i, i < in_shared ? keys4[i] : make_uint4(0u, 0u, 0u, 0u));
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u)
                if (kSharedQuads + u * kSelThreads + tid - lane < quads)
                    count_quad(kSharedQuads + u * kSelThreads + tid, held[u]);
#pragma unroll 1
            for (int i = kKeptQuads + tid; i - lane < quads; i += kSelThreads)
                count_quad(i, quad_again(i));
        }
        meet();                                  // every CTA's histogram is complete
        // thread t holds bins 2 t and 2 t + 1, summed over the cluster; suffix sums from the top bin down
        uint32_t b0 = 0, b1 = 0;
#pragma unroll 4
        for (int c = 0; c < csize; ++c) {
            const uint2 *at = reinterpret_cast<const uint2 *>(&sh.hist[d][2 * tid]);
            const uint2 v = csize > 1 ? *cluster.map_shared_rank(at, c) : *at;
            b0 += v.x;
            b1 += v.y;
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
        prefix |= sh.found_digit << shift;
        mask = 0xFFFFFFFFu << shift;
        want -= sh.found_above;
        ++used;
        if (sh.found_count == want)
            break;                               // the same in every thread of the cluster
    }
    // rows with (key & mask) above `prefix` stay, and the first `want` rows that equal it

    const uint32_t top = prefix | ~mask;         // the largest key of that prefix
    // Of four rows, bits 0-3: above the threshold; bits 4-7: at it.
    auto classes = [&](const uint4 &k) {
        const uint32_t gt = (uint32_t)(k.x > top) | (uint32_t)(k.y > top) << 1 | (uint32_t)(k.z > top) << 2 |
                            (uint32_t)(k.w > top) << 3;
        const uint32_t ge = (uint32_t)(k.x >= prefix) | (uint32_t)(k.y >= prefix) << 1 |
                            (uint32_t)(k.z >= prefix) << 2 | (uint32_t)(k.w >= prefix) << 3;
        return gt | (ge ^ gt) << 4;
    };
    // the quads in registers lie at other warps than those that walk over them: their classes go to a histogram that
    // no CTA reads any more
    uint8_t *flags = reinterpret_cast<uint8_t *>(sh.hist[used % 3]);
    if (quads > kSharedQuads) {
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u)
            flags[u * kSelThreads + tid] = (uint8_t)classes(held[u]);
        __syncthreads();
    }

    // ---- first walk: a warp's rows are contiguous, [w0, w1) of this CTA's, four a lane; those before wm lie below the
    // budget
    const int per_warp = (n + 4 * kSelThreads - 1) / (4 * kSelThreads) * 128;
    const int w0 = min(n, warp * per_warp), w1 = min(n, w0 + per_warp), wm = min(w1, max(w0, a.budget - lo));
    // classes of rows [r, r + 4), of those before w1, and which of them lie below the budget
    auto quad_classes = [&](int r, uint32_t &low) {
        const int i = r / 4;
        low = 0;
        if (r >= w1)
            return 0u;
        const uint32_t c = i < kSharedQuads  ? classes(keys4[i])
                           : i < kKeptQuads ? flags[i - kSharedQuads]
                                            : classes(quad_again(i));
        low = wm - r >= 4 ? 15u : (1u << max(0, wm - r)) - 1u;
        const uint32_t real = w1 - r >= 4 ? 15u : (1u << (w1 - r)) - 1u;
        return c & (real | real << 4);
    };
    // 128 rows from r0 on that are real, kept in shared memory and on one side of the budget need no masks
    auto plain = [&](int r0) { return r0 + 128 <= min(w1, 4 * kSharedQuads) && (r0 + 128 <= wm || r0 >= wm); };
    Counts mine = {0, 0, 0, 0};
#pragma unroll 2
    for (int r = w0 + 4 * lane; r - 4 * lane < w1; r += 128) {
        if (plain(r - 4 * lane)) {
            const uint4 k = keys4[r / 4];
            const uint32_t gt = (k.x > top) + (k.y > top) + (k.z > top) + (k.w > top);
            const uint32_t eq = (k.x >= prefix) + (k.y >= prefix) + (k.z >= prefix) + (k.w >= prefix) - gt;
            if (r - 4 * lane < wm) {
                mine.above_low += gt;
                mine.ties_low += eq;
            } else {
                mine.above_high += gt;
                mine.ties_high += eq;
            }
            continue;
        }
        uint32_t low;
        const uint32_t c = quad_classes(r, low), gt = c & 15u, eq = c >> 4;
        mine.above_low += __popc(gt & low);
        mine.ties_low += __popc(eq & low);
        mine.above_high += __popc(gt & ~low);
        mine.ties_high += __popc(eq & ~low);
    }
    mine.above_low = warp_sum_u32(mine.above_low);
    mine.ties_low = warp_sum_u32(mine.ties_low);
    mine.above_high = warp_sum_u32(mine.above_high);
    mine.ties_high = warp_sum_u32(mine.ties_high);
    if (lane == 0)
        sh.warp[warp] = mine;
    __syncthreads();
    const Counts other = sh.warp[lane];          // kSelWarps == 32
    const Counts all = {warp_sum_u32(other.above_low), warp_sum_u32(other.ties_low), warp_sum_u32(other.above_high),
                        warp_sum_u32(other.ties_high)};
    uint32_t tie0 = 0, hole0 = 0, tail0 = 0;
    if (csize > 1) {
        // where this CTA's lists start: the CTAs before it, in row order
        if (tid == 0)
            sh.cta = all;
        cluster.sync();
        Counts c = {0, 0, 0, 0};
        if (lane < csize)
            c = *cluster.map_shared_rank(&sh.cta, lane);
        cluster.barrier_arrive();                // this CTA has read the others' shared memory
        const int first = min(L, lane * chunk);
        const Part part = part_of(c, first, lane < csize ? min(chunk, L - first) : 0, a.budget, want, 0, lane);
        tie0 = __shfl_sync(kFull, part.ties_before, crank);
        hole0 = warp_sum_u32(lane < crank ? part.holes : 0u);
        tail0 = warp_sum_u32(lane < crank ? part.tails : 0u);
    }
    {
        // and where this warp's do
        const int first = min(n, lane * per_warp);
        const Part part = part_of(other, lo + first, min(per_warp, n - first), a.budget, want, tie0, lane);
        if (crank == csize - 1 && warp == 0) {
            const uint32_t moves = tail0 + warp_sum_u32(part.tails);
            if (lane == 0) {
                a.counts[pair] = (int32_t)moves;
                if (moves > (uint32_t)a.cap)
                    atomicOr(a.status, SK_DEV_INTERNAL);
            }
        }
        tie0 = __shfl_sync(kFull, part.ties_before, warp);
        hole0 += warp_sum_u32(lane < warp ? part.holes : 0u);
        tail0 += warp_sum_u32(lane < warp ? part.tails : 0u);
    }

    // ---- second walk: the lists, 128 rows at a time
    const uint32_t below = (1u << lane) - 1u;
    int32_t *dst = a.dst + (long long)pair * a.cap, *src = a.src + (long long)pair * a.cap;
#pragma unroll 1
    for (int r = w0 + 4 * lane; r - 4 * lane < w1; r += 128) {
        const int r0 = r - 4 * lane;
        if (plain(r0)) {                         // row r0 + 32 j + lane is this lane's: fewer instructions a row
            int32_t *list = r0 < wm ? dst : src;
            const uint32_t flip = r0 < wm ? kFull : 0u;
            uint32_t at = r0 < wm ? hole0 : tail0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t k = reinterpret_cast<const uint32_t *>(keys4)[r0 + 32 * j + lane];
                uint32_t stays = __ballot_sync(kFull, k > top);
                const uint32_t ties = __ballot_sync(kFull, k >= prefix) ^ stays;
                if (ties != 0) {                 // they stay in row order while there is room
                    stays |= __ballot_sync(kFull, (ties >> lane & 1u) && tie0 + __popc(ties & below) < want);
                    tie0 += __popc(ties);
                }
                const uint32_t listed = stays ^ flip, to = at + __popc(listed & below);
                if ((listed >> lane & 1u) && to < (uint32_t)a.cap)
                    list[to] = lo + r0 + 32 * j + lane;
                at += __popc(listed);
            }
            (r0 < wm ? hole0 : tail0) = at;
            continue;
        }
        uint32_t low;
        const uint32_t c = quad_classes(r, low);
        const uint32_t real = r >= w1 ? 0u : w1 - r >= 4 ? 15u : (1u << (w1 - r)) - 1u;
        uint32_t stays = c & 15u;
        if (__any_sync(kFull, c >> 4 != 0)) {    // ties stay in row order while there is room
            const uint32_t ties = __popc(c >> 4);
            uint32_t incl = ties;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t u = __shfl_up_sync(kFull, incl, o);
                incl += lane >= o ? u : 0u;
            }
            uint32_t room = want > tie0 + incl - ties ? want - (tie0 + incl - ties) : 0u;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool take = (c >> (4 + j) & 1u) && room > 0;
                stays |= take ? 1u << j : 0u;
                room -= take ? 1u : 0u;
            }
            tie0 += __shfl_sync(kFull, incl, 31);
        }
        const uint32_t holes = ~stays & low & real, tails = stays & ~low & real;
        // rows of either list in the lanes before, and in all
        const uint32_t num = __popc(holes) | __popc(tails) << 16;
        uint32_t incl = num;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(kFull, incl, o);
            incl += lane >= o ? u : 0u;
        }
        const uint32_t all_here = __shfl_sync(kFull, incl, 31);
        auto write = [&](int32_t *list, uint32_t rows, uint32_t to) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if ((rows >> j & 1u) && to < (uint32_t)a.cap)
                    list[to] = lo + r + j;
                to += rows >> j & 1u;
            }
        };
        if (r0 < wm)
            write(dst, holes, hole0 + (incl - num & 0xFFFFu));
        if (r0 + 128 > wm)
            write(src, tails, tail0 + (incl - num >> 16));
        hole0 += all_here & 0xFFFFu;
        tail0 += all_here >> 16;
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
                  const int32_t *__restrict__ block_table, int bt_stride, int num_blocks, int hkv, uint8_t *pages,
                  float *acc, int32_t *pos, int *status)
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
    // As many CTAs per cluster as there are SMs for, up to 8 (more need a whole GPC, which few clusters can have at a
    // time), or as many as keep all rows, up to 16; each has 4096 rows or more.  (32 clusters for up to 248k rows: 4
    // CTAs, which all run at once, 49 us; 5, 59 us; 6, 64; 8, 78.)
    const int pairs = bs * hkv;
    int c = num_sms / pairs;
    c = c < 8 ? c : 8;
    const int fit = (max_len + 4 * kKeptQuads - 1) / (4 * kKeptQuads);
    c = c > fit ? c : fit;
    c = c < 16 ? c : 16;
    c = c < (max_len + 4095) / 4096 ? c : (max_len + 4095) / 4096;
    c = c > 1 ? c : 1;
    const int chunk = ((max_len + c - 1) / c + 127) / 128 * 128;
    SelectArgs a{acc, pos, block_table, seq_lens, next_pos, src, dst, counts, new_lens, status,
                 bt_stride, num_blocks, hkv, budget, recent, cap, max_len};
    const size_t smem = (size_t)(chunk < 4 * kSharedQuads ? chunk : 4 * kSharedQuads) * 4;
    cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kSharedQuads * 16);
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
    // Up to 32 CTAs of 256 threads per SM over all pairs: four times what runs at once, so that pairs with many moves
    // are not left alone at the end (64 pairs of up to 6100 moves: 8 per SM 71.6 us, 16 69.7, 32 67.5, 64 70.1).
    const int fill = (num_sms * 32 + pairs - 1) / pairs;
    const int per_pair = want < fill ? want : fill;
    return launch_pdl(fp8 ? evict_move_kernel<true> : evict_move_kernel<false>,
                      dim3((unsigned)pairs * (unsigned)per_pair), dim3(kMoveThreads), 0, stream, src, dst, counts, cap,
                      per_pair, block_table, bt_stride, num_blocks, hkv, static_cast<uint8_t *>(pages),
                      acc, pos, status);
}

}  // namespace sk
