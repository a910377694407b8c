// Attention weight that each cached key has gathered:
//     acc[key p of (s, h)] += sum over the rows r = j * G + i of the group that see p of exp(score(r, p) - lse(r))
// with the scores of the attention and its log-sum-exp.  Only the K half of the pages is read.
//
// The product is taken as S^T [128 keys x rows] = K Q^T, so that a TMEM lane, and with it a thread, is one key: the sum
// over the rows is that thread's own running sum in fp32, in a fixed order, added to the key's weight once: the same
// bits every time, unless sequences share a block.
//
// Bound by HBM for a few rows (decode, verify: 256 or 128 bytes of K per key against up to 64 rows), by the
// exponentials and the tensor cores for a chunk (256 flops and one exponential per (row, key)).
//
// One CTA per SM works on groups of up to four tiles of 128 keys of one (sequence, head): tile i of a group belongs to
// softmax warpgroup i and its 128 TMEM columns.  Each CTA takes an equal share of the batch's cost, a contiguous run found
// from the lengths on the device.
//   few rows (MANY false): the rows are one Q block of 16, 32 or 64 rows that stays for the whole item while K tiles
//     stream through a ring; runs are cut between tiles.
//   many rows (MANY true): a group's K tiles stay (128 KB of bf16) while Q streams through in blocks of 128 rows, so
//     that a block's 32 KB meet 512 keys: with fewer the L2 could not deliver Q as fast as the tensor cores take it.  Runs
//     are cut inside a group, between Q blocks: cut between tiles they came out at one to three tiles each, which
//     left CTAs idle and a group's pipeline half empty (1190 and 1500 tokens over 18k and 8k keys of e4m3, 8 heads
//     a KV head: 184 us, now 125).  The sums of a group that several runs share meet in accum_join_kernel.
//
// Roles (640 threads): warp 0 copies K pages; warps 1 and 2 issue the products of every other tile of a group; warp 3
// finds the items (the parts of the run in one sequence and head) and publishes them, copies Q blocks (TMA: a box is
// whole tokens of the group's heads) and lays the rows' lse and scale beside them; warps 4-19 are the four softmax
// warpgroups.
//
// e4m3 pages: the products run as kind::f8f6f4 on the codes, with Q as two e4m3 terms and a power-of-two scale per row
// (prepared by a small kernel into a workspace; exact for bf16 elements within 2^-9 of the row's largest).
//
// Waits are bounded as in the attention kernels.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include <type_traits>

#include "sk_attn_util.cuh"
#include "sk_cache_ops.cuh"
#include "sk_sm100.cuh"

namespace sk {
namespace {

using namespace sm100;

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kKeys = 128;
constexpr int kGroup = 4;                            // tiles of a group, softmax warpgroups
constexpr int kThreads = 128 + kGroup * 128;
constexpr long long kDrainLimit = 4000000000LL;
constexpr int kMaxSmem = 232448;
constexpr int kAccumRuns = 256;                      // runs (SMs) at most
constexpr long long kAccumParts = 2LL * kAccumRuns * (kGroup * kKeys * 4 + (long long)sizeof(AccumPiece));
// Few rows, long runs: equal runs end up to a fifth apart (SMs see different shares of the bandwidth), so a last 16th
// of the batch goes out in short runs to the SMs that are free first (16 x 119k keys, 4 tokens: 182 us without, 173 with a
// 16th, 182 with an 8th).  Only where the tables' pages would make runs of so many tiles: the short runs are a start of a
// CTA each, 1 to 3 us in a batch that turns out too short for them (16 x 2052 keys under tables of 8192 blocks: 11.8 us
// against 8.9).
constexpr int kTailLeast = 96;
constexpr int kRing = 4;                             // items published ahead
template <int RB, bool MANY, bool FP8>
struct ACfg {
    static constexpr int kGroupBytes = FP8 ? 1024 : 2048;          // K of 8 tokens
    static constexpr int kKSlot = kKeys / 8 * kGroupBytes;
    static constexpr int kQSlot = RB * 256;
    static constexpr int kQSlots = MANY ? 3 : 2;
    static constexpr int kAuxEach = FP8 ? 2 * RB : RB;             // floats per Q block: -lse, and e4m3's scales
    static constexpr int kMisc = (FP8 ? 4 : 3) * 1024;
    static constexpr int kFit = (kMaxSmem - kQSlots * kQSlot - kMisc) / kKSlot;
    static constexpr int kKSlots = (kFit < 12 ? kFit : 12) / 2 * 2;        // every other one for either issuer
    static constexpr int kHalf = kKSlots / 2;
    static constexpr int kOffQ = kKSlots * kKSlot;
    static constexpr int kOffMisc = kOffQ + kQSlots * kQSlot;
    static constexpr int kSmemBytes = kOffMisc + kMisc;
    static constexpr int kPagesPerTile = kKeys / kPage;
    // misc area
    static constexpr int kBarKFull = 0;
    static constexpr int kBarKEmpty = 8 * kKSlots;
    static constexpr int kBarQFull = 16 * kKSlots;                 // [kQSlots]
    static constexpr int kBarQEmpty = kBarQFull + 8 * kQSlots;
    static constexpr int kBarAFull = kBarQEmpty + 8 * kQSlots;     // rows' lse and scale
    static constexpr int kBarAEmpty = kBarAFull + 8 * kQSlots;
    static constexpr int kBarS = kBarAEmpty + 8 * kQSlots;         // [kGroup] S complete
    static constexpr int kBarSFree = kBarS + 8 * kGroup;
    static constexpr int kBarDrain = kBarSFree + 8 * kGroup;
    static constexpr int kTmemSlot = kBarDrain + 16;
    static constexpr int kAbort = kTmemSlot + 4;
    static constexpr int kStart = (kAbort + 4 + 7) / 8 * 8;        // where the run starts
    static constexpr int kBarItem = kStart + 16;                   // [kRing] items published, and read
    static constexpr int kBarItemFree = kBarItem + 8 * kRing;
    static constexpr int kItems = (kBarItemFree + 8 * kRing + 15) / 16 * 16;
    static constexpr int kAux = 640;                               // float[kQSlots][kAuxEach], log2 units
    static_assert(kItems + kRing * 48 <= kAux && kAux + kQSlots * kAuxEach * 4 <= kMisc, "misc area");
    static_assert(kKSlots >= (MANY ? kGroup : 3) && kSmemBytes <= kMaxSmem && kOffQ % 1024 == 0 && kQSlot % 1024 == 0,
                  "shared memory");
};

// What a CTA works on at a time: Q blocks [q0, q1) against tiles [a, b) of one (sequence, head).
struct __align__(16) Item {
    int s, h, L, q_len, tok0, a, b, q0, q1;
    int slot;                                        // of the run's shared units, or -1: the sums are complete
    int ends;                                        // the unit's last rows are among them
    int pad;
};
static_assert(sizeof(Item) == 48, "the ring holds items of three 16-byte words");

// First Q block of a sequence with a row that sees tile `tile`: causal rows start at token p0 - (L - q).
__device__ __forceinline__ int first_block(const AccumParams &p, int L, int q_len, int tile)
{
    const int j = p.causal ? tile * kKeys - (L - q_len) : 0;
    return j > 0 ? j / p.tpb * p.nsub : 0;
}

// Q blocks of sequence s; 0 when it has nothing to do (and a bad one is reported).
__device__ __forceinline__ int blocks_of(const AccumParams &p, int s, int &L, int &q, int &tok0)
{
    L = __ldg(p.seq_lens + s);
    tok0 = __ldg(p.cu_q + s);
    const int end = __ldg(p.cu_q + s + 1);
    const bool bad = tok0 < 0 || end < tok0 || end > p.num_tokens || end - tok0 > p.max_q_len || L < 0 ||
                     (long long)L > (long long)p.bt_stride * kPage;
    if (bad) {
        atomicOr(p.status, SK_DEV_BAD_SEQ);
        L = 0;
    }
    q = bad ? 0 : end - tok0;
    return L > 0 ? (q + p.tpb - 1) / p.tpb * p.nsub : 0;
}

// Many rows: a unit is a group of four tiles against the Q blocks that see it.  It costs its tokens plus a fixed part (K
// tiles of the next unit are not there yet when one ends), times the tiles of a group and one.
struct Units {
    int L, q, tok0, nblk, units, w;
    long long fixed, ctx;
    __device__ __forceinline__ long long before(long long i) const
    {
        const int keys = kGroup * kKeys;
        const long long g1 = ctx < 0 ? 0 : ctx / keys + 1;           // first group that some rows do not see
        const long long unseen = i > g1 ? keys * ((i * (i - 1) - g1 * (g1 - 1)) / 2) - ctx * (i - g1) : 0;
        return (i * (fixed + q) - unseen) * w;
    }
};
// Q blocks.  (300 tokens over 3k keys, 2 KV heads: 16.3 us, with 2 18.1, with 3 20.5; 1190 and 1500 tokens over 18k and 8k:
// 125.2, 124.0, 125.8.)
constexpr int kUnitFixed = 1;

__device__ __forceinline__ Units units_of(const AccumParams &p, int s)
{
    Units u;
    u.nblk = blocks_of(p, s, u.L, u.q, u.tok0);
    const int tiles = (u.L + kKeys - 1) / kKeys;
    u.units = u.nblk > 0 ? (tiles + kGroup - 1) / kGroup : 0;
    u.w = min(tiles, kGroup) + 1;
    u.fixed = kUnitFixed * p.tpb;
    u.ctx = p.causal ? u.L - u.q : u.L;
    return u;
}

// Walks the units of a CTA's run [lo, hi) of the cost, cut in the rows where the run ends.
struct UnitWalk {
    const AccumParams &p;
    long long lo, hi, off;                           // the run, and where the current sequence starts
    int s, h, unit;
    bool loaded;
    Units q;
    __device__ UnitWalk(const AccumParams &pp, const Run &run, int s0)
        : p(pp), lo(run.lo), hi(run.hi), off(run.before), s(s0), h(0), unit(-1), loaded(false)
    {
    }
    __device__ __forceinline__ bool next(Item &it)
    {
        while (s < p.bs && off < hi) {
            if (!loaded) {
                q = units_of(p, s);
                loaded = true;
            }
            const long long head = q.before(q.units);
            if (h >= p.H_kv || q.units == 0) {
                off += head * p.H_kv;
                ++s;
                h = 0;
                unit = -1;
                loaded = false;
                continue;
            }
            const long long h0 = off + h * head;
            if (h0 + head <= lo) {
                ++h;
                continue;
            }
            if (unit < 0) {
                int left = 0, right = q.units - 1;   // the last unit that starts at lo or before
                while (left < right) {
                    const int mid = (left + right + 1) >> 1;
                    if (q.before(mid) <= lo - h0)
                        left = mid;
                    else
                        right = mid - 1;
                }
                unit = left;
            }
            const long long start = h0 + q.before(unit), cost = h0 + q.before(unit + 1) - start;
            if (start >= hi)
                return false;
            it.s = s;
            it.h = h;
            it.L = q.L;
            it.q_len = q.q;
            it.tok0 = q.tok0;
            it.a = unit * kGroup;
            it.b = min(it.a + kGroup, (q.L + kKeys - 1) / kKeys);
            // A cut near either end of the unit moves there, and where else it falls is rounded in fp32: alike in both
            // runs that it divides, and that is all that matters.
            const int f = first_block(p, q.L, q.q, it.a);
            const long long edge = q.fixed * q.w;
            auto block = [&](long long at) {
                const int n = q.nblk - f;
                return f + (at <= edge          ? 0
                            : at >= cost - edge ? n
                                                : max(0, min(n, (int)((float)n * __fdividef((float)at, (float)cost)))));
            };
            it.q0 = block(max(0LL, lo - start));
            it.q1 = block(hi - start);
            it.slot = it.q0 > f ? 0 : (it.q1 < q.nblk ? 1 : -1);
            it.ends = it.q1 == q.nblk;
            if (++unit == q.units) {
                ++h;
                unit = -1;
            }
            if (it.q0 < it.q1)
                return true;
        }
        return false;
    }
};

// Few rows: one Q block a sequence.  The tiles of a CTA's run, (sequence, head) after (sequence, head).
struct TileWalk {
    const AccumParams &p;
    long long lo, hi, off;                           // the run, and the current sequence's start, in tiles
    int s, h;
    __device__ TileWalk(const AccumParams &pp, const Run &run, int s0)
        : p(pp), lo(run.lo), hi(run.hi), off(run.before), s(s0), h(0)
    {
    }
    __device__ __forceinline__ bool next(Item &it)
    {
        while (s < p.bs && off < hi) {
            int L, q, tok0;
            const bool some = blocks_of(p, s, L, q, tok0) > 0;
            const int tiles = (L + kKeys - 1) / kKeys;
            if (some && h < p.H_kv) {
                const long long start = off + (long long)h * tiles;
                const int hh = h++;
                if (start >= hi)
                    return false;
                const long long a = max(0LL, lo - start), b = min((long long)tiles, hi - start);
                if (a < b) {
                    it.s = s;
                    it.h = hh;
                    it.L = L;
                    it.q_len = q;
                    it.tok0 = tok0;
                    it.a = (int)a;
                    it.b = (int)b;
                    it.q0 = 0;
                    it.q1 = 1;
                    it.slot = -1;
                    it.ends = 1;
                    return true;
                }
                continue;
            }
            off += some ? (long long)tiles * p.H_kv : 0;
            ++s;
            h = 0;
        }
        return false;
    }
};

template <int RB, bool MANY, bool FP8>
__global__ void __launch_bounds__(kThreads, 1)
accum_kernel(const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ CUtensorMap q_map,
             const AccumParams p)
{
    using C = ACfg<RB, MANY, FP8>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t sbase = smem_u32(smem);
    uint8_t *misc = smem + C::kOffMisc;
    const uint32_t mbase = sbase + C::kOffMisc;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(misc + C::kAbort);
    auto bar_kfull = [&](int i) { return mbase + C::kBarKFull + 8 * i; };
    auto bar_kempty = [&](int i) { return mbase + C::kBarKEmpty + 8 * i; };
    auto bar_qfull = [&](int i) { return mbase + C::kBarQFull + 8 * i; };
    auto bar_qempty = [&](int i) { return mbase + C::kBarQEmpty + 8 * i; };
    auto bar_afull = [&](int i) { return mbase + C::kBarAFull + 8 * i; };
    auto bar_aempty = [&](int i) { return mbase + C::kBarAEmpty + 8 * i; };
    auto bar_s = [&](int i) { return mbase + C::kBarS + 8 * i; };
    auto bar_sfree = [&](int i) { return mbase + C::kBarSFree + 8 * i; };
    auto bar_item = [&](int i) { return mbase + C::kBarItem + 8 * i; };
    auto bar_item_free = [&](int i) { return mbase + C::kBarItemFree + 8 * i; };
    Item *ring = reinterpret_cast<Item *>(misc + C::kItems);
    auto bar_drain = [&](int i) { return mbase + C::kBarDrain + 8 * i; };

    wait_prior_grid();
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kKSlots; ++i) {
            mbar_init(bar_kfull(i), 1);
            mbar_init(bar_kempty(i), 1);
        }
        for (int i = 0; i < C::kQSlots; ++i) {
            mbar_init(bar_qfull(i), 1);
            mbar_init(bar_qempty(i), 2);
            mbar_init(bar_afull(i), 1);
            mbar_init(bar_aempty(i), 4 * kGroup);
        }
        for (int i = 0; i < kGroup; ++i) {
            mbar_init(bar_s(i), 1);
            mbar_init(bar_sfree(i), 4);
        }
        for (int i = 0; i < kRing; ++i) {
            mbar_init(bar_item(i), 1);
            mbar_init(bar_item_free(i), 3 + 4 * kGroup);
        }
        mbar_init(bar_drain(0), 1);
        mbar_init(bar_drain(1), 1);
        *abort_flag = 0;
        fence_mbar_init();
        if (blockIdx.x == 0 && (__ldg(p.cu_q) != 0 || __ldg(p.cu_q + p.bs) != p.num_tokens))
            atomicOr(p.status, SK_DEV_BAD_SEQ);
    }
    if (warp == 1) {
        tmem_alloc(mbase + C::kTmemSlot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // this CTA's run of the batch's cost (found in the K slots' memory, before the first copy)
    const Run run = find_run<kThreads>(p.bs, blockIdx.x, p.runs, p.tail, kTailLeast, reinterpret_cast<long long *>(smem),
                                       reinterpret_cast<long long *>(misc + C::kStart), [&](int s) {
                                           if constexpr (MANY) {
                                               const Units u = units_of(p, s);
                                               return u.before(u.units) * p.H_kv;
                                           } else {
                                               int L, q, tok0;
                                               const bool some = blocks_of(p, s, L, q, tok0) > 0;
                                               return some ? (long long)((L + kKeys - 1) / kKeys) * p.H_kv : 0LL;
                                           }
                                       });
    fence_proxy_async_smem();                        // the copies come after these uses of the slots
    __syncthreads();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(misc + C::kTmemSlot);
    const bool any = (sbase & 1023u) == 0;
    if (!any && threadIdx.x == 0)
        atomicOr(p.status, SK_DEV_INTERNAL);
    // The next published item; false at the end of the run, or (ok becomes false) when the wait gave up.
    int read = 0;
    auto next_item = [&](Item &item, bool &ok) {
        const int i = read % kRing;
        ok = __all_sync(kFull, wait_bar(bar_item(i), (read / kRing) & 1, abort_flag, p.wait_limit));
        if (!ok)
            return false;
        item = ring[i];
        __syncwarp();
        if (lane == 0)
            mbar_arrive(bar_item_free(i));
        ++read;
        return item.s >= 0;
    };
    Item it;

    // groups of an item: its tiles in equal shares of up to four (many rows: one group)
    auto groups_of = [&](const Item &w) { return MANY ? 1 : (w.b - w.a + kGroup - 1) / kGroup; };
    auto group_at = [&](const Item &w, int ng, int g) {
        return MANY ? (g ? w.b : w.a) : w.a + (int)((long long)(w.b - w.a) * g / ng);
    };

    auto first_token = [&](int qb) { return p.nsub > 1 ? qb / p.nsub : qb * p.tpb; };      // (nsub > 1: tpb is 1)

    if (warp == 0) {
        // ============================================================ K pages
        if (lane == 0)
            prefetch_tensormap(&kv_map);
        int used[2] = {0, 0};                        // tiles issued for either issuer
        bool ok = true;
        while (ok && next_item(it, ok)) {
            const int page_end = (it.L + kPage - 1) / kPage;
            const int32_t *bt = p.block_table + (long long)it.s * p.bt_stride;
            auto block_at = [&](int t) {
                const int pg = t * C::kPagesPerTile + lane;
                return (lane < C::kPagesPerTile && t < it.b && pg < page_end) ? __ldg(bt + pg) : -1;
            };
            int blk[3] = {block_at(it.a), block_at(it.a + 1), block_at(it.a + 2)};
            const int ng = groups_of(it);
            int g = 0, e = 0, end = group_at(it, ng, 1);
            for (int t = it.a; t < it.b && ok; ++t, e ^= 1) {
                if (t == end) {
                    ++g;
                    end = group_at(it, ng, g + 1);
                    e = 0;
                }
                const int n = e ? used[1] : used[0];
                const int i = 2 * (n % C::kHalf) + e;
                if (n >= C::kHalf)
                    ok = wait_bar(bar_kempty(i), (n / C::kHalf - 1) & 1, abort_flag, p.wait_limit);
                ok = __all_sync(kFull, ok);
                if (!ok)
                    break;
                if (lane == 0)
                    mbar_arrive_expect_tx(bar_kfull(i), C::kKSlot);
                __syncwarp();
                if (lane < C::kPagesPerTile) {
                    int grp = -2;                    // whole box out of bounds: zero fill
                    if (t * C::kPagesPerTile + lane < page_end) {
                        if (blk[0] >= 0 && blk[0] < p.num_blocks)
                            grp = (blk[0] * p.H_kv + it.h) * 2;
                        else
                            atomicOr(p.status, SK_DEV_BAD_BLOCK);
                    }
                    tma_load_4d(sbase + i * C::kKSlot + lane * 2 * C::kGroupBytes, &kv_map, 0, 0, 0, grp, bar_kfull(i));
                }
                blk[0] = blk[1];
                blk[1] = blk[2];
                blk[2] = block_at(t + 3);
                used[0] += 1 - e;
                used[1] += e;
            }
        }
        if (!ok) {
            *abort_flag = 1;
            if (lane == 0)
                atomicOr(p.status, SK_DEV_TIMEOUT);
        }
        for (int e = 0; e < 2; ++e)
            for (int t = max(0, used[e] - C::kHalf); t < used[e]; ++t)
                wait_bar(bar_kfull(2 * (t % C::kHalf) + e), (t / C::kHalf) & 1, nullptr, kDrainLimit);
    } else if (warp <= 2) {
        // ============================================================ products: tiles 0 and 2 of a group, or 1 and 3
        // Either issuer has every other K slot for itself: a barrier shows only whether the last phase of a parity is
        // over, so each of a slot's phases has to be waited for by the same warp.
        const int e = warp - 1;
        constexpr uint32_t idesc = FP8 ? idesc_e4m3_f32(kKeys, RB, 0, 0) : idesc_bf16_f32(kKeys, RB, 0, 0);
        const uint64_t d_k0 = smem_desc_sw128(sbase, 16, C::kGroupBytes);
        const uint64_t d_q0 = smem_desc_sw128(sbase + C::kOffQ, 16, 1024);
        auto adv = [](uint64_t d, uint32_t bytes) { return d + (uint64_t)(bytes >> 4); };
        bool ok = true;
        int u = 0, v = 0;                            // own K tiles and Q blocks used up
        uint32_t uses[kGroup / 2] = {0, 0};          // products of each TMEM buffer of this issuer
        auto wait = [&](uint32_t bar, uint32_t parity) {
            if (ok)
                ok = wait_bar(bar, parity, abort_flag, p.wait_limit);
            ok = __all_sync(kFull, ok);
            if (ok)
                tc_fence_after();
            return ok;
        };
        while (ok && next_item(it, ok)) {
            const int ng = groups_of(it);
            for (int g = 0; g < ng && ok; ++g) {
                const int ta = group_at(it, ng, g), nt = group_at(it, ng, g + 1) - ta;
                for (int qb = it.q0; qb < it.q1 && ok; ++qb) {
                    const int qi = v % C::kQSlots;
                    if ((MANY || g == 0) && !wait(bar_qfull(qi), (v / C::kQSlots) & 1))
                        break;
#pragma unroll
                    for (int ii = 0; ii < kGroup / 2; ++ii) {
                        const int i = 2 * ii + e;
                        if (i >= nt || !ok)
                            continue;
                        const int ki = 2 * ((u + ii) % C::kHalf) + e;
                        if (qb == it.q0 && !wait(bar_kfull(ki), ((u + ii) / C::kHalf) & 1))
                            continue;
                        if (!MANY || qb >= first_block(p, it.L, it.q_len, ta + i)) {
                            if (uses[ii] > 0 && !wait(bar_sfree(i), (uses[ii] - 1) & 1))
                                continue;
                            const uint64_t k0 = adv(d_k0, (uint32_t)ki * C::kKSlot);
                            const uint64_t q0 = adv(d_q0, (uint32_t)qi * C::kQSlot);
                            const uint32_t sd = tmem + i * 128;
#pragma unroll
                            for (int hf = 0; hf < 2; ++hf) {
                                if constexpr (FP8)
                                    mma4_f8_ss<2, 2>(sd, k0, adv(q0, hf * (RB * 128)), idesc, hf);
                                else
                                    mma4_f16_ss<2, 2>(sd, adv(k0, hf * 1024), adv(q0, hf * (RB * 128)), idesc, hf);
                            }
                            mma_commit_warp(bar_s(i));
                            ++uses[ii];
                        }
                        if (qb + 1 == it.q1)
                            mma_commit_warp(bar_kempty(ki));
                    }
                    if (MANY || g + 1 == ng) {
                        mma_commit_warp(bar_qempty(qi));
                        ++v;
                    }
                }
                u += (nt + 1 - e) / 2;
            }
        }
        if (!ok) {
            *abort_flag = 1;
            if (lane == 0)
                atomicOr(p.status, SK_DEV_TIMEOUT);
        }
        mma_commit_warp(bar_drain(e));
        wait_bar(bar_drain(e), 0, nullptr, kDrainLimit);
    } else if (warp == 3) {
        // ============================================================ the items; Q blocks, and their rows' lse and scale
        using Walk = std::conditional_t<MANY, UnitWalk, TileWalk>;
        Walk walk(p, run, any ? run.s : p.bs);
        AccumPiece *shared = p.shared + 2 * blockIdx.x;      // this run's parts of units that others have a part of
        if (MANY && lane < 2)
            shared[lane].s = -1;
        __syncwarp();
        bool ok = true;
        int v = 0;
        for (int k = 0; ok; ++k) {
            const bool more = walk.next(it);
            if (!more)
                it.s = -1;
            if (k >= kRing)
                ok = wait_bar(bar_item_free(k % kRing), (k / kRing - 1) & 1, abort_flag, p.wait_limit);
            ok = __all_sync(kFull, ok);
            if (!ok)
                break;
            if (lane == 0) {
                ring[k % kRing] = it;
                if (MANY && more && it.slot >= 0)
                    shared[it.slot] = AccumPiece{it.s, it.h, it.a, it.ends};
                mbar_arrive(bar_item(k % kRing));
            }
            __syncwarp();
            if (!more)
                break;
            {
                for (int qb = it.q0; qb < it.q1 && ok; ++qb, ++v) {
                    const int qi = v % C::kQSlots;
                    const int j0 = first_token(qb), i0 = p.nsub > 1 ? (qb % p.nsub) * p.gb : 0;
                    const int hq0 = it.h * p.G + i0;
                    if (v >= C::kQSlots) {
                        ok = wait_bar(bar_qempty(qi), (v / C::kQSlots - 1) & 1, abort_flag, p.wait_limit);
                        if (ok)
                            ok = wait_bar(bar_aempty(qi), (v / C::kQSlots - 1) & 1, abort_flag, p.wait_limit);
                    }
                    ok = __all_sync(kFull, ok);
                    if (!ok)
                        break;
                    if (lane == 0) {
                        const uint32_t dst = sbase + C::kOffQ + qi * C::kQSlot;
                        mbar_arrive_expect_tx(bar_qfull(qi), (uint32_t)(p.gb * p.tpb * 256));
                        tma_load_3d(dst, &q_map, 0, hq0, it.tok0 + j0, bar_qfull(qi));
                        tma_load_3d(dst + RB * 128, &q_map, FP8 ? 128 : 64, hq0, it.tok0 + j0, bar_qfull(qi));
                    }
                    __syncwarp();
                    {
                        float *aux = reinterpret_cast<float *>(misc + C::kAux) + qi * C::kAuxEach;
                        for (int r = lane; r < RB; r += 32) {
                            const int jj = r / p.gb, ii = r - jj * p.gb;
                            float nl = -CUDART_INF_F;
                            [[maybe_unused]] float sc = 1.f;   // a masked -inf stays -inf
                            if (jj < p.tpb && j0 + jj < it.q_len && i0 + ii < p.G) {
                                const long long at = (long long)(it.tok0 + j0 + jj) * p.H_q + hq0 + ii;
                                nl = __ldg(p.lse + at) * -1.4426950408889634f;
                                nl = nl == CUDART_INF_F ? -CUDART_INF_F : nl;     // a row that sees nothing
                                if constexpr (FP8)
                                    sc = __ldg(p.q_scale + at) * p.score_scale_log2;
                            }
                            aux[r] = nl;
                            if constexpr (FP8)
                                aux[RB + r] = sc;
                        }
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(bar_afull(qi));
                    }
                }
            }
        }
        if (!ok) {
            *abort_flag = 1;
            if (lane == 0)
                atomicOr(p.status, SK_DEV_TIMEOUT);
        }
        for (int t = v > C::kQSlots ? v - C::kQSlots : 0; t < v; ++t)
            wait_bar(bar_qfull(t % C::kQSlots), (t / C::kQSlots) & 1, nullptr, kDrainLimit);
    } else {
        // ============================================================ sums of the exponentials
        const int wg = (warp >> 2) - 1;
        const int quarter = warp & 3;
        const int tau = quarter * 32 + lane;
        const uint32_t ts = tmem + wg * 128 + ((uint32_t)(quarter * 32) << 16);
        uint32_t uses = 0;
        int v = 0;
        bool ok = true;
        while (ok && next_item(it, ok)) {
            const int ng = groups_of(it);
            const int32_t *bt = p.block_table + (long long)it.s * p.bt_stride;
            for (int g = 0; g < ng && ok; ++g) {
                const int ta = group_at(it, ng, g), nt = group_at(it, ng, g + 1) - ta;
                const int key = (ta + wg) * kKeys + tau;
                const bool live = wg < nt && key < it.L;
                float *place = nullptr;              // where the key's sum goes
                if (live && it.slot >= 0)
                    place = p.part + (2LL * blockIdx.x + it.slot) * (kGroup * kKeys) + wg * kKeys + tau;
                else if (live) {
                    const int blk = __ldg(bt + key / kPage);
                    if (blk >= 0 && blk < p.num_blocks)
                        place = p.acc + ((long long)blk * p.H_kv + it.h) * kPage + key % kPage;
                }
                const int f = MANY ? first_block(p, it.L, it.q_len, ta + wg) : 0;
                const int jmin = p.causal ? key - (it.L - it.q_len) : 0;       // first token that sees the key
                float2 sum = make_float2(0.f, 0.f);
                for (int qb = it.q0; qb < it.q1 && ok; ++qb) {
                    const int qi = v % C::kQSlots;
                    // S is there long after the rows' lse: both barriers are tested at once (each test takes 200 cycles)
                    const bool work = wg < nt && qb >= f;
                    const bool early = work && sm100::mbar_test_wait(bar_s(wg), uses & 1);
                    if (MANY || g == 0)
                        ok = __all_sync(kFull, wait_bar(bar_afull(qi), (v / C::kQSlots) & 1, abort_flag,
                                                                 p.wait_limit));
                    if (ok && work) {
                        ok = early || wait_bar(bar_s(wg), uses & 1, abort_flag, p.wait_limit);
                        ++uses;
                        ok = __all_sync(kFull, ok);
                        if (ok) {
                            tc_fence_after();
                            const float *aux = reinterpret_cast<const float *>(misc + C::kAux) + qi * C::kAuxEach;
                            const int j0 = first_token(qb);
                            // rows [rmin, rows) of the block see this key
                            const int rmin = jmin > j0 ? (jmin - j0) * p.gb : 0;
                            const int rows = p.nsub > 1 ? min(p.gb, p.G - qb % p.nsub * p.gb)
                                                        : min(p.tpb, it.q_len - j0) * p.gb;
                            constexpr int kLd = RB < 64 ? RB : 64;
#pragma unroll
                            for (int c0 = 0; c0 < RB; c0 += kLd) {
                                if (c0 >= rows)
                                    break;
                                float x[kLd];
#pragma unroll
                                for (int c = 0; c < kLd; c += kLd < 32 ? kLd : 32)
                                    tmem_ld32<(kLd < 32 ? kLd : 32)>(ts + c0 + c, x + c);
                                tmem_wait_ld();
                                if (c0 + kLd >= rows) {              // the buffer's last read
                                    tc_fence_before();
                                    __syncwarp();
                                    if (lane == 0)
                                        mbar_arrive(bar_sfree(wg));
                                }
                                const bool whole = __all_sync(kFull, rmin <= c0) && c0 + kLd <= rows;
                                if (!whole) {
#pragma unroll
                                    for (int r = 0; r < kLd; ++r)
                                        x[r] = (c0 + r >= rmin && c0 + r < rows) ? x[r] : -CUDART_INF_F;
                                }
#pragma unroll
                                for (int r = 0; r < kLd; r += 4) {
                                    const float4 nl = *reinterpret_cast<const float4 *>(aux + c0 + r);
                                    float4 sc = make_float4(p.score_scale_log2, p.score_scale_log2, p.score_scale_log2,
                                                            p.score_scale_log2);
                                    if constexpr (FP8)
                                        sc = *reinterpret_cast<const float4 *>(aux + RB + c0 + r);
                                    const float2 d0 = ffma2(make_float2(x[r], x[r + 1]), make_float2(sc.x, sc.y),
                                                            make_float2(nl.x, nl.y));
                                    const float2 d1 = ffma2(make_float2(x[r + 2], x[r + 3]), make_float2(sc.z, sc.w),
                                                            make_float2(nl.z, nl.w));
                                    sum = fadd2(sum, make_float2(ex2_ftz(d0.x), ex2_ftz(d0.y)));
                                    sum = fadd2(sum, make_float2(ex2_ftz(d1.x), ex2_ftz(d1.y)));
                                }
                            }
                        }
                    }
                    if (ok && (MANY || g + 1 == ng)) {
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(bar_aempty(qi));
                        ++v;
                    }
                }
                // one addition per key (more only where sequences share a block)
                if (ok && place != nullptr) {
                    if (it.slot >= 0)
                        *place = sum.x + sum.y;
                    else
                        atomicAdd(place, sum.x + sum.y);
                }
                __syncwarp();
            }
        }
        if (!ok) {
            *abort_flag = 1;
            if (lane == 0)
                atomicOr(p.status, SK_DEV_TIMEOUT);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Adds up the parts of the units that several runs share: block r those of the unit whose last part is run r's first.
// Its other parts are the first ones of the runs before, back to the run that the unit starts in, whose last part it is;
// they are added in the rows' order, whatever the timing of the runs.
__global__ void __launch_bounds__(kGroup * kKeys) accum_join_kernel(const AccumParams p)
{
    __shared__ int slots[kAccumRuns], count;
    wait_prior_grid();
    const int index = blockIdx.x;
    const AccumPiece pc = p.shared[2 * index];
    if (pc.s < 0 || !pc.ends)
        return;
    if (threadIdx.x < 32) {
        const int n = shared_slots(index, [&](int slot) { return p.shared[slot].s >= 0; }, slots);
        if (threadIdx.x == 0)
            count = n;
    }
    const int key = pc.a * kKeys + threadIdx.x;
    const bool live = key < __ldg(p.seq_lens + pc.s);
    const int blk = live ? __ldg(p.block_table + (long long)pc.s * p.bt_stride + key / kPage) : -1;
    __syncthreads();
    if (blk < 0 || blk >= p.num_blocks)
        return;
    float sum = 0.f;
    for (int i = count - 1; i >= 0; --i)
        sum += p.part[(long long)slots[i] * (kGroup * kKeys) + threadIdx.x];
    atomicAdd(p.acc + ((long long)blk * p.H_kv + pc.h) * kPage + key % kPage, sum);
}

__global__ void __launch_bounds__(256) split_q_kernel(const uint16_t *__restrict__ q, long long rows,
                                                      uint8_t *__restrict__ codes, float *__restrict__ scale)
{
    wait_prior_grid();
    const int lane = threadIdx.x & 31;
    constexpr int kAtOnce = 4;
    const long long r0 = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * kAtOnce;
    uint2 raw[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
        raw[i] = r0 + i < rows ? __ldg(reinterpret_cast<const uint2 *>(q + (r0 + i) * kHeadDim) + lane)
                               : make_uint2(0u, 0u);
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
        if (r0 + i >= rows)
            break;
        uint32_t hi, lo;
        int e;
        split_q_row(raw[i], hi, lo, e);
        uint32_t *dst = reinterpret_cast<uint32_t *>(codes + (r0 + i) * 256);
        dst[lane] = hi;
        dst[32 + lane] = lo;
        if (lane == 0)
            scale[r0 + i] = ldexpf(1.f, -e);
    }
}

template <int RB, bool MANY, bool FP8>
cudaError_t launch_t(const CUtensorMap &kv_map, const CUtensorMap &q_map, const AccumParams &p, cudaStream_t stream)
{
    using C = ACfg<RB, MANY, FP8>;
    const cudaError_t e = cudaFuncSetAttribute(accum_kernel<RB, MANY, FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               C::kSmemBytes);
    if (e != cudaSuccess)
        return e;
    const cudaError_t l = launch_pdl(accum_kernel<RB, MANY, FP8>, dim3((unsigned)(p.runs + p.tail)), dim3(kThreads),
                                     C::kSmemBytes, stream, kv_map, q_map, p);
    if (!MANY || p.runs == 1 || l != cudaSuccess)
        return l;
    return launch_pdl(accum_join_kernel, dim3((unsigned)p.runs), dim3(kGroup * kKeys), 0, stream, p);
}

}  // namespace

cudaError_t launch_split_q(const uint16_t *q, long long rows, void *codes, cudaStream_t stream)
{
    uint8_t *c = static_cast<uint8_t *>(codes);
    return launch_pdl(split_q_kernel, dim3((unsigned)((rows + 31) / 32)), dim3(256), 0, stream, q, rows, c,
                      reinterpret_cast<float *>(c + rows * 256));
}

// Rows of a Q block: 16, 32 or 64 when that holds all of a sequence's rows (they then stay while K streams), else 128.
int accum_block_rows(int G, long long max_q_len)
{
    for (int rb = 16; rb <= 64; rb *= 2)
        if ((long long)G * max_q_len <= rb)
            return rb;
    return 128;
}

// Bytes of the workspace: for many rows the parts of shared units, and for e4m3 pages Q in two terms.
long long accum_workspace_bytes(int num_tokens, int H_q, int H_kv, int max_q_len, int kv_dtype)
{
    const bool many = accum_block_rows(H_q / H_kv, max_q_len) == 128;
    return (many ? kAccumParts : 0) + (kv_dtype == SK_KV_FP8_E4M3 ? (long long)num_tokens * H_q * (2 * kHeadDim + 4) : 0);
}

cudaError_t launch_accum(const AccumParams &params, int kv_dtype, void *workspace, int num_sms, cudaStream_t stream)
{
    const bool fp8 = kv_dtype == SK_KV_FP8_E4M3;
    AccumParams p = params;
    const int rb = accum_block_rows(p.G, p.max_q_len);
    p.gb = p.G < rb ? p.G : rb;
    p.nsub = (p.G + p.gb - 1) / p.gb;
    p.tpb = rb / p.gb;
    uint8_t *q_codes = static_cast<uint8_t *>(workspace);
    if (rb == 128) {
        p.part = static_cast<float *>(workspace);
        p.shared = reinterpret_cast<AccumPiece *>(p.part + 2LL * kAccumRuns * kGroup * kKeys);
        q_codes += kAccumParts;
    }
    const void *q = p.q;
    if (fp8) {
        const long long rows = (long long)p.num_tokens * p.H_q;
        const cudaError_t e = launch_split_q(p.q, rows, q_codes, stream);
        if (e != cudaSuccess)
            return e;
        q = q_codes;
        p.q_scale = reinterpret_cast<const float *>(q_codes + rows * 256);
    }
    p.runs = num_sms < kAccumRuns ? num_sms : kAccumRuns;
    const long long most = (long long)p.bs * p.H_kv * p.bt_stride / (kKeys / kPage);         // tiles of the tables' pages
    p.tail = rb < 128 && most >= (long long)kTailLeast * p.runs ? p.runs : 0;
    CUtensorMap kv_map, q_map;
    cudaError_t e = encode_page_map(&kv_map, p.kv, p.num_blocks, p.H_kv, fp8, fp8 ? 1 : 2);
    if (e == cudaSuccess)
        e = encode_q_map(&q_map, q, p.num_tokens, p.H_q, fp8, p.gb, p.tpb);
    if (e != cudaSuccess)
        return e;
    switch (rb * 2 + (fp8 ? 1 : 0)) {
    case 32:
        return launch_t<16, false, false>(kv_map, q_map, p, stream);
    case 33:
        return launch_t<16, false, true>(kv_map, q_map, p, stream);
    case 64:
        return launch_t<32, false, false>(kv_map, q_map, p, stream);
    case 65:
        return launch_t<32, false, true>(kv_map, q_map, p, stream);
    case 128:
        return launch_t<64, false, false>(kv_map, q_map, p, stream);
    case 129:
        return launch_t<64, false, true>(kv_map, q_map, p, stream);
    case 256:
        return launch_t<128, true, false>(kv_map, q_map, p, stream);
    default:
        return launch_t<128, true, true>(kv_map, q_map, p, stream);
    }
}

}  // namespace sk
