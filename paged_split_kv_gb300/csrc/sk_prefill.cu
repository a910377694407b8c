// Attention of a chunk of new tokens over the paged cache (bf16 or e4m3 pages) on the tcgen05 tensor cores.
//
// For the rows r = j * G + i (query token j, head i of the group) of one (sequence, KV head):
//     S = scale Q K^T over the keys p <= L - q + j,   O = softmax(S) V,   lse = log sum exp S
// with one pass over the keys: a running reference maximum and sum per row, O rescaled when the reference moves.
//
// Bound by the tensor cores: 4 * 128 flops per (row, key) against 512 bytes of K and V per key that 256 rows
// share.  One CTA takes 256 rows as two tiles A and B of 128 (the MMA's M) and streams the keys in tiles of
// 128 (its N): while the softmax of one row tile runs, the products of the other fill the tensor pipe.  For each row
// tile x, in issue order over the key tiles j:
//     O_x += P_x(j) V(j);  S_x = Q_x K(j+1)^T
// S_A, S_B, O_A and O_B fill the 512 TMEM columns; P overwrites
// S in half its columns, as bf16 (f16 for e4m3 pages), and is the A operand of PV straight from TMEM, so that
// probabilities never pass through shared memory.
// A row is one TMEM lane and so one thread: the row's maximum and sum need no exchange between threads.
//
// Roles (384 threads; 512 for e4m3 pages):
//   warp 0      copies: K and V of a key tile apart, 32 KB (16 KB e4m3) slots, one TMA copy per page and part, so
//               the ring holds two and a half (five) key tiles beside Q
//   warps 1, 2  issue the products of A and of B, each through one elected lane (warp 1 also allocates TMEM), and take
//               turns: one issuer for both was the bottleneck, its waits, 200 cycles each even for what is complete,
//               coming one after the other (3300 cycles per key tile against 2048 of products), and two that did not
//               take turns fell into step, both softmaxes at once (4000)
//   warp 3      finds the pieces of the CTA's share, publishes them to the others, copies their Q tiles
//   warps 4-7   softmax of A, its rescaling, its output
//   warps 8-11  the same for B
// S(j) complete implies PV(j - 1) complete (products of one issuer complete in issue order), so the softmax may rescale O
// at once; it does so only when scores beat the reference by far.
//
// e4m3 pages: QK runs as kind::f8f6f4 on the codes, with Q as two e4m3 terms and a power-of-two scale per row (exact for
// bf16 elements within 2^-9 of the row's largest), as two products into one S.  V's codes become f16 (exactly) in
// shared memory, by four more warps (12-15), and PV runs on f16.  (P as two e4m3 terms with V's codes as they are
// needs no conversion, but costs the softmax two more instructions per score: 325 against 266 us on 2432 tokens over
// 10.6k keys, 32/8 heads.)
//
// Division of the work: one CTA per SM with an equal share of the batch's cost, cut in the key axis where a share ends
// (below); what several CTAs have of a unit is joined by a second kernel.  Inside its share a CTA goes from unit to unit
// without a pause: the copies run ahead, Q comes by TMA when its last product is done, and a unit's output is written
// while the other row tile's products run.
//
// Every wait is bounded as in the decode kernel: on expiry SK_DEV_TIMEOUT is set and every role gives up; the
// producer waits for its copies and the issuer for its last commit before the CTA exits.
#include <cuda.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <math_constants.h>
#include <stdint.h>

#include <mutex>

#include "sk_attn_util.cuh"
#include "sk_cache_ops.cuh"
#include "sk_sm100.cuh"

namespace sk {
namespace {

using namespace sm100;

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kRows = 128;                           // rows of one tile (MMA M)
constexpr int kKeys = 128;                           // keys of one tile (MMA N)
constexpr long long kDrainLimit = 4000000000LL;      // cycles (~2 s): waits for work already issued
constexpr int kMaxSmem = 232448;
constexpr int kRing = 4;                             // pieces published ahead
template <bool FP8>
struct PCfg {
    static constexpr int kThreads = FP8 ? 512 : 384;
    // registers per thread after the reallocation: copies and products, softmax, e4m3's conversion of V; no more in all
    // than at launch (4 x 128, or 3 x 168)
    static constexpr int kRegsLaunch = FP8 ? 128 : 168;
    static constexpr int kRegsIssue = FP8 ? 64 : 72, kRegsSoftmax = FP8 ? 208 : 216, kRegsConvert = 32;
    static_assert(kRegsIssue + 2 * kRegsSoftmax + (FP8 ? kRegsConvert : 0) <= kThreads / 128 * kRegsLaunch, "registers");
    static constexpr int kQTile = kRows * 256;                     // bf16: two 64-dimension chunks; e4m3: hi and lo
    static constexpr int kGroupBytes = FP8 ? 1024 : 2048;          // K (or V) of 8 tokens, as copied
    static constexpr int kSlotBytes = kKeys / 8 * kGroupBytes;
    static constexpr int kVBytes = FP8 ? kKeys * 256 : 0;          // e4m3: V of a tile as f16, two of them
    static constexpr int kMisc = 1024;                             // barriers
    static constexpr int kSlots = (kMaxSmem - 2 * kQTile - 2 * kVBytes - kMisc) / kSlotBytes;
    static constexpr int kOffV = kSlots * kSlotBytes;
    static constexpr int kOffQ = kOffV + 2 * kVBytes;
    static constexpr int kOffMisc = kOffQ + 2 * kQTile;
    static constexpr int kSmemBytes = kOffMisc + kMisc;
    static constexpr int kPagesPerTile = kKeys / kPage;
    // The reference stands this far (in log2 units) below the score that sets it: 0 for bf16, whose precision is the same
    // at any size.  f16 rounds by a fixed 2^-25 below 2^-14: with probabilities of 2^8 for the row's largest scores
    // that is 2^-33 of its sum or less, instead of 2^-25, which a key far above many others made their whole weight.
    static constexpr float kAbove = FP8 ? 8.f : 0.f;
    // The sum of a tile's probabilities (relative to the reference) up to which they are as good as with the maximum
    // for reference: f16 ends at 65504 (128 equal scores sum to 2^15).
    static constexpr float kSumMost = FP8 ? 65504.f : 0x1p40f;
    // misc area
    static constexpr int kBarFull = 0;
    static constexpr int kBarEmpty = 8 * kSlots;
    static constexpr int kBarQ = 16 * kSlots;                      // [2] Q tile landed
    static constexpr int kBarQFree = kBarQ + 16;                   // [2] the last product that reads it complete
    static constexpr int kBarS = kBarQFree + 16;                       // [2] S complete
    static constexpr int kBarP = kBarS + 16;                       // [2] P written
    static constexpr int kBarO = kBarP + 16;                       // [2] last PV complete
    static constexpr int kBarTurn = kBarO + 16;                    // [2] the other issuer has issued its products
    static constexpr int kBarVFull = kBarTurn + 16;                // [2] e4m3: V of a tile as f16
    static constexpr int kBarVEmpty = kBarVFull + 16;              // [2]
    static constexpr int kBarDrain = kBarVEmpty + 16;              // [2]
    static constexpr int kTmemSlot = kBarDrain + 16;
    static constexpr int kAbort = kTmemSlot + 4;
    static constexpr int kStart = (kAbort + 4 + 7) / 8 * 8;        // where the run starts
    static constexpr int kBarPieceFull = kStart + 24;              // [kRing]
    static constexpr int kBarPieceEmpty = kBarPieceFull + 8 * kRing;
    static constexpr int kPieces = (kBarPieceEmpty + 8 * kRing + 15) / 16 * 16;   // Piece[kRing]
    static constexpr int kReaders = FP8 ? 15 : 11;                 // warps that read the pieces
    static_assert(kPieces + kRing * 48 <= kMisc, "misc area");
    static_assert(kSlots >= 3 && (!FP8 || kSlots % 2 == 0) && kSmemBytes <= kMaxSmem && kOffQ % 1024 == 0, "shared memory");
};

// TMEM map (columns)
constexpr int kColS = 0, kColO = 256;                // S_A, S_B, then O_A, O_B, 128 each

// ------------------------------------------------------------------ the work and its division
// A row tile is `tpb` query tokens times `gb` heads of the group (nsub tiles per token when the group has more than 128);
// a unit is two neighbouring row tiles of one (sequence, KV head), A and B, over all keys that its last token sees.
// Units cost their keys plus a fixed part; each CTA takes an equal share of the batch's cost, a contiguous run of units
// cut where the share ends, in the key axis too.  A unit inside one run goes straight to the output; the pieces of
// a unit that several runs share go to a slot each, as partial softmax states, and prefill_join_kernel joins them.
// A batch whose K and V are too large to stay in the L2 begins with whole units, dealt to the CTAs in turn, and only
// what is left over is shared out like that: CTAs that work at the same time then read the same heads (4096 tokens over
// 32k keys, 8 KV heads, 151 MB: 1433 us with 0.2 GB read from HBM, against 1543 us and 3.6 GB).  Dealing takes no account of
// what units cost, so it is done only where the largest costs at most 1.4 times the mean (no CTA then gets more
// than that times its share) or an eighth of a CTA's share.
struct Seq {
    int L, q_len, tok0, units;                       // units of one head
    long long base, step;                            // unit i costs base + step * (i + 1)
    __device__ __forceinline__ long long before(int i) const { return i * base + step * i * (i + 1) / 2; }
    __device__ __forceinline__ long long cost(int i) const { return base + step * (i + 1); }
};

constexpr double kL2Share = 60e6;                    // bytes of K and V that stay in the L2 (126 MB in two halves)
constexpr int kUnitFixed = 384;                      // cost of starting and finishing a unit, in keys

__device__ __forceinline__ Seq sequence(const PrefillParams &p, int s)
{
    Seq q;
    q.L = __ldg(p.seq_lens + s);
    q.tok0 = __ldg(p.cu_q + s);
    const int end = __ldg(p.cu_q + s + 1);
    const bool bad = q.tok0 < 0 || end < q.tok0 || end > p.num_tokens || end - q.tok0 > p.max_q_len || q.L < 0 ||
                     (long long)q.L > (long long)p.bt_stride * kPage;
    if (bad)
        atomicOr(p.status, SK_DEV_BAD_SEQ);
    q.q_len = bad ? 0 : end - q.tok0;
    q.units = ((q.q_len + p.tpb - 1) / p.tpb * p.nsub + 1) / 2;
    const bool rising = p.causal && p.nsub == 1;     // later units see more keys
    q.base = kUnitFixed + (rising ? max(0, q.L - q.q_len) : q.L);
    q.step = rising ? 2 * p.tpb : 0;
    return q;
}

using Piece = PrefillPiece;
static_assert(sizeof(Piece) == 48, "the ring holds pieces of three 16-byte words");

// First token and head (within the group) of row tile T.
__device__ __forceinline__ void tile_origin(const PrefillParams &p, int T, int &j0, int &i0)
{
    j0 = T * p.tpb;
    i0 = 0;
    if (p.nsub > 1) {
        j0 = T / p.nsub;                             // then a row tile is part of one token
        i0 = (T - j0 * p.nsub) * p.gb;
    }
}

// Key tiles that row tile T of a sequence needs (0 when it has no tokens).
__device__ __forceinline__ int tiles_of(const PrefillParams &p, int L, int q_len, int T)
{
    int j0, i0;
    tile_origin(p, T, j0, i0);
    if (j0 >= q_len)
        return 0;
    return (visible_keys(L, q_len, min(q_len, j0 + p.tpb) - 1, p.causal) + kKeys - 1) / kKeys;
}

// What a CTA has to do: whole units first, first + stride, ... below `dealt` (in the order of sequence, head, unit), then the
// pieces of the run [lo, hi) of the cost, which starts in sequence s, `before` in.
struct Share {
    long long lo, hi, before;
    int s, first, stride, dealt;
};

// Walks a share's pieces; called by a converged warp.
struct Walk {
    const PrefillParams &p;
    long long lo, hi, off;                           // the run, and where the current sequence starts
    int s, h, unit;
    int deal, stride, dealt, seek, passed;           // next unit dealt; the sequence that the search is at, units before it
    bool loaded;
    Seq q;
    __device__ Walk(const PrefillParams &pp, const Share &sh)
        : p(pp), lo(sh.lo), hi(sh.hi), off(sh.before), s(sh.s), h(0), unit(-1), deal(sh.first), stride(sh.stride),
          dealt(sh.dealt), seek(0), passed(0), loaded(false)
    {
    }
    __device__ __forceinline__ void fill(Piece &pc, int s_, int h_, int unit_, const Seq &sq, int &tA, int &tB) const
    {
        pc.s = s_;
        pc.h = h_;
        pc.unit = unit_;
        pc.L = sq.L;
        pc.q_len = sq.q_len;
        pc.tok0 = sq.tok0;
        tA = tiles_of(p, sq.L, sq.q_len, 2 * unit_);
        tB = tiles_of(p, sq.L, sq.q_len, 2 * unit_ + 1);
        pc.t = max(tA, tB);
    }
    // Unit number `deal`: 32 sequences at a time until the one that has it.
    __device__ __forceinline__ void dealt_unit(Piece &pc)
    {
        const int lane = threadIdx.x & 31;
        Seq sq;
        int own, incl;
        while (true) {
            sq = sequence(p, min(seek + lane, p.bs - 1));
            own = seek + lane < p.bs ? sq.units * p.H_kv : 0;
            incl = own;
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(kFull, incl, o);
                incl += lane >= o ? u : 0;
            }
            const int all = __shfl_sync(kFull, incl, 31);
            if (deal < passed + all)
                break;
            passed += all;
            seek += 32;
        }
        const int src = __ffs(__ballot_sync(kFull, deal < passed + incl)) - 1;
        const int index = deal - passed - __shfl_sync(kFull, incl - own, src);
        const int at = seek + src;
        Seq found = sequence(p, at);
        int tA, tB;
        fill(pc, at, index / found.units, index % found.units, found, tA, tB);
        pc.a = 0;
        pc.b = pc.t;
        pc.nA = tA;
        pc.nB = tB;
        deal += stride;
    }
    // This run's key tiles of a unit.  A cut near either end of the unit moves there (a piece costs its start, its end and
    // its share of the join), and where else it falls is rounded in fp32: alike in both runs that it divides, and that
    // is all that matters.
    __device__ __forceinline__ void cut(Piece &pc, long long start, long long cost) const
    {
        auto tile = [&](long long at) {
            return at <= kUnitFixed             ? 0
                   : at >= cost - kUnitFixed ? pc.t
                                             : max(0, min(pc.t, (int)((float)pc.t * __fdividef((float)at, (float)cost))));
        };
        pc.a = tile(max(0LL, lo - start));
        pc.b = tile(hi - start);
    }
    __device__ __forceinline__ bool next(Piece &pc)
    {
        if (deal < dealt) {
            dealt_unit(pc);
            return true;
        }
        while (s < p.bs && off < hi) {
            if (!loaded) {
                q = sequence(p, s);
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
                unit = 0;
                if (lo > h0) {                       // the last unit that starts at lo or before
                    int left = 0, right = q.units - 1;
                    while (left < right) {
                        const int mid = (left + right + 1) >> 1;
                        if (q.before(mid) <= lo - h0)
                            left = mid;
                        else
                            right = mid - 1;
                    }
                    unit = left;
                }
            }
            const long long start = h0 + q.before(unit);
            if (start >= hi)
                return false;
            int tA, tB;
            fill(pc, s, h, unit, q, tA, tB);
            cut(pc, start, q.cost(unit));
            if (++unit == q.units) {
                ++h;
                unit = -1;
            }
            pc.nA = max(0, min(pc.b, tA) - pc.a);
            pc.nB = max(0, min(pc.b, tB) - pc.a);
            // a unit without keys belongs to the run that it starts in
            if (pc.a < pc.b || (pc.t == 0 && start >= lo))
                return true;
        }
        return false;
    }
};

// The share of CTA `index` of `count`; every thread of the block calls it.  `part` (2 words of 64 bits per warp) and
// `found` (3) are shared memory; the share is there for all threads on return.
template <int kThreads>
__device__ __forceinline__ Share find_share(const PrefillParams &p, int index, int count, long long *part, long long *found)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.bs + kThreads - 1) / kThreads;
    const int s0 = min(p.bs, tid * per), s1 = min(p.bs, s0 + per);
    long long cost = 0;
    int units = 0;
    uint32_t largest = 0;                            // one unit's cost (its keys and the fixed part: below 2^32)
#pragma unroll 1
    for (int s = s0; s < s1; ++s) {
        const Seq q = sequence(p, s);
        cost += q.before(q.units) * p.H_kv;
        units += q.units * p.H_kv;
        if (q.units > 0)
            largest = max(largest, (uint32_t)q.cost(q.units - 1));
    }
    long long cost_to = cost, units_to = units;      // inclusive prefixes within the warp
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(kFull, cost_to, o);
        const long long w = __shfl_up_sync(kFull, units_to, o);
        cost_to += lane >= o ? u : 0;
        units_to += lane >= o ? w : 0;
    }
    largest = __reduce_max_sync(kFull, largest);
    if (lane == 31) {
        part[2 * warp] = cost_to;
        part[2 * warp + 1] = (long long)((unsigned long long)(largest >> 4) << 36 | units_to);
    }
    __syncthreads();
    long long total = 0, cost_before = cost_to - cost;
    // (offsets that overlap may give more units than an int holds; such a batch, which is reported, is not dealt out)
    long long all = 0, units_before = units_to - units;
#pragma unroll 1
    for (int w = 0; w < kThreads / 32; ++w) {
        const unsigned long long both = part[2 * w + 1];     // units, and a 16th of their largest cost
        const long long here = both & ((1ull << 36) - 1);
        cost_before += w < warp ? part[2 * w] : 0;
        units_before += w < warp ? here : 0;
        total += part[2 * w];
        all += here;
        largest = max(largest, (uint32_t)(both >> 36) << 4);
    }
    Share sh;
    sh.first = index;
    sh.stride = count;
    const bool alike = (float)largest * (float)all <= 1.4f * (float)total ||
                       (float)largest * (float)count * 8.f <= (float)total;
    sh.dealt = p.deal && alike && all <= INT_MAX ? (int)all / count * count : 0;
    // the cost of what is dealt, then the run's bounds, in one search each among this thread's sequences
    if (tid == 0)
        found[2] = sh.dealt == all ? total : 0;
    __syncthreads();
    if (sh.dealt > 0 && units > 0 && sh.dealt >= units_before && sh.dealt < units_before + units) {
        long long before = cost_before;
        int left = sh.dealt - (int)units_before;
#pragma unroll 1
        for (int s = s0; s < s1; ++s) {
            const Seq q = sequence(p, s);
            const int here = q.units * p.H_kv;
            if (left < here) {
                found[2] = before + (long long)(left / q.units) * q.before(q.units) + q.before(left % q.units);
                break;
            }
            left -= here;
            before += q.before(q.units) * p.H_kv;
        }
    }
    __syncthreads();
    const long long base = found[2], rest = total - base;
    // a little more than rest / count (a 64-bit division takes thousands of cycles in all threads)
    const long long each = (long long)((float)rest / (float)count * (1.f + 0x1p-20f)) + 1;
    sh.lo = min(total, base + each * index);
    sh.hi = min(total, base + each * (index + 1));
    if (cost > 0 && sh.lo >= cost_before && sh.lo < cost_before + cost) {
        long long before = cost_before;
        int s = s0;
#pragma unroll 1
        for (; s < s1 - 1; ++s) {
            const Seq q = sequence(p, s);
            const long long here = q.before(q.units) * p.H_kv;
            if (sh.lo < before + here)
                break;
            before += here;
        }
        found[0] = before;
        found[1] = s;
    }
    __syncthreads();
    sh.before = sh.lo < sh.hi ? found[0] : 0;
    sh.s = sh.lo < sh.hi ? (int)found[1] : p.bs;
    return sh;
}

template <bool FP8>
__global__ void __launch_bounds__(PCfg<FP8>::kThreads, 1)
prefill_kernel(const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ CUtensorMap q_map,
               const PrefillParams p)
{
    using C = PCfg<FP8>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t sbase = smem_u32(smem);
    uint8_t *misc = smem + C::kOffMisc;
    const uint32_t mbase = sbase + C::kOffMisc;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(misc + C::kAbort);
    auto bar_full = [&](int i) { return mbase + C::kBarFull + 8 * i; };
    auto bar_empty = [&](int i) { return mbase + C::kBarEmpty + 8 * i; };
    auto bar_q = [&](int x) { return mbase + C::kBarQ + 8 * x; };
    auto bar_qfree = [&](int x) { return mbase + C::kBarQFree + 8 * x; };
    auto bar_s = [&](int x) { return mbase + C::kBarS + 8 * x; };
    auto bar_p = [&](int x) { return mbase + C::kBarP + 8 * x; };
    auto bar_o = [&](int x) { return mbase + C::kBarO + 8 * x; };
    auto bar_turn = [&](int x) { return mbase + C::kBarTurn + 8 * x; };
    auto bar_vfull = [&](int i) { return mbase + C::kBarVFull + 8 * i; };
    auto bar_vempty = [&](int i) { return mbase + C::kBarVEmpty + 8 * i; };
    auto bar_drain = [&](int x) { return mbase + C::kBarDrain + 8 * x; };
    auto bar_piece = [&](int i) { return mbase + C::kBarPieceFull + 8 * i; };
    auto bar_piece_free = [&](int i) { return mbase + C::kBarPieceEmpty + 8 * i; };
    Piece *ring = reinterpret_cast<Piece *>(misc + C::kPieces);

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kSlots; ++i) {
            mbar_init(bar_full(i), 1);
            mbar_init(bar_empty(i), FP8 && (i & 1) ? 4 : 2);       // both issuers; e4m3's V: the converting warps
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(bar_q(x), 1);
            mbar_init(bar_qfree(x), 1);
            mbar_init(bar_s(x), 1);
            mbar_init(bar_p(x), 4);
            mbar_init(bar_o(x), 1);
            mbar_init(bar_turn(x), 1);
            mbar_init(bar_vfull(x), 4);
            mbar_init(bar_vempty(x), 2);
            mbar_init(bar_drain(x), 1);
        }
        for (int i = 0; i < kRing; ++i) {
            mbar_init(bar_piece(i), 1);
            mbar_init(bar_piece_free(i), C::kReaders);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(mbase + C::kTmemSlot, 512);
        tmem_relinquish();
    }
    wait_prior_grid();
    if (blockIdx.x == 0 && threadIdx.x == 0 && (__ldg(p.cu_q) != 0 || __ldg(p.cu_q + p.bs) != p.num_tokens))
        atomicOr(p.status, SK_DEV_BAD_SEQ);
    // found in the K and V slots' memory, before the first copy
    Share share = find_share<C::kThreads>(p, blockIdx.x, gridDim.x, reinterpret_cast<long long *>(smem),
                                          reinterpret_cast<long long *>(misc + C::kStart));
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(misc + C::kTmemSlot);
    const bool aligned = (sbase & 1023u) == 0;
    if (!aligned && threadIdx.x == 0)
        atomicOr(p.status, SK_DEV_INTERNAL);
    // The next published piece; false at the end of the run, or (ok becomes false) when the wait gave up.
    int read = 0;
    auto next_piece = [&](Piece &pc, bool &ok) {
        const int i = read % kRing;
        ok = __all_sync(kFull, wait_bar(bar_piece(i), (read / kRing) & 1, abort_flag, p.wait_limit));
        if (!ok)
            return false;
        pc = ring[i];
        __syncwarp();
        if (lane == 0)
            mbar_arrive(bar_piece_free(i));
        ++read;
        return pc.s >= 0;
    };
    Piece pc;

    if (warp < 4) {
        reg_dec<C::kRegsIssue>();
        if (warp == 0) {
            // ============================================================ K and V pages
            // slots hold, in turn, K(0), V(0), K(1), V(1), ... of piece after piece
            if (lane == 0)
                prefetch_tensormap(&kv_map);
            int u = 0;
            bool ok = true;
            while (ok && next_piece(pc, ok)) {
                const int page_end = (pc.L + kPage - 1) / kPage;
                const int32_t *bt = p.block_table + (long long)pc.s * p.bt_stride;
                auto block_at = [&](int t) {
                    const int pg = t * C::kPagesPerTile + lane;
                    return (lane < C::kPagesPerTile && t < pc.b && pg < page_end) ? __ldg(bt + pg) : -1;
                };
                int blk = block_at(pc.a), blk1 = block_at(pc.a + 1);
                for (int t = pc.a; t < pc.b && ok; ++t) {
                    const int blk2 = block_at(t + 2);
#pragma unroll
                    for (int part = 0; part < 2; ++part, ++u) {
                        const int i = u % C::kSlots;
                        if (u >= C::kSlots)
                            ok = wait_bar(bar_empty(i), (u / C::kSlots - 1) & 1, abort_flag, p.wait_limit);
                        ok = __all_sync(kFull, ok);
                        if (!ok)
                            break;
                        if (lane == 0)
                            mbar_arrive_expect_tx(bar_full(i), C::kSlotBytes);
                        __syncwarp();
                        if (lane < C::kPagesPerTile) {
                            int grp = -2;            // whole box out of bounds: zero fill
                            if (t * C::kPagesPerTile + lane < page_end) {
                                if (blk >= 0 && blk < p.num_blocks)
                                    grp = (blk * p.H_kv + pc.h) * 2;
                                else
                                    atomicOr(p.status, SK_DEV_BAD_BLOCK);
                            }
                            tma_load_4d(sbase + i * C::kSlotBytes + lane * 2 * C::kGroupBytes, &kv_map, 0, 0,
                                        part * (FP8 ? 1 : 2), grp, bar_full(i));
                        }
                    }
                    blk = blk1;
                    blk1 = blk2;
                }
            }
            if (!ok) {
                *abort_flag = 1;
                if (lane == 0)
                    atomicOr(p.status, SK_DEV_TIMEOUT);
            }
            // every copy issued lands before the CTA exits
            for (int t = u > C::kSlots ? u - C::kSlots : 0; t < u; ++t)
                wait_bar(bar_full(t % C::kSlots), (t / C::kSlots) & 1, nullptr, kDrainLimit);
        } else if (warp == 3) {
            // ============================================================ the pieces, and their Q tiles
            if (!aligned) {
                share.s = p.bs;
                share.dealt = 0;
            }
            Walk walk(p, share);
            Piece *shared = p.shared + 2 * blockIdx.x;   // this run's pieces of units that others have a part of
            if (lane < 2)
                shared[lane].s = -1;
            __syncwarp();
            int used[2] = {0, 0};                        // Q tiles copied
            bool ok = true, more = true;
            for (int k = 0; ok && more; ++k) {
                more = walk.next(pc);
                if (!more)
                    pc.s = -1;
                if (k >= kRing)
                    ok = wait_bar(bar_piece_free(k % kRing), (k / kRing - 1) & 1, abort_flag, p.wait_limit);
                ok = __all_sync(kFull, ok);
                if (!ok)
                    break;
                if (lane == 0) {
                    ring[k % kRing] = pc;
                    if (more && (pc.a > 0 || pc.b < pc.t))
                        shared[pc.a > 0 ? 0 : 1] = pc;
                    mbar_arrive(bar_piece(k % kRing));
                }
                __syncwarp();
                if (!more)
                    break;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (!ok || (x ? pc.nB : pc.nA) == 0)
                        continue;
                    if (used[x] > 0)
                        ok = wait_bar(bar_qfree(x), (used[x] - 1) & 1, abort_flag, p.wait_limit);
                    ok = __all_sync(kFull, ok);
                    if (ok && lane == 0) {
                        int j0, i0;
                        tile_origin(p, 2 * pc.unit + x, j0, i0);
                        const uint32_t dst = sbase + C::kOffQ + x * C::kQTile;
                        mbar_arrive_expect_tx(bar_q(x), (uint32_t)(p.gb * p.tpb * 256));
                        tma_load_3d(dst, &q_map, 0, pc.h * p.G + i0, pc.tok0 + j0, bar_q(x));
                        tma_load_3d(dst + kRows * 128, &q_map, FP8 ? 128 : 64, pc.h * p.G + i0, pc.tok0 + j0, bar_q(x));
                    }
                    __syncwarp();
                    used[x] += ok ? 1 : 0;
                }
            }
            if (!ok) {
                *abort_flag = 1;
                if (lane == 0)
                    atomicOr(p.status, SK_DEV_TIMEOUT);
            }
            for (int x = 0; x < 2; ++x)
                if (used[x] > 0)
                    wait_bar(bar_q(x), (used[x] - 1) & 1, nullptr, kDrainLimit);
        } else if (warp <= 2) {
            // ============================================================ products of row tile x
            constexpr uint32_t idesc_qk = FP8 ? idesc_e4m3_f32(kRows, kKeys, 0, 0) : idesc_bf16_f32(kRows, kKeys, 0, 0);
            constexpr uint32_t idesc_pv = FP8 ? idesc_f16_f32(kRows, kHeadDim, 0, 1)
                                              : idesc_bf16_f32(kRows, kHeadDim, 0, 1);
            const int x = warp - 1;
            const uint64_t d_k0 = smem_desc_sw128(sbase, 16, C::kGroupBytes);       // K-major K
            const uint64_t d_v0 = smem_desc_sw128(sbase + (FP8 ? C::kOffV : 0), 1024, 2048);    // dimension-major V
            const uint64_t d_q = smem_desc_sw128(sbase + C::kOffQ + x * C::kQTile, 16, 1024);   // K-major Q
            const uint32_t sd = tmem + kColS + x * 128, od = tmem + kColO + x * 128;
            auto adv = [](uint64_t d, uint32_t bytes) { return d + (uint64_t)(bytes >> 4); };
            bool ok = true;
            int u = 0, tiles = 0;                    // slots and key tiles before this piece
            int mine = 0, pieces = 0;                // this row tile's key tiles and pieces so far
            auto wait = [&](uint32_t bar, uint32_t parity) {
                if (ok)
                    ok = wait_bar(bar, parity, abort_flag, p.wait_limit);
                ok = __all_sync(kFull, ok);
                return ok;
            };
            auto wait_slot = [&](int i) { return wait(bar_full(i % C::kSlots), (i / C::kSlots) & 1); };
            // passes the turn with half of the products still to issue: the other issuer wakes up meanwhile
            auto pass_turn = [&]() {
                if (lane == 0)
                    mbar_arrive(bar_turn(1 - x));
                __syncwarp();
            };
            auto qk = [&](int slot, bool pass) {
                const uint64_t k0 = adv(d_k0, (uint32_t)(slot % C::kSlots) * C::kSlotBytes);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if constexpr (FP8)
                        mma4_f8_ss<2, 2>(sd, adv(d_q, h * (kRows * 128)), k0, idesc_qk, h);
                    else
                        mma4_f16_ss<2, 2>(sd, adv(d_q, h * (kRows * 128)), adv(k0, h * 1024), idesc_qk, h);
                    if (h == 0 && pass)
                        pass_turn();
                }
                mma_commit_warp(bar_s(x));
            };
            auto pv = [&](int j) {
                const uint64_t v0 = adv(d_v0, FP8 ? (uint32_t)((tiles + j) & 1) * C::kVBytes
                                                  : (uint32_t)((u + 2 * j + 1) % C::kSlots) * C::kSlotBytes);
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    mma4_f16_ts<8, 256>(od, sd + h * 64, adv(v0, h * 16384), idesc_pv, j > 0 || h > 0);
            };
            auto wait_v = [&](int j) {
                return FP8 ? wait(bar_vfull((tiles + j) & 1), ((tiles + j) >> 1) & 1) : wait_slot(u + 2 * j + 1);
            };
            // Both issuers pass every slot on, also those of tiles that only the other multiplies (they wait for them
            // all the same, so that neither is a turn of the ring ahead).
            while (ok && next_piece(pc, ok)) {
                const int n = pc.b - pc.a, nx = x ? pc.nB : pc.nA;
                if (n == 0)
                    continue;
                if (nx > 0 && !wait(bar_q(x), pieces & 1))
                    break;
                for (int j = -1; j < n && ok; ++j) {
                    // what has to have landed is checked while the softmax still works on the tile
                    if ((j >= 0 && !wait_v(j)) || (j + 1 < n && !wait_slot(u + 2 * j + 2)))
                        break;
                    if (j >= 0) {
                        // The row tiles take turns, so that one's softmax runs beside the other's products: A's products
                        // of a tile come after B's of the tile before, B's after A's of the same.  A row tile that has
                        // none there passes its turn on, so that neither is ever two turns ahead (a barrier shows only
                        // whether the last turn of a parity is over).
                        if ((x || tiles + j > 0) && !wait(bar_turn(x), (tiles + j - 1 + x) & 1))
                            break;
                        if (j < nx && !wait(bar_p(x), (mine + j) & 1))
                            break;
                    }
                    tc_fence_after();
                    if (j >= 0 && j < nx)
                        pv(j);
                    if (j + 1 < nx) {
                        qk(u + 2 * j + 2, j >= 0);
                        if (j + 2 == nx)
                            mma_commit_warp(bar_qfree(x));
                    } else if (j >= 0) {
                        if (j + 1 == nx)
                            mma_commit_warp(bar_o(x));
                        pass_turn();
                    }
                    if (j >= 0)
                        mma_commit_warp(FP8 ? bar_vempty((tiles + j) & 1) : bar_empty((u + 2 * j + 1) % C::kSlots));
                    if (j + 1 < n)
                        mma_commit_warp(bar_empty((u + 2 * j + 2) % C::kSlots));
                }
                u += 2 * n;
                tiles += n;
                mine += nx;
                pieces += nx > 0 ? 1 : 0;
            }
            if (!ok) {
                *abort_flag = 1;
                if (lane == 0)
                    atomicOr(p.status, SK_DEV_TIMEOUT);
            }
            // every product completes before TMEM is freed and shared memory is left
            mma_commit_warp(bar_drain(x));
            wait_bar(bar_drain(x), 0, nullptr, kDrainLimit);
        }
        __syncwarp();
    } else if (!FP8 || warp < 12) {
        // ================================================================ softmax of row tile x
        reg_inc<C::kRegsSoftmax>();
        const int x = (warp >> 2) - 1;
        const int quarter = warp & 3;
        const int tau = quarter * 32 + lane;                       // row of the tile, TMEM lane
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const uint32_t ts = tmem + kColS + x * 128 + lane_off, to = tmem + kColO + x * 128 + lane_off;
        int mine = 0, pieces = 0, u = 0;                           // this row tile's key tiles and pieces, slots so far
        bool failed = false;
        while (!failed) {
        // The piece stays in the ring, to be read again for the output, until that is written: in registers it would
        // spill the scores.
        const int place = read % kRing;
        volatile Piece *pc = ring + place;
        if (!__all_sync(kFull, wait_bar(bar_piece(place), (read / kRing) & 1, abort_flag, p.wait_limit))) {
            failed = true;
            break;
        }
        if (pc->s < 0)
            break;
        ++read;
        // this row: its token, and its head in the group
        auto row_at = [&](int &j, int &i) {
            tile_origin(p, 2 * pc->unit + x, j, i);
            const int jj = tau / p.gb;
            j += jj;
            i += tau - jj * p.gb;
            return jj < p.tpb && j < pc->q_len && i < p.G;
        };
        const int nx = x ? pc->nB : pc->nA;
        const int first_key = pc->a * kKeys, L = pc->L;
        int limit, least;                                          // keys that the row sees; that all of the warp's see
        float c = p.score_scale_log2;
        {
            int j, i;
            const bool live = row_at(j, i);
            limit = live ? visible_keys(L, pc->q_len, j, p.causal) : 0;
            least = __reduce_min_sync(kFull, live ? limit : INT_MAX);        // what padding rows hold is never used
            if (FP8 && live)
                c *= __ldg(p.q_scale + (long long)(pc->tok0 + j) * p.H_q + pc->h * p.G + i);
        }
        float m_ref = -CUDART_INF_F;
        bool anchored = false;                                     // every row that sees a key has a reference
        float2 l2 = make_float2(0.f, 0.f);
        for (int j = 0; j < nx; ++j) {
            const int key0 = first_key + j * kKeys;
            bool ok = wait_bar(bar_s(x), (mine + j) & 1, abort_flag, p.wait_limit);
            ok = __all_sync(kFull, ok);
            if (!ok) {
                failed = true;
                break;
            }
            tc_fence_after();
            float v[128];
#pragma unroll
            for (int cc = 0; cc < 128; cc += 32)
                tmem_ld32<32>(ts + cc, v + cc);
            tmem_wait_ld();
            const int lim = limit - key0;                          // columns [0, lim) are visible
            if (key0 + kKeys > least) {                            // uniform in the warp
#pragma unroll
                for (int i = 0; i < 128; ++i)
                    v[i] = i < lim ? v[i] : -CUDART_INF_F;
            }
            // the tile's largest score, in log2 units
            auto tile_top = [&]() {
                float mx[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
                for (int i = 4; i < 124; i += 8) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mx[k] = fmax3(mx[k], v[i + k], v[i + 4 + k]);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mx[k] = fmaxf(mx[k], v[124 + k]);
                return fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]) * c;
            };
            // moves the rows' reference up to kAbove below `top` and rescales what they have summed; `in_o`: O holds
            // something
            auto raise = [&](float top, bool in_o) {
                const float mn = fmaxf(m_ref, top - C::kAbove);
                const float alpha = m_ref == -CUDART_INF_F ? 0.f : exp2f(m_ref - mn);
                m_ref = mn;
                l2.x *= alpha;
                l2.y *= alpha;
                if (in_o) {
#pragma unroll 1
                    for (int cc = 0; cc < 128; cc += 32) {
                        float o[32];
                        tmem_ld32<32>(to + cc, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            o[i] *= alpha;
                        tmem_st32<32>(to + cc, o);
                    }
                }
            };
            // A row's first scores give it a reference: the largest of the first 16 will do (see below).
            if (!anchored) {
                if (__any_sync(kFull, m_ref == -CUDART_INF_F && lim > 0)) {
                    float top = v[0];
#pragma unroll
                    for (int i = 1; i < 15; i += 2)
                        top = fmax3(top, v[i], v[i + 1]);
                    raise(fmaxf(top, v[15]) * c, j > 0);
                }
                anchored = !__any_sync(kFull, m_ref == -CUDART_INF_F && limit > 0);
            }
            // rows past the sequence's end in its last page hold anything, and 0 * NaN would reach O: their V
            // becomes zeros, before either row tile multiplies it
            if (!FP8 && L < key0 + kKeys && (L & (kPage - 1)) != 0) {
                const int i = u + 2 * j + 1;
                ok = wait_bar(bar_full(i % C::kSlots), (i / C::kSlots) & 1, abort_flag, p.wait_limit);
                ok = __all_sync(kFull, ok);
                const int tok = key0 + tau;
                if (ok && tok >= L && tok < (L + kPage - 1) / kPage * kPage) {
                    uint8_t *row = smem + i % C::kSlots * C::kSlotBytes + (tau >> 3) * C::kGroupBytes +
                                   (tau & 7) * 128;
#pragma unroll
                    for (int cc = 0; cc < C::kGroupBytes / 1024; ++cc)
#pragma unroll
                        for (int u = 0; u < 8; ++u)
                            *reinterpret_cast<uint4 *>(row + cc * 1024 + u * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                if (!ok) {
                    *abort_flag = 1;                               // the other roles' waits end with it
                    atomicOr(p.status, SK_DEV_TIMEOUT);
                }
                __syncwarp();
            }
            // P overwrites the first columns of each half of S.  A row's reference need not follow its maximum while
            // the probabilities stay well inside their type's range, and the tile's sum shows whether some did not.
            // Only then is the maximum taken, the reference raised, O rescaled and the tile done again.  The same for a
            // row whose first 16 scores were all minus infinity: what it sums relative to no reference is not kept.
            const float2 c2 = make_float2(c, c);
            float2 h2;
#pragma unroll 1
            for (int again = 0; again < 2; ++again) {
                const float msub = m_ref == -CUDART_INF_F ? 0.f : m_ref;
                const float2 s2 = make_float2(-msub, -msub);
                h2 = make_float2(0.f, 0.f);
                float2 g2 = make_float2(0.f, 0.f);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int k = q * 32 + 2 * i;
                        const float2 d = ffma2(make_float2(v[k], v[k + 1]), c2, s2);
                        const float2 e = make_float2(ex2_ftz(d.x), ex2_ftz(d.y));
                        (i & 1 ? g2 : h2) = fadd2(i & 1 ? g2 : h2, e);
                        pk[i] = FP8 ? pack_f16x2(e.x, e.y) : pack_bf16x2(e.x, e.y);
                    }
                    tmem_st32_u<16>(ts + (q >> 1) * 64 + (q & 1) * 16, pk);
                }
                h2 = fadd2(h2, g2);
                const bool redo = limit > 0 && !(h2.x + h2.y <= C::kSumMost);
                if (again || !__any_sync(kFull, redo || (lim > 0 && m_ref == -CUDART_INF_F)))
                    break;
                tmem_wait_st();
                raise(tile_top(), j > 0);
            }
            l2 = fadd2(l2, h2);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar_p(x));
        }
        if (failed)
            break;
        // ---- the row's output, or its partial state (its place is found while the last products run).  A lane's row is
        // transposed within quads of lanes, so that a warp's store writes 64 contiguous bytes of eight rows (with 16 bytes
        // of 32 rows it took 5000 cycles)
        int jr, ir;
        const bool live = row_at(jr, ir);
        const bool whole = pc->a == 0 && pc->b == pc->t;
        const int qrow = live ? (pc->tok0 + jr) * p.H_q + pc->h * p.G + ir : -1;
        // a run has at most one piece that does not start its unit, and one more that does not end it
        const int part = (2 * blockIdx.x + (pc->a > 0 ? 0 : 1)) * (2 * kRows) + x * kRows + tau;
        const float l = l2.x + l2.y;
        const float mul = !whole ? p.v_scale : (l == 0.f ? 0.f : p.v_scale / l);
        int to_row[4];                                             // the quad's rows
#pragma unroll
        for (int i = 0; i < 4; ++i)
            to_row[i] = __shfl_sync(kFull, whole || !live ? qrow : part, (lane & ~3) + i);
        // a row that saw nothing is zero, whatever V holds
        const bool empty = __any_sync(kFull, nx == 0 || l == 0.f);
        uint8_t *dst = whole ? reinterpret_cast<uint8_t *>(p.out) : reinterpret_cast<uint8_t *>(p.part_o);
        const int row_bytes = whole ? kHeadDim * 2 : kHeadDim * 4;
        if (nx > 0) {
            const bool ok = wait_bar(bar_o(x), pieces & 1, abort_flag, p.wait_limit);
            if (!__all_sync(kFull, ok)) {
                failed = true;
                break;
            }
            tc_fence_after();
        }
#pragma unroll 1
        for (int cc = 0, at = (lane & 3) * 16; at < row_bytes; cc += whole ? 32 : 16, at += 64) {
            // 64 bytes of every row: 32 dimensions rounded, or 16 as they are
            float o[32];
            if (nx > 0) {
                tmem_ld32<16>(to + cc, o);
                if (whole)
                    tmem_ld32<16>(to + cc + 16, o + 16);
                tmem_wait_ld();
            }
#pragma unroll
            for (int i = 0; i < 32; ++i)
                o[i] = empty && (nx == 0 || l == 0.f) ? 0.f : o[i] * mul;
            uint4 w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                w[k] = whole ? make_uint4(pack_bf16x2(o[8 * k], o[8 * k + 1]), pack_bf16x2(o[8 * k + 2], o[8 * k + 3]),
                                          pack_bf16x2(o[8 * k + 4], o[8 * k + 5]), pack_bf16x2(o[8 * k + 6], o[8 * k + 7]))
                             : make_uint4(__float_as_uint(o[4 * k]), __float_as_uint(o[4 * k + 1]),
                                          __float_as_uint(o[4 * k + 2]), __float_as_uint(o[4 * k + 3]));
            quad_transpose(w, lane);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (to_row[i] >= 0)
                    *reinterpret_cast<uint4 *>(dst + (long long)to_row[i] * row_bytes + at) = w[i];
            __syncwarp();
        }
        if (live) {
            if (!whole) {
                p.part_m[part] = m_ref;
                p.part_l[part] = l;
            } else if (p.lse != nullptr) {
                p.lse[qrow] = l == 0.f ? -CUDART_INF_F : m_ref * 0.69314718055994531f + logf(l);
            }
        }
        // the next piece's first product into O waits for its P, which this thread writes after these reads
        tc_fence_before();
        mine += nx;
        pieces += nx > 0 ? 1 : 0;
        u += 2 * (pc->b - pc->a);
        __syncwarp();
        if (lane == 0)
            mbar_arrive(bar_piece_free(place));
        }
        if (failed) {
            *abort_flag = 1;
            if (lane == 0)
                atomicOr(p.status, SK_DEV_TIMEOUT);
        }
    } else {
        // ================================================================ e4m3: V codes to f16 (exact)
        reg_dec<C::kRegsConvert>();
        const int w = warp - 12;
        // a warp's load is four tokens' 128 codes, 16 a lane; token t's unit u lies at u ^ (t % 8) in its row.  The 16
        // dimensions become units 2 u and 2 u + 1 of f16, the upper half of the lanes storing the odd one first, so
        // that a store's lanes meet no bank twice
        const int u = lane & 7, sub = lane >> 3;
        int v = 0;                                                 // key tiles so far
        bool ok = true;
        while (ok && next_piece(pc, ok))
        for (int tile = pc.a; tile < pc.b; ++tile, ++v) {
            const int slot = (2 * v + 1) % C::kSlots, vb = v & 1;
            ok = wait_bar(bar_full(slot), ((2 * v + 1) / C::kSlots) & 1, abort_flag, p.wait_limit);
            if (ok && v >= 2)
                ok = wait_bar(bar_vempty(vb), ((v >> 1) - 1) & 1, abort_flag, p.wait_limit);
            ok = __all_sync(kFull, ok);
            if (!ok)
                break;
            const uint8_t *src = smem + slot * C::kSlotBytes;
            uint8_t *dst = smem + C::kOffV + vb * C::kVBytes;
            const int key0 = tile * kKeys;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int t = w * 32 + k * 4 + sub, x8 = t & 7;
                uint4 a = *reinterpret_cast<const uint4 *>(src + (t >> 3) * 1024 + x8 * 128 + ((u ^ x8) << 4));
                if (key0 + t >= pc.L)                               // past the end the page holds anything
                    a = make_uint4(0u, 0u, 0u, 0u);
                const uint4 lo = make_uint4(f16x2_of_e4m3(a.x), f16x2_of_e4m3(a.x >> 16), f16x2_of_e4m3(a.y),
                                            f16x2_of_e4m3(a.y >> 16));
                const uint4 hi = make_uint4(f16x2_of_e4m3(a.z), f16x2_of_e4m3(a.z >> 16), f16x2_of_e4m3(a.w),
                                            f16x2_of_e4m3(a.w >> 16));
                uint8_t *row = dst + (t >> 3) * 2048 + (u >> 2) * 1024 + x8 * 128;
                const int first = (2 * u & 7) + (u >> 2), second = first ^ 1;
                *reinterpret_cast<uint4 *>(row + ((first ^ x8) << 4)) = u >> 2 ? hi : lo;
                *reinterpret_cast<uint4 *>(row + ((second ^ x8) << 4)) = u >> 2 ? lo : hi;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar_vfull(vb));
                mbar_arrive(bar_empty(slot));
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

// Joins the pieces of the units that several runs share: block (run, part) those of the unit whose last piece is run's
// first.  Its other pieces are the first ones of the runs before, back to the run that the unit starts in, whose last piece
// it is.  They are taken in key order, whatever the timing of the runs.  With M = max m_i over the pieces with l_i > 0:
//     out = sum o_i 2^(m_i - M) / sum l_i 2^(m_i - M)
constexpr int kJoinThreads = 256, kJoinParts = 16;
constexpr int kMaxRuns = 1024;                       // runs (SMs) at most
constexpr int kJoinRows = 2 * kRows / kJoinParts / (kJoinThreads / 32);      // rows of one warp

__global__ void __launch_bounds__(kJoinThreads) prefill_join_kernel(const PrefillParams p)
{
    __shared__ int slots[kMaxRuns], count;
    wait_prior_grid();
    const int index = blockIdx.x / kJoinParts, part = blockIdx.x % kJoinParts;
    const Piece pc = p.shared[2 * index];
    if (pc.s < 0 || pc.b != pc.t)
        return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 0) {
        const int n = shared_slots(index, [&](int slot) { return p.shared[slot].s >= 0; }, slots);
        if (lane == 0)
            count = n;
    }
    __syncthreads();
    const int pieces = count;
    const int tok0 = __ldg(p.cu_q + pc.s);
    for (int k = 0; k < kJoinRows; ++k) {
        const int row = (part * (kJoinThreads / 32) + warp) * kJoinRows + k;     // of the unit's 256
        const int x = row / kRows, tau = row % kRows;
        int j0, i0;
        tile_origin(p, 2 * pc.unit + x, j0, i0);
        const int jj = tau / p.gb, ii = tau - jj * p.gb;
        if (!(jj < p.tpb && j0 + jj < pc.q_len && i0 + ii < p.G))
            continue;                                // uniform in the warp
        float M = -CUDART_INF_F, lam = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        constexpr int kAtOnce = 8;
        for (int g0 = 0; g0 < pieces; g0 += kAtOnce) {
            float m[kAtOnce], l[kAtOnce];
            float4 o[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                const long long slot = (long long)slots[max(pieces - 1 - g0 - i, 0)] * (2 * kRows) + row;
                m[i] = __ldg(p.part_m + slot);
                l[i] = g0 + i < pieces ? __ldg(p.part_l + slot) : 0.f;
                o[i] = __ldg(reinterpret_cast<const float4 *>(p.part_o + slot * kHeadDim) + lane);
            }
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                if (l[i] == 0.f)
                    continue;
                const float mn = fmaxf(M, m[i]), wa = M == -CUDART_INF_F ? 0.f : exp2f(M - mn), wb = exp2f(m[i] - mn);
                M = mn;
                lam = lam * wa + l[i] * wb;
                acc.x = acc.x * wa + o[i].x * wb;
                acc.y = acc.y * wa + o[i].y * wb;
                acc.z = acc.z * wa + o[i].z * wb;
                acc.w = acc.w * wa + o[i].w * wb;
            }
        }
        const float inv = lam == 0.f ? 0.f : 1.f / lam;
        const long long qrow = (long long)(tok0 + j0 + jj) * p.H_q + pc.h * p.G + i0 + ii;
        *reinterpret_cast<uint2 *>(p.out + qrow * kHeadDim + lane * 4) =
            make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
        if (lane == 0 && p.lse != nullptr)
            p.lse[qrow] = lam == 0.f ? -CUDART_INF_F : M * 0.69314718055994531f + logf(lam);
    }
}

template <bool FP8>
cudaError_t launch_t(const CUtensorMap &kv_map, const CUtensorMap &q_map, const PrefillParams &p, int runs,
                     cudaStream_t stream)
{
    const cudaError_t e = cudaFuncSetAttribute(prefill_kernel<FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               PCfg<FP8>::kSmemBytes);
    if (e != cudaSuccess)
        return e;
    // the warpgroups' shares after the reallocation may not exceed what the CTA was launched with
    static const int regs = [] {
        cudaFuncAttributes a{};
        return cudaFuncGetAttributes(&a, prefill_kernel<FP8>) == cudaSuccess ? a.numRegs : 0;
    }();
    if (regs < PCfg<FP8>::kRegsLaunch)
        return cudaErrorInvalidConfiguration;
    return launch_pdl(prefill_kernel<FP8>, dim3((unsigned)runs), dim3(PCfg<FP8>::kThreads), PCfg<FP8>::kSmemBytes,
                      stream, kv_map, q_map, p);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn()
{
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(ptr);
    });
    return fn;
}

}  // namespace

cudaError_t encode_page_map(CUtensorMap *map, const void *pages, long long num_blocks, int H_kv, bool fp8, int chunks)
{
    EncodeTiledFn enc = encode_fn();
    if (enc == nullptr)
        return cudaErrorNotSupported;
    const cuuint64_t row_bytes = (cuuint64_t)(2 * kHeadDim * (fp8 ? 1 : 2));
    const cuuint64_t dims[4] = {(cuuint64_t)(fp8 ? 128 : 64), 8, row_bytes / 128, (cuuint64_t)num_blocks * H_kv * 2};
    const cuuint64_t strides[3] = {row_bytes, 128, 8 * row_bytes};
    const cuuint32_t box[4] = {fp8 ? 128u : 64u, 8, (cuuint32_t)chunks, 2};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    const CUresult r = enc(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                           const_cast<void *>(pages), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t encode_q_map(CUtensorMap *map, const void *q, long long num_tokens, int H_q, bool fp8, int heads, int toks)
{
    EncodeTiledFn enc = encode_fn();
    if (enc == nullptr)
        return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {(cuuint64_t)(fp8 ? 256 : 128), (cuuint64_t)H_q, (cuuint64_t)num_tokens};
    const cuuint64_t strides[2] = {256, (cuuint64_t)H_q * 256};
    const cuuint32_t box[3] = {fp8 ? 128u : 64u, (cuuint32_t)heads, (cuuint32_t)toks};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = enc(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                           const_cast<void *>(q), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Bytes of the workspace: two pieces of 256 rows (o, m, l) per run with what they are pieces of, and for e4m3 pages Q in
// two terms.
long long prefill_workspace_bytes(int num_tokens, int H_q, int kv_dtype, int num_sms)
{
    const long long parts = 2LL * num_sms * (2 * kRows * (kHeadDim + 2) * 4 + (long long)sizeof(PrefillPiece));
    return parts + (kv_dtype == SK_KV_FP8_E4M3 ? (long long)num_tokens * H_q * (2 * kHeadDim + 4) : 0);
}

cudaError_t launch_prefill(const PrefillParams &params, int kv_dtype, long long max_seq_len, void *workspace, int num_sms,
                           cudaStream_t stream)
{
    const bool fp8 = kv_dtype == SK_KV_FP8_E4M3;
    PrefillParams p = params;
    p.gb = p.G < kRows ? p.G : kRows;
    p.nsub = (p.G + p.gb - 1) / p.gb;
    p.tpb = kRows / p.gb;
    const long long slots = 2LL * num_sms * 2 * kRows;
    p.part_o = static_cast<float *>(workspace);
    p.part_m = p.part_o + slots * kHeadDim;
    p.part_l = p.part_m + slots;
    p.shared = reinterpret_cast<PrefillPiece *>(p.part_l + slots);
    const void *q = p.q;
    if (fp8) {
        uint8_t *codes = reinterpret_cast<uint8_t *>(p.shared + 2 * num_sms);
        const long long rows = (long long)p.num_tokens * p.H_q;
        const cudaError_t e = launch_split_q(p.q, rows, codes, stream);
        if (e != cudaSuccess)
            return e;
        q = codes;
        p.q_scale = reinterpret_cast<const float *>(codes + rows * 256);
    }
    CUtensorMap kv_map, q_map;
    // one box of the pages: K (or V) of one page and head
    cudaError_t e = encode_page_map(&kv_map, p.kv, p.num_blocks, p.H_kv, fp8, fp8 ? 1 : 2);
    if (e == cudaSuccess)
        e = encode_q_map(&q_map, q, p.num_tokens, p.H_q, fp8, p.gb, p.tpb);
    if (e != cudaSuccess)
        return e;
    // A run per SM, but none of less than two key tiles on average: the number of units and of key tiles is bounded by
    // the tokens and by max_seq_len.
    const long long per_seq = ((long long)(p.max_q_len + p.tpb - 1) / p.tpb * p.nsub + 1) / 2 * p.bs;
    const long long by_tokens = ((long long)(p.num_tokens + p.tpb - 1) / p.tpb * p.nsub + 1) / 2 + p.bs;
    const long long units = (per_seq < by_tokens ? per_seq : by_tokens) * p.H_kv;
    const long long tiles = (max_seq_len + kKeys - 1) / kKeys;
    long long runs = units * (tiles < 2 ? 1 : tiles / 2);
    runs = runs < 1 ? 1 : (runs < num_sms ? runs : num_sms);
    runs = runs < kMaxRuns ? runs : kMaxRuns;
    p.deal = (double)p.bs * max_seq_len * p.H_kv * (fp8 ? 256 : 512) > kL2Share ? 1 : 0;
    e = fp8 ? launch_t<true>(kv_map, q_map, p, (int)runs, stream) : launch_t<false>(kv_map, q_map, p, (int)runs, stream);
    if (e != cudaSuccess || runs == 1)
        return e;
    return launch_pdl(prefill_join_kernel, dim3((unsigned)runs * kJoinParts), dim3(kJoinThreads), 0, stream, p);
}

}  // namespace sk
