// Attention with a sliding window and sinks for chunks of new tokens (prompts, parts of prompts, follow-up turns) over the
// paged cache (bf16 or e4m3 pages) on the tcgen05 tensor cores.
//
// For the rows r = j * G + i (query token j, head i of the group) of one (sequence, KV head), with P = L - q + j:
//     S = scale Q K^T over the keys p <= P with p < sinks or p > P - window,   O = softmax(S) V,   lse = log sum exp S
//
// The products are those of sk_paged_prefill_attn's kernel: 256 rows of a CTA as two tiles A and B of 128 (the MMA's M), keys
// in tiles of 128 (its N), S_A, S_B, O_A and O_B in the 512 TMEM columns, P over S in half its columns as the A operand of
// PV, a row one TMEM lane and so one thread.  For each row tile x, in issue order over the key tiles j:
//     O_x += P_x(j) V(j);  S_x = Q_x K(j+1)^T
// What differs is that a unit of work (256 rows over the keys that they see) is short: sinks + window + the unit's tokens,
// five key tiles for a window of 512.  Its bound is the tensor cores' 4 * 128 flops per (row, key); what costs beside them is
// a unit's start, its end, its masked tiles, and the code that these take: roles that together run through more of it than
// the instruction cache holds stall on it (with the softmax unrolled over 128 columns and a walk with sums of 64 bits, 107 KB,
// 2.3 warps waited for instructions for each that issued).  So the softmax takes half of a tile at a time, but
// for long units, and the shares are found and walked by one warp in 32 bits.
//
// Roles (384 threads; 512 for e4m3 pages):
//   warp 0      copies: K and V of a key tile apart, 32 KB (16 KB e4m3) slots, one TMA copy per page and part
//   warps 1, 2  issue the products of A and of B and take turns (warp 1 also allocates TMEM)
//   warp 3      finds the pieces of the CTA's share, publishes them to the others, copies their Q tiles
//   warps 4-7, 8-11  softmax of A and of B, its rescaling, its output
//   warps 12-15 (e4m3)  V's codes to f16 (exactly), for PV with P as f16
// S(j) complete implies PV(j - 1) complete (products of one issuer complete in issue order), so the softmax may rescale O
// at once; it does so only when scores beat the reference by far.
//
// P is rounded to V's type, bf16, as the product takes both of one (f16 on e4m3 pages); its sum is not: the output is off from
// 64 bits by 0.0023 of its size, where rounding the output alone is 0.0016 (f16: 0.0017).
//
// Every wait is bounded: on expiry SK_DEV_TIMEOUT is set and every role gives up, after its copies and products in flight.
//
// Measured: 4096 tokens over a window of 4096, 32/8 heads: 196 us, 1.40 PFLOP/s of the pairs that are seen.  24 prompts of up to
// 2000 tokens over 512, 16/2 heads: 112 us; 16001 tokens over 128: 53 us; 1919 tokens of four prompts over 2048 on e4m3 pages:
// 40 us.  A key tile takes 3050 cycles: the softmax of a row tile (1600) and its products (1024 for both of its own), one after
// the other, beside those of the other row tile; a unit's start and end take 5000 more, a call's first S 12000, on code that
// runs once in a while; the tensor pipe is busy 61 % of the first call, 41 % of the second.
#include <cuda.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <math_constants.h>
#include <stdint.h>

#include "sk_attn_util.cuh"
#include "sk_cache_ops.cuh"
#include "sk_sm100.cuh"
#include "sk_window_cost.cuh"

namespace sk {
namespace {

using namespace sm100;

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kRows = kChunkRows;                    // rows of one tile (MMA M)
constexpr int kKeys = kChunkKeys;                    // keys of one tile (MMA N)
constexpr uint32_t kDrainLimit = 4000000000u;        // cycles (~2 s): waits for work already issued
constexpr int kMaxSmem = 232448;
constexpr int kRing = 4;                             // pieces published ahead

// WIDE: a tile that a warp's rows all see is taken in one go, for units of many key tiles (kWideTiles)
template <bool FP8, bool WIDE>
struct CCfg {
    static constexpr int kThreads = FP8 ? 512 : 384;
    // registers per thread after the reallocation: copies and products, softmax, e4m3's conversion of V; no more in all
    // than at launch (4 x 128, or 3 x 168)
    static constexpr int kRegsLaunch = FP8 ? 128 : 168;
    static constexpr int kRegsIssue = FP8 ? 64 : 72, kRegsSoftmax = !FP8 ? 216 : WIDE ? 208 : 184,
                         kRegsConvert = WIDE ? 32 : 80;
    static constexpr int kLoads = WIDE ? 2 : 8;                    // of a tile's V, under way before the first is converted
    static_assert(kRegsIssue + 2 * kRegsSoftmax + (FP8 ? kRegsConvert : 0) <= kThreads / 128 * kRegsLaunch, "registers");
    static constexpr int kQTile = kRows * 256;                     // bf16: two 64-dimension chunks; e4m3: hi and lo
    static constexpr int kGroupBytes = FP8 ? 1024 : 2048;          // K (or V) of 8 tokens, as copied
    static constexpr int kSlotBytes = kKeys / 8 * kGroupBytes;
    static constexpr int kVBytes = FP8 ? kKeys * 256 : 0;          // e4m3: V of a tile as f16, two of them
    static constexpr int kMisc = 1024;                             // barriers
    // each softmax warp's rows on their way out, 64 dimensions of them at a time
    static constexpr int kOutWarp = 32 * 128;
    static constexpr int kSlots = (kMaxSmem - 2 * kQTile - 2 * kVBytes - 8 * kOutWarp - kMisc) / kSlotBytes;
    static constexpr int kOffV = kSlots * kSlotBytes;
    static constexpr int kOffOut = kOffV + 2 * kVBytes;
    static constexpr int kOffQ = kOffOut + 8 * kOutWarp;
    static constexpr int kOffMisc = kOffQ + 2 * kQTile;
    static constexpr int kSmemBytes = kOffMisc + kMisc;
    static constexpr int kPagesPerTile = kKeys / kPage;
    // The reference stands this far (in log2 units) below the score that sets it: 0 for bf16, whose precision is the same
    // at any size.  f16 rounds by a fixed 2^-25 below 2^-14: with probabilities of 2^8 for the row's largest scores
    // that is 2^-33 of its sum or less, instead of 2^-25, which a key far above many others made their whole weight.
    static constexpr float kAbove = FP8 ? 8.f : 0.f;
    // The sum of 64 probabilities (relative to the reference) up to which they are as good as with the maximum for
    // reference: f16 ends at 65504.
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
    static constexpr int kBarPieceFull = (kAbort + 4 + 7) / 8 * 8; // [kRing]
    static constexpr int kBarPieceEmpty = kBarPieceFull + 8 * kRing;
    static constexpr int kPieces = (kBarPieceEmpty + 8 * kRing + 15) / 16 * 16;   // Piece[kRing]
    static constexpr int kReaders = FP8 ? 15 : 11;                 // warps that read the pieces
    static_assert(kPieces + kRing * 64 <= kMisc, "misc area");
    static_assert(kSlots >= 3 && (!FP8 || kSlots % 2 == 0) && kSmemBytes <= kMaxSmem && kOffQ % 1024 == 0, "shared memory");
};

// TMEM map (columns)
constexpr int kColS = 0, kColO = 256;                // S_A, S_B, then O_A, O_B, 128 each

// ------------------------------------------------------------------ the work and its division
// A row tile is `tpb` query tokens times `gb` heads of the group (nsub tiles per token when the group has more than 128);
// a unit is two neighbouring row tiles of one (sequence, KV head), A and B, over all keys that its tokens see: the sinks'
// pages and the pages from the first row that its first token's window holds, numbered without the pages between (`gap` of
// them), so that a key tile is eight pages that some row needs and the sinks share theirs with the window's first pages.
// A unit costs its keys plus a fixed part: the cost rises over a prompt's first units, until the window is full.  Each CTA
// takes an equal share of the batch's cost, a contiguous run of units cut where the share ends, in the key axis too, and
// pieces of a unit that several runs share are joined by window_chunk_join_kernel.  A batch whose K and V are too large to
// stay in the L2 begins with whole units, dealt to the CTAs in turn, so that neighbours read the same window at the same
// time; what is left over is shared out.  Costs are counted in 2^shift keys, so that a batch's fits 32 bits.
constexpr double kL2Share = 60e6;                    // bytes of K and V that stay in the L2 (126 MB in two halves)
// Key tiles of a unit, on average, from which on a tile that a warp's rows all see is taken in one go instead of by halves.  That
// waits for the tensor memory and votes once, but its code beside that of the masked tiles costs units that change between
// them often.  Measured, in one go and by halves: 4096 tokens over a window of 4096 197 and 210 us (e4m3 pages 226 and 234),
// 2048 over 8192 190 and 204 (208 and 220), two prompts of 8000 over 4096, 16/2 heads, 287 and 300 (314 and 330); eight prompts
// of up to 4000 over 4096, 16 tiles on average, 147 and 147 (173 and 168), 24 of up to 2000 over 512 123 and 113 (172 and 152).
constexpr int kWideTiles = 23;

using Piece = ChunkPiece;
static_assert(sizeof(Piece) == 64, "the ring holds pieces of four 16-byte words");

// First token and head (within the group) of row tile T.
__device__ __forceinline__ void tile_origin(const WindowParams &p, int T, int &j0, int &i0)
{
    j0 = T * p.tpb;
    i0 = 0;
    if (p.nsub > 1) {
        j0 = T / p.nsub;                             // then a row tile is part of one token
        i0 = (T - j0 * p.nsub) * p.gb;
    }
}

struct WindowWalk {
    const WindowParams &p;
    const int lane, count;
    int s0;                                          // the 32 sequences that the lanes hold: what follows is lane's
    int L, q_len, tok0, units;                       // units of one head
    UnitCosts costs;                                 // of its units
    int head_cost;                                   // of one head's
    int units_to, cost_to;                           // of the lanes' sequences, all heads, up to this one's end
    int units_before, cost_done;                     // (uniform) of the sequences before s0
    int lo, hi;                                      // this CTA's run of the cost; of the units left over, a unit costs `count`
    int deal, dealt;                                 // next unit dealt, and how many units are dealt in all
    int s, h, unit;                                  // cursor of the run
    bool left_over, uncut, falls;                    // `falls`: some offset of the queries is below the one before

    __device__ __forceinline__ void load(int first)
    {
        s0 = first;
        const int at = s0 + lane;
        const int s_ = min(at, p.bs - 1);
        L = __ldg(p.seq_lens + s_);
        tok0 = __ldg(p.cu_q + s_);
        const int end = __ldg(p.cu_q + s_ + 1);
        const bool bad = tok0 < 0 || end < tok0 || end > p.num_tokens || end - tok0 > p.max_q_len || L < 0 ||
                         (long long)L > (long long)p.bt_stride * kPage;
        if (bad)
            atomicOr(p.status, SK_DEV_BAD_SEQ);
        falls |= end < tok0;
        q_len = bad ? 0 : end - tok0;
        units = at < p.bs ? ((q_len + p.tpb - 1) / p.tpb * p.nsub + 1) / 2 : 0;
        costs = unit_costs(max(0, L - q_len), p.sink_pages, kPage, p.window, p.tpb, p.slope, p.shift);
        head_cost = cost_before(units, costs, p.slope, p.shift);
        units_to = units * p.H_kv;
        cost_to = head_cost * p.H_kv;
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(kFull, units_to, o), y = __shfl_up_sync(kFull, cost_to, o);
            units_to += lane >= o ? x : 0;
            cost_to += lane >= o ? y : 0;
        }
    }
    __device__ __forceinline__ int of(int value, int src) const { return __shfl_sync(kFull, value, src); }
    // Moves on to the 32 sequences that hold unit (or cost) x; its lane.  There is one.
    __device__ __forceinline__ int seek(int x, bool by_cost)
    {
        while (true) {
            const int to = by_cost ? cost_done + cost_to : units_before + units_to;
            const uint32_t past = __ballot_sync(kFull, x < to);
            if (past != 0)
                return __ffs(past) - 1;
            units_before += of(units_to, 31);
            cost_done += of(cost_to, 31);
            load(s0 + 32);
        }
    }
    __device__ WindowWalk(const WindowParams &pp, int index, int runs, bool none)
        : p(pp), lane(threadIdx.x & 31), count(runs), units_before(0), cost_done(0), lo(0), hi(0), deal(index), dealt(0),
          s(0), h(0), unit(0), left_over(false), uncut(false), falls(false)
    {
        int total = 0, all = 0, largest = 0;
#pragma unroll 1
        for (int first = (p.bs - 1) / 32 * 32; first >= 0; first -= 32) {        // ends with the first 32
            load(first);
            total += of(cost_to, 31);
            all += of(units_to, 31);
            largest = max(largest, __reduce_max_sync(kFull, units > 0 ? cost_of(units - 1, costs, p.slope, p.shift) : 0));
        }
        // offsets that fall may give the same tokens to many sequences: more cost than the tokens come to
        if (none || (!p.bounded && __any_sync(kFull, falls)))
            return;
        const Division d = divide(total, all, largest, count, p.deal != 0, p.shift);
        uncut = d.uncut;
        if (d.deal) {
            // whole units in turn; each unit that is left over is shared by neighbours, as one of `count` parts
            dealt = all / count * count;
            left_over = true;
            lo = (all - dealt) * index;
            hi = lo + (all - dealt);
            unit = dealt + lo / count;
        } else {
            lo = min((long long)total, (long long)d.each * index);
            hi = min((long long)total, (long long)d.each * (index + 1));
        }
    }
    __device__ __forceinline__ bool next(Piece &pc)
    {
        while (true) {
            const bool whole = deal < dealt;
            if (!whole && lo >= hi)
                return false;
            const bool by_unit = whole || left_over;     // else the unit that lo lies in
            const int x = whole ? deal : by_unit ? unit : lo;
            const int src = seek(x, !by_unit);
            int start, cost = count;                     // the unit's place in the run's cost
            if (by_unit) {
                deal += whole ? count : 0;
                const int n = of(units, src), i = x - units_before - of(units_to - units * p.H_kv, src);
                pc.h = i / n;
                pc.unit = i - pc.h * n;
                start = (x - dealt) * count;
            } else {
                const int head = of(head_cost, src);
                const int in = x - cost_done - of(cost_to - head_cost * p.H_kv, src);
                pc.h = in / head;
                const int in_head = in - pc.h * head;
                const UnitCosts c{of(costs.base, src), of(costs.top, src), of(costs.rising, src)};
                auto upto = [&](int i) { return cost_before(i, c, p.slope, p.shift); };
                int left = 0, right = of(units, src) - 1, from = 0;      // `from`: upto(left)
#pragma unroll 1
                while (left < right) {
                    const int mid = (left + right + 1) >> 1, at = upto(mid);
                    if (at <= in_head) {
                        left = mid;
                        from = at;
                    } else {
                        right = mid - 1;
                    }
                }
                pc.unit = left;
                start = lo - in_head + from;
                cost = upto(left + 1) - from;
            }
            pc.s = s0 + src;
            pc.L = of(L, src);
            pc.q_len = of(q_len, src);
            pc.tok0 = of(tok0, src);
            // its two row tiles: their first tokens (the second's heads may be of the next token), what their rows see
            int j0, i0;
            tile_origin(p, 2 * pc.unit, j0, i0);
            const int j1 = p.nsub == 1 ? j0 + p.tpb : i0 + p.gb < p.nsub * p.gb ? j0 : j0 + 1;
            auto end = [&](int j) { return visible_keys(pc.L, pc.q_len, min(pc.q_len, j + p.tpb) - 1, 1); };
            pc.lo = max(0, visible_keys(pc.L, pc.q_len, j0, 1) - p.window);
            pc.hi = end(j1);
            pc.gap = max(0, pc.lo / kPage - p.sink_pages);
            auto tiles = [&](int j) { return j >= pc.q_len ? 0 : (end(j) - pc.gap * kPage + kKeys - 1) / kKeys; };
            const int tA = tiles(j0), tB = tiles(j1);
            pc.t = max(tA, tB);
            pc.a = 0;
            pc.b = pc.t;
            bool mine = true;
            if (!whole) {
                pc.a = cut_tile(lo - start, cost, pc.t, uncut);
                pc.b = cut_tile(hi - start, cost, pc.t, uncut);
                mine = pc.a < pc.b || (pc.t == 0 && lo == start);      // one without keys belongs to the run that starts it
                ++unit;
                lo = start + cost;                       // the next unit
            }
            pc.nA = max(0, min(pc.b, tA) - pc.a);
            pc.nB = max(0, min(pc.b, tB) - pc.a);
            if (mine)
                return true;
        }
    }
};

// The columns [from, to) of 32, as bits.
__device__ __forceinline__ uint32_t columns(int from, int to)
{
    const uint32_t below = to >= 32 ? 0xffffffffu : to <= 0 ? 0u : (1u << to) - 1u;
    return from >= 32 ? 0u : from <= 0 ? below : below & ~((1u << from) - 1u);
}

// 32 bytes of a row.
__device__ __forceinline__ void store32(void *dst, const uint32_t *w, bool wide)
{
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4 *>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// A packed pair as two floats.
template <bool F16>
__device__ __forceinline__ void unpack16x2(uint32_t v, float &lo, float &hi)
{
    if constexpr (F16) {
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
            : "=f"(lo), "=f"(hi)
            : "r"(v));
    } else {
        lo = __uint_as_float(v << 16);
        hi = __uint_as_float(v & 0xFFFF0000u);
    }
}

template <bool FP8, bool WIDE>
__global__ void __launch_bounds__(CCfg<FP8, WIDE>::kThreads, 1)
window_chunk_kernel(const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ CUtensorMap q_map,
                    const __grid_constant__ CUtensorMap out_map, const WindowParams p)
{
    using C = CCfg<FP8, WIDE>;
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
        ok = __all_sync(kFull, wait_short(bar_piece(i), (read / kRing) & 1, abort_flag, p.wait_limit));
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
                const int page_end = (pc.hi + kPage - 1) / kPage;      // the next page may be another's
                const int32_t *bt = p.block_table + (long long)pc.s * p.bt_stride;
                auto page_at = [&](int t) {
                    const int pg = t * C::kPagesPerTile + lane;
                    return pg >= p.sink_pages ? pg + pc.gap : pg;
                };
                auto block_at = [&](int t) {
                    const int pg = page_at(t);
                    return (lane < C::kPagesPerTile && t < pc.b && pg < page_end) ? __ldg(bt + pg) : -1;
                };
                int blk = block_at(pc.a), blk1 = block_at(pc.a + 1);
                for (int t = pc.a; t < pc.b && ok; ++t) {
                    const int blk2 = block_at(t + 2);
#pragma unroll 1
                    for (int part = 0; part < 2; ++part, ++u) {
                        const int i = u % C::kSlots;
                        if (u >= C::kSlots)
                            ok = wait_short(bar_empty(i), (u / C::kSlots - 1) & 1, abort_flag, p.wait_limit);
                        ok = __all_sync(kFull, ok);
                        if (!ok)
                            break;
                        if (lane == 0)
                            mbar_arrive_expect_tx(bar_full(i), C::kSlotBytes);
                        __syncwarp();
                        if (lane < C::kPagesPerTile) {
                            int grp = -2;            // whole box out of bounds: zero fill
                            if (page_at(t) < page_end) {
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
                wait_short(bar_full(t % C::kSlots), (t / C::kSlots) & 1, nullptr, kDrainLimit);
        } else if (warp == 3) {
            // ============================================================ the pieces, and their Q tiles
            WindowWalk walk(p, blockIdx.x, gridDim.x, !aligned);
            Piece *shared = p.units + 2 * blockIdx.x;   // this run's pieces of units that others have a part of
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
                    ok = wait_short(bar_piece_free(k % kRing), (k / kRing - 1) & 1, abort_flag, p.wait_limit);
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
                        ok = wait_short(bar_qfree(x), (used[x] - 1) & 1, abort_flag, p.wait_limit);
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
                    wait_short(bar_q(x), (used[x] - 1) & 1, nullptr, kDrainLimit);
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
                    ok = wait_short(bar, parity, abort_flag, p.wait_limit);
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
            wait_short(bar_drain(x), 0, nullptr, kDrainLimit);
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
        const int own_j = tau / p.gb;
        // The piece at work: its key tiles (and this row tile's), and where its row's output goes: token (-1: there is none), head,
        // whether the piece is the whole unit, and whether it starts it.
        int n = 0, nx = 0, tok = -1, head = 0, first_key = 0;
        bool whole = false, starts = false;
        // Keys are numbered without the gap: the row sees those below the sinks and those from low (0 where its window reaches the
        // sinks) on below limit; all of the warp's rows those from high on below least.  V's rows [dead_lo, dead_hi) and from
        // end on are no row's of the unit.
        int limit = 0, low = 0, least = 0, high = 0, end = 0, dead_hi = 0;
        const int dead_lo = p.sinks;
        float c = 0.f;
        // Takes the next piece; false at the run's end, and (failed becomes true) when the wait gave up.
        auto take = [&]() {
            const int place = read % kRing;
            failed = !__all_sync(kFull, wait_short(bar_piece(place), (read / kRing) & 1, abort_flag, p.wait_limit));
            const volatile Piece *pc = ring + place;
            if (failed || pc->s < 0)
                return false;
            ++read;
            n = pc->b - pc->a;
            nx = x ? pc->nB : pc->nA;
            first_key = pc->a * kKeys;
            starts = pc->a == 0;
            whole = starts && pc->b == pc->t;
            const int gap = pc->gap * kPage, q_len = pc->q_len;
            end = pc->hi - gap;
            dead_hi = pc->lo > p.sinks ? pc->lo - gap : 0;
            int j, i;
            tile_origin(p, 2 * pc->unit + x, j, i);
            j += own_j;
            i += tau - own_j * p.gb;
            const bool live = own_j < p.tpb && j < q_len && i < p.G;
            const int seen = live ? visible_keys(pc->L, q_len, j, 1) : 0;
            low = seen - p.window;
            low = low > p.sinks ? low - gap : 0;
            limit = max(0, seen - gap);
            tok = live ? pc->tok0 + j : -1;
            head = pc->h * p.G + i;
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar_piece_free(place));
            least = __reduce_min_sync(kFull, live ? limit : INT_MAX);            // what padding rows hold is never used
            high = __reduce_max_sync(kFull, low);
            c = p.score_scale_log2;
            if (FP8 && live)
                c *= __ldg(p.q_scale + (long long)tok * p.H_q + head);
            return true;
        };
        float m_ref = -CUDART_INF_F;
        float2 l2 = make_float2(0.f, 0.f);
        for (bool worked = false;; worked = true) {
            // The next piece is taken before the output of the one that was worked on, while its last products run (with that
            // after the output 24 prompts over a window of 512 took 111 us, 107 so).
            const int out_n = n, out_nx = nx, out_tok = tok, out_head = head;
            const bool out_whole = whole, out_starts = starts;
            const bool more = take();
            if (failed)
                break;
            if (worked) {
                // ---- the row's output, or its partial state
                const bool live = out_tok >= 0;
                const int qrow = out_tok * p.H_q + out_head;
                // a run has at most one piece that does not start its unit, and one more that does not end it
                const int part = (2 * blockIdx.x + (out_starts ? 1 : 0)) * (2 * kRows) + x * kRows + tau;
                const float l = l2.x + l2.y;
                const float mul = !out_whole ? p.v_scale : (l == 0.f ? 0.f : p.v_scale / l);
                if (out_nx > 0) {
                    const bool ok = wait_short(bar_o(x), pieces & 1, abort_flag, p.wait_limit);
                    if (!__all_sync(kFull, ok)) {
                        failed = true;
                        break;
                    }
                    tc_fence_after();
                }
                // A warp whose rows all exist and see something stages 64 dimensions of them at a time, swizzled, for a copy that
                // runs beside the next unit, and loads 32 dimensions while it rounds the 32 before.  (A lane's own row, 32 bytes a
                // store, took 4400 cycles a unit and row tile, the exchange between lanes below 5200, of 25000 that a unit of
                // five key tiles took.)
                const bool blind = out_nx == 0 || l == 0.f;
                if (out_whole && p.out_heads > 0 && !__any_sync(kFull, !live || blind)) {
                    uint8_t *stage = smem + C::kOffOut + (warp - 4) * C::kOutWarp;
                    const float2 mul2 = make_float2(mul, mul);
                    float o[2][32];
                    tmem_ld32<32>(to, o[0]);
                    if (lane == 0)                                     // the copy before has read the stage
                        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        tmem_wait_ld();
                        if (k < 3)
                            tmem_ld32<32>(to + 32 * k + 32, o[(k + 1) & 1]);
                        const float *y = o[k & 1];
                        uint32_t w[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float2 z = fmul2(make_float2(y[2 * i], y[2 * i + 1]), mul2);
                            w[i] = pack_bf16x2(z.x, z.y);
                        }
                        if (k == 2) {
                            if (lane == 0)
                                asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                            __syncwarp();
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            *reinterpret_cast<uint4 *>(stage + lane * 128 + ((((k & 1) * 4 + i) ^ (lane & 7)) << 4)) =
                                make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                        if (k & 1) {
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) {
                                asm volatile(
                                    "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                                        reinterpret_cast<uint64_t>(&out_map)),
                                    "r"(32 * k - 32), "r"(out_head), "r"(out_tok), "r"(smem_u32(stage))
                                    : "memory");
                                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                            }
                        }
                    }
                } else {
#pragma unroll 1
                    for (int cc = 0; cc < 128; cc += 32) {
                        float o[32];
                        if (out_nx > 0) {
                            tmem_ld32<32>(to + cc, o);
                            tmem_wait_ld();
                        }
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            o[i] = blind ? 0.f : o[i] * mul;
                        if (!out_whole) {
                            // four dimensions of 32 rows are 512 bytes: part_o is [slot][dimension / 4][row][4]
                            float4 *dst = reinterpret_cast<float4 *>(p.part_o) +
                                          (long long)(part / (2 * kRows)) * (32 * 2 * kRows) + (cc / 4) * (2 * kRows) +
                                          (x * kRows + tau);
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                dst[i * (2 * kRows)] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                        } else if (live) {
                            uint32_t w[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                w[i] = pack_bf16x2(o[2 * i], o[2 * i + 1]);
                            uint16_t *dst = p.out + (long long)qrow * kHeadDim + cc;
                            store32(dst, w, p.wide);
                            store32(dst + 16, w + 8, p.wide);
                        }
                        __syncwarp();
                    }
                }
                if (live) {
                    if (!out_whole) {
                        p.part_m[part] = m_ref;
                        p.part_l[part] = l;
                    } else if (p.lse != nullptr) {
                        p.lse[qrow] = l == 0.f ? -CUDART_INF_F : m_ref * 0.69314718055994531f + logf(l);
                    }
                }
                // the next piece's first product into O waits for its P, which this thread writes after these reads
                tc_fence_before();
                mine += out_nx;
                pieces += out_nx > 0 ? 1 : 0;
                u += 2 * out_n;
            }
            if (!more)
                break;
            const float2 c2 = make_float2(c, c);
            m_ref = -CUDART_INF_F;
            bool anchored = false;                                     // every row that sees a key has a reference
            l2 = make_float2(0.f, 0.f);
            for (int j = 0; j < nx; ++j) {
                const int key0 = first_key + j * kKeys;
                bool ok = wait_short(bar_s(x), (mine + j) & 1, abort_flag, p.wait_limit);
                ok = __all_sync(kFull, ok);
                if (!ok) {
                    failed = true;
                    break;
                }
                tc_fence_after();
                // page rows that no row of the unit sees may hold anything, and 0 * NaN would reach O: their V becomes zeros,
                // before either row tile multiplies it (the fence is below, when the stores are long done)
                bool zeroed = false;
                if constexpr (!FP8) {
                    const int tok = key0 + tau;
                    const bool dead = (tok >= end && tok < (end + kPage - 1) / kPage * kPage) || (tok >= dead_lo && tok < dead_hi);
                    zeroed = __any_sync(kFull, dead);
                    if (zeroed) {
                        const int i = u + 2 * j + 1;
                        ok = __all_sync(kFull, wait_short(bar_full(i % C::kSlots), (i / C::kSlots) & 1, abort_flag,
                                                          p.wait_limit));
                        if (!ok) {
                            failed = true;
                            break;
                        }
                        uint8_t *row = smem + i % C::kSlots * C::kSlotBytes + (tau >> 3) * C::kGroupBytes + (tau & 7) * 128;
                        if (dead) {
#pragma unroll 4
                            for (int cc = 0; cc < 16; ++cc)
                                *reinterpret_cast<uint4 *>(row + (cc >> 3) * 1024 + (cc & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                        }
                        __syncwarp();
                    }
                }
                // Scores, probabilities, their sum; P goes over the first columns of each half of S.  A row's reference need not
                // follow its maximum while the probabilities stay well inside their type's range, and their sum shows whether some
                // did not: then the reference moves by whole powers of two, so that what the row has summed and stored is rescaled
                // exactly.
                auto scale_o = [&](float alpha) {
#pragma unroll 1
                    for (int cc = 0; j > 0 && cc < 128; cc += 32) {        // O holds something
                        float o[32];
                        tmem_ld32<32>(to + cc, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            o[i] *= alpha;
                        tmem_st32<32>(to + cc, o);
                    }
                };
                if (WIDE && anchored && key0 + kKeys <= least && !(key0 < high && key0 + kKeys > p.sinks)) {
                    float v[128];
#pragma unroll
                    for (int cc = 0; cc < 128; cc += 32)
                        tmem_ld32<32>(ts + cc, v + cc);
                    tmem_wait_ld();
                    float2 h2;
#pragma unroll 1
                    for (int again = 0; again < 2; ++again) {
                        const float2 s2 = make_float2(-m_ref, -m_ref);
                        float2 g2 = make_float2(0.f, 0.f);
                        h2 = g2;
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
                        const bool over = limit > 0 && !(h2.x + h2.y <= C::kSumMost);
                        if (again || !__any_sync(kFull, over))
                            break;
                        float mx = fmax3(v[0], v[1], v[2]), my = v[3];
#pragma unroll
                        for (int i = 4; i < 128; i += 4) {
                            mx = fmax3(mx, v[i], v[i + 1]);
                            my = fmax3(my, v[i + 2], v[i + 3]);
                        }
                        const float by = over ? fmaxf(0.f, ceilf(fmaxf(mx, my) * c - C::kAbove - m_ref)) : 0.f;
                        const float alpha = by < 126.f ? __int_as_float((127 - (int)by) << 23) : 0.f;
                        m_ref += by;
                        l2.x *= alpha;
                        l2.y *= alpha;
                        tmem_wait_st();
                        scale_o(alpha);
                        tmem_wait_st();
                    }
                    l2 = fadd2(l2, h2);
                } else {
                    // half of the columns after the other
#pragma unroll 1
                    for (int half = 0; half < 2; ++half) {
                        const int k0 = key0 + 64 * half;
                        const uint32_t tp = ts + half * 64;
                        float v[64];
                        tmem_ld32<32>(tp, v);
                        tmem_ld32<32>(tp + 32, v + 32);
                        bool sees = true;
                        // uniform: some row does not see all of them
                        const bool masked = k0 + 64 > least || (k0 < high && k0 + 64 > p.sinks);
                        tmem_wait_ld();
                        if (masked) {
                            const int from = low - k0, to_ = limit - k0, sk = min(p.sinks, limit) - k0;
                            const uint32_t m0 = columns(from, to_) | columns(0, sk),
                                           m1 = columns(from - 32, to_ - 32) | columns(0, sk - 32);
                            sees = (m0 | m1) != 0;
                            if (!__any_sync(kFull, sees)) {
                                const uint32_t none[16] = {};
                                tmem_st32_u<16>(tp, none);
                                tmem_st32_u<16>(tp + 16, none);
                                continue;
                            }
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                v[i] = m0 & (1u << i) ? v[i] : -CUDART_INF_F;
                                v[32 + i] = m1 & (1u << i) ? v[32 + i] : -CUDART_INF_F;
                            }
                        }
                        auto largest = [&]() {
                            float mx = fmax3(v[0], v[1], v[2]), my = v[3];
#pragma unroll
                            for (int i = 4; i < 64; i += 4) {
                                mx = fmax3(mx, v[i], v[i + 1]);
                                my = fmax3(my, v[i + 2], v[i + 3]);
                            }
                            return fmaxf(mx, my) * c;
                        };
                        // a row's first scores give it a reference
                        if (!anchored && __any_sync(kFull, sees && m_ref == -CUDART_INF_F)) {
                            const float top = largest() - C::kAbove;
                            m_ref = m_ref == -CUDART_INF_F ? top : m_ref;
                        }
                        float2 h2;
                        uint32_t pk[32];
#pragma unroll 1
                        for (int again = 0; again < 2; ++again) {
                            const float msub = m_ref == -CUDART_INF_F ? 0.f : m_ref;
                            const float2 s2 = make_float2(-msub, -msub);
                            float2 g2 = make_float2(0.f, 0.f);
                            h2 = g2;
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                const float2 d = ffma2(make_float2(v[2 * i], v[2 * i + 1]), c2, s2);
                                const float2 e = make_float2(ex2_ftz(d.x), ex2_ftz(d.y));
                                (i & 1 ? g2 : h2) = fadd2(i & 1 ? g2 : h2, e);
                                pk[i] = FP8 ? pack_f16x2(e.x, e.y) : pack_bf16x2(e.x, e.y);
                            }
                            h2 = fadd2(h2, g2);
                            const bool over = limit > 0 && !(h2.x + h2.y <= C::kSumMost);
                            if (again || !__any_sync(kFull, over))
                                break;
                            // up by `by`, to kAbove below the largest score or just above it
                            const float by = over ? fmaxf(0.f, ceilf(largest() - C::kAbove - m_ref)) : 0.f;
                            const float alpha = by < 126.f ? __int_as_float((127 - (int)by) << 23) : 0.f;
                            m_ref += by;
                            l2.x *= alpha;
                            l2.y *= alpha;
                            tmem_wait_st();
#pragma unroll 1
                            for (int cc = 0; half > 0 && cc < 32; cc += 16) {      // the tile's probabilities so far
                                float w[16];
                                tmem_ld32<16>(ts + cc, w);
                                tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    float a, b;
                                    unpack16x2<FP8>(__float_as_uint(w[i]), a, b);
                                    w[i] = __uint_as_float(FP8 ? pack_f16x2(a * alpha, b * alpha)
                                                               : pack_bf16x2(a * alpha, b * alpha));
                                }
                                tmem_st32<16>(ts + cc, w);
                            }
                            scale_o(alpha);
                            tmem_wait_st();
                        }
                        tmem_st32_u<16>(tp, pk);
                        tmem_st32_u<16>(tp + 16, pk + 16);
                        l2 = fadd2(l2, h2);
                    }
                }
                if (!anchored)
                    anchored = !__any_sync(kFull, m_ref == -CUDART_INF_F && limit > 0);
                tmem_wait_st();
                if (zeroed)
                    fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar_p(x));
            }
            if (failed)
                break;
        }
        if (lane == 0)                                             // (its own copies: nothing is left in flight)
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        if (failed) {
            *abort_flag = 1;
            if (lane == 0)
                atomicOr(p.status, SK_DEV_TIMEOUT);
        }
    } else {
        // ================================================================ e4m3: V codes to f16 (exact)
        reg_dec<C::kRegsConvert>();
        const int w = warp - 12;
        // A warp has 32 tokens of a tile, in eight loads of four tokens' 128 codes, 16 a lane; all are under way before the
        // first is converted.  Token t's unit u lies at u ^ (t % 8) in its row.  The 16 dimensions become units 2 u and 2 u + 1
        // of f16, the upper half of the lanes storing the odd one first, so that a store's lanes meet no bank twice.
        const int u = lane & 7, sub = lane >> 3, first = (2 * u & 7) + (u >> 2);
        int from[2], to[2][2];                                     // of the tokens with t % 8 = sub and 4 + sub
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int x8 = 4 * e + sub;
            from[e] = w * 4 * 1024 + x8 * 128 + ((u ^ x8) << 4);
            to[e][0] = C::kOffV + w * 4 * 2048 + (u >> 2) * 1024 + x8 * 128 + ((first ^ x8) << 4);
            to[e][1] = C::kOffV + w * 4 * 2048 + (u >> 2) * 1024 + x8 * 128 + ((first ^ 1 ^ x8) << 4);
        }
        int v = 0;                                                 // key tiles so far
        bool ok = true;
        while (ok && next_piece(pc, ok)) {
            // rows that no row of the unit sees, as above
            const int end = pc.hi - pc.gap * kPage, dead_hi = pc.lo > p.sinks ? pc.lo - pc.gap * kPage : 0;
            for (int tile = pc.a; tile < pc.b; ++tile, ++v) {
                const int slot = (2 * v + 1) % C::kSlots, vb = v & 1;
                ok = wait_short(bar_full(slot), ((2 * v + 1) / C::kSlots) & 1, abort_flag, p.wait_limit);
                if (ok && v >= 2)
                    ok = wait_short(bar_vempty(vb), ((v >> 1) - 1) & 1, abort_flag, p.wait_limit);
                ok = __all_sync(kFull, ok);
                if (!ok)
                    break;
                const uint8_t *src = smem + slot * C::kSlotBytes;
                uint8_t *dst = smem + vb * C::kVBytes;
                // rows that no token sees may hold anything
                const bool dead = (tile + 1) * kKeys > end || (tile * kKeys < dead_hi && (tile + 1) * kKeys > p.sinks);
#pragma unroll
                for (int k0 = 0; k0 < 8; k0 += C::kLoads) {
                    uint4 a[C::kLoads];
#pragma unroll
                    for (int k = 0; k < C::kLoads; ++k)
                        a[k] = *reinterpret_cast<const uint4 *>(src + from[k & 1] + (k0 + k >> 1) * 1024);
                    if (dead) {
#pragma unroll
                        for (int k = 0; k < C::kLoads; ++k) {
                            const int vk = tile * kKeys + w * 32 + (k0 + k) * 4 + sub;
                            if (vk >= end || (vk >= p.sinks && vk < dead_hi))
                                a[k] = make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < C::kLoads; ++k) {
                        const uint4 lo = make_uint4(f16x2_of_e4m3(a[k].x), f16x2_of_e4m3(a[k].x >> 16),
                                                    f16x2_of_e4m3(a[k].y), f16x2_of_e4m3(a[k].y >> 16));
                        const uint4 hi = make_uint4(f16x2_of_e4m3(a[k].z), f16x2_of_e4m3(a[k].z >> 16),
                                                    f16x2_of_e4m3(a[k].w), f16x2_of_e4m3(a[k].w >> 16));
                        *reinterpret_cast<uint4 *>(dst + to[k & 1][0] + (k0 + k >> 1) * 2048) = u >> 2 ? hi : lo;
                        *reinterpret_cast<uint4 *>(dst + to[k & 1][1] + (k0 + k >> 1) * 2048) = u >> 2 ? lo : hi;
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar_vfull(vb));
                    mbar_arrive(bar_empty(slot));
                }
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

// Joins the pieces of the units that several runs share: block (run, rows) 32 rows of the unit whose last piece is that run's
// first, a lane its row, a warp 16 dimensions.  Its other pieces are the first ones of the runs before, back to the run that
// the unit starts in, whose last piece it is.  In key order, whatever the timing of the runs: with M = max m_i over the
// pieces with l_i > 0,
//     out = sum o_i 2^(m_i - M) / sum l_i 2^(m_i - M)
constexpr int kJoinThreads = 256;
constexpr int kMaxRuns = 1024;                       // runs (SMs) at most

__global__ void __launch_bounds__(kJoinThreads) window_chunk_join_kernel(const WindowParams p)
{
    __shared__ int slots[kMaxRuns], count;
    wait_prior_grid();
    const int index = blockIdx.x;
    const Piece pc = p.units[2 * index];
    if (pc.s < 0 || pc.b != pc.t)
        return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 0) {
        const int n = shared_slots(index, [&](int slot) { return p.units[slot].s >= 0; }, slots);
        if (lane == 0)
            count = n;
    }
    __syncthreads();
    const int pieces = count, row = blockIdx.y * 32 + lane;      // of the unit's 256
    int j, i;
    tile_origin(p, 2 * pc.unit + row / kRows, j, i);
    const int tau = row % kRows, jj = tau / p.gb;
    j += jj;
    i += tau - jj * p.gb;
    const bool live = jj < p.tpb && j < pc.q_len && i < p.G;
    if (!__any_sync(kFull, live))
        return;
    float M = -CUDART_INF_F, lam = 0.f;
    float4 acc[4] = {};
    constexpr int kAtOnce = 2;                       // (rarely are there more; four at once took 10.7 us for 122 units, two 7.3)
    for (int g0 = 0; g0 < pieces; g0 += kAtOnce) {
        float m[kAtOnce], l[kAtOnce];
        float4 o[kAtOnce][4];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const long long slot = slots[max(pieces - 1 - g0 - k, 0)];
            m[k] = __ldg(p.part_m + slot * (2 * kRows) + row);
            l[k] = g0 + k < pieces && live ? __ldg(p.part_l + slot * (2 * kRows) + row) : 0.f;
#pragma unroll
            for (int d = 0; d < 4; ++d)
                o[k][d] = __ldg(reinterpret_cast<const float4 *>(p.part_o) + (slot * 32 + warp * 4 + d) * (2 * kRows) + row);
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            if (l[k] == 0.f)
                continue;
            const float mn = fmaxf(M, m[k]), wa = M == -CUDART_INF_F ? 0.f : exp2f(M - mn), wb = exp2f(m[k] - mn);
            M = mn;
            lam = lam * wa + l[k] * wb;
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                acc[d].x = acc[d].x * wa + o[k][d].x * wb;
                acc[d].y = acc[d].y * wa + o[k][d].y * wb;
                acc[d].z = acc[d].z * wa + o[k][d].z * wb;
                acc[d].w = acc[d].w * wa + o[k][d].w * wb;
            }
        }
    }
    if (!live)
        return;
    const float inv = lam == 0.f ? 0.f : 1.f / lam;
    const long long qrow = (long long)(pc.tok0 + j) * p.H_q + pc.h * p.G + i;
    uint32_t w[8];
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        w[2 * d] = pack_bf16x2(acc[d].x * inv, acc[d].y * inv);
        w[2 * d + 1] = pack_bf16x2(acc[d].z * inv, acc[d].w * inv);
    }
    store32(p.out + qrow * kHeadDim + warp * 16, w, p.wide);
    if (warp == 0 && p.lse != nullptr)
        p.lse[qrow] = lam == 0.f ? -CUDART_INF_F : M * 0.69314718055994531f + logf(lam);
}

template <bool FP8, bool WIDE>
cudaError_t launch_t(const CUtensorMap &kv_map, const CUtensorMap &q_map, const CUtensorMap &out_map, const WindowParams &p,
                     int runs, cudaStream_t stream)
{
    using C = CCfg<FP8, WIDE>;
    const auto kernel = window_chunk_kernel<FP8, WIDE>;
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess)
        return e;
    // the warpgroups' shares after the reallocation may not exceed what the CTA was launched with
    static PerDevice registers;
    if (registers.get(device, [&] { return kernel_registers(kernel); }) < C::kRegsLaunch)
        return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(kernel, dim3((unsigned)runs), dim3(C::kThreads), C::kSmemBytes, stream,
                      kv_map, q_map, out_map, p);
}

}  // namespace

// Bytes of the workspace: two pieces of 256 rows (o, m, l) per run with what they are pieces of, and for e4m3 pages Q in
// two terms.
long long window_chunk_workspace_bytes(int num_tokens, int H_q, int kv_dtype, int num_sms)
{
    const long long parts = 2LL * num_sms * (2 * kRows * (kHeadDim + 2) * 4 + (long long)sizeof(ChunkPiece));
    return parts + (kv_dtype == SK_KV_FP8_E4M3 ? (long long)num_tokens * H_q * (2 * kHeadDim + 4) : 0);
}

cudaError_t launch_window_chunk(const WindowParams &params, int kv_dtype, long long max_seq_len, void *workspace, int num_sms,
                                cudaStream_t stream)
{
    const bool fp8 = kv_dtype == SK_KV_FP8_E4M3;
    WindowParams p = params;
    const ChunkShape shape = chunk_shape(p.G);
    p.gb = shape.gb;
    p.nsub = shape.nsub;
    p.tpb = shape.tpb;
    p.slope = shape.slope;
    const long long slots = 2LL * num_sms * 2 * kRows;
    p.part_o = static_cast<float *>(workspace);
    p.part_m = p.part_o + slots * kHeadDim;
    p.part_l = p.part_m + slots;
    p.units = reinterpret_cast<ChunkPiece *>(p.part_l + slots);
    p.wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
    const void *q = p.q;
    if (fp8) {
        uint8_t *codes = reinterpret_cast<uint8_t *>(p.units + 2 * num_sms);
        const long long rows = (long long)p.num_tokens * p.H_q;
        const cudaError_t e = launch_split_q(p.q, rows, codes, stream);
        if (e != cudaSuccess)
            return e;
        q = codes;
        p.q_scale = reinterpret_cast<const float *>(codes + rows * 256);
    }
    CUtensorMap kv_map, q_map, out_map{};
    // one box of the pages: K (or V) of one page and head
    cudaError_t e = encode_page_map(&kv_map, p.kv, p.num_blocks, p.H_kv, fp8, fp8 ? 1 : 2);
    if (e == cudaSuccess)
        e = encode_q_map(&q_map, q, p.num_tokens, p.H_q, fp8, p.gb, p.tpb);
    // a softmax warp's 32 rows are a box of the output where heads and tokens fill it
    if (e == cudaSuccess && (p.gb % 32 == 0 || 32 % p.gb == 0)) {
        p.out_heads = p.gb < 32 ? p.gb : 32;
        e = encode_q_map(&out_map, p.out, p.num_tokens, p.H_q, false, p.out_heads, 32 / p.out_heads);
    }
    if (e != cudaSuccess)
        return e;
    // A run per SM, but none of less than two key tiles on average: the number of units is bounded by the tokens, and that
    // of their key tiles by what a unit sees at most.
    const long long per_seq = ((long long)(p.max_q_len + p.tpb - 1) / p.tpb * p.nsub + 1) / 2 * p.bs;
    const long long by_tokens = ((long long)(p.num_tokens + p.tpb - 1) / p.tpb * p.nsub + 1) / 2 + p.bs;
    const long long units = (per_seq < by_tokens ? per_seq : by_tokens) * p.H_kv;
    p.sink_pages = (p.sinks + kPage - 1) / kPage;
    const long long most = (long long)p.sink_pages * kPage + p.window + 2 * p.tpb;
    const long long keys = max_seq_len < most ? max_seq_len : most;
    const long long tiles = (keys + kKeys - 1) / kKeys;
    long long runs = units * (tiles < 2 ? 1 : tiles / 2);
    runs = runs < 1 ? 1 : (runs < num_sms ? runs : num_sms);
    runs = runs < kMaxRuns ? runs : kMaxRuns;
    p.shift = cost_shift(units, most);
    p.bounded = (double)per_seq * p.H_kv * (kChunkFixed + kChunkEdge + (double)most) < (double)(1 << 30);
    p.deal = (double)p.bs * keys * p.H_kv * (fp8 ? 256 : 512) > kL2Share ? 1 : 0;
    // (a prompt's first units see less: on average keys / 2 less over its first `keys` tokens)
    const bool wide = keys > 0 && keys * (1. - 0.5 * keys / max_seq_len) >= kWideTiles * (double)kKeys;
    auto launch = fp8 ? (wide ? launch_t<true, true> : launch_t<true, false>)
                      : (wide ? launch_t<false, true> : launch_t<false, false>);
    e = launch(kv_map, q_map, out_map, p, (int)runs, stream);
    if (e != cudaSuccess || runs == 1)
        return e;
    return launch_pdl(window_chunk_join_kernel, dim3((unsigned)runs, 2 * kRows / 32), dim3(kJoinThreads), 0, stream, p);
}

}  // namespace sk
