// Attention with a sliding window and sinks for decode and verify steps: up to 64 rows (query tokens times heads of a group)
// of a (sequence, KV head) over the pages of its sinks and its window, on the tcgen05 tensor cores.
//
// For the rows r = j * G + i (query token j, head i of the group), with P = L - q + j the token's own row:
//     S = scale Q K^T over the keys p <= P with p < sinks or p > P - window,   O = softmax(S) V,   lse = log sum exp S
//
// Bound by HBM: 512 bytes of K and V (256 for e4m3 pages) per key, once.  A window bounds what a unit, one (sequence, KV
// head), can cost, so that no plan of segments is needed.  The batch's key tiles (128 keys: eight pages, the sinks' first,
// then those from the page with the first row that the window of the first token holds) stand in one line, unit after unit,
// and each CTA, one per SM, takes an equal run of it.  Inside its run a CTA goes from unit to unit without a pause; what
// several runs have of a unit is joined by a second kernel.  A batch of few units is divided otherwise: a unit has a
// cluster of CTAs, as many as fit, which share its key tiles and join their states through shared memory.
//
// The products take the keys as M, so that nothing but the padding of the rows to 16, 32 or 64 is wasted:
//     S^T[128 keys x R] = K Q^T,   O^T[128 dimensions x R] += V^T P^T
//
// Roles (384 threads; 512 for e4m3 pages):
//   warp 0      walks the run, publishes its pieces to the others and copies their pages: one TMA copy per page (8 KB, e4m3
//               4 KB) into 128-byte-swizzled atoms that are the operands K and V^T
//   warp 1      issues QK (and allocates TMEM), warp 2 PV
//   warp 3      bf16: copies Q
//   warps 4-7, 8-11  softmax of the even and of the odd key tiles, each group with its own O, reference and sums: a group
//               has the time of two tiles for one, and the groups meet only at a unit's end, where their states are joined.
//               A thread is a key (its TMEM lane).  A row's reference is its largest score of the group's first tile;
//               it moves only when a later score beats it by far, on which the group's threads vote once per tile.
//               P^T goes over the tile's own K, which QK no longer needs.  It is rounded to V's type, bf16, as the product
//               takes both of one (f16 on e4m3 pages); its sum is not.  The output is then off from 64 bits by 0.0023 of its
//               size, where rounding the output alone is 0.0016 (f16: 0.0017).
//   warps 12-15 (e4m3)  Q as two e4m3 terms, and V's codes to f16 (exactly): PV runs on f16 with P as f16
// e4m3 pages: QK runs on the codes, with Q as two e4m3 terms and a power-of-two scale per row, two products into one S.
//
// Every wait is bounded; on expiry SK_DEV_TIMEOUT is set and every role gives up, after its copies and products in flight.
//
// Measured (calls replayed from a graph): 128 tokens over a window of 4096, 32/8 heads, 2150 MB: 312 us, 6.9 TB/s (e4m3 pages
// 209 us, 5.1: a copy of a page costs the SM's copy unit 130 cycles and 3.3 for each 128 bytes, whatever else it does).  64 ragged
// ones over 1024, 269 MB: 53 us, of which the join is 4 and the pages stream at 6.8 TB/s.  One token over 4096, 17 MB: 10.5 us;
// 16 times 4 tokens over 4096 on e4m3 pages with 2 KV heads, 35 MB: 20.4 us.  These two are a chain: launch, block ids, pages,
// products and softmax of few tiles, end, join, on code that is fetched as it is first run.
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
constexpr int kKeys = 128;                           // keys of a tile (MMA M)
constexpr int kPagesPerTile = kKeys / kPage;
constexpr uint32_t kDrainLimit = 4000000000u;        // cycles (~2 s): waits for work already issued
constexpr int kMaxSmem = 232448;
constexpr int kRing = 8;                             // pieces published ahead
constexpr int kUnitFixed = 1;                        // cost of starting and finishing a unit, in key tiles
template <int RP, bool FP8>
struct WCfg {
    static_assert(RP == 16 || RP == 32 || RP == 64, "rows: 16, 32 or 64");
    static constexpr int kThreads = FP8 ? 512 : 384;
    // registers per thread after the reallocation; no more in all than at launch (4 x 128, or 3 x 168)
    static constexpr int kRegsLaunch = FP8 ? 128 : 168;
    static constexpr int kRegsIssue = FP8 ? 56 : 72, kRegsSoftmax = !FP8 ? 216 : RP == 64 ? 192 : 176,
                         kRegsConvert = RP == 64 ? 72 : 104;
    static_assert(kRegsIssue + 2 * kRegsSoftmax + (FP8 ? kRegsConvert : 0) <= kThreads / 128 * kRegsLaunch, "registers");
    static constexpr int kGroupBytes = FP8 ? 2048 : 4096;          // 8 tokens as copied: 128-byte chunks of K, then of V
    static constexpr int kPageBytes = 2 * kGroupBytes;
    static constexpr int kOffV = FP8 ? 1024 : 2048;                // V's first chunk in a group
    static constexpr int kStageBytes = kKeys / 8 * kGroupBytes;
    static constexpr int kQBytes = RP * 256;                       // bf16: two 64-dimension chunks; e4m3: hi and lo
    static constexpr int kV16Bytes = FP8 ? kKeys * 256 : 0;        // e4m3: V of a tile as f16, two of them
    static constexpr int kMisc = 3072;
    static constexpr int kStages = (kMaxSmem - 2 * kQBytes - 2 * kV16Bytes - kMisc) / kStageBytes;
    static constexpr int kOffV16 = kStages * kStageBytes;
    static constexpr int kOffQ = kOffV16 + 2 * kV16Bytes;
    static constexpr int kOffSums = kOffQ + 64 * RP;               // a cluster's part: float[2][RP], past the unit's-end scratch
    static constexpr int kOffMisc = kOffQ + 2 * kQBytes;
    static constexpr int kSmemBytes = kOffMisc + kMisc;
    // TMEM columns: S buffers (even and odd tiles in turn), then O of the even and of the odd tiles
    static constexpr int kSBufs = 4;
    static constexpr int kColO = kSBufs * RP;
    static constexpr int kTmemNeed = kColO + 2 * RP;
    static constexpr int kTmemCols = kTmemNeed <= 128 ? 128 : kTmemNeed <= 256 ? 256 : 512;
    static_assert(kTmemNeed <= 512, "TMEM columns");
    // The reference stands this far (log2 units) below the score that sets it, and moves when a score is kMost above it.
    // bf16 is as precise at any size.  f16 ends at 2^16 and rounds by a fixed 2^-25 below 2^-14: with 2^8 or more for a row's
    // largest score that is 2^-33 of its sum.
    static constexpr float kAbove = FP8 ? 8.f : 0.f;
    static constexpr float kMost = FP8 ? 15.f : 40.f;
    // misc area
    static constexpr int kBarFull = 0;                             // [kStages]
    static constexpr int kBarEmpty = kBarFull + 8 * kStages;       // [kStages]
    static constexpr int kBarP = kBarEmpty + 8 * kStages;          // [kStages] P written
    static constexpr int kBarS = kBarP + 8 * kStages;              // [kSBufs] S complete
    static constexpr int kBarSFree = kBarS + 8 * kSBufs;           // [kSBufs]
    static constexpr int kBarQ = kBarSFree + 8 * kSBufs;           // [2] Q written
    static constexpr int kBarQFree = kBarQ + 16;                   // [2] its last product complete, its memory not used
    static constexpr int kBarV = kBarQFree + 16;                   // [2] e4m3: V of a tile as f16
    static constexpr int kBarVFree = kBarV + 16;                   // [2]
    static constexpr int kBarO = kBarVFree + 16;                   // a piece's last PV complete
    static constexpr int kBarOFree = kBarO + 8;                    // O read
    static constexpr int kBarDrain = kBarOFree + 8;                // [2]
    static constexpr int kBarPiece = kBarDrain + 16;               // [kRing]
    static constexpr int kBarPieceFree = kBarPiece + 8 * kRing;    // [kRing]
    static constexpr int kTmemSlot = kBarPieceFree + 8 * kRing;
    static constexpr int kAbort = kTmemSlot + 4;
    static constexpr int kFound = (kAbort + 4 + 7) / 8 * 8;        // where the run starts
    static constexpr int kPieces = (kFound + 16 + 15) / 16 * 16;   // WindowPiece[kRing]
    static constexpr int kUnit = kPieces + 48 * kRing;             // WindowPiece: the cluster's unit
    static constexpr int kNeg = kUnit + 48;                  // float[2][RP] minus the reference of a group's rows (log2)
    static constexpr int kDelta = kNeg + 8 * RP;                   // float[2][RP] what it changes by
    static constexpr int kAlpha = kDelta + 8 * RP;                 // float[2][RP] 2^delta; float2[2][RP / 2] at a unit's end
    static constexpr int kScale = kAlpha + 8 * RP;                 // float[2][RP] e4m3: score scale of a Q buffer's rows
    static_assert(kScale + (FP8 ? 8 * RP : 0) <= kMisc, "misc area");
    static constexpr int kReaders = FP8 ? 14 : 11;                 // warps that read the pieces
    static_assert(kStages >= 3 && kSmemBytes <= kMaxSmem && kOffQ % 1024 == 0, "shared memory");
};

// ------------------------------------------------------------------ the work and its division
struct Seq {
    int L, q_len, tok0, gap, t;                      // gap: pages between the sinks and the window; t: key tiles
};

__device__ __forceinline__ Seq sequence(const WindowParams &p, int s)
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
    const int lo = max(0, q.L - q.q_len + 1 - p.window);           // the first row of the first token's window
    q.gap = max(0, min(lo, q.L) / kPage - p.sink_pages);
    q.t = bad ? 0 : (q.L - q.gap * kPage + kKeys - 1) / kKeys;
    return q;
}

using Piece = WindowPiece;
static_assert(sizeof(Piece) == 48, "the ring holds pieces of three 16-byte words");

// Sum (or maximum) of each of N values across the 32 lanes: lane l ends with that of value l / (32 / N) in v[0].
template <int N, int OFF, bool MAX>
__device__ __forceinline__ void reduce_step(float *v, int lane)
{
    if constexpr (N >= 2) {
        const bool upper = (lane & OFF) != 0;
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float send = upper ? v[i] : v[i + N / 2], keep = upper ? v[i + N / 2] : v[i];
            const float got = __shfl_xor_sync(kFull, send, OFF);
            v[i] = MAX ? fmaxf(keep, got) : keep + got;
        }
        if constexpr (OFF > 1)
            reduce_step<N / 2, OFF / 2, MAX>(v, lane);
    } else {
        const float got = __shfl_xor_sync(kFull, v[0], OFF);
        v[0] = MAX ? fmaxf(v[0], got) : v[0] + got;
        if constexpr (OFF > 1)
            reduce_step<1, OFF / 2, MAX>(v, lane);
    }
}

// min(a / b, most) for a >= 0, b > 0 and most < 2^24 (a division of 64 bits takes a thousand cycles).
__device__ __forceinline__ int quotient(long long a, long long b, int most)
{
    if (a >= b * most)
        return most;
    int x = (int)__fdividef((float)a, (float)b);     // within 2^-22 of the quotient, which is below 2^24
    while (x * b > a)
        --x;
    while ((x + 1) * b <= a)
        ++x;
    return x;
}

// Row r of a unit among the rows of q: the token's, times H_q, and the head.
__device__ __forceinline__ long long unit_row(const WindowParams &p, const Piece &pc, int r)
{
    const int j = r * p.inv_G >> 16;                 // r / G
    return (long long)(pc.tok0 + j) * p.H_q + pc.h * p.G + (r - j * p.G);
}

// The run of CTA `index` of `count` for a batch of at most 32 sequences and a cost below 2^31; called by a warp.  (The whole
// CTA's search, with its barriers before the first copy, takes 0.4 us longer for 40 sequences, and 0.6 less for 100 than a
// warp's, 32 at a time.)
__device__ __forceinline__ Run small_run(const WindowParams &p, int index, int count)
{
    const int lane = threadIdx.x & 31;
    const Seq q = sequence(p, min(lane, p.bs - 1));
    const int mine = lane < p.bs && q.q_len > 0 ? p.H_kv * (q.t + kUnitFixed) : 0;
    int upto = mine;                                 // of the sequences up to this lane's
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(kFull, upto, o);
        upto += lane >= o ? x : 0;
    }
    const int total = __shfl_sync(kFull, upto, 31), each = (total + count - 1) / count;
    Run r;
    r.lo = min((long long)total, (long long)each * index);
    r.hi = min((long long)total, (long long)each * (index + 1));
    const uint32_t past = __ballot_sync(kFull, r.lo < upto);
    const int src = past ? __ffs(past) - 1 : 0;      // the sequence that lo lies in
    r.s = past ? src : p.bs;
    r.before = __shfl_sync(kFull, upto - mine, src);
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Shared memory of CTA `rank` of the cluster at the address that `local` has in this one.
__device__ __forceinline__ uint32_t of_rank(uint32_t local, int rank)
{
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(local), "r"(rank));
    return a;
}

template <int RP, bool FP8>
__global__ void __launch_bounds__(WCfg<RP, FP8>::kThreads, 1)
window_step_kernel(const __grid_constant__ CUtensorMap kv_map, const WindowParams p)
{
    using C = WCfg<RP, FP8>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t sbase = smem_u32(smem);
    uint8_t *misc = smem + C::kOffMisc;
    const uint32_t mbase = sbase + C::kOffMisc;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(misc + C::kAbort);
    auto bar = [&](int at, int i) { return mbase + at + 8 * i; };
    Piece *ring = reinterpret_cast<Piece *>(misc + C::kPieces);

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(bar(C::kBarFull, i), 1);
            mbar_init(bar(C::kBarEmpty, i), 1);
            mbar_init(bar(C::kBarP, i), 4);
        }
        for (int i = 0; i < C::kSBufs; ++i) {
            mbar_init(bar(C::kBarS, i), 1);
            mbar_init(bar(C::kBarSFree, i), 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(C::kBarQ, i), FP8 ? 4 : 1);
            mbar_init(bar(C::kBarQFree, i), 1 + 8);
            mbar_init(bar(C::kBarV, i), 4);
            mbar_init(bar(C::kBarVFree, i), 1);
            mbar_init(bar(C::kBarDrain, i), 1);
        }
        mbar_init(bar(C::kBarO, 0), 1);
        mbar_init(bar(C::kBarOFree, 0), 8);
        for (int i = 0; i < kRing; ++i) {
            mbar_init(bar(C::kBarPiece, i), 1);
            mbar_init(bar(C::kBarPieceFree, i), C::kReaders);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(mbase + C::kTmemSlot, C::kTmemCols);
        tmem_relinquish();
    }
    wait_prior_grid();
    if (blockIdx.x == 0 && threadIdx.x == 0 && (__ldg(p.cu_q) != 0 || __ldg(p.cu_q + p.bs) != p.num_tokens))
        atomicOr(p.status, SK_DEV_BAD_SEQ);
    // A large batch's runs are found by the whole CTA, in the stages' memory, before the first copy; else warp 0 finds its own.
    Run run{0, 0, 0, p.bs};
    if (!p.small && p.split == 0)
        run = find_run<C::kThreads>(p.bs, blockIdx.x, gridDim.x, 0, 0, reinterpret_cast<long long *>(smem),
                                    reinterpret_cast<long long *>(misc + C::kFound), [&](int s) {
                                        const Seq q = sequence(p, s);
                                        return q.q_len > 0 ? (long long)p.H_kv * (q.t + kUnitFixed) : 0LL;
                                    });
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(misc + C::kTmemSlot);
    const bool aligned = (sbase & 1023u) == 0;
    if (!aligned && threadIdx.x == 0)
        atomicOr(p.status, SK_DEV_INTERNAL);
    auto wait = [&](uint32_t b, uint32_t parity) {
        return __all_sync(kFull, wait_short(b, parity, abort_flag, p.wait_limit)) != 0;
    };
    auto give_up = [&]() {
        *abort_flag = 1;
        if (lane == 0)
            atomicOr(p.status, SK_DEV_TIMEOUT);
    };
    // The next published piece; false at the end of the run, or (ok becomes false) when the wait gave up.
    int read = 0;
    auto next_piece = [&](Piece &pc, bool &ok) {
        const int i = read % kRing;
        ok = wait(bar(C::kBarPiece, i), (read / kRing) & 1);
        if (!ok)
            return false;
        pc = ring[i];
        __syncwarp();
        if (lane == 0)
            mbar_arrive(bar(C::kBarPieceFree, i));
        ++read;
        return pc.s >= 0;
    };
    Piece pc;
    bool ok = true;

    if (warp < 4) {
        reg_dec<C::kRegsIssue>();
        if (warp == 0) {
            // ============================================================ the pieces and their pages
            if (lane == 0)
                prefetch_tensormap(&kv_map);
            if (p.small && p.split == 0)
                run = small_run(p, blockIdx.x, gridDim.x);
            if (!aligned)
                run.s = p.bs;                            // nothing is done
            Piece *shared = p.shared + 2 * blockIdx.x;   // this run's pieces of units that others have a part of
            if (lane < 2 && p.split == 0)
                shared[lane].s = -1;
            __syncwarp();
            // equal shares: all runs are as long as the ones before this, or as this
            const long long share = blockIdx.x > 0 ? run.lo / blockIdx.x : run.hi;
            Seq q;
            int s = run.s, h = -1, count = 0;
            long long off = run.before;                  // where sequence s starts
            // The next piece, published; its s is -1 at the run's end (and after a wait that gave up).
            auto next = [&]() {
                bool more = false;
                if (p.split > 0 && h < 0) {              // this CTA's part of its cluster's unit, once
                    const uint32_t unit = blockIdx.x / (uint32_t)p.split, rank = blockIdx.x - unit * p.split;
                    s = unit / (uint32_t)p.H_kv;
                    h = unit - s * p.H_kv;
                    q = sequence(p, s);
                    pc.s = s;
                    pc.h = h;
                    pc.L = q.L;
                    pc.q_len = q.q_len;
                    pc.tok0 = q.tok0;
                    pc.gap = q.gap;
                    pc.t = q.q_len > 0 ? q.t : 0;
                    // the first ranks have one tile more where they do not come out even
                    const int each = (uint32_t)pc.t / (uint32_t)p.split, rest = pc.t - each * p.split;
                    pc.a = rank * each + min((int)rank, rest);
                    pc.b = pc.a + each + ((int)rank < rest ? 1 : 0);
                    if (lane == 0)
                        *reinterpret_cast<Piece *>(misc + C::kUnit) = pc;
                    more = aligned && (pc.a < pc.b || (pc.t == 0 && rank == 0 && q.q_len > 0));
                }
                while (p.split == 0 && s < p.bs && off < run.hi) {
                    if (h < 0) {
                        q = sequence(p, s);
                        h = 0;
                        if (q.q_len > 0 && run.lo > off)     // the head that the run starts in
                            h = quotient(run.lo - off, q.t + kUnitFixed, p.H_kv);
                    }
                    const int unit = q.t + kUnitFixed;
                    if (q.q_len == 0 || h >= p.H_kv) {
                        off += q.q_len > 0 ? (long long)unit * p.H_kv : 0;
                        ++s;
                        h = -1;
                        continue;
                    }
                    const long long start = off + (long long)h * unit;
                    if (start >= run.hi)
                        break;
                    // tile i stands at start + kUnitFixed + i
                    const long long first = start + kUnitFixed;
                    pc.s = s;
                    pc.h = h++;
                    pc.L = q.L;
                    pc.q_len = q.q_len;
                    pc.tok0 = q.tok0;
                    pc.gap = q.gap;
                    pc.t = q.t;
                    pc.a = (int)max(0LL, min((long long)q.t, run.lo - first));
                    pc.b = (int)max(0LL, min((long long)q.t, run.hi - first));
                    // a unit without keys belongs to the run that it starts in
                    more = pc.a < pc.b || (q.t == 0 && start >= run.lo);
                    pc.first = more && pc.a > 0 ? quotient(first, share, blockIdx.x) : blockIdx.x;
                    if (more)
                        break;
                }
                if (!more)
                    pc.s = -1;
                const int i = count % kRing;
                if (count >= kRing)
                    ok = wait(bar(C::kBarPieceFree, i), (count / kRing - 1) & 1);
                if (!ok) {
                    pc.s = -1;
                    return;
                }
                ++count;
                if (lane == 0) {
                    ring[i] = pc;
                    if (more && pc.b - pc.a < pc.t && p.split == 0)
                        shared[pc.a > 0 ? 0 : 1] = pc;
                    mbar_arrive(bar(C::kBarPiece, i));
                }
                __syncwarp();
            };
            // Block ids of four tiles of a piece, from tile t on, one page a lane.  (A tile's eight at a time, two tiles ahead,
            // each copy waited a thousand cycles for the register moves of the ids read last.)
            auto page_of = [&](const Piece &x, int v) { return v >= p.sink_pages ? v + x.gap : v; };
            auto blocks_at = [&](const Piece &x, int t) {
                const int v = t * kPagesPerTile + lane, pg = page_of(x, v);
                return v < x.b * kPagesPerTile && pg * kPage < x.L
                           ? __ldg(p.block_table + (long long)x.s * p.bt_stride + pg) : -1;
            };
            int u = 0;                                   // tiles so far
            int blocks = -1;
            pc = Piece{};                                // begins with a piece of no tiles
            while (ok && pc.s >= 0) {
                // the piece after this one is found, and its first blocks are read, once the first copies are out
                const Piece now = pc;
                const int turn = min(now.b, now.a + C::kStages);
                int after = -1, more = blocks_at(now, now.a + 4);
                for (int t = now.a; t <= now.b; ++t) {
                    if (t == turn) {
                        next();
                        if (pc.s >= 0)
                            after = blocks_at(pc, pc.a);
                    }
                    if (t == now.b)
                        break;
                    const int k = (t - now.a) & 3;
                    if (k == 0 && t > now.a) {
                        blocks = more;
                        more = blocks_at(now, t + 4);
                    }
                    const int blk = __shfl_sync(kFull, blocks, k * kPagesPerTile + (lane & (kPagesPerTile - 1)));
                    const int i = u % C::kStages;
                    if (u >= C::kStages && ok)
                        ok = wait(bar(C::kBarEmpty, i), (u / C::kStages - 1) & 1);
                    if (!ok)
                        break;
                    if (lane == 0)
                        mbar_arrive_expect_tx(bar(C::kBarFull, i), C::kStageBytes);
                    __syncwarp();
                    if (lane < kPagesPerTile) {
                        int grp = -2;                    // whole box out of bounds: zero fill
                        if (page_of(now, t * kPagesPerTile + lane) * kPage < now.L) {
                            if (blk >= 0 && blk < p.num_blocks)
                                grp = (blk * p.H_kv + now.h) * 2;
                            else
                                atomicOr(p.status, SK_DEV_BAD_BLOCK);
                        }
                        tma_load_4d(sbase + i * C::kStageBytes + lane * C::kPageBytes, &kv_map, 0, 0, 0, grp,
                                    bar(C::kBarFull, i));
                    }
                    ++u;
                }
                blocks = after;
            }
            if (!ok)
                give_up();
            // every copy issued lands before the CTA exits
            for (int t = u > C::kStages ? u - C::kStages : 0; t < u; ++t)
                wait_short(bar(C::kBarFull, t % C::kStages), (t / C::kStages) & 1, nullptr, kDrainLimit);
        } else if (warp == 3) {
            // ============================================================ bf16: Q, K-major with the 128-byte swizzle
            int copied = 0;
            while (!FP8 && ok && next_piece(pc, ok)) {
                if (pc.a == pc.b)
                    continue;
                const int buf = copied & 1;
                if (copied >= 2)
                    ok = wait(bar(C::kBarQFree, buf), ((copied >> 1) - 1) & 1);
                if (!ok)
                    break;
                ++copied;
                const int R = p.G * pc.q_len, unit = lane & 15;
#pragma unroll 4
                for (int r = lane >> 4; r < RP; r += 2) {      // two rows at a time, 16 bytes a lane; zeros past the rows
                    const uint32_t dst = sbase + C::kOffQ + buf * C::kQBytes + (unit >> 3) * (RP * 128) + r * 128 +
                                         (((unit & 7) ^ (r & 7)) << 4);
                    const int rr = min(r, R - 1);
                    const uint16_t *src = p.q + unit_row(p, pc, rr) * kHeadDim + unit * 8;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                                 "r"(r < R ? 16 : 0)
                                 : "memory");
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(C::kBarQ, buf));
            }
            if (!ok)
                give_up();
        } else if (warp == 1) {
            // ============================================================ S^T = K Q^T
            constexpr uint32_t idesc = FP8 ? idesc_e4m3_f32(kKeys, RP, 0, 0) : idesc_bf16_f32(kKeys, RP, 0, 0);
            const uint64_t d_k = smem_desc_sw128(sbase, 16, C::kGroupBytes);
            const uint64_t d_q = smem_desc_sw128(sbase + C::kOffQ, 16, 1024);
            int u = 0, pieces = 0;
            while (ok && next_piece(pc, ok)) {
                const int n = pc.b - pc.a, buf = pieces & 1;
                if (n == 0)
                    continue;
                ok = wait(bar(C::kBarQ, buf), (pieces >> 1) & 1);
                const uint64_t q0 = d_q + (uint64_t)(buf * C::kQBytes >> 4);
                for (int j = 0; j < n && ok; ++j, ++u) {
                    const int b = u % C::kSBufs, st = u % C::kStages;
                    if (u >= C::kSBufs)
                        ok = wait(bar(C::kBarSFree, b), (u / C::kSBufs - 1) & 1);
                    if (ok)
                        ok = wait(bar(C::kBarFull, st), (u / C::kStages) & 1);
                    if (!ok)
                        break;
                    tc_fence_after();
                    const uint32_t sd = tmem + b * RP;
                    const uint64_t k0 = d_k + (uint64_t)(st * C::kStageBytes >> 4);
                    if constexpr (FP8) {
                        mma4_f8_ss<2, 2>(sd, k0, q0, idesc, 0);
                        mma4_f8_ss<2, 2>(sd, k0, q0 + (RP * 128 >> 4), idesc, 1);
                    } else {
                        mma4_f16_ss<2, 2>(sd, k0, q0, idesc, 0);
                        mma4_f16_ss<2, 2>(sd, k0 + (1024 >> 4), q0 + (RP * 128 >> 4), idesc, 1);
                    }
                    mma_commit_warp(bar(C::kBarS, b));
                    if (j + 1 == n)
                        mma_commit_warp(bar(C::kBarQFree, buf));
                }
                ++pieces;
            }
            if (!ok)
                give_up();
            // every product completes before TMEM is freed and shared memory is left
            mma_commit_warp(bar(C::kBarDrain, 0));
            wait_short(bar(C::kBarDrain, 0), 0, nullptr, kDrainLimit);
        } else {
            // ============================================================ O^T += V^T P^T
            constexpr uint32_t idesc = FP8 ? idesc_f16_f32(kHeadDim, RP, 1, 1) : idesc_bf16_f32(kHeadDim, RP, 1, 1);
            constexpr int kVGroup = FP8 ? 2048 : C::kGroupBytes;
            constexpr int kStepV = 2 * kVGroup >> 4, kStepP = 2 * C::kGroupBytes >> 4;    // 16 keys
            const uint64_t d_p = smem_desc_sw128(sbase, 1024, C::kGroupBytes);
            const uint64_t d_v = smem_desc_sw128(sbase + (FP8 ? C::kOffV16 : C::kOffV), 1024, kVGroup);
            int u = 0, pieces = 0;
            while (ok && next_piece(pc, ok)) {
                const int n = pc.b - pc.a;
                if (n == 0)
                    continue;
                if (pieces > 0)                          // both O are read
                    ok = wait(bar(C::kBarOFree, 0), (pieces - 1) & 1);
                for (int j = 0; j < n && ok; ++j, ++u) {
                    const int st = u % C::kStages;
                    ok = wait(bar(C::kBarP, st), (u / C::kStages) & 1);
                    if (FP8 && ok)
                        ok = wait(bar(C::kBarV, u & 1), (u >> 1) & 1);
                    if (!ok)
                        break;
                    tc_fence_after();
                    const uint32_t od = tmem + C::kColO + (u & 1) * RP;
                    const uint64_t p0 = d_p + (uint64_t)(st * C::kStageBytes >> 4);
                    const uint64_t v0 = d_v + (uint64_t)((FP8 ? (u & 1) * C::kV16Bytes : st * C::kStageBytes) >> 4);
                    mma4_f16_ss<kStepV, kStepP>(od, v0, p0, idesc, j >= 2);
                    mma4_f16_ss<kStepV, kStepP>(od, v0 + 4 * kStepV, p0 + 4 * kStepP, idesc, 1);
                    mma_commit_warp(bar(C::kBarEmpty, st));
                    if (FP8)
                        mma_commit_warp(bar(C::kBarVFree, u & 1));
                }
                if (ok)
                    mma_commit_warp(bar(C::kBarO, 0));
                ++pieces;
            }
            if (!ok)
                give_up();
            mma_commit_warp(bar(C::kBarDrain, 1));
            wait_short(bar(C::kBarDrain, 1), 0, nullptr, kDrainLimit);
        }
        __syncwarp();
    } else if (!FP8 || warp < 12) {
        // ================================================================ softmax of the tiles of parity g
        reg_inc<C::kRegsSoftmax>();
        const int g = (warp >> 2) - 1;
        const int tw = warp & 3;                                   // warp of the group, and its TMEM lane quarter
        const int tau = tw * 32 + lane;                            // key of the tile (S), dimension (O)
        const uint32_t lane_off = (uint32_t)(tw * 32) << 16;
        const uint32_t group_bar = 1 + g, both_bar = 3;
        constexpr int kLd = RP >= 32 ? 32 : RP;                    // TMEM columns per load
        float *neg = reinterpret_cast<float *>(misc + C::kNeg) + g * RP;
        float *delta = reinterpret_cast<float *>(misc + C::kDelta) + g * RP;
        float *alpha = reinterpret_cast<float *>(misc + C::kAlpha) + g * RP;
        int u = 0, pieces = 0;
        bool failed = false;
        while (true) {
            // all eight warps agree on whether there is a piece
            const int place = read % kRing;
            if (!failed)
                failed = !wait(bar(C::kBarPiece, place), (read / kRing) & 1);
            if (named_bar_or(both_bar, 256, failed)) {
                failed = true;
                break;
            }
            ++read;
            pc = ring[place];
            if (pc.s < 0)
                break;
            const int n = pc.b - pc.a, R = p.G * pc.q_len;
            const int own0 = pc.L - pc.q_len;                      // the first token's own row
            const int lo = max(0, own0 + 1 - p.window);            // no token sees rows from the sinks to here
            const float *scale = reinterpret_cast<const float *>(misc + C::kScale) + (pieces & 1) * RP;
            float lsum[RP];
#pragma unroll
            for (int r = 0; r < RP; ++r)
                lsum[r] = 0.f;
            bool open = true;                                      // some row has no reference yet
            if (FP8 && n > 0 && !wait(bar(C::kBarQ, pieces & 1), (pieces >> 1) & 1))     // (the rows' scales)
                failed = true;
            for (int j = (u ^ g) & 1; j < n; j += 2) {
                const int v = u + j;                               // this tile's number
                const int b = v % C::kSBufs, st = v % C::kStages;
                const int vk = (pc.a + j) * kKeys + tau;
                const int key = vk >= p.sink_pages * kPage ? vk + pc.gap * kPage : vk;
                // the rows [rmin, rmax) see this thread's key
                int jmin = key - own0, jmax = key < p.sinks ? pc.q_len : jmin + p.window;
                jmin = max(0, min(jmin, pc.q_len));
                jmax = max(0, min(jmax, pc.q_len));
                const int rmin = jmin * p.G, rmax = jmax * p.G;
                float x[RP];
                ok = !failed && wait(bar(C::kBarS, b), (v / C::kSBufs) & 1);
                // x = the key's scores (log2 units) less the rows' references; -inf where a row does not see it (padding rows
                // are 0).  A row without a reference has 0 for one.
                bool move = open;
                if (ok) {
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < RP; c += kLd)
                        tmem_ld32<kLd>(tmem + b * RP + c + lane_off, x + c);
                    tmem_wait_ld();
                    if (rmin > 0 || rmax < R) {
#pragma unroll
                        for (int r = 0; r < RP; ++r)
                            x[r] = r >= rmin && r < rmax ? x[r] : -CUDART_INF_F;
                    }
                    float top = -CUDART_INF_F;
#pragma unroll
                    for (int r = 0; r < RP; r += 4) {
                        float4 c4 = make_float4(p.score_scale_log2, p.score_scale_log2, p.score_scale_log2,
                                                p.score_scale_log2);
                        if constexpr (FP8)
                            c4 = *reinterpret_cast<const float4 *>(scale + r);
                        float4 n4 = *reinterpret_cast<const float4 *>(neg + r);
                        if (j < 2)
                            n4 = make_float4(0.f, 0.f, 0.f, 0.f);
                        const float2 a = ffma2(make_float2(x[r], x[r + 1]), make_float2(c4.x, c4.y), make_float2(n4.x, n4.y));
                        const float2 c = ffma2(make_float2(x[r + 2], x[r + 3]), make_float2(c4.z, c4.w),
                                               make_float2(n4.z, n4.w));
                        x[r] = a.x;
                        x[r + 1] = a.y;
                        x[r + 2] = c.x;
                        x[r + 3] = c.y;
                        top = fmaxf(fmax3(top, a.x, a.y), fmaxf(c.x, c.y));
                    }
                    move = open || top > C::kMost;
                }
                // one vote per tile: does a reference move, or has a wait failed?  Only then a second one tells which.
                if (named_bar_or(group_bar, 128, move || !ok)) {
                    if (named_bar_or(group_bar, 128, !ok)) {
                        failed = true;
                        break;
                    }
                    // the tile's largest score of each row, by way of the tile's dead K
                    float *red = reinterpret_cast<float *>(smem + st * C::kStageBytes);
#pragma unroll
                    for (int c0 = 0; c0 < RP; c0 += 32) {
                        float mine = 0.f;
#pragma unroll
                        for (int r = 0; r < (RP < 32 ? RP : 32); ++r) {
                            float most;
                            asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(most) : "f"(x[c0 + r]));
                            mine = lane == r ? most : mine;
                        }
                        if (RP >= 32 || lane < RP)
                            red[tw * RP + c0 + lane] = mine;
                    }
                    named_bar_sync(group_bar, 128);
                    bool none = false;
                    if (tau < RP) {
                        const float top = fmaxf(fmaxf(red[tau], red[RP + tau]), fmaxf(red[2 * RP + tau], red[3 * RP + tau]));
                        const float old = j < 2 ? 0.f : neg[tau];
                        const bool had = j >= 2 && alpha[tau] >= 0.f;      // a row's alpha is -1 until it has a reference
                        // x is relative to the old reference: the new one stands kAbove below top, but no lower than the old
                        float by = top - C::kAbove;
                        by = had ? fmaxf(by, 0.f) : by;
                        none = by == -CUDART_INF_F && tau < R;
                        by = by == -CUDART_INF_F ? 0.f : by;
                        delta[tau] = -by;
                        neg[tau] = old - by;
                        alpha[tau] = none || (!had && top == -CUDART_INF_F) ? -1.f : had ? ex2_ftz(-by) : 0.f;
                    }
                    open = named_bar_or(group_bar, 128, none);
                    if (j >= 2) {
#pragma unroll
                        for (int r = 0; r < RP; ++r)
                            lsum[r] *= fmaxf(alpha[r], 0.f);
                        // O holds the group's tiles before this one: its last product is complete once that tile's stage
                        // is free.  (The stage's next tile is past this one, so its phase cannot be over.)
                        const int prev = v - 2;
                        const bool done = wait(bar(C::kBarEmpty, prev % C::kStages), (prev / C::kStages) & 1);
                        if (done) {
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < RP; c += 16) {
                                float o[16];
                                const uint32_t col = tmem + C::kColO + g * RP + c + lane_off;
                                tmem_ld32<16>(col, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int r = 0; r < 16; ++r)
                                    o[r] *= fmaxf(alpha[c + r], 0.f);
                                tmem_st32<16>(col, o);
                            }
                            tmem_wait_st();
                        } else {
                            failed = true;                         // the next vote, or the unit's end, takes all out
                            *abort_flag = 1;
                        }
                    }
#pragma unroll
                    for (int r = 0; r < RP; r += 4) {
                        const float4 d4 = *reinterpret_cast<const float4 *>(delta + r);
                        x[r] += d4.x;
                        x[r + 1] += d4.y;
                        x[r + 2] += d4.z;
                        x[r + 3] += d4.w;
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(C::kBarSFree, b));
                // P^T over the tile's K: key t's rows at (t / 8) groups, t % 8 rows of 128 bytes, swizzled units
                uint8_t *prow = smem + st * C::kStageBytes + (tau >> 3) * C::kGroupBytes + (tau & 7) * 128;
#pragma unroll
                for (int r = 0; r < RP; r += 8) {
                    uint32_t w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 e = make_float2(ex2_ftz(x[r + 2 * k]), ex2_ftz(x[r + 2 * k + 1]));
                        const float2 l = fadd2(make_float2(lsum[r + 2 * k], lsum[r + 2 * k + 1]), e);
                        lsum[r + 2 * k] = l.x;
                        lsum[r + 2 * k + 1] = l.y;
                        w[k] = FP8 ? pack_f16x2(e.x, e.y) : pack_bf16x2(e.x, e.y);
                    }
                    *reinterpret_cast<uint4 *>(prow + (((r >> 3) ^ (tau & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
                // a row of a page that no token sees may hold anything, and 0 * NaN would reach O: its V becomes zeros
                if (!FP8 && ((key >= p.sinks && key < lo) || (key >= pc.L && key < (pc.L + kPage - 1) / kPage * kPage))) {
#pragma unroll
                    for (int c = 0; c < 16; ++c)
                        *reinterpret_cast<uint4 *>(prow + C::kOffV + (c >> 3) * 1024 + (c & 7) * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(C::kBarP, st));
            }
            // ---- the unit's end: both groups are here, all their products of Q are complete
            if (named_bar_or(both_bar, 256, failed)) {
                failed = true;
                break;
            }
            const bool whole = n == pc.t;
            // group g writes the rows [g RP / 2, (g + 1) RP / 2)
            constexpr int kHalf = RP / 2;
            const int r0 = g * kHalf;
            float2 *weight = reinterpret_cast<float2 *>(misc + C::kAlpha) + r0;
            // where a part of a unit goes: a cluster's to the stages' memory once the last product is complete, its sums to
            // that of its Q
            const int part = (2 * blockIdx.x + (pc.a > 0 ? 0 : 1)) * RP;
            float *part_o = p.split > 0 ? reinterpret_cast<float *>(smem) : p.part_o + (long long)part * kHeadDim;
            float *part_m = p.split > 0 ? reinterpret_cast<float *>(smem + C::kOffSums) : p.part_m + part;
            float *part_l = p.split > 0 ? part_m + RP : p.part_l + part;
            auto out_row = [&](int r) { return unit_row(p, pc, r); };
            if (n > 0) {
                float *red = reinterpret_cast<float *>(smem + C::kOffQ + (pieces & 1) * C::kQBytes);     // [2][4][RP]
#pragma unroll
                for (int c0 = 0; c0 < RP; c0 += kLd) {
                    float y[kLd];
#pragma unroll
                    for (int r = 0; r < kLd; ++r)
                        y[r] = lsum[c0 + r];
                    reduce_step<kLd, 16, false>(y, lane);
                    red[(g * 4 + tw) * RP + c0 + lane / (32 / kLd)] = y[0];
                }
                named_bar_sync(both_bar, 256);
                if (tau < kHalf) {
                    const int r = r0 + tau;
                    const float *negs = reinterpret_cast<const float *>(misc + C::kNeg);
                    float l[2], m[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float *x = red + k * 4 * RP + r;
                        l[k] = (x[0] + x[RP]) + (x[2 * RP] + x[3 * RP]);
                        m[k] = l[k] == 0.f ? -CUDART_INF_F : -negs[k * RP + r];
                    }
                    const float M = fmaxf(m[0], m[1]);
                    const float w0 = l[0] == 0.f ? 0.f : exp2f(m[0] - M), w1 = l[1] == 0.f ? 0.f : exp2f(m[1] - M);
                    const float sum = l[0] * w0 + l[1] * w1;
                    const float mul = !whole ? p.v_scale : sum == 0.f ? 0.f : p.v_scale / sum;
                    weight[tau] = make_float2(w0 * mul, w1 * mul);
                    if (r < R) {
                        if (!whole) {
                            part_m[r] = M;
                            part_l[r] = sum;
                        } else if (p.lse != nullptr) {
                            p.lse[out_row(r)] = sum == 0.f ? -CUDART_INF_F : M * 0.69314718055994531f + logf(sum);
                        }
                    }
                }
                named_bar_sync(group_bar, 128);
                if (!wait(bar(C::kBarO, 0), pieces & 1))
                    failed = true;
                if (!failed) {
                    tc_fence_after();
                    constexpr int kCols = kHalf >= 16 ? 16 : 8;
#pragma unroll 1
                    for (int c = 0; c < kHalf && r0 + c < R; c += kCols) {
                        float o[kCols], o1[kCols];
                        const uint32_t col = tmem + C::kColO + r0 + c + lane_off;
                        tmem_ld32<kCols>(col, o);
                        tmem_ld32<kCols>(col + RP, o1);
                        tmem_wait_ld();
#pragma unroll
                        for (int r = 0; r < kCols; ++r) {
                            const float2 w = weight[c + r];        // a weight of 0: that O may hold anything
                            o[r] = (w.x == 0.f ? 0.f : o[r] * w.x) + (w.y == 0.f ? 0.f : o1[r] * w.y);
                        }
                        // 4 x 4 transposes within lane quads: lane 4 a + b ends with row 4 k + b of a block of four and
                        // dimensions 4 a .. 4 a + 3 of the warp's 32
                        const bool b0 = (lane & 1) != 0, b1 = (lane & 2) != 0;
                        const int dim = tw * 32 + (lane & ~3);
#pragma unroll
                        for (int k = 0; k < kCols / 4; ++k) {
                            const float x0 = o[4 * k], x1 = o[4 * k + 1], x2 = o[4 * k + 2], x3 = o[4 * k + 3];
                            const float own_a = b1 ? x2 : x0, own_b = b1 ? x3 : x1;
                            const float got_a = __shfl_xor_sync(kFull, b1 ? x0 : x2, 2);
                            const float got_b = __shfl_xor_sync(kFull, b1 ? x1 : x3, 2);
                            const float la = b1 ? got_a : own_a, lb = b1 ? got_b : own_b;
                            const float ha = b1 ? own_a : got_a, hb = b1 ? own_b : got_b;
                            const float rl = __shfl_xor_sync(kFull, b0 ? la : lb, 1);
                            const float rh = __shfl_xor_sync(kFull, b0 ? ha : hb, 1);
                            const float kl = b0 ? lb : la, kh = b0 ? hb : ha;
                            const float4 y = make_float4(b0 ? rl : kl, b0 ? kl : rl, b0 ? rh : kh, b0 ? kh : rh);
                            const int r = r0 + c + 4 * k + (lane & 3);
                            if (r < R) {
                                if (whole)
                                    *reinterpret_cast<uint2 *>(p.out + out_row(r) * kHeadDim + dim) =
                                        make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
                                else
                                    *reinterpret_cast<float4 *>(part_o + r * kHeadDim + dim) = y;
                            }
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(C::kBarOFree, 0));
                    mbar_arrive(bar(C::kBarQFree, pieces & 1));
                }
                ++pieces;
            } else {
                // no keys: zeros
                for (int r = g * 4 + tw; r < R; r += 8) {
                    *reinterpret_cast<uint2 *>(p.out + out_row(r) * kHeadDim + lane * 4) = make_uint2(0u, 0u);
                    if (lane == 0 && p.lse != nullptr)
                        p.lse[out_row(r)] = -CUDART_INF_F;
                }
            }
            u += n;
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar(C::kBarPieceFree, place));
        }
        if (failed)
            give_up();
        if (p.split > 1) {
            // the cluster's parts of its unit, in key order: this CTA joins the rows of its rank, a warp a row
            __syncwarp();
            cluster_sync();
            const Piece unit = *reinterpret_cast<const Piece *>(misc + C::kUnit);
            const int R = p.G * unit.q_len, rank = blockIdx.x % (uint32_t)p.split, parts = min(p.split, unit.t);
            for (int r = rank + p.split * (warp - 4); unit.t > 1 && r < R; r += p.split * 8) {
                float M = -CUDART_INF_F, lam = 0.f;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
                for (int k0 = 0; k0 < parts; k0 += 4) {
                    float m[4], l[4];
                    float4 o[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t base = of_rank(sbase, min(k0 + k, parts - 1));
                        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(m[k]) : "r"(base + C::kOffSums + r * 4));
                        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(l[k]) : "r"(base + C::kOffSums + RP * 4 + r * 4));
                        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                     : "=f"(o[k].x), "=f"(o[k].y), "=f"(o[k].z), "=f"(o[k].w)
                                     : "r"(base + r * 512 + lane * 16));
                        l[k] = k0 + k < parts ? l[k] : 0.f;
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (l[k] == 0.f)
                            continue;
                        const float mn = fmaxf(M, m[k]), wa = M == -CUDART_INF_F ? 0.f : exp2f(M - mn),
                                    wb = exp2f(m[k] - mn);
                        M = mn;
                        lam = lam * wa + l[k] * wb;
                        acc.x = acc.x * wa + o[k].x * wb;
                        acc.y = acc.y * wa + o[k].y * wb;
                        acc.z = acc.z * wa + o[k].z * wb;
                        acc.w = acc.w * wa + o[k].w * wb;
                    }
                }
                const float inv = lam == 0.f ? 0.f : 1.f / lam;
                const long long row = unit_row(p, unit, r);
                *reinterpret_cast<uint2 *>(p.out + row * kHeadDim + lane * 4) =
                    make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
                if (lane == 0 && p.lse != nullptr)
                    p.lse[row] = lam == 0.f ? -CUDART_INF_F : M * 0.69314718055994531f + logf(lam);
            }
            __syncwarp();
            cluster_sync();                                        // the others have read this CTA's memory
        }
    } else {
        // ================================================================ e4m3: V codes to f16 (exact)
        reg_dec<C::kRegsConvert>();
        const int w = warp - 12;
        // A warp has 32 keys of a tile, in eight loads of four keys' 128 codes, 16 a lane; all are under way before the first
        // is converted (one at a time, a tile took 2000 cycles and was what the kernel waited for).  Key t's unit lies at
        // unit ^ (t % 8) in its row.  The 16 dimensions become units 2 unit and 2 unit + 1 of f16, the upper half of the lanes
        // storing the odd one first, so that a store's lanes meet no bank twice.
        const int unit = lane & 7, sub = lane >> 3, one = (2 * unit & 7) + (unit >> 2);
        int from[2], to[2][2];                                     // of the keys with t % 8 = sub and 4 + sub
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int x8 = 4 * e + sub;
            from[e] = C::kOffV + w * 4 * C::kGroupBytes + x8 * 128 + ((unit ^ x8) << 4);
            to[e][0] = C::kOffV16 + w * 4 * 2048 + (unit >> 2) * 1024 + x8 * 128 + ((one ^ x8) << 4);
            to[e][1] = C::kOffV16 + w * 4 * 2048 + (unit >> 2) * 1024 + x8 * 128 + ((one ^ 1 ^ x8) << 4);
        }
        int u = 0, copied = 0;
        while (ok && next_piece(pc, ok)) {
            if (pc.a == pc.b)
                continue;
            const int buf = copied & 1;
            if (copied >= 2)
                ok = wait(bar(C::kBarQFree, buf), ((copied >> 1) - 1) & 1);
            if (!ok)
                break;
            ++copied;
            // a quarter of the rows each, two at a time, 8 elements a lane; zeros past the rows
            const int R = p.G * pc.q_len;
            uint8_t *qs = smem + C::kOffQ + buf * C::kQBytes;
            float *scale = reinterpret_cast<float *>(misc + C::kScale) + buf * RP;
            constexpr int kLoads = RP >= 32 ? 4 : RP / 8;              // in flight
#pragma unroll 1
            for (int r0 = w * (RP / 4); r0 < (w + 1) * (RP / 4); r0 += 2 * kLoads) {
                uint4 x[kLoads];
#pragma unroll
                for (int k = 0; k < kLoads; ++k) {
                    const int r = r0 + 2 * k + (lane >> 4);
                    x[k] = r < R ? __ldg(reinterpret_cast<const uint4 *>(p.q + unit_row(p, pc, r) * kHeadDim) + (lane & 15))
                                 : make_uint4(0u, 0u, 0u, 0u);
                }
#pragma unroll
                for (int k = 0; k < kLoads; ++k) {
                    const int r = r0 + 2 * k + (lane >> 4);
                    uint2 hi, lo;
                    const int e = split_q_half_row(x[k], hi, lo);
                    const uint32_t at = r * 128 + (((((lane & 15) >> 1) ^ (r & 7)) << 4) | ((lane & 1) << 3));
                    *reinterpret_cast<uint2 *>(qs + at) = hi;
                    *reinterpret_cast<uint2 *>(qs + RP * 128 + at) = lo;
                    if ((lane & 15) == 0)
                        scale[r] = p.score_scale_log2 * __int_as_float((127 - e) << 23);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar(C::kBarQ, buf));
            // keys as numbered without the gap: those from the sinks to dead_hi and from end on are no token's
            const int lo = max(0, pc.L - pc.q_len + 1 - p.window), end = pc.L - pc.gap * kPage;
            const int dead_hi = lo > p.sinks ? lo - pc.gap * kPage : 0;
            for (int t = pc.a; t < pc.b; ++t, ++u) {
                const int st = u % C::kStages, vb = u & 1;
                ok = wait(bar(C::kBarFull, st), (u / C::kStages) & 1);
                if (ok && u >= 2)
                    ok = wait(bar(C::kBarVFree, vb), ((u >> 1) - 1) & 1);
                if (!ok)
                    break;
                const uint8_t *src = smem + st * C::kStageBytes;
                uint8_t *dst = smem + vb * C::kV16Bytes;
                uint4 a[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    a[k] = *reinterpret_cast<const uint4 *>(src + from[k & 1] + (k >> 1) * C::kGroupBytes);
                // rows that no token sees may hold anything
                if ((t + 1) * kKeys > end || (t * kKeys < dead_hi && (t + 1) * kKeys > p.sinks)) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int vk = t * kKeys + w * 32 + k * 4 + sub;
                        if (vk >= end || (vk >= p.sinks && vk < dead_hi))
                            a[k] = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint4 lo16 = make_uint4(f16x2_of_e4m3(a[k].x), f16x2_of_e4m3(a[k].x >> 16),
                                                  f16x2_of_e4m3(a[k].y), f16x2_of_e4m3(a[k].y >> 16));
                    const uint4 hi16 = make_uint4(f16x2_of_e4m3(a[k].z), f16x2_of_e4m3(a[k].z >> 16),
                                                  f16x2_of_e4m3(a[k].w), f16x2_of_e4m3(a[k].w >> 16));
                    *reinterpret_cast<uint4 *>(dst + to[k & 1][0] + (k >> 1) * 2048) = unit >> 2 ? hi16 : lo16;
                    *reinterpret_cast<uint4 *>(dst + to[k & 1][1] + (k >> 1) * 2048) = unit >> 2 ? lo16 : hi16;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(C::kBarV, vb));
            }
        }
        if (!ok)
            give_up();
    }

    if (p.split > 1 && (warp < 4 || warp >= 12)) {                 // (the softmax warps' two are above)
        __syncwarp();
        cluster_sync();
        cluster_sync();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

// Joins the pieces of the units that several runs share: block `index` those of the unit whose last piece is that run's
// first, four rows of them, one a warp.  The unit's other pieces are the first ones of the runs before, and the last one of the
// run that it starts in.  In key order, whatever the timing: with M = max m_i over the pieces with l_i > 0,
//     out = sum o_i 2^(m_i - M) / sum l_i 2^(m_i - M)
constexpr int kJoinRows = 4;                         // rows (warps) of a block
constexpr int kMaxRuns = 1024;                       // runs (SMs) at most

__global__ void __launch_bounds__(32 * kJoinRows) window_join_kernel(const WindowParams p)
{
    wait_prior_grid();
    const int index = blockIdx.x;
    const Piece pc = p.shared[2 * index];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = blockIdx.y * kJoinRows + warp;
    if (pc.s < 0 || pc.b != pc.t || r >= p.G * pc.q_len)
        return;
    const int pieces = index - pc.first + 1;
    float M = -CUDART_INF_F, lam = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kAtOnce = 8;
    for (int g0 = 0; g0 < pieces; g0 += kAtOnce) {
        float m[kAtOnce], l[kAtOnce];
        float4 o[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int run = pc.first + min(g0 + i, pieces - 1);
            const long long slot = (2LL * run + (run == pc.first ? 1 : 0)) * p.rows + r;
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
    const long long row = unit_row(p, pc, r);
    *reinterpret_cast<uint2 *>(p.out + row * kHeadDim + lane * 4) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (lane == 0 && p.lse != nullptr)
        p.lse[row] = lam == 0.f ? -CUDART_INF_F : M * 0.69314718055994531f + logf(lam);
}

template <int RP, bool FP8>
cudaError_t launch_t(const CUtensorMap &kv_map, WindowParams p, long long tiles, int num_sms, cudaStream_t stream)
{
    using C = WCfg<RP, FP8>;
    const auto kernel = window_step_kernel<RP, FP8>;
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
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    // clusters of each size that run at the same time; none where the query fails
    static PerDevice most_clusters[kMaxSplit + 1];
    int fit[kMaxSplit + 1] = {};
    cfg.numAttrs = 2;
    for (int c = 2; c <= kMaxSplit; ++c) {
        cfg.gridDim = dim3((unsigned)c);
        attr[1].val.clusterDim.x = (unsigned)c;
        fit[c] = most_clusters[c].get(device, [&] {
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess)
                return n;
            cudaGetLastError();
            return -1;
        });
    }
    const long long units = (long long)p.bs * p.H_kv, runs = step_runs(units, tiles, num_sms);
    p.split = step_cluster(units, tiles, num_sms, fit);
    const unsigned grid = (unsigned)(p.split > 0 ? units * p.split : runs);
    cfg.gridDim = dim3(grid);
    attr[1].val.clusterDim.x = (unsigned)(p.split > 1 ? p.split : 1);
    cfg.numAttrs = p.split > 1 ? 2 : 1;
    const cudaError_t rc = cudaLaunchKernelEx(&cfg, kernel, kv_map, p);
    if (rc != cudaSuccess || p.split > 0)
        return rc;
    return launch_pdl(window_join_kernel, dim3(grid, (unsigned)((p.G * p.max_q_len + kJoinRows - 1) / kJoinRows)),
                      dim3(32 * kJoinRows), 0, stream, p);
}

int padded_rows(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

}  // namespace

// Rows of a (sequence, KV head) up to which this kernel is the faster one: for 64 rows it takes 22 us where the chunk kernel
// takes 29 (64 sequences of two KV heads over a window of 1024), 99 against 111 over 8192, on e4m3 pages 77 against 103; it
// has no room for more.
bool window_step_takes(long long rows) { return rows <= 64; }

// Two pieces of the padded rows (o, m, l) per run, with what they are pieces of.
long long window_step_workspace_bytes(int rows, int num_sms)
{
    return 2LL * num_sms * ((long long)padded_rows(rows) * (kHeadDim + 2) * 4 + (long long)sizeof(WindowPiece));
}

cudaError_t launch_window_step(const WindowParams &params, int kv_dtype, long long max_seq_len, void *workspace,
                               int num_sms, cudaStream_t stream)
{
    const bool fp8 = kv_dtype == SK_KV_FP8_E4M3;
    WindowParams p = params;
    p.rows = padded_rows(p.G * p.max_q_len);
    p.sink_pages = (p.sinks + kPage - 1) / kPage;
    const long long slots = 2LL * num_sms * p.rows;
    p.part_o = static_cast<float *>(workspace);
    p.part_m = p.part_o + slots * kHeadDim;
    p.part_l = p.part_m + slots;
    p.shared = reinterpret_cast<WindowPiece *>(p.part_l + slots);
    CUtensorMap kv_map;
    cudaError_t e = encode_page_map(&kv_map, p.kv, p.num_blocks, p.H_kv, fp8, fp8 ? 2 : 4);
    if (e != cudaSuccess)
        return e;
    const long long most = (long long)p.sink_pages * kPage + p.window + p.max_q_len + kPage;
    const long long keys = max_seq_len < most ? max_seq_len : most;
    const long long tiles = (keys + kKeys - 1) / kKeys;
    p.inv_G = (65536 + p.G - 1) / p.G;               // r / G = r * inv_G >> 16 for the rows r < 64
    p.small = p.bs <= 32 && (long long)p.bs * p.H_kv * (most / kKeys + 1 + kUnitFixed) + num_sms < INT_MAX;
    auto launch = p.rows == 16 ? (fp8 ? launch_t<16, true> : launch_t<16, false>)
                  : p.rows == 32 ? (fp8 ? launch_t<32, true> : launch_t<32, false>)
                                 : (fp8 ? launch_t<64, true> : launch_t<64, false>);
    return launch(kv_map, p, tiles, num_sms < kMaxRuns ? num_sms : kMaxRuns, stream);
}

}  // namespace sk
