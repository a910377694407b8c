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
// Roles (384 threads):
//   warp 0      copies: K and V of a key tile apart, 32 KB (16 KB e4m3) slots, one TMA copy per page and part, so
//               the ring holds two and a half (five) key tiles beside Q
//   warps 1, 2  issue the products of A and of B, each through one elected lane (warp 1 also allocates TMEM); one issuer
//               for both was the bottleneck: its waits, 200 cycles each even for what is complete, came one after the
//               other (3300 cycles per key tile against 2048 of products)
//   warps 4-7   Q tile A into shared memory; softmax of A, its rescaling, its output
//   warps 8-11  the same for B
// S(j) complete implies PV(j - 1) complete (products of one issuer complete in issue order), so the softmax may rescale O
// at once; it does so only when scores beat the reference by far.
//
// e4m3 pages: QK runs as kind::f8f6f4 on the codes, with Q as two e4m3 terms and a power-of-two scale per row (exact for
// bf16 elements within 2^-9 of the row's largest), as two products into one S.  V's codes become f16 (exactly) in
// shared memory, by four more warps (12-15), and PV runs on f16.  (P as two e4m3 terms with V's codes as they are
// needs no conversion, but costs the softmax two more instructions per score: 263 against TODO us on 4 chunks of up to
// 1024 tokens over 16k keys.)
//
// Few row tiles on a long axis: the keys of every row tile are split over `nsplit` CTAs that write partial
// softmax states, joined by the library's merge.
//
// Every wait is bounded as in the decode kernel: on expiry SK_DEV_TIMEOUT is set and every role gives up; the
// producer waits for its copies and the issuer for its last commit before the CTA exits.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include <mutex>

#include "sk_attn_util.cuh"
#include "sk_internal.cuh"
#include "sk_sm100.cuh"

namespace sk {
namespace {

using namespace sm100;

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kRows = 128;                           // rows of one tile (MMA M)
constexpr int kKeys = 128;                           // keys of one tile (MMA N)
constexpr long long kDrainLimit = 4000000000LL;      // cycles (~2 s): waits for work already issued
constexpr int kMaxSmem = 232448;
template <bool FP8>
struct PCfg {
    static constexpr int kThreads = FP8 ? 512 : 384;
    // registers per thread after the reallocation: copies and products, softmax, e4m3's conversion of V; no more in all
    // than at launch (4 x 128, or 3 x 168)
    static constexpr int kRegsLaunch = FP8 ? 128 : 168;
    static constexpr int kRegsIssue = FP8 ? 80 : 104, kRegsSoftmax = FP8 ? 192 : 200, kRegsConvert = 48;
    static_assert(kRegsIssue + 2 * kRegsSoftmax + (FP8 ? kRegsConvert : 0) <= kThreads / 128 * kRegsLaunch, "registers");
    static constexpr int kQTile = kRows * 256;                     // bf16: two 64-dimension chunks; e4m3: hi and lo
    static constexpr int kGroupBytes = FP8 ? 1024 : 2048;          // K (or V) of 8 tokens, as copied
    static constexpr int kSlotBytes = kKeys / 8 * kGroupBytes;
    static constexpr int kVBytes = FP8 ? kKeys * 256 : 0;          // e4m3: V of a tile as f16, two of them
    static constexpr int kMisc = 3072;                             // barriers, then kCrow
    static constexpr int kSlots = (kMaxSmem - 2 * kQTile - 2 * kVBytes - kMisc) / kSlotBytes;
    static constexpr int kOffV = kSlots * kSlotBytes;
    static constexpr int kOffQ = kOffV + 2 * kVBytes;
    static constexpr int kOffMisc = kOffQ + 2 * kQTile;
    static constexpr int kSmemBytes = kOffMisc + kMisc;
    static constexpr int kPagesPerTile = kKeys / kPage;
    // The sum of a tile's probabilities (relative to the reference) up to which they are as good as with the maximum
    // for reference: bf16 keeps its precision at any size, f16 ends at 2^16.
    static constexpr float kSumMost = FP8 ? 0x1p15f : 0x1p40f;
    // misc area
    static constexpr int kBarFull = 0;
    static constexpr int kBarEmpty = 8 * kSlots;
    static constexpr int kBarQ = 16 * kSlots;                      // [2]
    static constexpr int kBarS = kBarQ + 16;                       // [2] S complete
    static constexpr int kBarP = kBarS + 16;                       // [2] P written
    static constexpr int kBarO = kBarP + 16;                       // [2] last PV complete
    static constexpr int kBarTurn = kBarO + 16;                    // [2] the other issuer has issued its products
    static constexpr int kBarVFull = kBarTurn + 16;                // [2] e4m3: V of a tile as f16
    static constexpr int kBarVEmpty = kBarVFull + 16;              // [2]
    static constexpr int kBarDrain = kBarVEmpty + 16;              // [2]
    static constexpr int kTmemSlot = kBarDrain + 16;
    static constexpr int kAbort = kTmemSlot + 4;
    static constexpr int kCrow = 512;                              // float[256]: score scale of each row (e4m3)
    static_assert(kAbort + 4 <= kCrow && kCrow + 1024 <= kMisc, "misc area");
    static_assert(kSlots >= 3 && (!FP8 || kSlots % 2 == 0) && kSmemBytes <= kMaxSmem && kOffQ % 1024 == 0, "shared memory");
};

// TMEM map (columns)
constexpr int kColS = 0, kColO = 256;                // S_A, S_B, then O_A, O_B, 128 each

template <bool FP8>
__global__ void __launch_bounds__(PCfg<FP8>::kThreads, 1)
prefill_kernel(const __grid_constant__ CUtensorMap kv_map, const PrefillParams p)
{
    using C = PCfg<FP8>;
    extern __shared__ __align__(1024) uint8_t smem[];

    wait_prior_grid();
    if (blockIdx.x == 0 && threadIdx.x == 0 && (__ldg(p.cu_q) != 0 || __ldg(p.cu_q + p.bs) != p.num_tokens))
        atomicOr(p.status, SK_DEV_BAD_SEQ);
    // row blocks of one (sequence, head) are neighbours, the longest first, so that they share K and V in L2
    int b = blockIdx.x;
    const int g = b % p.nsplit;
    b /= p.nsplit;
    const int rb = p.row_blocks - 1 - b % p.row_blocks;
    b /= p.row_blocks;
    const int h = b % p.H_kv;
    const int s = b / p.H_kv;
    const int L = __ldg(p.seq_lens + s);
    const int tok0 = __ldg(p.cu_q + s);
    const int q_len = __ldg(p.cu_q + s + 1) - tok0;
    const uint32_t sbase = smem_u32(smem);
    if (q_len < 0 || q_len > p.max_q_len || tok0 < 0 || tok0 + q_len > p.num_tokens || L < 0 ||
        (long long)L > (long long)p.bt_stride * kPage || (sbase & 1023u) != 0) {
        if (threadIdx.x == 0)
            atomicOr(p.status, (sbase & 1023u) != 0 ? SK_DEV_INTERNAL : SK_DEV_BAD_SEQ);
        return;
    }
    const int R_all = p.G * q_len;
    const int row0 = rb * 2 * kRows;
    if (row0 >= R_all)
        return;
    const int rowsA = min(kRows, R_all - row0), rowsB = max(0, min(kRows, R_all - row0 - kRows));

    // key tiles: the row block's tiles are cut into nsplit ranges; a row tile stops where its last row does
    auto tiles_of = [&](int first, int rows) {
        if (rows <= 0)
            return 0;
        return (visible_keys(L, q_len, (first + rows - 1) / p.G, p.causal) + kKeys - 1) / kKeys;
    };
    const int tA = tiles_of(row0, rowsA), tB = tiles_of(row0 + kRows, rowsB);
    const int t_all = max(tA, tB);
    const int t0 = (int)((long long)t_all * g / p.nsplit), t1 = (int)((long long)t_all * (g + 1) / p.nsplit);
    const int nA = max(0, min(t1, tA) - t0), nB = max(0, min(t1, tB) - t0);
    const int n = max(nA, nB);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t *misc = smem + C::kOffMisc;
    const uint32_t mbase = sbase + C::kOffMisc;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(misc + C::kAbort);
    auto bar_full = [&](int i) { return mbase + C::kBarFull + 8 * i; };
    auto bar_empty = [&](int i) { return mbase + C::kBarEmpty + 8 * i; };
    auto bar_q = [&](int x) { return mbase + C::kBarQ + 8 * x; };
    auto bar_s = [&](int x) { return mbase + C::kBarS + 8 * x; };
    auto bar_p = [&](int x) { return mbase + C::kBarP + 8 * x; };
    auto bar_o = [&](int x) { return mbase + C::kBarO + 8 * x; };
    auto bar_vfull = [&](int i) { return mbase + C::kBarVFull + 8 * i; };
    auto bar_vempty = [&](int i) { return mbase + C::kBarVEmpty + 8 * i; };
    auto bar_turn = [&](int x) { return mbase + C::kBarTurn + 8 * x; };
    auto bar_drain = [&](int x) { return mbase + C::kBarDrain + 8 * x; };

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kSlots; ++i) {
            mbar_init(bar_full(i), 1);
            mbar_init(bar_empty(i), FP8 && (i & 1) ? 4 : 2);       // both issuers; e4m3's V: the converting warps
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(bar_q(x), 4);
            mbar_init(bar_s(x), 1);
            mbar_init(bar_p(x), 4);
            mbar_init(bar_o(x), 1);
            mbar_init(bar_turn(x), 1);
            mbar_init(bar_vfull(x), 4);
            mbar_init(bar_vempty(x), 2);
            mbar_init(bar_drain(x), 1);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(mbase + C::kTmemSlot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(misc + C::kTmemSlot);

    if (warp < 4) {
        reg_dec<C::kRegsIssue>();
        if (warp == 0) {
            // ============================================================ copies
            // slot i holds, in turn, K(0), V(0), K(1), V(1), ...
            if (lane == 0)
                prefetch_tensormap(&kv_map);
            const int page0 = t0 * C::kPagesPerTile, page_end = (L + kPage - 1) / kPage;
            const int32_t *bt = p.block_table + (long long)s * p.bt_stride;
            auto block_at = [&](int j) {
                const int pg = page0 + j * C::kPagesPerTile + lane;
                return (lane < C::kPagesPerTile && j < n && pg < page_end) ? __ldg(bt + pg) : -1;
            };
            int blk = block_at(0), blk1 = block_at(1);
            int issued = 0;
            bool ok = true;
            for (int u = 0; u < 2 * n && ok; ++u) {
                const int j = u >> 1, part = u & 1, i = u % C::kSlots;
                if (u >= C::kSlots)
                    ok = wait_bar(bar_empty(i), (u / C::kSlots - 1) & 1, abort_flag, p.wait_limit);
                ok = __all_sync(kFull, ok);
                if (!ok)
                    break;
                if (lane == 0)
                    mbar_arrive_expect_tx(bar_full(i), C::kSlotBytes);
                __syncwarp();
                if (lane < C::kPagesPerTile) {
                    int grp = -2;                    // whole box out of bounds: zero fill
                    if (page0 + j * C::kPagesPerTile + lane < page_end) {
                        if (blk >= 0 && blk < p.num_blocks)
                            grp = (blk * p.H_kv + h) * 2;
                        else
                            atomicOr(p.status, SK_DEV_BAD_BLOCK);
                    }
                    tma_load_4d(sbase + i * C::kSlotBytes + lane * 2 * C::kGroupBytes, &kv_map, 0, 0,
                                part * (FP8 ? 1 : 2), grp, bar_full(i));
                }
                issued = u + 1;
                if (part) {
                    blk = blk1;
                    blk1 = block_at(j + 2);
                }
            }
            if (!ok) {
                *abort_flag = 1;
                if (lane == 0)
                    atomicOr(p.status, SK_DEV_TIMEOUT);
            }
            // every copy issued lands before the CTA exits
            for (int u = issued > C::kSlots ? issued - C::kSlots : 0; u < issued; ++u)
                mbar_wait_bounded(bar_full(u % C::kSlots), (u / C::kSlots) & 1, nullptr, kDrainLimit);
        } else if (warp <= 2) {
            // ============================================================ products of row tile x
            constexpr uint32_t idesc_qk = FP8 ? idesc_e4m3_f32(kRows, kKeys, 0, 0) : idesc_bf16_f32(kRows, kKeys, 0, 0);
            constexpr uint32_t idesc_pv = FP8 ? idesc_f16_f32(kRows, kHeadDim, 0, 1)
                                              : idesc_bf16_f32(kRows, kHeadDim, 0, 1);
            const int x = warp - 1;
            const int nx = x ? nB : nA;
            const uint64_t d_k0 = smem_desc_sw128(sbase, 16, C::kGroupBytes);       // K-major K
            const uint64_t d_v0 = smem_desc_sw128(sbase + (FP8 ? C::kOffV : 0), 1024, 2048);    // dimension-major V
            const uint64_t d_q = smem_desc_sw128(sbase + C::kOffQ + x * C::kQTile, 16, 1024);   // K-major Q
            const uint32_t sd = tmem + kColS + x * 128, od = tmem + kColO + x * 128;
            auto adv = [](uint64_t d, uint32_t bytes) { return d + (uint64_t)(bytes >> 4); };
            bool ok = true;
            auto wait = [&](uint32_t bar, uint32_t parity) {
                if (ok)
                    ok = wait_bar(bar, parity, abort_flag, p.wait_limit);
                ok = __all_sync(kFull, ok);
                return ok;
            };
            auto wait_slot = [&](int u) { return wait(bar_full(u % C::kSlots), (u / C::kSlots) & 1); };
            // passes the turn with half of the products still to issue: the other issuer wakes up meanwhile
            auto pass_turn = [&]() {
                if (lane == 0)
                    mbar_arrive(bar_turn(1 - x));
                __syncwarp();
            };
            auto qk = [&](int j) {
                const uint32_t so = (uint32_t)(2 * j % C::kSlots) * C::kSlotBytes;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    if constexpr (FP8)
                        mma_f8_ss_warp(sd, adv(d_q, (k >> 2) * (kRows * 128) + (k & 3) * 32),
                                       adv(d_k0, so + (k & 3) * 32), idesc_qk, k > 0 ? 1u : 0u);
                    else
                        mma_f16_ss_warp(sd, adv(d_q, (k >> 2) * (kRows * 128) + (k & 3) * 32),
                                        adv(d_k0, so + (k >> 2) * 1024 + (k & 3) * 32), idesc_qk, k > 0 ? 1u : 0u);
                    if (k == 3 && j > 0)
                        pass_turn();
                }
                mma_commit_warp(bar_s(x));
            };
            auto pv = [&](int j) {
                const uint32_t so = FP8 ? (uint32_t)(j & 1) * C::kVBytes : (uint32_t)((2 * j + 1) % C::kSlots) * C::kSlotBytes;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    mma_f16_ts_warp(od, sd + (k >> 2) * 64 + (k & 3) * 8, adv(d_v0, so + k * 4096), idesc_pv,
                                    (j > 0 || k > 0) ? 1u : 0u);
            };
            auto wait_v = [&](int j) { return FP8 ? wait(bar_vfull(j & 1), (j >> 1) & 1) : wait_slot(2 * j + 1); };
            // Both issuers pass every slot on, also those of tiles that only the other multiplies (they wait for them
            // all the same, so that neither is a turn of the ring ahead).
            if (n > 0 && (nx == 0 || wait(bar_q(x), 0)) && wait_slot(0)) {
                tc_fence_after();
                if (nx > 0)
                    qk(0);
                mma_commit_warp(bar_empty(0));
            }
            for (int j = 0; j < n && ok; ++j) {
                // what has to have landed is checked while the softmax still works on the tile
                if (!wait_v(j) || (j + 1 < n && !wait_slot(2 * j + 2)))
                    break;
                if (j < nx) {
                    // the row tiles take turns, so that one's softmax runs beside the other's products
                    if (x == 0 ? (j > 0 && j - 1 < nB && !wait(bar_turn(0), (j - 1) & 1))
                               : (j < nA && !wait(bar_turn(1), j & 1)))
                        break;
                    if (!wait(bar_p(x), j & 1))
                        break;
                    tc_fence_after();
                    pv(j);
                    if (j + 1 < nx) {
                        qk(j + 1);
                    } else {
                        mma_commit_warp(bar_o(x));
                        pass_turn();
                    }
                }
                mma_commit_warp(FP8 ? bar_vempty(j & 1) : bar_empty((2 * j + 1) % C::kSlots));
                if (j + 1 < n)
                    mma_commit_warp(bar_empty((2 * j + 2) % C::kSlots));
            }
            if (!ok) {
                *abort_flag = 1;
                if (lane == 0)
                    atomicOr(p.status, SK_DEV_TIMEOUT);
            }
            // every product completes before TMEM is freed and shared memory is left
            mma_commit_warp(bar_drain(x));
            mbar_wait_bounded(bar_drain(x), 0, nullptr, kDrainLimit);
        }
        __syncwarp();
    } else if (!FP8 || warp < 12) {
        // ================================================================ softmax of row tile x
        reg_inc<C::kRegsSoftmax>();
        const int x = (warp >> 2) - 1;
        const int quarter = warp & 3;
        const int tau = quarter * 32 + lane;                       // row of the tile, TMEM lane
        const int nx = x ? nB : nA;
        const int rows = x ? rowsB : rowsA;
        const int rx0 = row0 + x * kRows;                          // first row of the tile
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const uint32_t ts = tmem + kColS + x * 128 + lane_off, to = tmem + kColO + x * 128 + lane_off;
        float *crow = reinterpret_cast<float *>(misc + C::kCrow) + x * kRows;

        // ---- Q rows of this warp into shared memory (K-major, 128-byte swizzle); zeros past the rows
        uint8_t *qs = smem + C::kOffQ + x * C::kQTile;
        if (nx > 0) {
            if constexpr (!FP8) {
                uint4 v[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const int r = quarter * 32 + k * 2 + (lane >> 4), unit = lane & 15;
                    v[k] = make_uint4(0u, 0u, 0u, 0u);
                    if (r < rows) {
                        const int j = (rx0 + r) / p.G, i = rx0 + r - j * p.G;
                        v[k] = __ldg(reinterpret_cast<const uint4 *>(
                            p.q + ((long long)(tok0 + j) * p.H_q + h * p.G + i) * kHeadDim + unit * 8));
                    }
                }
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const int r = quarter * 32 + k * 2 + (lane >> 4), unit = lane & 15;
                    *reinterpret_cast<uint4 *>(qs + (unit >> 3) * (kRows * 128) + r * 128 +
                                               (((unit & 7) ^ (r & 7)) << 4)) = v[k];
                }
            } else {
                uint2 raw[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    const int r = quarter * 32 + k;
                    raw[k] = make_uint2(0u, 0u);
                    if (r < rows) {
                        const int j = (rx0 + r) / p.G, i = rx0 + r - j * p.G;
                        raw[k] = __ldg(reinterpret_cast<const uint2 *>(
                            p.q + ((long long)(tok0 + j) * p.H_q + h * p.G + i) * kHeadDim + lane * 4));
                    }
                }
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    const int r = quarter * 32 + k;
                    uint32_t hi, lo;
                    int e;
                    split_q_row(raw[k], hi, lo, e);
                    const uint32_t off = (uint32_t)(r * 128 + ((((lane >> 2) ^ (r & 7)) << 4) | ((lane & 3) << 2)));
                    *reinterpret_cast<uint32_t *>(qs + off) = hi;
                    *reinterpret_cast<uint32_t *>(qs + kRows * 128 + off) = lo;
                    if (lane == 0)
                        crow[r] = p.score_scale_log2 * ldexpf(1.f, -e);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar_q(x));
        }
        const float c = FP8 ? (nx > 0 ? crow[tau] : 0.f) : p.score_scale_log2;

        const int r = rx0 + tau;                                   // this thread's row
        const int jq = r / p.G, iq = r - jq * p.G;
        const bool live = tau < rows;
        const int limit = live ? visible_keys(L, q_len, jq, p.causal) : 0;
        const int least = __reduce_min_sync(kFull, limit);         // keys that every row of the warp sees
        float m_ref = -CUDART_INF_F;
        bool anchored = false;                                     // every row that sees a key has a reference
        float2 l2 = make_float2(0.f, 0.f);
        bool failed = false;
        for (int j = 0; j < nx; ++j) {
            const int key0 = (t0 + j) * kKeys;
            bool ok = wait_bar(bar_s(x), j & 1, abort_flag, p.wait_limit);
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
            // moves the rows' reference up to `top` and rescales what they have summed; `in_o`: O holds something
            auto raise = [&](float top, bool in_o) {
                const float mn = fmaxf(m_ref, top);
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
            // only a row's first scores need their maximum before they are exponentiated (see below)
            if (!anchored) {
                if (__any_sync(kFull, m_ref == -CUDART_INF_F && lim > 0))
                    raise(tile_top(), j > 0);
                anchored = !__any_sync(kFull, m_ref == -CUDART_INF_F && limit > 0);
            }
            // rows past the sequence's end in its last page hold anything, and 0 * NaN would reach O: their V
            // becomes zeros, before either row tile multiplies it
            if (!FP8 && L < key0 + kKeys && (L & (kPage - 1)) != 0) {
                ok = mbar_wait_bounded(bar_full((2 * j + 1) % C::kSlots), ((2 * j + 1) / C::kSlots) & 1, abort_flag,
                                       p.wait_limit);
                ok = __all_sync(kFull, ok);
                const int tok = key0 + tau;
                if (ok && tok >= L && tok < (L + kPage - 1) / kPage * kPage) {
                    uint8_t *row = smem + (2 * j + 1) % C::kSlots * C::kSlotBytes + (tau >> 3) * C::kGroupBytes +
                                   (tau & 7) * 128;
#pragma unroll
                    for (int cc = 0; cc < C::kGroupBytes / 1024; ++cc)
#pragma unroll
                        for (int u = 0; u < 8; ++u)
                            *reinterpret_cast<uint4 *>(row + cc * 1024 + u * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                if (!ok)
                    *abort_flag = 1;                               // the other roles' waits end with it
            }
            // P overwrites the first columns of each half of S.  A row's reference need not follow its maximum while
            // the probabilities stay well inside their type's range, and the tile's sum shows whether some did not.
            // Only then is the maximum taken, the reference raised, O rescaled and the tile done again.
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
                if (again || !__any_sync(kFull, !(h2.x + h2.y <= C::kSumMost)))
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
        if (!failed && nx > 0) {
            bool ok = mbar_wait_bounded(bar_o(x), 0, abort_flag, p.wait_limit);
            failed = !__all_sync(kFull, ok);
        }
        if (failed) {
            *abort_flag = 1;
        } else if (rows > 0) {
            tc_fence_after();
            const float l = l2.x + l2.y;
            const long long qrow = (long long)(tok0 + jq) * p.H_q + h * p.G + iq;
            const long long slot = ((long long)(tok0 + jq) * p.nsplit + g) * p.H_q + h * p.G + iq;
            const float mul = p.nsplit > 1 ? p.v_scale : (l == 0.f ? 0.f : p.v_scale / l);
#pragma unroll
            for (int cc = 0; cc < 128; cc += 32) {
                float o[32];
                if (nx > 0) {
                    tmem_ld32<32>(to + cc, o);
                    tmem_wait_ld();
                }
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    o[i] = (nx > 0 && !(l == 0.f)) ? o[i] * mul : 0.f;
                if (!live)
                    continue;
                if (p.nsplit > 1) {
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        *reinterpret_cast<float4 *>(p.part_o + slot * kHeadDim + cc + i) =
                            make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; i += 8)
                        *reinterpret_cast<uint4 *>(p.out + qrow * kHeadDim + cc + i) =
                            make_uint4(pack_bf16x2(o[i], o[i + 1]), pack_bf16x2(o[i + 2], o[i + 3]),
                                       pack_bf16x2(o[i + 4], o[i + 5]), pack_bf16x2(o[i + 6], o[i + 7]));
                }
            }
            if (live) {
                const float ln2 = 0.69314718055994531f;
                if (p.nsplit > 1) {
                    p.part_m[slot] = l > 0.f ? m_ref * ln2 : -CUDART_INF_F;
                    p.part_l[slot] = l;
                } else if (p.lse != nullptr) {
                    p.lse[qrow] = l == 0.f ? -CUDART_INF_F : m_ref * ln2 + logf(l);
                }
            }
        }
    } else {
        // ================================================================ e4m3: V codes to f16 (exact)
        reg_dec<C::kRegsConvert>();
        const int w = warp - 12;
        // a warp's load is four tokens' 128 codes, 16 a lane; token t's unit u lies at u ^ (t % 8) in its row.  The 16
        // dimensions become units 2 u and 2 u + 1 of f16, the upper half of the lanes storing the odd one first, so
        // that a store's lanes meet no bank twice
        const int u = lane & 7, sub = lane >> 3;
        for (int j = 0; j < n; ++j) {
            const int slot = (2 * j + 1) % C::kSlots, vb = j & 1;
            bool ok = wait_bar(bar_full(slot), ((2 * j + 1) / C::kSlots) & 1, abort_flag, p.wait_limit);
            if (ok && j >= 2)
                ok = wait_bar(bar_vempty(vb), ((j >> 1) - 1) & 1, abort_flag, p.wait_limit);
            if (!__all_sync(kFull, ok)) {
                *abort_flag = 1;
                break;
            }
            const uint8_t *src = smem + slot * C::kSlotBytes;
            uint8_t *dst = smem + C::kOffV + vb * C::kVBytes;
            const int key0 = (t0 + j) * kKeys;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int t = w * 32 + k * 4 + sub, x8 = t & 7;
                uint4 a = *reinterpret_cast<const uint4 *>(src + (t >> 3) * 1024 + x8 * 128 + ((u ^ x8) << 4));
                if (key0 + t >= L)                                 // past the end the page holds anything
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
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <bool FP8>
cudaError_t launch_t(const CUtensorMap &map, const PrefillParams &p, cudaStream_t stream)
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
    const dim3 grid((unsigned)p.nsplit * p.row_blocks * p.H_kv * p.bs);
    return launch_pdl(prefill_kernel<FP8>, grid, dim3(PCfg<FP8>::kThreads), PCfg<FP8>::kSmemBytes, stream, map, p);
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

// CTAs that share the keys of a row block: the number with the least estimated time.  A CTA takes kFixed to start and
// finish and kTile per key tile (us); the GPU works off `units` row blocks (at most; with ragged query lengths the
// tokens' own count bounds them) num_sms at a time, the last round half full on average; a split adds the merge, whose
// partial states (520 bytes per row, head and split) are written and read.
int prefill_nsplit(int bs, int num_tokens, int max_q_len, int H_q, int H_kv, int max_seq_len, int num_sms)
{
    constexpr double kFixed = 4.0, kTile = 1.25, kMerge = 3.0, kBytesPerUs = 5e6;
    const long long G = H_q / H_kv;
    const long long most = (G * max_q_len + kPrefillRows - 1) / kPrefillRows * bs;
    const long long have = (G * num_tokens + kPrefillRows - 1) / kPrefillRows + bs;
    const double units = (double)(most < have ? most : have) * H_kv;
    const int tiles = (max_seq_len + kKeys - 1) / kKeys;
    int best = 1;
    double best_t = 1e300;
    for (int n = 1; n <= 64 && (n == 1 || n <= tiles); ++n) {
        const double cta = kFixed + kTile * ((tiles + n - 1) / n), rounds = units * n / num_sms;
        double t = cta * (rounds <= 1.0 ? 1.0 : rounds + 0.5);
        if (n > 1)
            t += kMerge + 2.0 * n * num_tokens * H_q * 520.0 / kBytesPerUs;
        if (t < best_t * (n > 1 ? 0.97 : 1.0)) {
            best_t = t;
            best = n;
        }
    }
    return best;
}

cudaError_t launch_prefill(const PrefillParams &p, int kv_dtype, cudaStream_t stream)
{
    const bool fp8 = kv_dtype == SK_KV_FP8_E4M3;
    CUtensorMap map;
    // one box: K (or V) of one page and head
    const cudaError_t e = encode_page_map(&map, p.kv, p.num_blocks, p.H_kv, fp8, fp8 ? 1 : 2);
    if (e != cudaSuccess)
        return e;
    return fp8 ? launch_t<true>(map, p, stream) : launch_t<false>(map, p, stream);
}

}  // namespace sk
