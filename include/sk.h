/*
 * sk.h -- C ABI of libsk: length-aware split-KV paged decode/verify attention
 * for one GB300 (sm_103a).
 *
 * The method (SGLang PR 39172, "[AMD] gfx950 assembly attention: length-aware
 * split-KV for dynamic workload") runs in three device steps per attention
 * call:
 *   1. sk_build_plan        picks one segment length T from the batch's
 *                           sequence lengths and writes a compact work list
 *                           of (sequence, segment) items plus a per-query-
 *                           token segment count (Modifications, first item).
 *   2. sk_paged_decode_attn one CTA per (sequence, segment, kv head) work item
 *                           gathers K/V from standard pages and emits a
 *                           partial softmax state per query row
 *                           (Modifications, second item).
 *   3. sk_merge_segments    merges each token's segments by log-sum-exp,
 *                           reading only that token's segment count
 *                           (Modifications, third item).
 * A NULL plan selects the fixed split of the Motivation section (used for
 * bs == 1, where it already gives 64 segments).
 *
 * Around them, on the same pages: the writes of new tokens (sk_reshape_and_cache, or with rotary positions
 * sk_rope_and_cache, of several axes sk_rope_axes_and_cache), attention of many new tokens at once
 * (sk_paged_prefill_attn), attention with a sliding window and sinks (sk_paged_window_attn), and a cache bounded by
 * eviction (sk_accum_attn_weights, sk_evict_select, sk_evict_move).
 *
 * Conventions for every call:
 *  - Pointers marked "device" are device memory owned by the caller; the
 *    library keeps no reference after the call returns.  It allocates no
 *    device memory of its own: its only device storage is one status word
 *    per device and the fixed scratch array of
 *    sk_paged_decode_attention_static (both static __device__ variables).
 *  - Work is enqueued asynchronously on `stream` (a cudaStream_t; NULL is the
 *    legacy default stream).  No call synchronises, so the whole path can be
 *    captured into a CUDA graph.  Every kernel is launched with programmatic
 *    stream serialization: it may start while the kernel before it on the
 *    stream finishes, and waits for that kernel's completion (and its writes)
 *    before it reads anything, so stream order is kept.
 *  - Invalid arguments are caught on the host before anything is launched
 *    and return a negative sk_status; sk_last_error() then describes the
 *    problem.  Conditions only the device can see (a block id outside
 *    [0, num_blocks), a query length above max_q_len, an inconsistent
 *    cu_seqlens_q, a wait that timed out) set bits in the device status word
 *    and the affected work is skipped; read them with sk_get_device_status().
 *    cu_seqlens_q must be non-decreasing with cu[0] == 0 and cu[bs] ==
 *    num_tokens; otherwise SK_DEV_BAD_SEQ is set, tokens outside [cu[0],
 *    cu[bs]) get 0 segments from the plan (output 0, lse -inf), and on the
 *    fixed split their outputs are undefined.
 *  - Supported shapes: head_dim == 128, page_size == 16, 1 <= bs <= 32767
 *    (so seq << 16 stays positive), num_q_heads % num_kv_heads == 0.
 */
#ifndef SK_H_
#define SK_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SK_OK = 0,
    SK_CACHED = 1,            /* sk_build_plan: cache hit, nothing launched */
    SK_ERR_INVALID = -1,      /* bad pointer, size or stride */
    SK_ERR_CAPACITY = -2,     /* plan_capacity too small */
    SK_ERR_UNSUPPORTED = -3,  /* shape outside the supported set */
    SK_ERR_CUDA = -4,         /* a CUDA runtime call failed */
    SK_ERR_TIMEOUT = -5       /* sk_get_device_status: a bounded wait inside a kernel expired */
} sk_status;

typedef enum {
    SK_KV_BF16 = 0,           /* pages hold bf16 */
    SK_KV_FP8_E4M3 = 1        /* pages hold OCP e4m3fn codes (vLLM RFC 59111, Proposed Change:
                                 OCP e4m3fn, not MI300's fnuz), value = code * scale */
} sk_kv_dtype;

/* Bits of the device status word (sk_get_device_status). */
#define SK_DEV_BAD_BLOCK 0x1   /* a block-table entry outside [0, num_blocks) was skipped */
#define SK_DEV_BAD_SEQ 0x2     /* q_len > max_q_len, L > block_table_stride * page, or bad cu_seqlens_q */
#define SK_DEV_TIMEOUT 0x4     /* a bounded wait inside a kernel expired; its work item was abandoned */
#define SK_DEV_INTERNAL 0x8    /* a kernel precondition failed (e.g. shared-memory alignment); item skipped */

/* Tokens per plan tile.  The plan counts segment lengths in tiles:
 * plan[0] = tiles per segment, so a segment spans plan[0] * sk_tile_tokens()
 * tokens (SGLang PR 39172, Modifications: "tiles per segment come from
 * plan[0]").  Returns 64. */
int sk_tile_tokens(void);

/* Smallest valid plan_capacity for a batch: 1 + max(B, bs) with
 * B = floor(num_sms / num_kv_heads), the plan's budget of work items (SGLang PR
 * 39172, Modifications: total segments capped at num_CUs / kv_heads; a batch
 * with more non-empty sequences than B takes one segment each, so up to bs
 * items).  Host-only arithmetic; SK_ERR_INVALID for bs outside [1, 32767] or
 * a non-positive head or SM count. */
int sk_plan_capacity(int bs, int num_kv_heads, int num_sms);

/* Segment count of the fixed split (SGLang PR 39172, Motivation):
 * max(1, min(seg_max, pow2floor(num_sms / (bs * num_kv_heads)))), pow2floor
 * of a value below 1 being 0.  Host-only arithmetic. */
int sk_fixed_nseg(int bs, int num_kv_heads, int num_sms, int seg_max);

/* Build the length-aware plan on the device (SGLang PR 39172, Modifications).
 *
 *   tiles_s = ceil(seq_lens[s] / sk_tile_tokens())
 *   B       = floor(num_sms / num_kv_heads)
 *   T       = smallest t >= 1 with sum_s ceil(tiles_s / t) <= B and
 *             max_s ceil(tiles_s / t) <= seg_max; if no t qualifies (more
 *             non-empty sequences than B) T = max_s tiles_s, one segment per
 *             non-empty sequence; T = 1 when every sequence is empty.
 *
 * Outputs (device, caller-owned):
 *   plan     int32[plan_capacity]: plan[0] = T; plan[1+k] = (s << 16) | g for
 *            every segment g < ceil(tiles_s / T) of every sequence s, in
 *            (s ascending, g ascending) order; -1 in every later slot.
 *   tok_nseg int32[num_tokens]: tok_nseg[t] = segment count of t's sequence.
 * Inputs (device): seq_lens int32[bs] (KV length including this step's query
 *   tokens), cu_seqlens_q int32[bs+1] (query-token offsets, cu[bs] ==
 *   num_tokens).
 * plan_capacity must be >= sk_plan_capacity(bs, num_kv_heads, num_sms) =
 * 1 + max(B, bs); larger values are allowed.
 *
 * Plan cache: the plan is built once per forward and reused by every layer.
 * The cache key is (seq_lens, seq_lens_version, cu_seqlens_q,
 * cu_seqlens_q_version, bs, num_tokens, num_kv_heads, num_sms, seg_max, plan,
 * plan_capacity, tok_nseg, whether `stream` is capturing).  A hit returns
 * SK_CACHED and launches nothing: the caller's plan/tok_nseg buffers still hold
 * the result.  The version arguments let a caller mark in-place changes (the
 * Python binding passes tensor._version).  sk_plan_cache_reset() clears the
 * cache; call it at the start of every forward.
 * Returns SK_OK (plan kernel enqueued), SK_CACHED, or a negative sk_status. */
int sk_build_plan(const int32_t *seq_lens, uint64_t seq_lens_version,
                  const int32_t *cu_seqlens_q, uint64_t cu_seqlens_q_version,
                  int bs, int num_tokens, int num_kv_heads, int num_sms, int seg_max,
                  int32_t *plan, int plan_capacity, int32_t *tok_nseg, void *stream);

/* Clear the plan cache (SGLang PR 39172, Modifications: the cache is cleared
 * at the start of every forward). */
void sk_plan_cache_reset(void);

/* Number of plan kernels launched by this process so far (cache misses). */
long long sk_plan_launch_count(void);

/* Split-KV paged attention (SGLang PR 39172, Modifications, second item).
 *
 * Grid: with a plan, (plan_capacity - 1) * num_kv_heads * row_blocks CTAs,
 * row_blocks = ceil(G * max_q_len / 64) when that exceeds 64 rows (else 1);
 * CTA b takes row block b % row_blocks (rows [64 rb, 64 rb + 64) of the item)
 * of work item i = (b / row_blocks) / num_kv_heads and KV head
 * h = (b / row_blocks) % num_kv_heads, reads w = plan[1+i], and exits at once
 * when w == -1 or the block is past the item's rows.  Sequence s = w >> 16,
 * segment g = w & 0xFFFF covers keys [g*T, min((g+1)*T, L_s)) with
 * T = plan[0] * sk_tile_tokens().  With plan == NULL the fixed split runs:
 * nseg = sk_fixed_nseg(bs, num_kv_heads, num_sms, seg_max) segments per
 * sequence of ceil(tiles_s / nseg) tiles each (trailing ones may be empty);
 * the grid is bs * nseg * num_kv_heads.
 *
 * Layouts (device):
 *   q            bf16 [num_tokens, num_q_heads, head_dim], token-major via
 *                cu_seqlens_q.  Query head hq uses KV head hq / G, G =
 *                num_q_heads / num_kv_heads.
 *   kv_pages     [num_blocks, num_kv_heads, page_size, 2*head_dim]: standard
 *                pages (vLLM RFC 59111, Background): per head, each token
 *                row holds K in [0, D) and V in [D, 2D).  bf16 or e4m3fn.
 *   block_table  int32 [bs, block_table_stride]; key p of sequence s lives in
 *                block block_table[s*stride + p/page_size], row p % page_size.
 *   seq_lens, cu_seqlens_q as for sk_build_plan; plan as written by it.
 * Masking: with causal != 0, query token j of sequence s (q_s tokens) sees
 *   keys p <= L_s - q_s + j; otherwise all L_s keys.
 * Scores: sm_scale * k_scale * <q, k>; values are multiplied by v_scale (the
 *   two scales apply to fp8 pages only and are ignored for bf16).
 * max_q_len: an upper bound on every q_s (at least 1 when num_tokens > 0); it
 *   sizes the kernel's row tile and row blocks (rows per work item = G * q_s).
 *   G * max_q_len above 65536, or num_blocks * num_kv_heads above 2^30, is
 *   SK_ERR_UNSUPPORTED.
 * Outputs (device, fp32): for every query token t of the item's sequence,
 *   every query head hq of KV head h, and the item's segment g:
 *     part_m[(t*seg_max + g)*num_q_heads + hq]  reference value m (score units)
 *     part_l[same]                               l = sum_p exp(score_p - m)
 *     part_o[same * head_dim + d]                o = v_scale * sum_p exp(score_p - m) * V_p[d]
 *   over the keys of the segment that the row sees.  A row that sees none of
 *   them gets (m, l, o) = (-inf, 0, 0).  m is not required to be the maximum
 *   score; m + log(l) and o / l are the segment's unique log-sum-exp and output.
 *   Arrays are [num_tokens, seg_max, num_q_heads(, head_dim)]; only segments
 *   that exist are written.
 * q, kv_pages and part_o must be 16-byte aligned (SK_ERR_INVALID otherwise).
 * Returns SK_OK or a negative sk_status. */
int sk_paged_decode_attn(const void *q, const void *kv_pages, int kv_dtype, float k_scale,
                         float v_scale, const int32_t *block_table, int block_table_stride,
                         int num_blocks, int page_size, const int32_t *seq_lens,
                         const int32_t *cu_seqlens_q, const int32_t *plan, int plan_capacity,
                         int bs, int num_tokens, int max_q_len, int num_q_heads, int num_kv_heads,
                         int head_dim, float sm_scale, int causal, int num_sms, int seg_max,
                         float *part_o, float *part_m, float *part_l, void *stream);

/* Merge segment partials by log-sum-exp (SGLang PR 39172, Modifications,
 * third item: the reduce reads only its token's segment count).
 * For token t and query head hq with n = tok_nseg[t] (or fixed_nseg when
 * tok_nseg == NULL) segments, over segments with l > 0:
 *   M = max m_g,  Lambda = sum l_g exp(m_g - M),
 *   out = sum o_g exp(m_g - M) / Lambda   (bf16, round to nearest even),
 *   lse = M + log(Lambda)                  (fp32, optional).
 * No contributing segment: out = 0, lse = -inf.
 * out bf16 [num_tokens, num_q_heads, head_dim]; lse fp32 [num_tokens,
 * num_q_heads] or NULL.  Partials as written by sk_paged_decode_attn.
 * part_o must be 16-byte and out 8-byte aligned (SK_ERR_INVALID otherwise).
 * Returns SK_OK or a negative sk_status. */
int sk_merge_segments(const float *part_o, const float *part_m, const float *part_l,
                      const int32_t *tok_nseg, int fixed_nseg, int num_tokens, int num_q_heads,
                      int head_dim, int seg_max, void *out, float *lse, void *stream);

/* KV write: store this step's K and V rows into standard pages through a
 * slot mapping (the writer of the backends that keep standard pages, vLLM RFC
 * 59111, Background: per head, a token row holds K and V side by side).
 *
 * For token t and KV head h with slot = slot_mapping[t] >= 0:
 *   kv_pages[slot / page_size][h][slot % page_size][0 : D)  = K[t][h][:]
 *   kv_pages[slot / page_size][h][slot % page_size][D : 2D) = V[t][h][:]
 * bf16 pages receive the input bits unchanged.  e4m3fn pages
 * (kv_dtype == SK_KV_FP8_E4M3) receive each value divided by k_scale (K) or
 * v_scale (V) in IEEE binary32 and rounded to the nearest e4m3fn code, ties
 * to even, magnitudes above 448 (and infinities) saturated to 448, NaN kept
 * as NaN; sk_paged_decode_attn then multiplies the codes back by the same
 * scales.
 * A negative slot writes nothing for that token.  A slot at or past
 * num_blocks * page_size writes nothing and sets SK_DEV_BAD_BLOCK in the
 * device status word.  Two tokens with the same slot leave that row
 * undefined (either token's values).
 *
 * Layouts (device, caller-owned): key, value bf16 [num_tokens, num_kv_heads,
 * head_dim]; slot_mapping int64 [num_tokens]; kv_pages [num_blocks,
 * num_kv_heads, page_size, 2*head_dim] of bf16 or e4m3fn, written in place.
 * key, value and kv_pages must be 16-byte aligned; head_dim must be 128 and
 * page_size 16.  Asynchronous on `stream`, no allocation, capture safe.
 * Returns SK_OK or a negative sk_status. */
int sk_reshape_and_cache(const void *key, const void *value, const int64_t *slot_mapping,
                         int num_tokens, int num_kv_heads, int head_dim, void *kv_pages, int kv_dtype,
                         float k_scale, float v_scale, int num_blocks, int page_size, void *stream);

/* Standard -> shuffled page conversion (vLLM RFC 59111, Proposed Change,
 * Convert: the per-block view/permute that turns standard pages into ROCm
 * AITER's shuffled pages).  With x = 16 / element size (8 for bf16, 16 for
 * e4m3fn), for every block blk listed in block_ids (all num_blocks blocks when
 * block_ids == NULL, num_ids then ignored), head h, token row n, dimension d:
 *   k_shuf[blk][h][d / x][n][d % x] = kv_pages[blk][h][n][d]
 *   v_shuf[blk][h][n / x][d][n % x] = kv_pages[blk][h][n][D + d]
 * Other blocks of k_shuf and v_shuf are left alone.  An id outside
 * [0, num_blocks) is skipped and sets SK_DEV_BAD_BLOCK in the device status.
 *
 * Layouts (device, caller-owned): kv_pages [num_blocks, num_kv_heads,
 * page_size, 2*head_dim] (kv_dtype bf16 or e4m3fn, bytes copied as they are);
 * k_shuf [num_blocks, num_kv_heads, head_dim / x, page_size, x];
 * v_shuf [num_blocks, num_kv_heads, page_size / x, head_dim, x]; block_ids
 * int32 [num_ids] or NULL.  All three arrays 16-byte aligned; head_dim 128,
 * page_size 16.  Asynchronous on `stream`, no allocation, capture safe.
 * Returns SK_OK or a negative sk_status. */
int sk_std_to_shuffled(const void *kv_pages, int kv_dtype, const int32_t *block_ids, int num_ids,
                       int num_blocks, int num_kv_heads, int head_dim, int page_size, void *k_shuf,
                       void *v_shuf, void *stream);

/* Attention of a chunk of new tokens over the paged cache: prefill, chunked prefill, a follow-up turn on a
 * long conversation, cross attention (causal == 0).  The result of sk_paged_decode_attn + sk_merge_segments, by
 * a kernel for many query rows: the softmax runs over all of a sequence's keys in one pass, without a plan.
 *
 *   out[t][hq] = sum_p softmax(score)_p V_p,  lse[t][hq] = log sum_p exp(score_p)
 * with scores sm_scale * k_scale * <q, k> over the keys that token t sees (the masking, layouts and scales of
 * sk_paged_decode_attn; the chunk's own keys are already in the pages and counted in seq_lens).  A token that
 * sees no key gets out = 0 and lse = -inf.  Query lengths may differ and may be 0; with no tokens at all nothing is launched,
 * and q, out and lse may be NULL.  max_q_len bounds the query lengths (more sets SK_DEV_BAD_SEQ and skips the sequence,
 * whose rows are then undefined).  Rows past cu_seqlens_q[bs], if that is below num_tokens (which sets SK_DEV_BAD_SEQ), are
 * left as they were.  At most 2^26 blocks a sequence and 2^24 (sequence, KV head) pairs, here and in the three calls
 * of eviction.
 *
 * The work is divided evenly over the SMs, in the key axis too, so few query rows on a long cache use the whole
 * GPU, beside many short sequences as well; in a batch larger than the L2 whose units of 256 rows cost alike, or are
 * many, whole units go out first, which is nearly as even.  max_seq_len, an upper bound on the lengths, decides how many
 * CTAs a small call launches and how the work is divided; a wrong one costs time only.  workspace (device, 16-byte
 * aligned): sk_prefill_workspace_bytes(num_tokens, num_q_heads, kv_dtype) bytes; its contents do not matter, and
 * calls that may overlap need one each.  q, kv_pages and out are 16-byte aligned; lse may be NULL.  Probabilities
 * round to bf16 (for e4m3fn pages to f16, by 2^-11 of themselves or 2^-33 of the row's sum, whichever is more); sums
 * are fp32; the same bits every time on the same device.  With e4m3fn pages q is two e4m3 terms per element, as for
 * sk_accum_attn_weights.  A key that a row does not see weighs exactly 0 there: a NaN or an infinity in its K does not
 * matter, one in its V may reach the row as 0 times it.  (The page rows past a sequence's end may hold anything.)
 * Returns SK_OK or a negative sk_status. */
int sk_paged_prefill_attn(const void *q, const void *kv_pages, int kv_dtype, float k_scale, float v_scale,
                          const int32_t *block_table, int block_table_stride, int num_blocks, int page_size,
                          const int32_t *seq_lens, const int32_t *cu_seqlens_q, int bs, int num_tokens, int max_q_len,
                          int num_q_heads, int num_kv_heads, int head_dim, float sm_scale, int causal, int max_seq_len,
                          void *workspace, int64_t workspace_bytes, void *out, float *lse, void *stream);

/* Attention with a sliding window and sinks, of one token a sequence up to whole prompts: the query token in row
 * P = seq_lens[s] - q_s + j of its sequence (j < q_s, its query length) sees the rows r <= P with
 *   r < sinks  or  r > P - window,
 * so its last `window` rows, its own among them, and the first `sinks` ones (window >= 1, sinks >= 0; with a window of
 * at least seq_lens[s] it is causal attention over the whole cache).  Everything else as for sk_paged_prefill_attn with
 * causal set: arguments, layouts, outputs, roundings, workspace rules and status bits.  A row with P < 0 sees nothing:
 * its output is 0, its lse -inf.  Rows are counted along the block table, so a cache that sk_evict_move has reordered
 * has no window.
 *
 * Pages that no query token of the sequence sees are not read, and their block table entries are not looked at: a
 * server may hand them back and leave anything there.  They are the whole pages between row sinks and row
 * seq_lens[s] - q_s + 1 - window.  Rows in pages that are read, but that no token of the call sees, may hold anything as
 * well.  The rule on a NaN or an infinity in V that sk_paged_prefill_attn gives holds for rows that only some
 * tokens of the call see.  Where cu_seqlens_q falls somewhere, which sets SK_DEV_BAD_SEQ, the sequences whose offsets are in
 * order are worked on all the same, or, in a large batch, none is.
 *
 * Up to 64 query rows of a (sequence, KV head), max_q_len * num_q_heads / num_kv_heads, are a step's: its cost is divided by
 * key tiles over the SMs, or, for few sequences, each (sequence, KV head) has a cluster of CTAs.  More are a chunk's.
 *
 * workspace (device, 16-byte aligned): sk_window_workspace_bytes(num_tokens, num_q_heads, num_kv_heads, max_q_len,
 * kv_dtype) bytes.  max_seq_len as for sk_paged_prefill_attn.  Asynchronous on `stream`, no allocation, capture safe.
 * Returns SK_OK or a negative sk_status. */
int sk_paged_window_attn(const void *q, const void *kv_pages, int kv_dtype, float k_scale, float v_scale,
                         const int32_t *block_table, int block_table_stride, int num_blocks, int page_size,
                         const int32_t *seq_lens, const int32_t *cu_seqlens_q, int bs, int num_tokens, int max_q_len,
                         int num_q_heads, int num_kv_heads, int head_dim, float sm_scale, int window, int sinks,
                         int max_seq_len, void *workspace, int64_t workspace_bytes, void *out, float *lse,
                         void *stream);

/* Bytes of workspace of sk_paged_window_attn on the current device.  A negative sk_status for bad sizes or if a CUDA call
 * fails. */
int64_t sk_window_workspace_bytes(int num_tokens, int num_q_heads, int num_kv_heads, int max_q_len, int kv_dtype);

/* Bytes of workspace of sk_paged_prefill_attn on the current device (two partial states of 256 rows per SM, and for
 * e4m3fn pages q in two terms).  A negative sk_status for bad sizes or if a CUDA call fails. */
int64_t sk_prefill_workspace_bytes(int num_tokens, int num_q_heads, int kv_dtype);

/* Attention weight gathered by each cached key: for every sequence s, KV head h and key p < seq_lens[s],
 *   acc_pages (place of p) += sum over query tokens t of s that see p, and heads hq of the group of h, of
 *                             exp(score(t, hq, p) - lse[t][hq])
 * with the scores and the masking of sk_paged_decode_attn (max_q_len as there) and `lse` as written by the
 * attention calls (fp32 [num_tokens, num_q_heads], natural logarithm): each (t, hq) adds weights that sum to 1
 * over its keys.  A row whose lse is -inf adds nothing.  Places of no key, and those of blocks outside
 * [0, num_blocks) (which set SK_DEV_BAD_BLOCK), are left as they were.  Where sequences share a block, all add to
 * it (in no fixed order; otherwise the same bits every time).
 *
 * acc_pages fp32 [num_blocks, num_kv_heads, page_size], updated in place.  workspace (device, 16-byte aligned):
 * sk_accum_workspace_bytes(num_tokens, num_q_heads, num_kv_heads, max_q_len, kv_dtype) bytes, 0 for bf16 pages and at
 * most 64 rows (max_q_len times the heads of a group; then it may be NULL); its contents do not matter, and calls that
 * may overlap need one each.  q and kv_pages are 16-byte aligned.
 * Scores and sums are fp32; with e4m3fn pages q is two e4m3 terms per element, exact for elements of at least
 * 2^-9 of the row's largest (an infinite element saturates: it counts as 896, beside the others as they are).  Asynchronous on `stream`, no allocation, capture safe.
 * Returns SK_OK or a negative sk_status. */
int sk_accum_attn_weights(const void *q, const void *kv_pages, int kv_dtype, float k_scale,
                          const int32_t *block_table, int block_table_stride, int num_blocks, int page_size,
                          const int32_t *seq_lens, const int32_t *cu_seqlens_q, int bs, int num_tokens, int max_q_len,
                          int num_q_heads, int num_kv_heads, int head_dim, float sm_scale, int causal,
                          const float *lse, float *acc_pages, void *workspace, int64_t workspace_bytes, void *stream);

/* Bytes of workspace of sk_accum_attn_weights.  Host-only arithmetic; a negative sk_status for bad sizes. */
int64_t sk_accum_workspace_bytes(int num_tokens, int num_q_heads, int num_kv_heads, int max_q_len, int kv_dtype);

/* How sk_rope_frequencies fits the frequencies w_i = base^(-2 i / rot_dim) to contexts `factor` times
 * longer than the trained ones. */
typedef enum {
    SK_ROPE_PLAIN = 0,        /* w_i */
    SK_ROPE_LINEAR = 1,       /* w_i / factor (positions interpolated) */
    SK_ROPE_BASE = 2,         /* base * factor^(rot_dim / (rot_dim - 2)) in place of base */
    SK_ROPE_BANDS = 3         /* by the turns r = original_len * w_i / (2 pi) that a frequency makes in the trained
                                 context: w_i / factor up to `low` turns, w_i from `high` on, a linear blend between */
} sk_rope_scaling;

/* Frequencies of the rotary positions, on the host, in 64 bits: freqs[rot_dim / 2] (host, caller-owned),
 * and in *attn_factor (may be NULL) the factor that goes with them (0.1 ln(factor) + 1 for
 * SK_ROPE_BANDS, else 1).  original_len, low and high are read for SK_ROPE_BANDS only.
 * Returns SK_OK, or SK_ERR_INVALID (odd rot_dim, base <= 1, factor < 1, high <= low). */
int sk_rope_frequencies(int rot_dim, double base, int scaling, double factor, double original_len, double low,
                        double high, double *freqs, double *attn_factor);

/* Rotary positions with the KV write: turns this step's q and k, and stores k and v like
 * sk_reshape_and_cache.
 *
 * For token t at position p = positions[t], pair i < rot_dim / 2 of a head is elements (2 i, 2 i + 1)
 * (interleaved != 0) or (i, i + rot_dim / 2), and
 *   a' = attn_factor (a cos(p w_i) - b sin(p w_i)),  b' = attn_factor (b cos(p w_i) + a sin(p w_i))
 * with w_i = freqs[i] radians per position; elements from rot_dim on pass through unchanged.
 *   q_out[t]           every query head of q, turned
 *   kv_pages (slot t)  K: every KV head of key, turned; V: value; bf16 pages round once from the fp32
 *                      result, e4m3fn pages take the fp32 result divided by k_scale (v_scale)
 *                      and rounded like sk_reshape_and_cache
 *   acc_pages (slot t), pos_pages (slot t)  0 and p (its low 32 bits) for every KV head, where the arrays are given
 * A negative slot writes q_out only.  A slot at or past num_blocks * page_size writes q_out only and sets
 * SK_DEV_BAD_BLOCK.  Two tokens with the same slot leave that row undefined.  Angles are taken
 * in 64 bits modulo a revolution, so far positions lose no more than the rounding of freqs; positions may be
 * negative.
 *
 * Layouts (device, caller-owned): q bf16 [num_tokens, num_q_heads, 128] with q_stride elements between
 * tokens (heads contiguous; a view of a fused projection will do), key and value likewise with
 * num_kv_heads; strides are multiples of 8.  q_out is contiguous and may be q itself (when that is
 * contiguous).  positions, slot_mapping int64 [num_tokens]; freqs float64 [rot_dim / 2] (device);
 * rot_dim a multiple of 16 up to 128.  kv_pages as for sk_reshape_and_cache.  acc_pages fp32 and pos_pages
 * int32 [num_blocks, num_kv_heads, page_size], or NULL.  q, key, value, q_out and kv_pages are 16-byte
 * aligned.  Asynchronous on `stream`, no allocation, capture safe.
 * Returns SK_OK or a negative sk_status. */
int sk_rope_and_cache(const void *q, const void *key, const void *value, int64_t q_stride, int64_t key_stride,
                      int64_t value_stride, const int64_t *positions, const double *freqs, int rot_dim,
                      int interleaved, float attn_factor, const int64_t *slot_mapping, int num_tokens,
                      int num_q_heads, int num_kv_heads, int head_dim, void *q_out, void *kv_pages, int kv_dtype,
                      float k_scale, float v_scale, int num_blocks, int page_size, float *acc_pages,
                      int32_t *pos_pages, void *stream);

/* Axes of sk_rope_axes_and_cache at most. */
#define SK_MAX_AXES 4

/* Which axis turns each pair of a rotary embedding with several axes (such as time, height and width), on the host:
 * axes[rot_dim / 2] (host, caller-owned).  sections[a], a < num_axes, is how many pairs axis a has; they add up to
 * rot_dim / 2.  cycled == 0: the axes' pairs follow one another (axis 0 has the first sections[0]).  cycled != 0: pair i
 * belongs to axis i mod num_axes while that axis has pairs left, and what is left at the end to axis 0.
 * Returns SK_OK, or SK_ERR_INVALID (odd rot_dim, sections that do not add up or, cycled, do not go round). */
int sk_rope_axes(int rot_dim, int num_axes, const int *sections, int cycled, uint8_t *axes);

/* The rotary write with several axes: sk_rope_and_cache where pair i of token t turns by the angle
 * p w_i with p = positions[axes[i]][t], its position on the pair's axis.  Text tokens have the same position on
 * every axis; an image or video patch has its place in the grid.
 *
 * positions int64 [num_axes][num_tokens] with positions_stride elements between axes (a view of a wider buffer will do;
 * 0 where all axes share one row of positions, as text does);
 * axes uint8 [rot_dim / 2] (device), from sk_rope_axes or the caller's own; 1 <= num_axes <= SK_MAX_AXES.  pos_pages, where
 * given, receives the position on axis 0.
 *
 * A cache that is evicted from needs the token's place in its sequence there: sk_evict_select takes the rows at or past
 * next_pos - recent for the latest, and of more of them than fit keeps the lower.  On a time axis all patches of an image
 * have one position, so that an image within `recent` can push out the text behind it.  So give the places an axis of
 * their own, the first, that turns no pair: positions [place, time, height, width] with sections {0, ...}, or with the
 * axes of sk_rope_axes plus 1, and next_pos in places.
 *
 * An axis of num_axes or more sets SK_DEV_BAD_SEQ, and its pair does not
 * turn (it is multiplied by attn_factor).  Everything else as for sk_rope_and_cache. */
int sk_rope_axes_and_cache(const void *q, const void *key, const void *value, int64_t q_stride, int64_t key_stride,
                           int64_t value_stride, const int64_t *positions, int64_t positions_stride, int num_axes,
                           const double *freqs, const uint8_t *axes, int rot_dim, int interleaved, float attn_factor,
                           const int64_t *slot_mapping, int num_tokens, int num_q_heads, int num_kv_heads,
                           int head_dim, void *q_out, void *kv_pages, int kv_dtype, float k_scale, float v_scale,
                           int num_blocks, int page_size, float *acc_pages, int32_t *pos_pages, void *stream);

/* Eviction of cached rows by gathered attention weight, first step: which rows stay.
 *
 * A sequence with L = seq_lens[s] > budget keeps `budget` rows of every KV head.  Row r of (s, h) has the
 * weight acc_pages and the position pos_pages at its place in the pages.  Rows with a position of at least
 * next_pos[s] - recent rank first (next_pos: the position that the sequence's next token will have), then
 * rows rank by weight, larger first; equal ranks go to the lower row; NaN ranks like -inf.  The first
 * `budget` rows stay.  (Positions that rise along a sequence have at most `recent` such rows.  Where they repeat, as on
 * the time axis of an image, there can be more than fit, and the lower rows stay, not the latest: see
 * sk_rope_axes_and_cache.)
 *   counts[s][h]                n = how many rows at or past `budget` stay
 *   src_rows[s][h][m], m < n    the m-th of them, ascending
 *   dst_rows[s][h][m], m < n    the m-th row below `budget` that does not stay, ascending
 *   new_lens[s]                 min(L, budget)
 * Entries from n on are left as they were.  sk_evict_move then moves src_rows[m] to dst_rows[m].  Rows
 * below `budget` that stay do not move, so the rows of a head are not in order of position after it; the
 * attention of this library does not depend on the order of rows that every query token sees.  A sequence
 * with L <= budget has n = 0.  Each sequence is ranked by itself: one whose blocks another sequence shares (a common
 * prefix) needs blocks of its own before it is evicted, see sk_evict_move.  L above max_seq_len (or below 0) sets SK_DEV_BAD_SEQ: n = 0, new_lens = L.
 * A row in a block outside [0, num_blocks) ranks like -inf and sets SK_DEV_BAD_BLOCK.
 *
 * acc_pages fp32, pos_pages int32 [num_blocks, num_kv_heads, page_size], 16-byte aligned; src_rows, dst_rows int32 [bs,
 * num_kv_heads, capacity], capacity >= sk_evict_capacity(budget, max_seq_len); counts int32 [bs,
 * num_kv_heads]; new_lens int32 [bs], not seq_lens itself.  max_seq_len: an upper bound on the lengths; it
 * sizes the launch.  0 <= recent <= budget.  Asynchronous on `stream`, no allocation,
 * capture safe, the same result whatever the timing.
 * Returns SK_OK or a negative sk_status. */
int sk_evict_select(const float *acc_pages, const int32_t *pos_pages, const int32_t *block_table,
                    int block_table_stride, int num_blocks, int page_size, const int32_t *seq_lens,
                    const int32_t *next_pos, int bs, int num_kv_heads, int budget, int recent, int max_seq_len,
                    int capacity, int32_t *src_rows, int32_t *dst_rows, int32_t *counts, int32_t *new_lens,
                    void *stream);

/* Smallest capacity of the move lists: max(1, min(budget, max_seq_len - budget)).  Host-only arithmetic;
 * SK_ERR_INVALID for budget < 1 or a negative length. */
int sk_evict_capacity(int budget, int max_seq_len);

/* Eviction, second step: for every (s, h) and m < counts[s][h], copies row src_rows[s][h][m] of the pages
 * (K and V of that head), of acc_pages and of pos_pages to row dst_rows[s][h][m].  All moves run at once,
 * so no row of the pages may be both a source and a destination and no destination may be listed twice, over all
 * sequences.  sk_evict_select's lists are so where the sequences share no blocks.  Where they do (a common prefix), the
 * moves of a sequence that is evicted overwrite rows that the others read, and moves of two sequences race; nothing
 * reports it.  So give a sequence over its budget its own copy of shared blocks first.  Sources keep their contents.  A row outside [0, block_table_stride *
 * page_size), or a count outside [0, capacity], sets SK_DEV_BAD_SEQ, a block outside [0, num_blocks)
 * SK_DEV_BAD_BLOCK; such a move is skipped (of a count above the capacity, the listed moves run).
 * kv_pages [num_blocks, num_kv_heads, 16, 256] bf16 or e4m3fn, 16-byte aligned.  Asynchronous on `stream`,
 * no allocation, capture safe.  Returns SK_OK or a negative sk_status. */
int sk_evict_move(const int32_t *src_rows, const int32_t *dst_rows, const int32_t *counts, int capacity, int bs,
                  int num_kv_heads, int head_dim, const int32_t *block_table, int block_table_stride, int num_blocks,
                  int page_size, void *kv_pages, int kv_dtype, float *acc_pages, int32_t *pos_pages, void *stream);

/* The whole attention call -- plan (use_plan != 0) or fixed split, split-KV
 * attention, merge -- without any device allocation, for callers that cannot
 * allocate: a host engine that owns all device memory through its own
 * allocator and forbids plug-ins to call cudaMalloc, or a C caller without a
 * caching allocator that cannot afford cudaMalloc/cudaFree (which may
 * synchronise the device) in a serving step.  The pages have no counterpart
 * to this call; it exists for those callers only.
 *
 * The caller passes inputs and outputs as for sk_build_plan,
 * sk_paged_decode_attn and sk_merge_segments (same meanings and layouts;
 * out bf16 [num_tokens, num_q_heads, 128], lse fp32 or NULL).  The plan,
 * per-token segment counts and segment partials live in one file-scope
 * device array of sk_static_scratch_bytes() = 32 MiB per GPU that loads the
 * library, held until exit.  A call needs about
 * num_tokens * seg_max * num_q_heads * 520 bytes plus the plan; larger calls
 * return SK_ERR_CAPACITY and launch nothing.  The plan is rebuilt on every
 * call (no plan cache).  All calls share the array and it keeps the last
 * call's contents (nothing in it needs to start at zero); calls whose kernels
 * overlap on the GPU race on it, so serialise them.  The first call on a
 * device looks up the array's address (cudaGetSymbolAddress, once per
 * device); make that first call before any stream capture.
 * Returns SK_OK or a negative sk_status. */
int sk_paged_decode_attention_static(const void *q, const void *kv_pages, int kv_dtype,
                                     float k_scale, float v_scale, const int32_t *block_table,
                                     int block_table_stride, int num_blocks, int page_size,
                                     const int32_t *seq_lens, const int32_t *cu_seqlens_q,
                                     int use_plan, int bs, int num_tokens, int max_q_len,
                                     int num_q_heads, int num_kv_heads, int head_dim,
                                     float sm_scale, int causal, int num_sms, int seg_max,
                                     void *out, float *lse, void *stream);

/* Size in bytes of the static scratch array used by
 * sk_paged_decode_attention_static. */
size_t sk_static_scratch_bytes(void);

/* Synchronise `stream`, read the device status word of the current device
 * and clear it when `clear` != 0.
 * Returns SK_ERR_TIMEOUT when SK_DEV_TIMEOUT is set (a bounded wait expired and
 * its work item was abandoned, so some partials and outputs of the calls since
 * the last clear are missing); otherwise the mask of SK_DEV_* bits, 0 when
 * clean; another negative sk_status if a CUDA call fails.  The whole mask read
 * by the last call on this thread, timeout bit included, is
 * sk_last_device_status(). */
int sk_get_device_status(void *stream, int clear);

/* The mask of SK_DEV_* bits that the last sk_get_device_status call on this
 * thread read (0 before the first call). */
int sk_last_device_status(void);

/* Limit, in SM clock cycles, of each wait of the attention kernels (decode and
 * verify, chunk attention, windowed attention, whose limit is at most the
 * default, attention weights) that can give up (for a copy to
 * land, a product to complete, another role to finish its part of a tile).
 * It applies to the launches made after the call;
 * cycles < 0 restores the default of 4e9 (about two seconds).  Returns the
 * previous limit.  Waits for work a CTA has already issued -- its copies and
 * products in flight, before the CTA exits -- keep the default whatever this
 * limit is.  This is a test hook: a limit far below the memory latency makes
 * waits expire in an unchanged kernel, so the timeout path (SK_DEV_TIMEOUT,
 * then SK_ERR_TIMEOUT from sk_get_device_status) can be exercised without
 * faulting or hanging anything.  Process-wide; not for concurrent use with
 * other calls. */
long long sk_set_wait_limit(long long cycles);

/* Message for the last negative status returned on this thread. */
const char *sk_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* SK_H_ */
