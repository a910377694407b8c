// Launchers and parameters of the cache operators around the attention path: rotary write, chunk attention, gathered
// attention weights, eviction.
#pragma once

#include "sk_internal.cuh"

namespace sk {

// Chunk attention: a piece of a unit of work (two row tiles of one sequence and KV head), key tiles [a, b) of its t.
struct PrefillPiece {
    int s, h, unit, L, q_len, tok0;
    int t, a, b;
    int nA, nB;                  // tiles of [a, b) that row tiles A and B need
    int pad;
};

// Attention of a chunk of new tokens, resolved on the host.
struct PrefillParams {
    const uint16_t *q;           // bf16 bits [NT, H_q, D]
    const float *q_scale;        // e4m3 pages: 2^-e of each row of the split Q (set by the launcher)
    const void *kv;              // pages
    const int32_t *block_table, *seq_lens, *cu_q;
    uint16_t *out;               // bf16 bits [NT, H_q, D]
    float *lse;                  // [NT, H_q] or NULL
    float *part_o, *part_m, *part_l;   // partial states of the pieces (set by the launcher) ...
    PrefillPiece *shared;        // ... and what they are pieces of, two per run
    int *status;
    int64_t num_blocks;
    int bt_stride, bs, num_tokens, max_q_len;
    int H_q, H_kv, G;
    int gb, tpb, nsub;           // heads and tokens of a row tile, row tiles per token (set by the launcher)
    int deal;                    // whole units are dealt to the CTAs first (set by the launcher)
    int causal;
    float score_scale_log2;      // sm_scale * k_scale * log2(e)
    float v_scale;
    long long wait_limit;
};
long long prefill_workspace_bytes(int num_tokens, int H_q, int kv_dtype, int num_sms);
cudaError_t launch_prefill(const PrefillParams &p, int kv_dtype, long long max_seq_len, void *workspace, int num_sms,
                           cudaStream_t stream);

// A run's part of a unit that others share: the keys from tile a on of a sequence and head, and whether it has the unit's
// last rows.
struct AccumPiece {
    int s, h, a, ends;
};

// Gathered attention weights, resolved on the host.
struct AccumParams {
    const uint16_t *q;           // bf16 bits [NT, H_q, D]
    const float *q_scale;        // e4m3 pages: 2^-e of each row of the split Q (set by the launcher)
    const void *kv;              // pages
    const int32_t *block_table, *seq_lens, *cu_q;
    const float *lse;            // [NT, H_q]
    float *acc;                  // [NB, H_kv, 16]
    int *status;
    int64_t num_blocks;
    int bt_stride, bs, num_tokens, max_q_len;
    int H_q, H_kv, G;
    int gb, tpb, nsub;           // heads and tokens of a Q block, blocks per token (set by the launcher)
    int causal;
    float score_scale_log2;
    long long wait_limit;
    int runs, tail;              // equal shares of the cost, and short ones after them (set by the launcher)
    float *part;                 // workspace, set by the launcher: sums of shared units, and what they are parts of
    AccumPiece *shared;
};
long long accum_workspace_bytes(int num_tokens, int H_q, int H_kv, int max_q_len, int kv_dtype);
cudaError_t launch_accum(const AccumParams &p, int kv_dtype, void *workspace, int num_sms, cudaStream_t stream);

cudaError_t launch_rope_cache(const uint16_t *q, const uint16_t *k, const uint16_t *v, long long q_stride,
                              long long k_stride, long long v_stride, const int64_t *pos, const double *freqs,
                              const int64_t *slots, int num_tokens, int hq, int hkv, int rot, int interleaved,
                              float factor, uint16_t *q_out, void *pages, int kv_dtype, float k_scale, float v_scale,
                              long long num_blocks, float *acc, int32_t *pos_pages, int *status, int num_sms,
                              cudaStream_t stream);
cudaError_t launch_evict_select(const float *acc, const int32_t *pos, const int32_t *block_table, int bt_stride,
                                int num_blocks, const int32_t *seq_lens, const int32_t *next_pos, int bs, int hkv,
                                int budget, int recent, int max_len, int cap, int32_t *src, int32_t *dst,
                                int32_t *counts, int32_t *new_lens, int *status, int num_sms, cudaStream_t stream);
cudaError_t launch_evict_move(const int32_t *src, const int32_t *dst, const int32_t *counts, int cap, int bs, int hkv,
                              const int32_t *block_table, int bt_stride, int num_blocks, void *pages, int kv_dtype,
                              float *acc, int32_t *pos, int *status, int num_sms, cudaStream_t stream);

}  // namespace sk
