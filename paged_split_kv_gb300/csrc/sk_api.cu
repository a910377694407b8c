// C ABI of libsk: argument validation, the plan cache, the device status
// word and kernel dispatch.  See include/sk.h for the contract of each call.
#include <cuda_runtime.h>
#include <math.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <atomic>
#include <mutex>

#include "sk.h"
#include "sk_cache_ops.cuh"
#include "sk_internal.cuh"
#include "sk_window_cost.cuh"

namespace sk {

// One status word per device; kernels OR SK_DEV_* bits into it.
__device__ int g_device_status;

namespace {

thread_local char g_msg[512];

int fail(int code, const char *fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_msg, sizeof g_msg, fmt, ap);
    va_end(ap);
    return code;
}

int cuda_fail(cudaError_t e, const char *what)
{
    return fail(SK_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

constexpr int kMaxDevices = 64;
int *g_status_ptr[kMaxDevices];
std::mutex g_status_mutex;

// Address of this device's status word (looked up once per device).
// SM count of the current device, read once per device.
int sm_count(int *out)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return cuda_fail(e, "cudaGetDevice");
    if (dev < 0 || dev >= kMaxDevices)
        return fail(SK_ERR_UNSUPPORTED, "device ordinal %d out of range", dev);
    static std::atomic<int> cached[kMaxDevices];
    int v = cached[dev].load();
    if (v == 0) {
        e = cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess)
            return cuda_fail(e, "cudaDeviceGetAttribute(SM count)");
        cached[dev].store(v);
    }
    *out = v;
    return SK_OK;
}

int status_ptr(int **out)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return cuda_fail(e, "cudaGetDevice");
    if (dev < 0 || dev >= kMaxDevices)
        return fail(SK_ERR_UNSUPPORTED, "device ordinal %d out of range", dev);
    std::lock_guard<std::mutex> lock(g_status_mutex);
    if (g_status_ptr[dev] == nullptr) {
        void *p = nullptr;
        e = cudaGetSymbolAddress(&p, g_device_status);
        if (e != cudaSuccess)
            return cuda_fail(e, "cudaGetSymbolAddress(status)");
        g_status_ptr[dev] = static_cast<int *>(p);
    }
    *out = g_status_ptr[dev];
    return SK_OK;
}

// ---------------------------------------------------------------- plan cache
struct PlanKey {
    const void *seq_lens;
    uint64_t seq_lens_version;
    const void *cu_q;
    uint64_t cu_q_version;
    int bs, num_tokens, num_kv_heads, num_sms, seg_max;
    const void *plan;
    int plan_capacity;
    const void *tok_nseg;
    int capturing;
    int device;
};

bool same_key(const PlanKey &a, const PlanKey &b)
{
    return a.seq_lens == b.seq_lens && a.seq_lens_version == b.seq_lens_version && a.cu_q == b.cu_q &&
           a.cu_q_version == b.cu_q_version && a.bs == b.bs && a.num_tokens == b.num_tokens &&
           a.num_kv_heads == b.num_kv_heads && a.num_sms == b.num_sms && a.seg_max == b.seg_max &&
           a.plan == b.plan && a.plan_capacity == b.plan_capacity && a.tok_nseg == b.tok_nseg &&
           a.capturing == b.capturing && a.device == b.device;
}

constexpr int kCacheSlots = 8;
PlanKey g_cache[kCacheSlots];
int g_cache_used = 0;
int g_cache_next = 0;
std::mutex g_cache_mutex;
std::atomic<long long> g_plan_launches{0};

}  // namespace

int device_status_word(int **out) { return status_ptr(out); }

namespace {
std::atomic<long long> g_wait_limit{kDefaultWaitLimit};
thread_local int g_last_device_status = 0;

// Plan buffer length: the plan's T, then up to max(B, bs) work items, B = floor(num_sms /
// num_kv_heads) (SGLang PR 39172, Modifications: the total segment count is capped at
// num_CUs / kv_heads, and a batch with more non-empty sequences than that takes one each).
long long capacity_of(int bs, int num_kv_heads, int num_sms)
{
    const long long budget = (long long)num_sms / num_kv_heads;
    return 1 + (budget > bs ? budget : bs);
}
}  // namespace

long long wait_limit() { return g_wait_limit.load(); }

int set_error(int code, const char *msg) { return fail(code, "%s", msg); }

}  // namespace sk

using namespace sk;

extern "C" {

int sk_tile_tokens(void) { return kTile; }

int sk_fixed_nseg(int bs, int num_kv_heads, int num_sms, int seg_max)
{
    long long denom = (long long)bs * num_kv_heads;
    long long q = denom > 0 && num_sms > 0 ? (long long)num_sms / denom : 0;
    long long p = 0;
    if (q >= 1) {
        p = 1;
        while (p * 2 <= q)
            p *= 2;
    }
    if (p > seg_max)
        p = seg_max;
    return p < 1 ? 1 : (int)p;
}

const char *sk_last_error(void) { return g_msg; }

int sk_plan_capacity(int bs, int num_kv_heads, int num_sms)
{
    if (bs < 1 || bs > 32767 || num_kv_heads < 1 || num_sms < 1)
        return fail(SK_ERR_INVALID, "sk_plan_capacity: bs=%d num_kv_heads=%d num_sms=%d", bs, num_kv_heads,
                    num_sms);
    const long long c = capacity_of(bs, num_kv_heads, num_sms);
    if (c > 0x7FFFFFFFLL)
        return fail(SK_ERR_INVALID, "sk_plan_capacity: capacity overflows int");
    return (int)c;
}

long long sk_set_wait_limit(long long cycles)
{
    return g_wait_limit.exchange(cycles < 0 ? kDefaultWaitLimit : cycles);
}

int sk_last_device_status(void) { return g_last_device_status; }

void sk_plan_cache_reset(void)
{
    std::lock_guard<std::mutex> lock(g_cache_mutex);
    g_cache_used = 0;
    g_cache_next = 0;
}

long long sk_plan_launch_count(void) { return g_plan_launches.load(); }

int sk_build_plan(const int32_t *seq_lens, uint64_t seq_lens_version, const int32_t *cu_seqlens_q,
                  uint64_t cu_seqlens_q_version, int bs, int num_tokens, int num_kv_heads,
                  int num_sms, int seg_max, int32_t *plan, int plan_capacity, int32_t *tok_nseg,
                  void *stream)
{
    if (seq_lens == nullptr || cu_seqlens_q == nullptr || plan == nullptr)
        return fail(SK_ERR_INVALID, "sk_build_plan: null seq_lens, cu_seqlens_q or plan");
    if (bs < 1 || bs > 32767)
        return fail(SK_ERR_INVALID, "sk_build_plan: bs=%d outside [1, 32767]", bs);
    if (num_tokens < 0 || (num_tokens > 0 && tok_nseg == nullptr))
        return fail(SK_ERR_INVALID, "sk_build_plan: num_tokens=%d with tok_nseg=%p", num_tokens,
                    (void *)tok_nseg);
    if (num_kv_heads < 1 || num_sms < 1)
        return fail(SK_ERR_INVALID, "sk_build_plan: num_kv_heads=%d num_sms=%d", num_kv_heads, num_sms);
    if (seg_max < 1 || seg_max > 0xFFFF)
        return fail(SK_ERR_INVALID, "sk_build_plan: seg_max=%d outside [1, 65535]", seg_max);
    const int budget = num_sms / num_kv_heads;
    if (plan_capacity < capacity_of(bs, num_kv_heads, num_sms))
        return fail(SK_ERR_CAPACITY, "sk_build_plan: plan_capacity=%d < 1 + max(B=%d, bs=%d)",
                    plan_capacity, budget, bs);

    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    cudaError_t e = cudaStreamIsCapturing(st, &cap);
    if (e != cudaSuccess)
        return cuda_fail(e, "cudaStreamIsCapturing");
    int dev = 0;
    e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return cuda_fail(e, "cudaGetDevice");

    PlanKey key{seq_lens, seq_lens_version, cu_seqlens_q, cu_seqlens_q_version, bs, num_tokens,
                num_kv_heads, num_sms, seg_max, plan, plan_capacity, tok_nseg,
                cap != cudaStreamCaptureStatusNone ? 1 : 0, dev};
    {
        std::lock_guard<std::mutex> lock(g_cache_mutex);
        for (int i = 0; i < g_cache_used; ++i)
            if (same_key(g_cache[i], key))
                return SK_CACHED;
    }
    int *status = nullptr;
    int rc = status_ptr(&status);
    if (rc != SK_OK)
        return rc;
    e = launch_plan(seq_lens, cu_seqlens_q, bs, num_tokens, budget, seg_max, plan, plan_capacity,
                    tok_nseg, status, st);
    if (e != cudaSuccess)
        return cuda_fail(e, "plan kernel launch");
    g_plan_launches.fetch_add(1);
    {
        std::lock_guard<std::mutex> lock(g_cache_mutex);
        // a plan buffer holds one plan: drop entries that wrote to the same buffers
        int w = 0;
        for (int i = 0; i < g_cache_used; ++i)
            if (g_cache[i].plan != plan && g_cache[i].tok_nseg != tok_nseg)
                g_cache[w++] = g_cache[i];
        g_cache_used = w;
        if (g_cache_used < kCacheSlots) {
            g_cache[g_cache_used++] = key;
        } else {
            g_cache[g_cache_next] = key;
            g_cache_next = (g_cache_next + 1) % kCacheSlots;
        }
    }
    return SK_OK;
}

}  // extern "C"

namespace sk {

// Checks the arguments of an attention call and resolves the kernel's parameters; launches
// nothing.  *rp_out is the row tile of the launch, 0 when there is nothing to launch.
int prepare_attn(const void *q, const void *kv_pages, int kv_dtype, float k_scale, float v_scale,
                 const int32_t *block_table, int block_table_stride, int num_blocks, int page_size,
                 const int32_t *seq_lens, const int32_t *cu_seqlens_q, const int32_t *plan,
                 int plan_capacity, int bs, int num_tokens, int max_q_len, int num_q_heads,
                 int num_kv_heads, int head_dim, float sm_scale, int causal, int num_sms, int seg_max,
                 float *part_o, float *part_m, float *part_l, AttnParams *params, int *rp_out)
{
    if (q == nullptr || kv_pages == nullptr || block_table == nullptr || seq_lens == nullptr ||
        cu_seqlens_q == nullptr || part_o == nullptr || part_m == nullptr || part_l == nullptr)
        return fail(SK_ERR_INVALID, "sk_paged_decode_attn: null pointer argument");
    if (kv_dtype != SK_KV_BF16 && kv_dtype != SK_KV_FP8_E4M3)
        return fail(SK_ERR_INVALID, "sk_paged_decode_attn: kv_dtype=%d", kv_dtype);
    if (head_dim != kHeadDim)
        return fail(SK_ERR_UNSUPPORTED, "sk_paged_decode_attn: head_dim=%d (only 128)", head_dim);
    if (page_size != kPage)
        return fail(SK_ERR_UNSUPPORTED, "sk_paged_decode_attn: page_size=%d (only 16)", page_size);
    if (bs < 1 || bs > 32767)
        return fail(SK_ERR_INVALID, "sk_paged_decode_attn: bs=%d outside [1, 32767]", bs);
    if (num_tokens < 0 || max_q_len < 0 || (num_tokens > 0 && max_q_len < 1) || block_table_stride < 1 ||
        num_blocks < 1)
        return fail(SK_ERR_INVALID,
                    "sk_paged_decode_attn: num_tokens=%d max_q_len=%d stride=%d num_blocks=%d",
                    num_tokens, max_q_len, block_table_stride, num_blocks);
    if (num_q_heads < 1 || num_kv_heads < 1 || num_q_heads % num_kv_heads != 0)
        return fail(SK_ERR_INVALID, "sk_paged_decode_attn: %d query heads, %d kv heads", num_q_heads,
                    num_kv_heads);
    if (num_sms < 1 || seg_max < 1 || seg_max > 0xFFFF)
        return fail(SK_ERR_INVALID, "sk_paged_decode_attn: num_sms=%d seg_max=%d", num_sms, seg_max);
    if (!(sm_scale > 0.f) || (kv_dtype == SK_KV_FP8_E4M3 && !(k_scale > 0.f && v_scale > 0.f)))
        return fail(SK_ERR_INVALID, "sk_paged_decode_attn: scales must be positive");
    if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(kv_pages) |
         reinterpret_cast<uintptr_t>(part_o)) & 15)
        return fail(SK_ERR_INVALID, "sk_paged_decode_attn: q, kv_pages and part_o must be 16-byte aligned");
    int num_items;
    int fixed = 0;
    if (plan != nullptr) {
        const long long need = capacity_of(bs, num_kv_heads, num_sms);
        if (plan_capacity < need)
            return fail(SK_ERR_CAPACITY, "sk_paged_decode_attn: plan_capacity=%d < %lld", plan_capacity,
                        need);
        num_items = plan_capacity - 1;
    } else {
        fixed = sk_fixed_nseg(bs, num_kv_heads, num_sms, seg_max);
        num_items = bs * fixed;
    }
    const long long rows_ll = (long long)(num_q_heads / num_kv_heads) * max_q_len;
    const int rows_max = rows_ll > 0x7FFFFFFFLL ? 0x7FFFFFFF : (int)rows_ll;
    const int rp = attn_tc_rows(kv_dtype, rows_max, num_blocks, num_kv_heads);
    if (num_tokens > 0 && rp == 0)
        return fail(SK_ERR_UNSUPPORTED,
                    "sk_paged_decode_attn: %d rows per work item (G * max_q_len) or %d blocks x %d heads "
                    "exceed the kernel's limits (65536 rows; 2^30 block-heads)",
                    rows_max, num_blocks, num_kv_heads);
    const int row_blocks = rp > 0 ? (rows_max + rp - 1) / rp : 1;
    if ((long long)num_items * num_kv_heads * row_blocks > 0x7FFFFFFFLL)
        return fail(SK_ERR_INVALID, "sk_paged_decode_attn: grid too large");
    *rp_out = 0;
    if (num_tokens == 0)
        return SK_OK;

    int *status = nullptr;
    int rc = status_ptr(&status);
    if (rc != SK_OK)
        return rc;

    AttnParams &p = *params;
    p.q = static_cast<const uint16_t *>(q);
    p.kv = kv_pages;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.cu_q = cu_seqlens_q;
    p.plan = plan;
    p.part_o = part_o;
    p.part_m = part_m;
    p.part_l = part_l;
    p.status = status;
    p.num_blocks = num_blocks;
    p.bt_stride = block_table_stride;
    p.bs = bs;
    p.num_tokens = num_tokens;
    p.max_q_len = max_q_len;
    p.H_q = num_q_heads;
    p.H_kv = num_kv_heads;
    p.G = num_q_heads / num_kv_heads;
    p.seg_max = seg_max;
    p.fixed_nseg = fixed;
    p.num_items = num_items;
    p.causal = causal ? 1 : 0;
    const float log2e = 1.4426950408889634f;
    p.score_scale_log2 = sm_scale * (kv_dtype == SK_KV_FP8_E4M3 ? k_scale : 1.f) * log2e;
    p.v_scale = kv_dtype == SK_KV_FP8_E4M3 ? v_scale : 1.f;
    p.wait_limit = wait_limit();

    p.row_blocks = row_blocks;
    *rp_out = rp;
    return SK_OK;
}

// Checks the arguments of a merge call; launches nothing.
int check_merge(const float *part_o, const float *part_m, const float *part_l, const int32_t *tok_nseg,
                int fixed_nseg, int num_tokens, int num_q_heads, int head_dim, int seg_max, const void *out)
{
    if (part_o == nullptr || part_m == nullptr || part_l == nullptr || out == nullptr)
        return fail(SK_ERR_INVALID, "sk_merge_segments: null pointer argument");
    if (head_dim != kHeadDim)
        return fail(SK_ERR_UNSUPPORTED, "sk_merge_segments: head_dim=%d (only 128)", head_dim);
    if (num_tokens < 0 || num_q_heads < 1 || seg_max < 1 || seg_max > 0xFFFF)
        return fail(SK_ERR_INVALID, "sk_merge_segments: num_tokens=%d num_q_heads=%d seg_max=%d",
                    num_tokens, num_q_heads, seg_max);
    if (tok_nseg == nullptr && (fixed_nseg < 0 || fixed_nseg > seg_max))
        return fail(SK_ERR_INVALID, "sk_merge_segments: fixed_nseg=%d outside [0, seg_max]", fixed_nseg);
    if ((reinterpret_cast<uintptr_t>(part_o) & 15) || (reinterpret_cast<uintptr_t>(out) & 7))
        return fail(SK_ERR_INVALID, "sk_merge_segments: part_o must be 16-byte and out 8-byte aligned");
    return SK_OK;
}

int launch_prepared_attn(const AttnParams &p, int kv_dtype, int rp, void *stream)
{
    cudaError_t e = launch_attn_tc(p, kv_dtype, rp, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess)
        return cuda_fail(e, "attention kernel launch");
    return SK_OK;
}

}  // namespace sk

extern "C" {

int sk_paged_decode_attn(const void *q, const void *kv_pages, int kv_dtype, float k_scale,
                         float v_scale, const int32_t *block_table, int block_table_stride,
                         int num_blocks, int page_size, const int32_t *seq_lens,
                         const int32_t *cu_seqlens_q, const int32_t *plan, int plan_capacity,
                         int bs, int num_tokens, int max_q_len, int num_q_heads, int num_kv_heads,
                         int head_dim, float sm_scale, int causal, int num_sms, int seg_max,
                         float *part_o, float *part_m, float *part_l, void *stream)
{
    AttnParams p;
    int rp = 0;
    const int rc = prepare_attn(q, kv_pages, kv_dtype, k_scale, v_scale, block_table, block_table_stride,
                                num_blocks, page_size, seq_lens, cu_seqlens_q, plan, plan_capacity, bs,
                                num_tokens, max_q_len, num_q_heads, num_kv_heads, head_dim, sm_scale,
                                causal, num_sms, seg_max, part_o, part_m, part_l, &p, &rp);
    if (rc != SK_OK || rp == 0)
        return rc;
    return launch_prepared_attn(p, kv_dtype, rp, stream);
}

int sk_merge_segments(const float *part_o, const float *part_m, const float *part_l,
                      const int32_t *tok_nseg, int fixed_nseg, int num_tokens, int num_q_heads,
                      int head_dim, int seg_max, void *out, float *lse, void *stream)
{
    const int rc = check_merge(part_o, part_m, part_l, tok_nseg, fixed_nseg, num_tokens, num_q_heads,
                               head_dim, seg_max, out);
    if (rc != SK_OK)
        return rc;
    cudaError_t e = launch_merge(part_o, part_m, part_l, tok_nseg, fixed_nseg, num_tokens, num_q_heads,
                                 seg_max, static_cast<uint16_t *>(out), lse,
                                 static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess)
        return cuda_fail(e, "merge kernel launch");
    return SK_OK;
}

int sk_reshape_and_cache(const void *key, const void *value, const int64_t *slot_mapping,
                         int num_tokens, int num_kv_heads, int head_dim, void *kv_pages, int kv_dtype,
                         float k_scale, float v_scale, int num_blocks, int page_size, void *stream)
{
    if (num_tokens < 0 || num_kv_heads < 1 || num_blocks < 1)
        return fail(SK_ERR_INVALID, "sk_reshape_and_cache: num_tokens=%d num_kv_heads=%d num_blocks=%d",
                    num_tokens, num_kv_heads, num_blocks);
    if (kv_dtype != SK_KV_BF16 && kv_dtype != SK_KV_FP8_E4M3)
        return fail(SK_ERR_INVALID, "sk_reshape_and_cache: kv_dtype=%d", kv_dtype);
    if (head_dim != kHeadDim)
        return fail(SK_ERR_UNSUPPORTED, "sk_reshape_and_cache: head_dim=%d (only 128)", head_dim);
    if (page_size != kPage)
        return fail(SK_ERR_UNSUPPORTED, "sk_reshape_and_cache: page_size=%d (only 16)", page_size);
    if (kv_dtype == SK_KV_FP8_E4M3 && !(k_scale > 0.f && v_scale > 0.f && k_scale < INFINITY && v_scale < INFINITY))
        return fail(SK_ERR_INVALID, "sk_reshape_and_cache: scales must be positive and finite");
    if (num_tokens == 0)
        return SK_OK;
    if (key == nullptr || value == nullptr || slot_mapping == nullptr || kv_pages == nullptr)
        return fail(SK_ERR_INVALID, "sk_reshape_and_cache: null pointer argument");
    if ((reinterpret_cast<uintptr_t>(key) | reinterpret_cast<uintptr_t>(value) |
         reinterpret_cast<uintptr_t>(kv_pages)) & 15)
        return fail(SK_ERR_INVALID, "sk_reshape_and_cache: key, value and kv_pages must be 16-byte aligned");
    int *status = nullptr;
    int rc = status_ptr(&status);
    if (rc != SK_OK)
        return rc;
    int sms = 0;
    rc = sm_count(&sms);
    if (rc != SK_OK)
        return rc;
    cudaError_t e = launch_kv_write(static_cast<const uint16_t *>(key), static_cast<const uint16_t *>(value),
                                    slot_mapping, num_tokens, num_kv_heads, num_blocks, kv_pages, kv_dtype,
                                    k_scale, v_scale, status, sms, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess)
        return cuda_fail(e, "kv write kernel launch");
    return SK_OK;
}

int sk_std_to_shuffled(const void *kv_pages, int kv_dtype, const int32_t *block_ids, int num_ids,
                       int num_blocks, int num_kv_heads, int head_dim, int page_size, void *k_shuf,
                       void *v_shuf, void *stream)
{
    if (num_blocks < 1 || num_kv_heads < 1 || (block_ids != nullptr && num_ids < 0))
        return fail(SK_ERR_INVALID, "sk_std_to_shuffled: num_blocks=%d num_kv_heads=%d num_ids=%d", num_blocks,
                    num_kv_heads, num_ids);
    if (kv_dtype != SK_KV_BF16 && kv_dtype != SK_KV_FP8_E4M3)
        return fail(SK_ERR_INVALID, "sk_std_to_shuffled: kv_dtype=%d", kv_dtype);
    if (head_dim != kHeadDim)
        return fail(SK_ERR_UNSUPPORTED, "sk_std_to_shuffled: head_dim=%d (only 128)", head_dim);
    if (page_size != kPage)
        return fail(SK_ERR_UNSUPPORTED, "sk_std_to_shuffled: page_size=%d (only 16)", page_size);
    if (kv_pages == nullptr || k_shuf == nullptr || v_shuf == nullptr)
        return fail(SK_ERR_INVALID, "sk_std_to_shuffled: null pointer argument");
    if ((reinterpret_cast<uintptr_t>(kv_pages) | reinterpret_cast<uintptr_t>(k_shuf) |
         reinterpret_cast<uintptr_t>(v_shuf)) & 15)
        return fail(SK_ERR_INVALID, "sk_std_to_shuffled: kv_pages, k_shuf and v_shuf must be 16-byte aligned");
    if (block_ids != nullptr && num_ids == 0)
        return SK_OK;
    int *status = nullptr;
    int rc = status_ptr(&status);
    if (rc != SK_OK)
        return rc;
    int sms = 0;
    rc = sm_count(&sms);
    if (rc != SK_OK)
        return rc;
    cudaError_t e = launch_std_to_shuffled(kv_pages, kv_dtype, block_ids, num_ids, num_blocks, num_kv_heads, k_shuf,
                                           v_shuf, status, sms, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess)
        return cuda_fail(e, "shuffle kernel launch");
    return SK_OK;
}

static constexpr int kMaxStride = 1 << 26;       // blocks a sequence: row numbers stay below 2^30
static constexpr int kMaxPairs = 1 << 24;        // (sequence, KV head) pairs

int sk_rope_frequencies(int rot_dim, double base, int scaling, double factor, double original_len, double low,
                        double high, double *freqs, double *attn_factor)
{
    if (rot_dim < 2 || (rot_dim & 1) || freqs == nullptr)
        return fail(SK_ERR_INVALID, "sk_rope_frequencies: rot_dim=%d, freqs=%p", rot_dim, (void *)freqs);
    if (!(base > 1.0 && base < INFINITY) || !(factor >= 1.0 && factor < INFINITY))
        return fail(SK_ERR_INVALID, "sk_rope_frequencies: base=%g must exceed 1 and factor=%g be at least 1", base,
                    factor);
    if (scaling < SK_ROPE_PLAIN || scaling > SK_ROPE_BANDS)
        return fail(SK_ERR_INVALID, "sk_rope_frequencies: scaling=%d", scaling);
    if (scaling == SK_ROPE_BASE && rot_dim < 4)
        return fail(SK_ERR_INVALID, "sk_rope_frequencies: a rescaled base needs rot_dim of 4 or more");
    if (scaling == SK_ROPE_BANDS && !(original_len > 0.0 && original_len < INFINITY && low >= 0.0 && high > low &&
                                      high < INFINITY))
        return fail(SK_ERR_INVALID, "sk_rope_frequencies: original_len=%g low=%g high=%g", original_len, low, high);
    const double pi2 = 6.283185307179586476925;
    if (scaling == SK_ROPE_BASE)
        base *= pow(factor, (double)rot_dim / (rot_dim - 2));
    for (int i = 0; i < rot_dim / 2; ++i) {
        double w = pow(base, -2.0 * i / rot_dim);
        if (scaling == SK_ROPE_LINEAR) {
            w /= factor;
        } else if (scaling == SK_ROPE_BANDS) {
            double keep = (original_len * w / pi2 - low) / (high - low);
            keep = keep < 0.0 ? 0.0 : (keep > 1.0 ? 1.0 : keep);
            w = (1.0 - keep) * (w / factor) + keep * w;
        }
        freqs[i] = w;
    }
    if (attn_factor != nullptr)
        *attn_factor = scaling == SK_ROPE_BANDS ? 0.1 * log(factor) + 1.0 : 1.0;
    return SK_OK;
}

// Both rotary writes: `axes` NULL for the one with a single axis.
static int rope_call(const char *name, const void *q, const void *key, const void *value, int64_t q_stride,
                     int64_t key_stride, int64_t value_stride, const int64_t *positions, int64_t pos_stride,
                     int num_axes, const uint8_t *axes, const double *freqs, int rot_dim, int interleaved,
                     float attn_factor, const int64_t *slot_mapping, int num_tokens, int num_q_heads, int num_kv_heads,
                     int head_dim, void *q_out, void *kv_pages, int kv_dtype, float k_scale, float v_scale,
                     int num_blocks, int page_size, float *acc_pages, int32_t *pos_pages, void *stream)
{
    if (num_tokens < 0 || num_q_heads < 1 || num_kv_heads < 1 || num_blocks < 1)
        return fail(SK_ERR_INVALID, "%s: num_tokens=%d num_q_heads=%d num_kv_heads=%d num_blocks=%d", name,
                    num_tokens, num_q_heads, num_kv_heads, num_blocks);
    if (num_q_heads > (1 << 20) || num_kv_heads > (1 << 20))
        return fail(SK_ERR_UNSUPPORTED, "%s: %d query heads, %d kv heads", name, num_q_heads, num_kv_heads);
    if (kv_dtype != SK_KV_BF16 && kv_dtype != SK_KV_FP8_E4M3)
        return fail(SK_ERR_INVALID, "%s: kv_dtype=%d", name, kv_dtype);
    if (head_dim != kHeadDim)
        return fail(SK_ERR_UNSUPPORTED, "%s: head_dim=%d (only 128)", name, head_dim);
    if (page_size != kPage)
        return fail(SK_ERR_UNSUPPORTED, "%s: page_size=%d (only 16)", name, page_size);
    if (rot_dim < 16 || rot_dim > kHeadDim || rot_dim % 16 != 0)
        return fail(SK_ERR_UNSUPPORTED, "%s: rot_dim=%d (multiples of 16 up to 128)", name, rot_dim);
    if (!(attn_factor > 0.f && attn_factor < INFINITY))
        return fail(SK_ERR_INVALID, "%s: attn_factor must be positive and finite", name);
    if (kv_dtype == SK_KV_FP8_E4M3 && !(k_scale > 0.f && v_scale > 0.f && k_scale < INFINITY && v_scale < INFINITY))
        return fail(SK_ERR_INVALID, "%s: scales must be positive and finite", name);
    if (num_tokens == 0)
        return SK_OK;
    if (q == nullptr || key == nullptr || value == nullptr || positions == nullptr || freqs == nullptr ||
        slot_mapping == nullptr || q_out == nullptr || kv_pages == nullptr)
        return fail(SK_ERR_INVALID, "%s: null pointer argument", name);
    if (q_stride < (int64_t)num_q_heads * kHeadDim || key_stride < (int64_t)num_kv_heads * kHeadDim ||
        value_stride < (int64_t)num_kv_heads * kHeadDim || ((q_stride | key_stride | value_stride) & 7))
        return fail(SK_ERR_INVALID,
                    "%s: token strides %lld, %lld, %lld must cover the heads and be multiples of 8", name,
                    (long long)q_stride, (long long)key_stride, (long long)value_stride);
    if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(key) | reinterpret_cast<uintptr_t>(value) |
         reinterpret_cast<uintptr_t>(q_out) | reinterpret_cast<uintptr_t>(kv_pages)) & 15)
        return fail(SK_ERR_INVALID, "%s: q, key, value, q_out and kv_pages must be 16-byte aligned", name);
    int *status = nullptr;
    int sms = 0;
    int rc = status_ptr(&status);
    if (rc == SK_OK)
        rc = sm_count(&sms);
    if (rc != SK_OK)
        return rc;
    const auto *qp = static_cast<const uint16_t *>(q), *kp = static_cast<const uint16_t *>(key),
               *vp = static_cast<const uint16_t *>(value);
    auto *qo = static_cast<uint16_t *>(q_out);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int inter = interleaved ? 1 : 0;
    const cudaError_t e =
        axes == nullptr
            ? launch_rope_cache(qp, kp, vp, q_stride, key_stride, value_stride, positions, freqs, slot_mapping, num_tokens,
                                num_q_heads, num_kv_heads, rot_dim, inter, attn_factor, qo, kv_pages, kv_dtype, k_scale,
                                v_scale, num_blocks, acc_pages, pos_pages, status, sms, st)
            : launch_rope_axes(qp, kp, vp, q_stride, key_stride, value_stride, positions, pos_stride, num_axes, freqs,
                               axes, slot_mapping, num_tokens, num_q_heads, num_kv_heads, rot_dim, inter, attn_factor, qo,
                               kv_pages, kv_dtype, k_scale, v_scale, num_blocks, acc_pages, pos_pages, status, sms, st);
    if (e != cudaSuccess)
        return cuda_fail(e, "rope kernel launch");
    return SK_OK;
}

int sk_rope_and_cache(const void *q, const void *key, const void *value, int64_t q_stride, int64_t key_stride,
                      int64_t value_stride, const int64_t *positions, const double *freqs, int rot_dim,
                      int interleaved, float attn_factor, const int64_t *slot_mapping, int num_tokens,
                      int num_q_heads, int num_kv_heads, int head_dim, void *q_out, void *kv_pages, int kv_dtype,
                      float k_scale, float v_scale, int num_blocks, int page_size, float *acc_pages,
                      int32_t *pos_pages, void *stream)
{
    return rope_call("sk_rope_and_cache", q, key, value, q_stride, key_stride, value_stride, positions, 0, 1, nullptr,
                     freqs, rot_dim, interleaved, attn_factor, slot_mapping, num_tokens, num_q_heads, num_kv_heads,
                     head_dim, q_out, kv_pages, kv_dtype, k_scale, v_scale, num_blocks, page_size, acc_pages,
                     pos_pages, stream);
}

int sk_rope_axes(int rot_dim, int num_axes, const int *sections, int cycled, uint8_t *axes)
{
    if (rot_dim < 2 || (rot_dim & 1) || num_axes < 1 || num_axes > SK_MAX_AXES || sections == nullptr || axes == nullptr)
        return fail(SK_ERR_INVALID, "sk_rope_axes: rot_dim=%d num_axes=%d (1 to %d) sections=%p axes=%p", rot_dim,
                    num_axes, SK_MAX_AXES, (const void *)sections, (void *)axes);
    const int half = rot_dim / 2;
    long long total = 0;
    for (int a = 0; a < num_axes; ++a) {
        if (sections[a] < 0)
            return fail(SK_ERR_INVALID, "sk_rope_axes: section %d has %d pairs", a, sections[a]);
        total += sections[a];
    }
    if (total != half)
        return fail(SK_ERR_INVALID, "sk_rope_axes: the sections hold %lld pairs, rot_dim=%d has %d", total, rot_dim, half);
    if (!cycled) {
        for (int a = 0, i = 0; a < num_axes; ++a)
            for (int n = 0; n < sections[a]; ++n)
                axes[i++] = (uint8_t)a;
        return SK_OK;
    }
    // pair i belongs to axis i mod num_axes while that axis has pairs left, and to the first axis after that
    int count[SK_MAX_AXES] = {};
    for (int i = 0; i < half; ++i) {
        const int a = i % num_axes;
        axes[i] = (uint8_t)(i / num_axes < sections[a] ? a : 0);
        ++count[axes[i]];
    }
    for (int a = 0; a < num_axes; ++a)
        if (count[a] != sections[a])
            return fail(SK_ERR_INVALID, "sk_rope_axes: %d pairs cannot go round %d axes with %d for axis %d (the first "
                        "axis takes what is left, so it has at least as many as the others)", half, num_axes,
                        sections[a], a);
    return SK_OK;
}

int sk_rope_axes_and_cache(const void *q, const void *key, const void *value, int64_t q_stride, int64_t key_stride,
                           int64_t value_stride, const int64_t *positions, int64_t positions_stride, int num_axes,
                           const double *freqs, const uint8_t *axes, int rot_dim, int interleaved, float attn_factor,
                           const int64_t *slot_mapping, int num_tokens, int num_q_heads, int num_kv_heads,
                           int head_dim, void *q_out, void *kv_pages, int kv_dtype, float k_scale, float v_scale,
                           int num_blocks, int page_size, float *acc_pages, int32_t *pos_pages, void *stream)
{
    if (num_axes < 1 || num_axes > SK_MAX_AXES)
        return fail(SK_ERR_INVALID, "sk_rope_axes_and_cache: num_axes=%d (1 to %d)", num_axes, SK_MAX_AXES);
    if (positions_stride < num_tokens && positions_stride != 0 && num_axes > 1)
        return fail(SK_ERR_INVALID, "sk_rope_axes_and_cache: positions_stride=%lld is neither 0 nor num_tokens=%d or more",
                    (long long)positions_stride, num_tokens);
    if (axes == nullptr)
        return fail(SK_ERR_INVALID, "sk_rope_axes_and_cache: null pointer argument");
    return rope_call("sk_rope_axes_and_cache", q, key, value, q_stride, key_stride, value_stride, positions,
                     positions_stride, num_axes, axes, freqs, rot_dim, interleaved, attn_factor, slot_mapping,
                     num_tokens, num_q_heads, num_kv_heads, head_dim, q_out, kv_pages, kv_dtype, k_scale, v_scale,
                     num_blocks, page_size, acc_pages, pos_pages, stream);
}

int sk_evict_capacity(int budget, int max_seq_len)
{
    if (budget < 1 || max_seq_len < 0)
        return fail(SK_ERR_INVALID, "sk_evict_capacity: budget=%d max_seq_len=%d", budget, max_seq_len);
    const int over = max_seq_len > budget ? max_seq_len - budget : 0;
    return over < budget ? (over > 0 ? over : 1) : budget;
}

int sk_evict_select(const float *acc_pages, const int32_t *pos_pages, const int32_t *block_table,
                    int block_table_stride, int num_blocks, int page_size, const int32_t *seq_lens,
                    const int32_t *next_pos, int bs, int num_kv_heads, int budget, int recent, int max_seq_len,
                    int capacity, int32_t *src_rows, int32_t *dst_rows, int32_t *counts, int32_t *new_lens,
                    void *stream)
{
    if (bs < 1 || bs > 32767 || num_kv_heads < 1 || num_blocks < 1 || block_table_stride < 1)
        return fail(SK_ERR_INVALID, "sk_evict_select: bs=%d num_kv_heads=%d num_blocks=%d stride=%d", bs, num_kv_heads,
                    num_blocks, block_table_stride);
    if (page_size != kPage)
        return fail(SK_ERR_UNSUPPORTED, "sk_evict_select: page_size=%d (only 16)", page_size);
    if (budget < 1 || recent < 0 || recent > budget || max_seq_len < 0)
        return fail(SK_ERR_INVALID, "sk_evict_select: budget=%d, recent=%d (at most the budget), max_seq_len=%d",
                    budget, recent, max_seq_len);
    if ((long long)bs * num_kv_heads > kMaxPairs || block_table_stride > kMaxStride || max_seq_len > kMaxStride * kPage)
        return fail(SK_ERR_UNSUPPORTED, "sk_evict_select: %d sequences of %d heads (at most 2^24), %d blocks a sequence "
                    "(2^26), max_seq_len=%d (2^30)", bs, num_kv_heads, block_table_stride, max_seq_len);
    if (capacity < sk_evict_capacity(budget, max_seq_len))
        return fail(SK_ERR_CAPACITY, "sk_evict_select: capacity=%d below min(budget, max_seq_len - budget) = %d",
                    capacity, sk_evict_capacity(budget, max_seq_len));
    if (acc_pages == nullptr || pos_pages == nullptr || block_table == nullptr || seq_lens == nullptr ||
        next_pos == nullptr || src_rows == nullptr || dst_rows == nullptr || counts == nullptr || new_lens == nullptr)
        return fail(SK_ERR_INVALID, "sk_evict_select: null pointer argument");
    if ((reinterpret_cast<uintptr_t>(acc_pages) | reinterpret_cast<uintptr_t>(pos_pages)) & 15)
        return fail(SK_ERR_INVALID, "sk_evict_select: acc_pages and pos_pages must be 16-byte aligned");
    int *status = nullptr;
    int sms = 0;
    int rc = status_ptr(&status);
    if (rc == SK_OK)
        rc = sm_count(&sms);
    if (rc != SK_OK)
        return rc;
    cudaError_t e = launch_evict_select(acc_pages, pos_pages, block_table, block_table_stride, num_blocks, seq_lens,
                                        next_pos, bs, num_kv_heads, budget, recent, max_seq_len, capacity, src_rows,
                                        dst_rows, counts, new_lens, status, sms, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess)
        return cuda_fail(e, "eviction select kernel launch");
    return SK_OK;
}

int sk_evict_move(const int32_t *src_rows, const int32_t *dst_rows, const int32_t *counts, int capacity, int bs,
                  int num_kv_heads, int head_dim, const int32_t *block_table, int block_table_stride, int num_blocks,
                  int page_size, void *kv_pages, int kv_dtype, float *acc_pages, int32_t *pos_pages, void *stream)
{
    if (bs < 1 || bs > 32767 || num_kv_heads < 1 || num_blocks < 1 || block_table_stride < 1 || capacity < 1)
        return fail(SK_ERR_INVALID, "sk_evict_move: bs=%d num_kv_heads=%d num_blocks=%d stride=%d capacity=%d", bs,
                    num_kv_heads, num_blocks, block_table_stride, capacity);
    if (kv_dtype != SK_KV_BF16 && kv_dtype != SK_KV_FP8_E4M3)
        return fail(SK_ERR_INVALID, "sk_evict_move: kv_dtype=%d", kv_dtype);
    if (head_dim != kHeadDim)
        return fail(SK_ERR_UNSUPPORTED, "sk_evict_move: head_dim=%d (only 128)", head_dim);
    if (page_size != kPage)
        return fail(SK_ERR_UNSUPPORTED, "sk_evict_move: page_size=%d (only 16)", page_size);
    if ((long long)bs * num_kv_heads > kMaxPairs || block_table_stride > kMaxStride)
        return fail(SK_ERR_UNSUPPORTED, "sk_evict_move: %d sequences of %d heads (at most 2^24), %d blocks a sequence "
                    "(2^26)", bs, num_kv_heads, block_table_stride);
    if (src_rows == nullptr || dst_rows == nullptr || counts == nullptr || block_table == nullptr ||
        kv_pages == nullptr || acc_pages == nullptr || pos_pages == nullptr)
        return fail(SK_ERR_INVALID, "sk_evict_move: null pointer argument");
    if (reinterpret_cast<uintptr_t>(kv_pages) & 15)
        return fail(SK_ERR_INVALID, "sk_evict_move: kv_pages must be 16-byte aligned");
    int *status = nullptr;
    int sms = 0;
    int rc = status_ptr(&status);
    if (rc == SK_OK)
        rc = sm_count(&sms);
    if (rc != SK_OK)
        return rc;
    cudaError_t e = launch_evict_move(src_rows, dst_rows, counts, capacity, bs, num_kv_heads, block_table,
                                      block_table_stride, num_blocks, kv_pages, kv_dtype, acc_pages, pos_pages,
                                      status, sms, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess)
        return cuda_fail(e, "eviction move kernel launch");
    return SK_OK;
}

int64_t sk_prefill_workspace_bytes(int num_tokens, int num_q_heads, int kv_dtype)
{
    if (num_tokens < 0 || num_q_heads < 1 || (kv_dtype != SK_KV_BF16 && kv_dtype != SK_KV_FP8_E4M3))
        return fail(SK_ERR_INVALID, "sk_prefill_workspace_bytes: num_tokens=%d num_q_heads=%d kv_dtype=%d", num_tokens,
                    num_q_heads, kv_dtype);
    int sms = 0;
    const int rc = sm_count(&sms);
    return rc != SK_OK ? rc : prefill_workspace_bytes(num_tokens, num_q_heads, kv_dtype, sms);
}

// Attention of new tokens over the pages: the whole cache (window 0), or the last `window` rows and the first `sinks`.
static int chunk_call(const char *name, const void *q, const void *kv_pages, int kv_dtype, float k_scale, float v_scale,
                      const int32_t *block_table, int block_table_stride, int num_blocks, int page_size,
                      const int32_t *seq_lens, const int32_t *cu_seqlens_q, int bs, int num_tokens, int max_q_len,
                      int num_q_heads, int num_kv_heads, int head_dim, float sm_scale, int causal, int window,
                      int sinks, int max_seq_len, void *workspace, int64_t workspace_bytes, void *out, float *lse,
                      void *stream)
{
    if (kv_pages == nullptr || block_table == nullptr || seq_lens == nullptr || cu_seqlens_q == nullptr ||
        (num_tokens != 0 && (q == nullptr || out == nullptr)))       // arrays of no tokens may have no address
        return fail(SK_ERR_INVALID, "%s: null pointer argument", name);
    if (kv_dtype != SK_KV_BF16 && kv_dtype != SK_KV_FP8_E4M3)
        return fail(SK_ERR_INVALID, "%s: kv_dtype=%d", name, kv_dtype);
    if (head_dim != kHeadDim)
        return fail(SK_ERR_UNSUPPORTED, "%s: head_dim=%d (only 128)", name, head_dim);
    if (page_size != kPage)
        return fail(SK_ERR_UNSUPPORTED, "%s: page_size=%d (only 16)", name, page_size);
    if (bs < 1 || bs > 32767)
        return fail(SK_ERR_INVALID, "%s: bs=%d outside [1, 32767]", name, bs);
    if (num_tokens < 0 || max_q_len < 0 || (num_tokens > 0 && max_q_len < 1) || block_table_stride < 1 ||
        num_blocks < 1)
        return fail(SK_ERR_INVALID, "%s: num_tokens=%d max_q_len=%d stride=%d num_blocks=%d", name,
                    num_tokens, max_q_len, block_table_stride, num_blocks);
    if (num_q_heads < 1 || num_kv_heads < 1 || num_q_heads % num_kv_heads != 0)
        return fail(SK_ERR_INVALID, "%s: %d query heads, %d kv heads", name, num_q_heads, num_kv_heads);
    if (max_seq_len < 0)
        return fail(SK_ERR_INVALID, "%s: max_seq_len=%d", name, max_seq_len);
    if (!(sm_scale > 0.f && sm_scale < INFINITY) ||
        (kv_dtype == SK_KV_FP8_E4M3 && !(k_scale > 0.f && v_scale > 0.f && k_scale < INFINITY && v_scale < INFINITY)))
        return fail(SK_ERR_INVALID, "%s: scales must be positive and finite", name);
    if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(kv_pages) | reinterpret_cast<uintptr_t>(out) |
         reinterpret_cast<uintptr_t>(workspace)) & 15)
        return fail(SK_ERR_INVALID, "%s: q, kv_pages, out and workspace must be 16-byte aligned", name);
    const int G = num_q_heads / num_kv_heads;
    if ((long long)num_q_heads * max_q_len > 0x3FFFFFFFLL || (long long)num_q_heads * num_tokens > 0x7FFFFFFFLL ||
        (long long)num_blocks * num_kv_heads * 2 > 0x7FFFFFFFLL)
        return fail(SK_ERR_UNSUPPORTED, "%s: %d blocks of %d heads or %d query tokens of %d heads "
                    "exceed the kernel's limits (2^30)", name, num_blocks, num_kv_heads, max_q_len, num_q_heads);
    if (block_table_stride > kMaxStride || (long long)bs * num_kv_heads > kMaxPairs)
        return fail(SK_ERR_UNSUPPORTED, "%s: %d blocks a sequence (at most 2^26), %d sequences of %d "
                    "heads (2^24)", name, block_table_stride, bs, num_kv_heads);
    if (num_tokens == 0)
        return SK_OK;
    int *status = nullptr;
    int sms = 0;
    int rc = status_ptr(&status);
    if (rc == SK_OK)
        rc = sm_count(&sms);
    if (rc != SK_OK)
        return rc;
    const bool step = window > 0 && window_step_takes((long long)G * max_q_len);
    const int64_t need = step         ? window_step_workspace_bytes(G * max_q_len, sms)
                         : window > 0 ? window_chunk_workspace_bytes(num_tokens, num_q_heads, kv_dtype, sms)
                                      : prefill_workspace_bytes(num_tokens, num_q_heads, kv_dtype, sms);
    if (workspace == nullptr || workspace_bytes < need)
        return fail(SK_ERR_CAPACITY, "%s: workspace of %lld bytes, %lld needed", name,
                    (long long)workspace_bytes, (long long)need);
    const bool fp8 = kv_dtype == SK_KV_FP8_E4M3;
    auto fill = [&](auto &p) {
        p.q = static_cast<const uint16_t *>(q);
        p.kv = kv_pages;
        p.block_table = block_table;
        p.seq_lens = seq_lens;
        p.cu_q = cu_seqlens_q;
        p.out = static_cast<uint16_t *>(out);
        p.lse = lse;
        p.status = status;
        p.num_blocks = num_blocks;
        p.bt_stride = block_table_stride;
        p.bs = bs;
        p.num_tokens = num_tokens;
        p.max_q_len = max_q_len;
        p.H_q = num_q_heads;
        p.H_kv = num_kv_heads;
        p.G = G;
        p.score_scale_log2 = sm_scale * (fp8 ? k_scale : 1.f) * 1.4426950408889634f;
        p.v_scale = fp8 ? v_scale : 1.f;
    };
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (window > 0) {
        WindowParams p{};
        fill(p);
        p.window = rows_in_table(window, block_table_stride, kPage);
        p.sinks = rows_in_table(sinks, block_table_stride, kPage);
        p.wait_limit = (uint32_t)(wait_limit() < kDefaultWaitLimit ? wait_limit() : kDefaultWaitLimit);
        e = step ? launch_window_step(p, kv_dtype, max_seq_len, workspace, sms, st)
                 : launch_window_chunk(p, kv_dtype, max_seq_len, workspace, sms, st);
    } else {
        PrefillParams p{};
        fill(p);
        p.causal = causal ? 1 : 0;
        p.wait_limit = wait_limit();
        e = launch_prefill(p, kv_dtype, max_seq_len, workspace, sms, st);
    }
    if (e != cudaSuccess)
        return cuda_fail(e, "chunk attention kernel launch");
    return SK_OK;
}

int sk_paged_prefill_attn(const void *q, const void *kv_pages, int kv_dtype, float k_scale, float v_scale,
                          const int32_t *block_table, int block_table_stride, int num_blocks, int page_size,
                          const int32_t *seq_lens, const int32_t *cu_seqlens_q, int bs, int num_tokens, int max_q_len,
                          int num_q_heads, int num_kv_heads, int head_dim, float sm_scale, int causal, int max_seq_len,
                          void *workspace, int64_t workspace_bytes, void *out, float *lse, void *stream)
{
    return chunk_call("sk_paged_prefill_attn", q, kv_pages, kv_dtype, k_scale, v_scale, block_table,
                      block_table_stride, num_blocks, page_size, seq_lens, cu_seqlens_q, bs, num_tokens, max_q_len,
                      num_q_heads, num_kv_heads, head_dim, sm_scale, causal, 0, 0, max_seq_len, workspace,
                      workspace_bytes, out, lse, stream);
}

int64_t sk_window_workspace_bytes(int num_tokens, int num_q_heads, int num_kv_heads, int max_q_len, int kv_dtype)
{
    if (num_tokens < 0 || max_q_len < 0 || num_q_heads < 1 || num_kv_heads < 1 || num_q_heads % num_kv_heads != 0 ||
        (kv_dtype != SK_KV_BF16 && kv_dtype != SK_KV_FP8_E4M3))
        return fail(SK_ERR_INVALID, "sk_window_workspace_bytes: num_tokens=%d num_q_heads=%d num_kv_heads=%d max_q_len=%d "
                    "kv_dtype=%d", num_tokens, num_q_heads, num_kv_heads, max_q_len, kv_dtype);
    const long long rows = (long long)max_q_len * (num_q_heads / num_kv_heads);
    int sms = 0;
    const int rc = sm_count(&sms);
    if (rc != SK_OK)
        return rc;
    return window_step_takes(rows) ? window_step_workspace_bytes((int)rows, sms)
                                   : window_chunk_workspace_bytes(num_tokens, num_q_heads, kv_dtype, sms);
}

int sk_paged_window_attn(const void *q, const void *kv_pages, int kv_dtype, float k_scale, float v_scale,
                         const int32_t *block_table, int block_table_stride, int num_blocks, int page_size,
                         const int32_t *seq_lens, const int32_t *cu_seqlens_q, int bs, int num_tokens, int max_q_len,
                         int num_q_heads, int num_kv_heads, int head_dim, float sm_scale, int window, int sinks,
                         int max_seq_len, void *workspace, int64_t workspace_bytes, void *out, float *lse, void *stream)
{
    if (window < 1 || sinks < 0)
        return fail(SK_ERR_INVALID, "sk_paged_window_attn: window=%d (at least 1), sinks=%d (at least 0)", window, sinks);
    return chunk_call("sk_paged_window_attn", q, kv_pages, kv_dtype, k_scale, v_scale, block_table,
                      block_table_stride, num_blocks, page_size, seq_lens, cu_seqlens_q, bs, num_tokens, max_q_len,
                      num_q_heads, num_kv_heads, head_dim, sm_scale, 1, window, sinks, max_seq_len, workspace,
                      workspace_bytes, out, lse, stream);
}

int64_t sk_accum_workspace_bytes(int num_tokens, int num_q_heads, int num_kv_heads, int max_q_len, int kv_dtype)
{
    if (num_tokens < 0 || max_q_len < 0 || num_q_heads < 1 || num_kv_heads < 1 || num_q_heads % num_kv_heads != 0 ||
        (kv_dtype != SK_KV_BF16 && kv_dtype != SK_KV_FP8_E4M3))
        return fail(SK_ERR_INVALID, "sk_accum_workspace_bytes: num_tokens=%d num_q_heads=%d num_kv_heads=%d max_q_len=%d "
                    "kv_dtype=%d", num_tokens, num_q_heads, num_kv_heads, max_q_len, kv_dtype);
    return accum_workspace_bytes(num_tokens, num_q_heads, num_kv_heads, max_q_len, kv_dtype);
}

int sk_accum_attn_weights(const void *q, const void *kv_pages, int kv_dtype, float k_scale,
                          const int32_t *block_table, int block_table_stride, int num_blocks, int page_size,
                          const int32_t *seq_lens, const int32_t *cu_seqlens_q, int bs, int num_tokens, int max_q_len,
                          int num_q_heads, int num_kv_heads, int head_dim, float sm_scale, int causal,
                          const float *lse, float *acc_pages, void *workspace, int64_t workspace_bytes, void *stream)
{
    if (kv_pages == nullptr || block_table == nullptr || seq_lens == nullptr || cu_seqlens_q == nullptr ||
        acc_pages == nullptr || (num_tokens != 0 && (q == nullptr || lse == nullptr)))
        return fail(SK_ERR_INVALID, "sk_accum_attn_weights: null pointer argument");
    if (kv_dtype != SK_KV_BF16 && kv_dtype != SK_KV_FP8_E4M3)
        return fail(SK_ERR_INVALID, "sk_accum_attn_weights: kv_dtype=%d", kv_dtype);
    if (head_dim != kHeadDim)
        return fail(SK_ERR_UNSUPPORTED, "sk_accum_attn_weights: head_dim=%d (only 128)", head_dim);
    if (page_size != kPage)
        return fail(SK_ERR_UNSUPPORTED, "sk_accum_attn_weights: page_size=%d (only 16)", page_size);
    if (bs < 1 || bs > 32767)
        return fail(SK_ERR_INVALID, "sk_accum_attn_weights: bs=%d outside [1, 32767]", bs);
    if (num_tokens < 0 || max_q_len < 0 || (num_tokens > 0 && max_q_len < 1) || block_table_stride < 1 ||
        num_blocks < 1)
        return fail(SK_ERR_INVALID, "sk_accum_attn_weights: num_tokens=%d max_q_len=%d stride=%d num_blocks=%d",
                    num_tokens, max_q_len, block_table_stride, num_blocks);
    if (num_q_heads < 1 || num_kv_heads < 1 || num_q_heads % num_kv_heads != 0)
        return fail(SK_ERR_INVALID, "sk_accum_attn_weights: %d query heads, %d kv heads", num_q_heads, num_kv_heads);
    if (!(sm_scale > 0.f && sm_scale < INFINITY) ||
        (kv_dtype == SK_KV_FP8_E4M3 && !(k_scale > 0.f && k_scale < INFINITY)))
        return fail(SK_ERR_INVALID, "sk_accum_attn_weights: scales must be positive and finite");
    if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(kv_pages)) & 15)
        return fail(SK_ERR_INVALID, "sk_accum_attn_weights: q and kv_pages must be 16-byte aligned");
    if ((long long)num_blocks * num_kv_heads * 2 > 0x7FFFFFFFLL || (long long)num_q_heads * max_q_len > 0x3FFFFFFFLL)
        return fail(SK_ERR_UNSUPPORTED, "sk_accum_attn_weights: %d blocks of %d heads or %d query tokens of %d heads "
                    "exceed the kernel's limits (2^30)", num_blocks, num_kv_heads, max_q_len, num_q_heads);
    if (block_table_stride > kMaxStride || (long long)bs * num_kv_heads > kMaxPairs)
        return fail(SK_ERR_UNSUPPORTED, "sk_accum_attn_weights: %d blocks a sequence (at most 2^26), %d sequences of %d "
                    "heads (2^24)", block_table_stride, bs, num_kv_heads);
    const int64_t need = sk_accum_workspace_bytes(num_tokens, num_q_heads, num_kv_heads, max_q_len, kv_dtype);
    if (workspace_bytes < need || (need > 0 && workspace == nullptr))
        return fail(SK_ERR_CAPACITY, "sk_accum_attn_weights: workspace of %lld bytes, %lld needed",
                    (long long)workspace_bytes, (long long)need);
    if (reinterpret_cast<uintptr_t>(workspace) & 15)
        return fail(SK_ERR_INVALID, "sk_accum_attn_weights: workspace must be 16-byte aligned");
    if (num_tokens == 0)
        return SK_OK;
    int *status = nullptr;
    int sms = 0;
    int rc = status_ptr(&status);
    if (rc == SK_OK)
        rc = sm_count(&sms);
    if (rc != SK_OK)
        return rc;
    AccumParams p{};
    p.q = static_cast<const uint16_t *>(q);
    p.kv = kv_pages;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.cu_q = cu_seqlens_q;
    p.lse = lse;
    p.acc = acc_pages;
    p.status = status;
    p.num_blocks = num_blocks;
    p.bt_stride = block_table_stride;
    p.bs = bs;
    p.num_tokens = num_tokens;
    p.max_q_len = max_q_len;
    p.H_q = num_q_heads;
    p.H_kv = num_kv_heads;
    p.G = num_q_heads / num_kv_heads;
    p.causal = causal ? 1 : 0;
    p.score_scale_log2 = sm_scale * (kv_dtype == SK_KV_FP8_E4M3 ? k_scale : 1.f) * 1.4426950408889634f;
    p.wait_limit = wait_limit();
    cudaError_t e = launch_accum(p, kv_dtype, workspace, sms, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess)
        return cuda_fail(e, "attention weight kernel launch");
    return SK_OK;
}

int sk_get_device_status(void *stream, int clear)
{
    int *status = nullptr;
    int rc = status_ptr(&status);
    if (rc != SK_OK)
        return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int value = 0;
    cudaError_t e = cudaMemcpyAsync(&value, status, sizeof value, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess && clear)
        e = cudaMemsetAsync(status, 0, sizeof(int), st);
    if (e == cudaSuccess)
        e = cudaStreamSynchronize(st);
    if (e != cudaSuccess)
        return cuda_fail(e, "reading the device status word");
    g_last_device_status = value;
    if (value & SK_DEV_TIMEOUT)
        return fail(SK_ERR_TIMEOUT, "a bounded wait inside a kernel expired (device status 0x%x)", value);
    return value;
}

}  // extern "C"
