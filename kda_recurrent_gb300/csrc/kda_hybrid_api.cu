// C ABI of the operators beside KDA layers (linear attention with a decay for each head,
// paged attention of one token, cache eviction): argument checks on the host, then dispatch.
#include <math.h>

#include "kda_internal.cuh"

using namespace kda;

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int from_cuda(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

// What a cache's shape may be: 32-bit token positions and item counts, 64-bit cache offsets.
int cache_shape(int32_t batch, int32_t num_kv_heads, int32_t max_pages, int32_t page_size) {
    if (batch < 0 || num_kv_heads < 1 || max_pages < 1 || page_size < 1) return KDA_ERR_INVALID_ARG;
    if (page_size < 8 || page_size > 1024 || (page_size & (page_size - 1)) != 0) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)max_pages * page_size > 0x3fffffffLL || (int64_t)batch * num_kv_heads > 0xffffffLL ||
        (int64_t)num_kv_heads * page_size * kHeadDim > 0x3fffffffLL)
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

int attn_shape(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads, int32_t max_pages, int32_t page_size) {
    if (num_q_heads < 1 || num_kv_heads < 1 || num_q_heads % num_kv_heads != 0) return KDA_ERR_INVALID_ARG;
    const int bad = cache_shape(batch, num_kv_heads, max_pages, page_size);
    if (bad != KDA_OK) return bad;
    return (int64_t)batch * num_q_heads > 0xffffffLL ? KDA_ERR_UNSUPPORTED : KDA_OK;
}

int linear_prefill_shape(int32_t num_seqs, int32_t total_tokens, int32_t num_heads) {
    if (num_seqs < 0 || total_tokens < 0 || num_heads < 1) return KDA_ERR_INVALID_ARG;
    if ((int64_t)total_tokens * num_heads > ((int64_t)1 << 40) / kHeadDim) return KDA_ERR_UNSUPPORTED;
    return (int64_t)num_seqs * num_heads > 0x7fffffffLL / kHeadDim ? KDA_ERR_UNSUPPORTED : KDA_OK;
}

// Checks the cache's sizes and pointers and fills `c`.
int paged_cache(PagedCache *c, void *k_cache, void *v_cache, int64_t k_page_stride, int64_t v_page_stride,
                int64_t num_pages, int32_t page_size, const int32_t *block_table, int32_t max_pages,
                const int32_t *seq_lens, int32_t batch, int32_t num_kv_heads) {
    if (num_pages < 1) return KDA_ERR_INVALID_ARG;
    const int bad = cache_shape(batch, num_kv_heads, max_pages, page_size);
    if (bad != KDA_OK) return bad;
    const int64_t page = (int64_t)num_kv_heads * page_size * kHeadDim;
    if (k_page_stride < page || v_page_stride < page) return KDA_ERR_INVALID_ARG;
    if (k_page_stride % 8 != 0 || v_page_stride % 8 != 0) return KDA_ERR_MISALIGNED;
    if (num_pages > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED;
    const int64_t stride = k_page_stride > v_page_stride ? k_page_stride : v_page_stride;
    if (stride > ((int64_t)1 << 60) / num_pages) return KDA_ERR_UNSUPPORTED;
    if (batch == 0) return KDA_OK;
    if (!k_cache || !v_cache || !block_table || !seq_lens) return KDA_ERR_INVALID_ARG;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(block_table, 4) || !aligned(seq_lens, 4))
        return KDA_ERR_MISALIGNED;
    c->k = static_cast<__nv_bfloat16 *>(k_cache);
    c->v = static_cast<__nv_bfloat16 *>(v_cache);
    c->k_page_stride = k_page_stride;
    c->v_page_stride = v_page_stride;
    c->num_pages = num_pages;
    c->block_table = block_table;
    c->seq_lens = seq_lens;
    c->batch = batch;
    c->num_kv_heads = num_kv_heads;
    c->max_pages = max_pages;
    c->page_size = page_size;
    c->page_shift = 0;
    while ((1 << c->page_shift) < page_size) ++c->page_shift;
    c->capacity = max_pages * page_size;
    return KDA_OK;
}

}  // namespace

extern "C" {

int kda_linear_prefill(const void *q, const void *k, const void *v, const float *log_decay, int32_t decay_per_token,
                       const int32_t *cu_seqlens, const float *init_state, void *out, float *final_state,
                       int32_t num_seqs, int32_t total_tokens, int32_t num_heads, float scale, void *workspace,
                       int64_t workspace_bytes, kda_stream_t stream) {
    if (!isfinite(scale) || (decay_per_token != 0 && decay_per_token != 1)) return KDA_ERR_INVALID_ARG;
    const int bad = linear_prefill_shape(num_seqs, total_tokens, num_heads);
    if (bad != KDA_OK) return bad;
    if (num_seqs == 0) return total_tokens == 0 ? KDA_OK : KDA_ERR_INVALID_ARG;
    if (cu_seqlens == nullptr) return KDA_ERR_INVALID_ARG;
    if (total_tokens > 0 && (!q || !k || !v || !log_decay || !out)) return KDA_ERR_INVALID_ARG;
    if (total_tokens == 0 && final_state == nullptr) return KDA_OK;
    const void *p16[] = {q, k, v, out, init_state, final_state, workspace};
    for (const void *p : p16)
        if (p && !aligned(p, 16)) return KDA_ERR_MISALIGNED;
    if (!aligned(log_decay, 4) || !aligned(cu_seqlens, 4)) return KDA_ERR_MISALIGNED;
    if (workspace != nullptr) {
        int32_t sms = 0;
        const int st = sm_count_of_current_device(&sms);
        if (st != KDA_OK) return st;
        if (workspace_bytes < linear_prefill_workspace_bytes(num_seqs, total_tokens, num_heads, sms))
            return KDA_ERR_INVALID_ARG;
    }
    LinearPrefillArgs a;
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.k = static_cast<const __nv_bfloat16 *>(k);
    a.v = static_cast<const __nv_bfloat16 *>(v);
    a.log_decay = log_decay;
    a.decay_token_stride = decay_per_token ? num_heads : 0;
    a.cu_seqlens = cu_seqlens;
    a.init_state = init_state;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.final_state = final_state;
    a.num_seqs = num_seqs;
    a.total_tokens = total_tokens;
    a.num_heads = num_heads;
    a.scale = scale;
    a.ws = workspace;
    if (device_status_ptr(&a.status) != cudaSuccess) return KDA_ERR_CUDA;
    return from_cuda(launch_linear_prefill(a, reinterpret_cast<cudaStream_t>(stream)));
}

int64_t kda_linear_prefill_workspace_size(int32_t num_seqs, int32_t total_tokens, int32_t num_heads,
                                          int32_t sm_count) {
    if (sm_count < 0) return KDA_ERR_INVALID_ARG;
    const int bad = linear_prefill_shape(num_seqs, total_tokens, num_heads);
    if (bad != KDA_OK) return bad;
    if (sm_count == 0) {
        const int st = sm_count_of_current_device(&sm_count);
        if (st != KDA_OK) return st;
    }
    return linear_prefill_workspace_bytes(num_seqs, total_tokens, num_heads, sm_count);
}

int kda_linear_decode(const void *q, const void *k, const void *v, const float *log_decay, int32_t decay_per_row,
                      const int32_t *slot_idx, void *state_pool, int64_t num_slots, int32_t state_dtype, void *out,
                      int32_t rows, int32_t num_heads, float scale, kda_stream_t stream) {
    if (rows < 0 || num_heads < 1 || num_slots < 1) return KDA_ERR_INVALID_ARG;
    if (state_dtype != KDA_STATE_F32 && state_dtype != KDA_STATE_BF16) return KDA_ERR_INVALID_ARG;
    if (!isfinite(scale) || (decay_per_row != 0 && decay_per_row != 1)) return KDA_ERR_INVALID_ARG;
    if ((int64_t)rows * num_heads > 0x7fffffffLL / 8) return KDA_ERR_UNSUPPORTED;
    if (num_slots > ((int64_t)1 << 62) / ((int64_t)num_heads * kHeadDim * kHeadDim * 4)) return KDA_ERR_UNSUPPORTED;
    if (rows == 0) return KDA_OK;
    if (!q || !k || !v || !log_decay || !slot_idx || !state_pool || !out) return KDA_ERR_INVALID_ARG;
    const void *p16[] = {q, k, v, out, state_pool};
    for (const void *p : p16)
        if (!aligned(p, 16)) return KDA_ERR_MISALIGNED;
    if (!aligned(log_decay, 4) || !aligned(slot_idx, 4)) return KDA_ERR_MISALIGNED;
    LinearDecodeArgs a;
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.k = static_cast<const __nv_bfloat16 *>(k);
    a.v = static_cast<const __nv_bfloat16 *>(v);
    a.log_decay = log_decay;
    a.decay_row_stride = decay_per_row ? num_heads : 0;
    a.slot_idx = slot_idx;
    a.state_pool = state_pool;
    a.num_slots = num_slots;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.rows = rows;
    a.num_heads = num_heads;
    a.state_dtype = state_dtype;
    a.scale = scale;
    if (device_status_ptr(&a.status) != cudaSuccess) return KDA_ERR_CUDA;
    return from_cuda(launch_linear_decode(a, reinterpret_cast<cudaStream_t>(stream)));
}

int64_t kda_attn_decode_workspace_size(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads, int32_t max_pages,
                                       int32_t page_size, int32_t with_weight, int32_t sm_count) {
    if (sm_count < 0) return KDA_ERR_INVALID_ARG;
    const int bad = attn_shape(batch, num_q_heads, num_kv_heads, max_pages, page_size);
    if (bad != KDA_OK) return bad;
    if (sm_count == 0) {
        const int st = sm_count_of_current_device(&sm_count);
        if (st != KDA_OK) return st;
    }
    return attn_decode_workspace_bytes(batch, num_q_heads, num_kv_heads, (int64_t)max_pages * page_size,
                                       with_weight != 0, sm_count);
}

int kda_attn_decode(const void *q, const void *k_cache, const void *v_cache, int64_t k_page_stride,
                    int64_t v_page_stride, int64_t num_pages, int32_t page_size, const int32_t *block_table,
                    int32_t max_pages, const int32_t *seq_lens, void *out, float *lse, float *weight, int32_t batch,
                    int32_t num_q_heads, int32_t num_kv_heads, float scale, void *workspace, int64_t workspace_bytes,
                    kda_stream_t stream) {
    if (!isfinite(scale)) return KDA_ERR_INVALID_ARG;
    int bad = attn_shape(batch, num_q_heads, num_kv_heads, max_pages, page_size);
    if (bad != KDA_OK) return bad;
    AttnDecodeArgs a;
    bad = paged_cache(&a.c, const_cast<void *>(k_cache), const_cast<void *>(v_cache), k_page_stride,
                                v_page_stride, num_pages, page_size, block_table, max_pages, seq_lens, batch,
                                num_kv_heads);
    if (bad != KDA_OK) return bad;
    if (batch == 0) return KDA_OK;
    if (!q || !out || !workspace) return KDA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 16) || !aligned(lse, 4) || !aligned(weight, 16))
        return KDA_ERR_MISALIGNED;
    int32_t sms = 0;
    const int st = sm_count_of_current_device(&sms);
    if (st != KDA_OK) return st;
    if (workspace_bytes < attn_decode_workspace_bytes(batch, num_q_heads, num_kv_heads, a.c.capacity,
                                                      weight != nullptr, sms))
        return KDA_ERR_INVALID_ARG;
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.lse = lse;
    a.weight = weight;
    a.num_q_heads = num_q_heads;
    a.group = num_q_heads / num_kv_heads;
    a.scale = scale;
    a.ws = workspace;
    if (device_status_ptr(&a.status) != cudaSuccess) return KDA_ERR_CUDA;
    return from_cuda(launch_attn_decode(a, reinterpret_cast<cudaStream_t>(stream)));
}

int kda_cache_evict(void *k_cache, void *v_cache, int64_t k_page_stride, int64_t v_page_stride, int64_t num_pages,
                    int32_t page_size, const int32_t *block_table, const int32_t *dst_table, int32_t max_pages,
                    const int32_t *seq_lens, const float *weight, float *dst_weight, int32_t *new_lens, int32_t *kept,
                    int32_t batch, int32_t num_kv_heads, int32_t budget, int32_t sink, int32_t recent,
                    kda_stream_t stream) {
    if (budget < 1 || sink < 0 || recent < 0 || (int64_t)sink + recent > budget) return KDA_ERR_INVALID_ARG;
    CacheEvictArgs a;
    const int bad = paged_cache(&a.c, k_cache, v_cache, k_page_stride, v_page_stride, num_pages, page_size,
                                block_table, max_pages, seq_lens, batch, num_kv_heads);
    if (bad != KDA_OK) return bad;
    if (batch == 0) return KDA_OK;
    if (!weight || !dst_weight || !new_lens || !kept) return KDA_ERR_INVALID_ARG;
    if (!aligned(weight, 16) || !aligned(dst_weight, 16) || !aligned(new_lens, 4) || !aligned(kept, 4) ||
        !aligned(dst_table, 4))
        return KDA_ERR_MISALIGNED;
    a.dst_table = dst_table ? dst_table : block_table;
    a.weight = weight;
    a.dst_weight = dst_weight;
    a.new_lens = new_lens;
    a.kept = kept;
    a.budget = budget;
    a.sink = sink;
    a.recent = recent;
    if (device_status_ptr(&a.status) != cudaSuccess) return KDA_ERR_CUDA;
    return from_cuda(launch_cache_evict(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
