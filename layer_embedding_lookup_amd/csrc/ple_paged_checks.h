// The argument checks that the paged caches' entry points share (ple_fp4_api.cpp, ple_8bit_api.cpp).
#pragma once

#include <string.h>

#include "ple_8bit_launch.h"
#include "ple_api.h"

namespace ple {

inline int validate_cache_memory(const ple_kv4_cache* c) {
    const void* p[4] = {c->k_codes, c->k_scales, c->v_codes, c->v_scales};
    for (const void* x : p)
        if (x == nullptr || !aligned16(x))
            return fail(PLE_ERR_INVALID_ARGUMENT, "cache codes or scales are NULL or not 16-byte aligned");
    if (c->k_scale == nullptr || c->v_scale == nullptr || !aligned4(c->k_scale) || !aligned4(c->v_scale))
        return fail(PLE_ERR_INVALID_ARGUMENT, "k_scale or v_scale is NULL or misaligned");
    return PLE_OK;
}

inline int validate_cache_memory(const ple_kv8_cache* c) {
    if (c->k_codes == nullptr || c->v_codes == nullptr || !aligned16(c->k_codes) || !aligned16(c->v_codes))
        return fail(PLE_ERR_INVALID_ARGUMENT, "cache codes are NULL or not 16-byte aligned");
    if (c->k_scales == nullptr || c->v_scales == nullptr || !aligned4(c->k_scales) || !aligned4(c->v_scales))
        return fail(PLE_ERR_INVALID_ARGUMENT, "k_scales or v_scales is NULL or misaligned");
    return PLE_OK;
}

template <class Cache>
int validate_cache(const Cache* c) {
    if (c == nullptr) return fail(PLE_ERR_INVALID_ARGUMENT, "cache descriptor is NULL");
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
        return fail(PLE_ERR_UNSUPPORTED, "head_dim %d is not 64, 128 or 256", c->head_dim);
    if (c->num_kv_heads < 1 || c->num_kv_heads > 1024)
        return fail(PLE_ERR_INVALID_ARGUMENT, "num_kv_heads %d outside 1..1024", c->num_kv_heads);
    if (c->page_size < 16 || c->page_size > 65536 || c->page_size % 16 != 0)
        return fail(PLE_ERR_UNSUPPORTED, "page_size %d is not a multiple of 16 in 16..65536", c->page_size);
    if (c->num_pages < 1 || c->num_pages >= ((int64_t)1 << 31) ||
        c->num_pages * c->num_kv_heads * (c->page_size / 16) >= ((int64_t)1 << 31))
        return fail(PLE_ERR_UNSUPPORTED, "%lld pages are none, or more than the cache can number",
                    (long long)c->num_pages);
    return validate_cache_memory(c);
}

template <class Cache>
int validate_batch(const ple_kv4_batch* b, const Cache* c) {
    if (b == nullptr) return fail(PLE_ERR_INVALID_ARGUMENT, "batch descriptor is NULL");
    if (b->num_tokens < 0 || b->num_tokens > PLE_MAX_TOKENS)
        return fail(PLE_ERR_INVALID_ARGUMENT, "num_tokens %lld outside 0..%d", (long long)b->num_tokens, PLE_MAX_TOKENS);
    if (b->num_reqs < 0) return fail(PLE_ERR_INVALID_ARGUMENT, "num_reqs < 0");
    if (b->num_reqs == 0 && b->num_tokens > 0)
        return fail(PLE_ERR_INVALID_ARGUMENT, "num_tokens > 0 with num_reqs == 0");
    if (b->max_request_tokens < 0 || b->max_seq_len < 0)
        return fail(PLE_ERR_INVALID_ARGUMENT, "max_request_tokens or max_seq_len < 0");
    if (b->num_tokens == 0) return PLE_OK;
    if (b->table_width < 1 || (int64_t)b->table_width * c->page_size >= ((int64_t)1 << 30))
        return fail(PLE_ERR_UNSUPPORTED, "a page table of %d pages of %d tokens covers none, or 2^30 tokens or more",
                    b->table_width, c->page_size);
    if (b->query_start_loc == nullptr || b->seq_lens == nullptr || b->page_table == nullptr ||
        !aligned4(b->query_start_loc) || !aligned4(b->seq_lens) || !aligned4(b->page_table))
        return fail(PLE_ERR_INVALID_ARGUMENT, "query_start_loc, seq_lens or page_table is NULL or misaligned");
    return PLE_OK;
}

inline int check_rows(const char* name, const uint16_t* p, int64_t stride, int64_t least) {
    if (p == nullptr || !aligned16(p)) return fail(PLE_ERR_INVALID_ARGUMENT, "%s is NULL or not 16-byte aligned", name);
    if (stride < least || stride % 8 != 0 || stride > ((int64_t)1 << 32))
        return fail(PLE_ERR_INVALID_ARGUMENT, "%s stride %lld is below %lld, not a multiple of 8 or above 2^32", name,
                    (long long)stride, (long long)least);
    return PLE_OK;
}

template <class Cache>
int validate_query_heads(int32_t hq, const Cache* c) {
    if (hq < 1 || hq > 1024 || hq % c->num_kv_heads != 0)
        return fail(PLE_ERR_INVALID_ARGUMENT, "num_q_heads %d outside 1..1024 or not a multiple of num_kv_heads %d", hq,
                    c->num_kv_heads);
    return PLE_OK;
}

// The checks that size the attention's launch and workspace, and its plan.
template <class Cache>
int plan_attention(int32_t num_q_heads, const Cache* cache, const ple_kv4_batch* batch, int32_t window,
                   PagedAttentionArgs<Cache>* a, void (*plan)(PagedAttentionArgs<Cache>&),
                   int64_t (*threads)(const PagedAttentionArgs<Cache>&)) {
    int rc = validate_cache(cache);
    if (rc) return rc;
    rc = validate_batch(batch, cache);
    if (rc) return rc;
    rc = validate_query_heads(num_q_heads, cache);
    if (rc) return rc;
    if (window < 0) return fail(PLE_ERR_INVALID_ARGUMENT, "window < 0");
    memset(a, 0, sizeof(*a));
    if (batch->num_tokens == 0) return PLE_OK;
    a->cache = *cache;
    a->batch = *batch;
    a->num_q_heads = num_q_heads;
    a->group = num_q_heads / cache->num_kv_heads;
    a->window = window < (1 << 30) ? window : 0;  // wider than any sequence: none
    plan(*a);
    if (threads(*a) > kMostThreads)
        return fail(PLE_ERR_UNSUPPORTED, "%d requests of up to %d query tiles need a launch of 2^32 threads or more; pass "
                    "max_request_tokens", batch->num_reqs, a->tiles);
    return PLE_OK;
}

// The rest of an attention call's checks; `need`: bytes of workspace by the plan.
template <class Cache>
int check_attention(const uint16_t* q, int64_t q_stride, const Cache* cache, const ple_kv4_batch* batch,
                    int32_t num_q_heads, float scale, const uint16_t* out, const float* lse, const void* workspace,
                    size_t workspace_bytes, size_t need) {
    if (!(scale > 0.f) || scale > 1e30f) return fail(PLE_ERR_INVALID_ARGUMENT, "scale must be positive and at most 1e30");
    if (batch->num_tokens == 0) return PLE_OK;
    int rc = check_rows("q", q, q_stride, (int64_t)num_q_heads * cache->head_dim);
    if (rc) return rc;
    if (out == nullptr || !aligned16(out)) return fail(PLE_ERR_INVALID_ARGUMENT, "out is NULL or not 16-byte aligned");
    if (lse != nullptr && !aligned4(lse)) return fail(PLE_ERR_INVALID_ARGUMENT, "lse is misaligned");
    if (need > 0 && (workspace == nullptr || !aligned16(workspace)))
        return fail(PLE_ERR_INVALID_ARGUMENT, "workspace is NULL or not 16-byte aligned");
    if (need > workspace_bytes)
        return fail(PLE_ERR_WORKSPACE, "workspace holds %zu bytes, %zu needed", workspace_bytes, need);
    return PLE_OK;
}

template <class Cache>
int check_append(const Cache* cache, const ple_kv4_batch* batch, const uint16_t* k, int64_t k_stride, const uint16_t* v,
                 int64_t v_stride, const uint16_t* q, int64_t q_stride, int32_t num_q_heads, const uint16_t* q_out,
                 const float* inv_freq, int32_t rot_dim) {
    int rc = validate_cache(cache);
    if (rc) return rc;
    rc = validate_batch(batch, cache);
    if (rc) return rc;
    const int D = cache->head_dim;
    if (rot_dim < 0 || rot_dim > D || rot_dim % 16 != 0)
        return fail(PLE_ERR_UNSUPPORTED, "rot_dim %d is not a multiple of 16 in 0..%d", rot_dim, D);
    if (rot_dim > 0 && (inv_freq == nullptr || !aligned4(inv_freq)))
        return fail(PLE_ERR_INVALID_ARGUMENT, "inv_freq is NULL or misaligned");
    if ((q == nullptr) != (q_out == nullptr)) return fail(PLE_ERR_INVALID_ARGUMENT, "q and q_out go together");
    if (q != nullptr) {
        rc = validate_query_heads(num_q_heads, cache);
        if (rc) return rc;
    }
    if (batch->num_tokens == 0) return PLE_OK;
    rc = check_rows("k", k, k_stride, (int64_t)cache->num_kv_heads * D);
    if (rc) return rc;
    rc = check_rows("v", v, v_stride, (int64_t)cache->num_kv_heads * D);
    if (rc) return rc;
    if (q != nullptr) {
        rc = check_rows("q", q, q_stride, (int64_t)num_q_heads * D);
        if (rc) return rc;
        if (!aligned16(q_out)) return fail(PLE_ERR_INVALID_ARGUMENT, "q_out is not 16-byte aligned");
        if (q_out == q) return fail(PLE_ERR_INVALID_ARGUMENT, "q_out must not alias q");
    }
    return PLE_OK;
}

template <class Cache>
int check_read(const Cache* cache, const ple_kv4_batch* batch, const uint16_t* k_out, const uint16_t* v_out) {
    int rc = validate_cache(cache);
    if (rc) return rc;
    rc = validate_batch(batch, cache);
    if (rc) return rc;
    if (batch->num_tokens == 0) return PLE_OK;
    if (k_out == nullptr || v_out == nullptr || !aligned16(k_out) || !aligned16(v_out))
        return fail(PLE_ERR_INVALID_ARGUMENT, "k_out or v_out is NULL or not 16-byte aligned");
    return PLE_OK;
}

}  // namespace ple
