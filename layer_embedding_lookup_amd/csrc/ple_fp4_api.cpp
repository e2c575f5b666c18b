// The C entry points of the 4-bit decode operators (ple_fp4.h): argument checks, then launches.
#include <string.h>

#include "ple_api.h"
#include "ple_fp4_launch.h"

using namespace ple;

namespace {

bool aligned2(const void* p) { return ((uintptr_t)p & 1u) == 0; }

int validate_weight(const ple_w4_weight* w) {
    if (w == nullptr) return fail(PLE_ERR_INVALID_ARGUMENT, "weight descriptor is NULL");
    if (w->format != PLE_W4_NVFP4 && w->format != PLE_W4_INT4)
        return fail(PLE_ERR_UNSUPPORTED, "weight format %d is not one of the PLE_W4_* formats", w->format);
    if (w->out_dim < 1 || w->out_dim > (1 << 24))
        return fail(PLE_ERR_INVALID_ARGUMENT, "out_dim %d outside 1..2^24", w->out_dim);
    if (w->k_dim < 1 || w->k_dim > (1 << 20)) return fail(PLE_ERR_INVALID_ARGUMENT, "k_dim %d outside 1..2^20", w->k_dim);
    const bool nv = w->format == PLE_W4_NVFP4;
    if (nv ? w->group != 16 : (w->group != 32 && w->group != 64 && w->group != 128))
        return fail(PLE_ERR_UNSUPPORTED, "group of %d elements (NVFP4: 16; INT4: 32, 64 or 128)", w->group);
    if (w->k_dim % (nv ? 32 : w->group) != 0)
        return fail(PLE_ERR_UNSUPPORTED, "k_dim %d is not a multiple of %d", w->k_dim, nv ? 32 : w->group);
    if (w->codes == nullptr || !aligned16(w->codes))
        return fail(PLE_ERR_INVALID_ARGUMENT, "weight codes are NULL or not 16-byte aligned");
    if (w->scales == nullptr || !aligned2(w->scales))
        return fail(PLE_ERR_INVALID_ARGUMENT, "weight scales are NULL or not 2-byte aligned");
    if (nv && (w->tensor_scale == nullptr || !aligned4(w->tensor_scale)))
        return fail(PLE_ERR_INVALID_ARGUMENT, "an NVFP4 weight needs a 4-byte aligned tensor_scale");
    if (nv && w->zeros != nullptr) return fail(PLE_ERR_INVALID_ARGUMENT, "an NVFP4 weight has no zero points");
    if (!nv && w->tensor_scale != nullptr) return fail(PLE_ERR_INVALID_ARGUMENT, "an INT4 weight has no tensor_scale");
    return PLE_OK;
}

int validate_cache(const ple_kv4_cache* c) {
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
    const void* p[4] = {c->k_codes, c->k_scales, c->v_codes, c->v_scales};
    for (const void* x : p)
        if (x == nullptr || !aligned16(x))
            return fail(PLE_ERR_INVALID_ARGUMENT, "cache codes or scales are NULL or not 16-byte aligned");
    if (c->k_scale == nullptr || c->v_scale == nullptr || !aligned4(c->k_scale) || !aligned4(c->v_scale))
        return fail(PLE_ERR_INVALID_ARGUMENT, "k_scale or v_scale is NULL or misaligned");
    return PLE_OK;
}

int validate_batch(const ple_kv4_batch* b, const ple_kv4_cache* c) {
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

int validate_rows(const char* name, const uint16_t* p, int64_t stride, int64_t least) {
    if (p == nullptr || !aligned16(p)) return fail(PLE_ERR_INVALID_ARGUMENT, "%s is NULL or not 16-byte aligned", name);
    if (stride < least || stride % 8 != 0 || stride > ((int64_t)1 << 32))
        return fail(PLE_ERR_INVALID_ARGUMENT, "%s stride %lld is below %lld, not a multiple of 8 or above 2^32", name,
                    (long long)stride, (long long)least);
    return PLE_OK;
}

int validate_query_heads(int32_t hq, const ple_kv4_cache* c) {
    if (hq < 1 || hq > 1024 || hq % c->num_kv_heads != 0)
        return fail(PLE_ERR_INVALID_ARGUMENT, "num_q_heads %d outside 1..1024 or not a multiple of num_kv_heads %d", hq,
                    c->num_kv_heads);
    return PLE_OK;
}

// The checks that size the attention's launch and workspace, and its plan.
int plan_attention(int32_t num_q_heads, const ple_kv4_cache* cache, const ple_kv4_batch* batch, int32_t window,
                   Kv4AttentionArgs* a) {
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
    plan_kv4_attention(*a);
    if (kv4_attention_threads(*a) > kMostThreads)
        return fail(PLE_ERR_UNSUPPORTED, "%d requests of up to %d query tiles need a launch of 2^32 threads or more; pass "
                    "max_request_tokens", batch->num_reqs, a->tiles);
    return PLE_OK;
}

}  // namespace

extern "C" {

int ple_w4_linear(const uint16_t* x, int64_t x_stride, const ple_w4_weight* w, int64_t num_tokens, uint16_t* out,
                  void* stream) {
    int rc = validate_weight(w);
    if (rc) return rc;
    if (num_tokens < 0 || num_tokens > PLE_MAX_TOKENS)
        return fail(PLE_ERR_INVALID_ARGUMENT, "num_tokens outside 0..%d", PLE_MAX_TOKENS);
    if ((num_tokens + 63) / 64 * ((w->out_dim + 63) / 64) > (1 << 22))
        return fail(PLE_ERR_UNSUPPORTED, "w4_linear of %lld x %d outputs exceeds 2^22 tiles", (long long)num_tokens,
                    w->out_dim);
    if (num_tokens == 0) return ok();
    rc = validate_rows("x", x, x_stride, w->k_dim);
    if (rc) return rc;
    if (out == nullptr || !aligned16(out)) return fail(PLE_ERR_INVALID_ARGUMENT, "out is NULL or not 16-byte aligned");
    rc = check_device();
    if (rc) return rc;
    const hipError_t e = launch_w4_linear(x, x_stride, *w, num_tokens, out, (hipStream_t)stream);
    return e == hipSuccess ? ok() : hip_fail(e, "w4_linear launch");
}

int ple_kv4_append(const ple_kv4_cache* cache, const ple_kv4_batch* batch, const uint16_t* k, int64_t k_stride,
                   const uint16_t* v, int64_t v_stride, const uint16_t* q, int64_t q_stride, int32_t num_q_heads,
                   uint16_t* q_out, const float* inv_freq, int32_t rot_dim, int32_t interleaved, void* stream) {
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
    if (batch->num_tokens == 0) return ok();
    rc = validate_rows("k", k, k_stride, (int64_t)cache->num_kv_heads * D);
    if (rc) return rc;
    rc = validate_rows("v", v, v_stride, (int64_t)cache->num_kv_heads * D);
    if (rc) return rc;
    if (q != nullptr) {
        rc = validate_rows("q", q, q_stride, (int64_t)num_q_heads * D);
        if (rc) return rc;
        if (!aligned16(q_out)) return fail(PLE_ERR_INVALID_ARGUMENT, "q_out is not 16-byte aligned");
        if (q_out == q) return fail(PLE_ERR_INVALID_ARGUMENT, "q_out must not alias q");
    }
    rc = check_device();
    if (rc) return rc;
    const Kv4AppendArgs a = {*cache, *batch, {q, k, v}, {q_stride, k_stride, v_stride}, q_out, inv_freq,
                             q != nullptr ? num_q_heads : 0, rot_dim, interleaved != 0};
    const hipError_t e = launch_kv4_append(a, (hipStream_t)stream);
    return e == hipSuccess ? ok() : hip_fail(e, "kv4_append launch");
}

int ple_kv4_read(const ple_kv4_cache* cache, const ple_kv4_batch* batch, uint16_t* k_out, uint16_t* v_out,
                 void* stream) {
    int rc = validate_cache(cache);
    if (rc) return rc;
    rc = validate_batch(batch, cache);
    if (rc) return rc;
    if (batch->num_tokens == 0) return ok();
    if (k_out == nullptr || v_out == nullptr || !aligned16(k_out) || !aligned16(v_out))
        return fail(PLE_ERR_INVALID_ARGUMENT, "k_out or v_out is NULL or not 16-byte aligned");
    rc = check_device();
    if (rc) return rc;
    const hipError_t e = launch_kv4_read(*cache, *batch, k_out, v_out, (hipStream_t)stream);
    return e == hipSuccess ? ok() : hip_fail(e, "kv4_read launch");
}

size_t ple_kv4_attention_workspace_bytes(int32_t num_q_heads, const ple_kv4_cache* cache, const ple_kv4_batch* batch,
                                         int32_t window) {
    Kv4AttentionArgs a;
    if (plan_attention(num_q_heads, cache, batch, window, &a) != PLE_OK || batch->num_tokens == 0) return 0;
    return kv4_attention_part_bytes(a);
}

int ple_kv4_attention(const uint16_t* q, int64_t q_stride, int32_t num_q_heads, const ple_kv4_cache* cache,
                      const ple_kv4_batch* batch, int32_t window, float scale, uint16_t* out, float* lse,
                      void* workspace, size_t workspace_bytes, void* stream) {
    Kv4AttentionArgs a;
    int rc = plan_attention(num_q_heads, cache, batch, window, &a);
    if (rc) return rc;
    if (!(scale > 0.f) || scale > 1e30f) return fail(PLE_ERR_INVALID_ARGUMENT, "scale must be positive and at most 1e30");
    if (batch->num_tokens == 0) return ok();
    rc = validate_rows("q", q, q_stride, (int64_t)num_q_heads * cache->head_dim);
    if (rc) return rc;
    if (out == nullptr || !aligned16(out)) return fail(PLE_ERR_INVALID_ARGUMENT, "out is NULL or not 16-byte aligned");
    if (lse != nullptr && !aligned4(lse)) return fail(PLE_ERR_INVALID_ARGUMENT, "lse is misaligned");
    const size_t need = kv4_attention_part_bytes(a);
    if (need > 0 && (workspace == nullptr || !aligned16(workspace)))
        return fail(PLE_ERR_INVALID_ARGUMENT, "workspace is NULL or not 16-byte aligned");
    if (need > workspace_bytes)
        return fail(PLE_ERR_WORKSPACE, "workspace holds %zu bytes, %zu needed", workspace_bytes, need);
    rc = check_device();
    if (rc) return rc;
    a.q = q;
    a.q_stride = q_stride;
    a.out = out;
    a.lse = lse;
    a.part = (float*)workspace;
    a.scale = scale;
    const hipError_t e = launch_kv4_attention(a, (hipStream_t)stream);
    return e == hipSuccess ? ok() : hip_fail(e, "kv4_attention launch");
}

}  // extern "C"
