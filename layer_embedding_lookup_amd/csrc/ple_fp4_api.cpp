// The C entry points of the 4-bit decode operators (ple_fp4.h): argument checks, then launches.
#include "ple_paged_checks.h"

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
    rc = check_rows("x", x, x_stride, w->k_dim);
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
    int rc = check_append(cache, batch, k, k_stride, v, v_stride, q, q_stride, num_q_heads, q_out, inv_freq, rot_dim);
    if (rc) return rc;
    if (batch->num_tokens == 0) return ok();
    rc = check_device();
    if (rc) return rc;
    const Kv4AppendArgs a = {*cache, *batch, {q, k, v}, {q_stride, k_stride, v_stride}, q_out, inv_freq,
                             q != nullptr ? num_q_heads : 0, rot_dim, interleaved != 0};
    const hipError_t e = launch_kv4_append(a, (hipStream_t)stream);
    return e == hipSuccess ? ok() : hip_fail(e, "kv4_append launch");
}

int ple_kv4_read(const ple_kv4_cache* cache, const ple_kv4_batch* batch, uint16_t* k_out, uint16_t* v_out,
                 void* stream) {
    int rc = check_read(cache, batch, k_out, v_out);
    if (rc) return rc;
    if (batch->num_tokens == 0) return ok();
    rc = check_device();
    if (rc) return rc;
    const hipError_t e = launch_kv4_read(*cache, *batch, k_out, v_out, (hipStream_t)stream);
    return e == hipSuccess ? ok() : hip_fail(e, "kv4_read launch");
}

size_t ple_kv4_attention_workspace_bytes(int32_t num_q_heads, const ple_kv4_cache* cache, const ple_kv4_batch* batch,
                                         int32_t window) {
    Kv4AttentionArgs a;
    if (plan_attention(num_q_heads, cache, batch, window, &a, plan_kv4_attention, kv4_attention_threads) != PLE_OK ||
        batch->num_tokens == 0)
        return 0;
    return kv4_attention_part_bytes(a);
}

int ple_kv4_attention(const uint16_t* q, int64_t q_stride, int32_t num_q_heads, const ple_kv4_cache* cache,
                      const ple_kv4_batch* batch, int32_t window, float scale, uint16_t* out, float* lse,
                      void* workspace, size_t workspace_bytes, void* stream) {
    Kv4AttentionArgs a;
    int rc = plan_attention(num_q_heads, cache, batch, window, &a, plan_kv4_attention, kv4_attention_threads);
    if (rc) return rc;
    rc = check_attention(q, q_stride, cache, batch, num_q_heads, scale, out, lse, workspace, workspace_bytes,
                         batch->num_tokens == 0 ? 0 : kv4_attention_part_bytes(a));
    if (rc) return rc;
    if (batch->num_tokens == 0) return ok();
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
