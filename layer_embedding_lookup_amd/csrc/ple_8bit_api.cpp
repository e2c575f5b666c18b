// The C entry points of the 8-bit decode operators (ple_8bit.h): argument checks, then launches.
#include "ple_paged_checks.h"

using namespace ple;

namespace {

int validate_count(int64_t T) {
    if (T < 0 || T > PLE_MAX_TOKENS)
        return fail(PLE_ERR_INVALID_ARGUMENT, "num_tokens %lld outside 0..%d", (long long)T, PLE_MAX_TOKENS);
    return PLE_OK;
}

int validate_inputs(const char* name, int32_t n) {
    if (n < 16 || n > PLE_W8_MAX_K || n % 16 != 0)
        return fail(PLE_ERR_UNSUPPORTED, "%s %d is not a multiple of 16 in 16..%d", name, n, PLE_W8_MAX_K);
    return PLE_OK;
}

}  // namespace

extern "C" {

int ple_rms_norm8(const uint16_t* x, int64_t x_stride, const uint16_t* residual, const uint16_t* weight,
                  int64_t num_tokens, int32_t n, float eps, int8_t* codes, float* scales, uint16_t* residual_out,
                  void* stream) {
    int rc = validate_inputs("n", n);
    if (rc) return rc;
    rc = validate_count(num_tokens);
    if (rc) return rc;
    if (!(eps > 0.f) || eps > 1e30f) return fail(PLE_ERR_INVALID_ARGUMENT, "eps must be positive and at most 1e30");
    if ((residual == nullptr) != (residual_out == nullptr))
        return fail(PLE_ERR_INVALID_ARGUMENT, "residual and residual_out go together");
    if (num_tokens == 0) return ok();
    rc = check_rows("x", x, x_stride, n);
    if (rc) return rc;
    if (weight == nullptr || !aligned16(weight)) return fail(PLE_ERR_INVALID_ARGUMENT, "weight is NULL or not 16-byte aligned");
    if (codes == nullptr || !aligned16(codes)) return fail(PLE_ERR_INVALID_ARGUMENT, "codes is NULL or not 16-byte aligned");
    if (scales == nullptr || !aligned4(scales)) return fail(PLE_ERR_INVALID_ARGUMENT, "scales is NULL or misaligned");
    if (!aligned16(residual) || !aligned16(residual_out))
        return fail(PLE_ERR_INVALID_ARGUMENT, "residual or residual_out is not 16-byte aligned");
    if (residual_out == x && x_stride != n)
        return fail(PLE_ERR_INVALID_ARGUMENT, "residual_out is x, whose rows are %lld elements apart", (long long)x_stride);
    rc = check_device();
    if (rc) return rc;
    const RmsNorm8Args a = {x, x_stride, residual, weight, num_tokens, n, eps, codes, scales, residual_out};
    const hipError_t e = launch_rms_norm8(a, (hipStream_t)stream);
    return e == hipSuccess ? ok() : hip_fail(e, "rms_norm8 launch");
}

int ple_w8_linear(const int8_t* x, int64_t x_stride, const float* x_scales, const ple_w8_weight* w, int64_t num_tokens,
                  uint16_t* out, void* stream) {
    if (w == nullptr) return fail(PLE_ERR_INVALID_ARGUMENT, "weight descriptor is NULL");
    if (w->out_dim < 1 || w->out_dim > (1 << 24))
        return fail(PLE_ERR_INVALID_ARGUMENT, "out_dim %d outside 1..2^24", w->out_dim);
    int rc = validate_inputs("k_dim", w->k_dim);
    if (rc) return rc;
    if (w->codes == nullptr || !aligned16(w->codes))
        return fail(PLE_ERR_INVALID_ARGUMENT, "weight codes are NULL or not 16-byte aligned");
    if (w->scales == nullptr || !aligned4(w->scales))
        return fail(PLE_ERR_INVALID_ARGUMENT, "weight scales are NULL or misaligned");
    rc = validate_count(num_tokens);
    if (rc) return rc;
    if ((num_tokens + 63) / 64 * ((w->out_dim + 63) / 64) > (1 << 22))
        return fail(PLE_ERR_UNSUPPORTED, "w8_linear of %lld x %d outputs exceeds 2^22 tiles", (long long)num_tokens,
                    w->out_dim);
    if (num_tokens == 0) return ok();
    if (x == nullptr || !aligned16(x)) return fail(PLE_ERR_INVALID_ARGUMENT, "x is NULL or not 16-byte aligned");
    if (x_stride < w->k_dim || x_stride % 16 != 0 || x_stride > (1 << 22))
        return fail(PLE_ERR_INVALID_ARGUMENT, "x stride %lld is below %d, not a multiple of 16 or above 2^22",
                    (long long)x_stride, w->k_dim);
    if (x_scales == nullptr || !aligned4(x_scales)) return fail(PLE_ERR_INVALID_ARGUMENT, "x_scales is NULL or misaligned");
    if (out == nullptr || !aligned16(out)) return fail(PLE_ERR_INVALID_ARGUMENT, "out is NULL or not 16-byte aligned");
    rc = check_device();
    if (rc) return rc;
    const W8Args a = {x,  w->codes, x_scales, w->scales, (int32_t)num_tokens, w->k_dim, w->out_dim, (int32_t)x_stride,
                      out};
    const hipError_t e = launch_w8_linear(a, (hipStream_t)stream);
    return e == hipSuccess ? ok() : hip_fail(e, "w8_linear launch");
}

int ple_kv8_append(const ple_kv8_cache* cache, const ple_kv8_batch* batch, const uint16_t* k, int64_t k_stride,
                   const uint16_t* v, int64_t v_stride, const uint16_t* q, int64_t q_stride, int32_t num_q_heads,
                   uint16_t* q_out, const float* inv_freq, int32_t rot_dim, int32_t interleaved, void* stream) {
    int rc = check_append(cache, batch, k, k_stride, v, v_stride, q, q_stride, num_q_heads, q_out, inv_freq, rot_dim);
    if (rc) return rc;
    if (batch->num_tokens == 0) return ok();
    if (kv8_append_blocks(*cache, *batch, q != nullptr ? num_q_heads : 0) > kMostBlocks)
        return fail(PLE_ERR_UNSUPPORTED, "%d requests need a launch of more than 2^34 blocks", batch->num_reqs);
    rc = check_device();
    if (rc) return rc;
    const Kv8AppendArgs a = {*cache, *batch, {q, k, v}, {q_stride, k_stride, v_stride}, q_out, inv_freq,
                             q != nullptr ? num_q_heads : 0, rot_dim, interleaved != 0};
    const hipError_t e = launch_kv8_append(a, (hipStream_t)stream);
    return e == hipSuccess ? ok() : hip_fail(e, "kv8_append launch");
}

int ple_kv8_read(const ple_kv8_cache* cache, const ple_kv8_batch* batch, uint16_t* k_out, uint16_t* v_out,
                 void* stream) {
    int rc = check_read(cache, batch, k_out, v_out);
    if (rc) return rc;
    if (batch->num_tokens == 0) return ok();
    if (kv8_read_blocks(*cache, *batch) > kMostBlocks)
        return fail(PLE_ERR_UNSUPPORTED, "%d requests need a launch of more than 2^34 blocks", batch->num_reqs);
    rc = check_device();
    if (rc) return rc;
    const hipError_t e = launch_kv8_read(*cache, *batch, k_out, v_out, (hipStream_t)stream);
    return e == hipSuccess ? ok() : hip_fail(e, "kv8_read launch");
}

size_t ple_kv8_attention_workspace_bytes(int32_t num_q_heads, const ple_kv8_cache* cache, const ple_kv8_batch* batch,
                                         int32_t window) {
    Kv8AttentionArgs a;
    if (plan_attention(num_q_heads, cache, batch, window, &a, plan_kv8_attention, kv8_attention_threads) != PLE_OK ||
        batch->num_tokens == 0)
        return 0;
    return kv8_attention_part_bytes(a);
}

int ple_kv8_attention(const uint16_t* q, int64_t q_stride, int32_t num_q_heads, const ple_kv8_cache* cache,
                      const ple_kv8_batch* batch, int32_t window, float scale, uint16_t* out, float* lse,
                      void* workspace, size_t workspace_bytes, void* stream) {
    Kv8AttentionArgs a;
    int rc = plan_attention(num_q_heads, cache, batch, window, &a, plan_kv8_attention, kv8_attention_threads);
    if (rc) return rc;
    rc = check_attention(q, q_stride, cache, batch, num_q_heads, scale, out, lse, workspace, workspace_bytes,
                         batch->num_tokens == 0 ? 0 : kv8_attention_part_bytes(a));
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
    const hipError_t e = launch_kv8_attention(a, (hipStream_t)stream);
    return e == hipSuccess ? ok() : hip_fail(e, "kv8_attention launch");
}

}  // extern "C"
