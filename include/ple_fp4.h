/*
 * ple_fp4.h - C ABI of libple's 4-bit decode operators on MI355X (gfx950):
 *   ple_w4_linear      products with 4-bit weights and group scales
 *   ple_kv4_append     keys and values, rotated by position, into a paged 4-bit cache
 *   ple_kv4_read       the rows of new tokens back out of that cache
 *   ple_kv4_attention  attention over that cache (decode, verify windows, prefill chunks)
 *
 * The conventions of ple.h hold here too: error codes and ple_error_message(),
 * checks before any HIP call, caller-owned memory, calls that only enqueue on
 * `stream`, bf16 passed as uint16_t.  Device pointers are 16-byte aligned
 * unless a field says otherwise.
 *
 * 4-bit formats
 *   e2m1   sign, two exponent bits (bias 1), one mantissa bit: 0 .5 1 1.5 2 3 4 6
 *   codes  two per byte, element 2i in the low nibble of byte i
 *   e4m3   OCP float8 e4m3fn (0x7F and 0xFF are NaN)
 */
#ifndef PLE_FP4_H
#define PLE_FP4_H

#include "ple.h"

#ifdef __cplusplus
extern "C" {
#endif

#define PLE_W4_NVFP4 0 /* e2m1 codes, an e4m3 scale per 16 elements, one fp32 scale for the tensor */
#define PLE_W4_INT4 1  /* unsigned codes 0..15, a bf16 scale and optionally a zero point per group */

/*
 * A weight matrix W [out_dim][k_dim]:
 *   NVFP4: W[o][i] = e2m1(code) * e4m3(scales[o][i / 16]) * tensor_scale[0]
 *   INT4:  W[o][i] = (code - zero[o][i / group]) * bf16(scales[o][i / group])
 * The library only reads it, during the enqueued work.
 */
typedef struct ple_w4_weight {
    const uint8_t* codes;      /* device [out_dim][k_dim/2] */
    const void* scales;        /* device; NVFP4: uint8_t [out_dim][k_dim/16], 2-byte aligned;
                                  INT4: bf16 [out_dim][k_dim/group], 2-byte aligned */
    const uint8_t* zeros;      /* device, INT4: [out_dim][k_dim/group], values 0..15, any alignment;
                                  NULL = 8 everywhere.  NVFP4: NULL */
    const float* tensor_scale; /* device [1], 4-byte aligned, NVFP4; NULL for INT4 */
    int32_t format;            /* PLE_W4_* */
    int32_t out_dim;           /* O, 1 .. 2^24 */
    int32_t k_dim;             /* K, at most 2^20; a multiple of 32 (NVFP4) or of group (INT4) */
    int32_t group;             /* NVFP4: 16; INT4: 32, 64 or 128 */
} ple_w4_weight;

/*
 * out[t][o] = bf16(sum_i x[t][i] * W[o][i]), sums in fp32.
 * x: device bf16, row t at x + t * x_stride elements (x_stride >= K, a
 * multiple of 8); out: device bf16 [T][O].  0 <= T <= PLE_MAX_TOKENS and
 * ceil(T/64) * ceil(O/64) <= 2^22 (else PLE_ERR_UNSUPPORTED).  NVFP4
 * weights enter the products exactly and tensor_scale multiplies the fp32
 * sum.  INT4: code - zero enters exactly and the group scale multiplies the
 * group's fp32 sum.
 */
int ple_w4_linear(const uint16_t* x, int64_t x_stride, const ple_w4_weight* w, int64_t num_tokens, uint16_t* out,
                  void* stream);

/*
 * A paged cache of 4-bit keys and values.  Token j of a request lives in page
 * page_table[r][j / page_size] at place j % page_size:
 *   key[d] = e2m1(code) * e4m3(k_scales[page][head][place / 16][d / 16][place % 16]) * k_scale[head]
 * and values likewise.
 */
typedef struct ple_kv4_cache {
    uint8_t* k_codes;     /* device [num_pages][num_kv_heads][page_size][head_dim/2] */
    uint8_t* k_scales;    /* device [num_pages][num_kv_heads][page_size/16][head_dim/16][16] */
    uint8_t* v_codes;
    uint8_t* v_scales;
    const float* k_scale; /* device [num_kv_heads], 4-byte aligned, positive */
    const float* v_scale;
    int64_t num_pages;    /* >= 1; num_pages * num_kv_heads * page_size / 16 < 2^31 */
    int32_t num_kv_heads; /* 1 .. 1024 */
    int32_t page_size;    /* a multiple of 16, at most 65536 */
    int32_t head_dim;     /* D: 64, 128 or 256 */
    int32_t reserved;
} ple_kv4_cache;

/*
 * One ragged batch: request r has the new tokens [query_start_loc[r],
 * query_start_loc[r+1]) of the call's T and, with them, seq_lens[r] tokens in
 * all, so new token t stands at position seq_lens[r] - (query_start_loc[r+1] - t).
 * That holds for a request that runs past T too, whose first tokens the call
 * has, and for a sequence longer than its row of the page table covers.
 * Positions past what the row covers, and those whose table entry lies outside
 * [0, num_pages), are on no page: append drops what would go there, read gives
 * zeros and attention leaves those tokens out.  query_start_loc has to be
 * non-decreasing; tokens before query_start_loc[0] or from query_start_loc[R]
 * on (a batch padded to a captured graph's T) belong to no request: append
 * drops their keys and values and leaves their queries unrotated, read gives
 * zeros and attention rows that see nothing.
 */
typedef struct ple_kv4_batch {
    const int32_t* query_start_loc; /* device [R+1] */
    const int32_t* seq_lens;        /* device [R] */
    const int32_t* page_table;      /* device [R][table_width] */
    int64_t num_tokens;             /* 0 <= T <= PLE_MAX_TOKENS */
    int32_t num_reqs;               /* R >= 0 (R == 0 requires T == 0) */
    int32_t table_width;            /* >= 1; table_width * page_size < 2^30 */
    int32_t max_request_tokens;     /* hint, 0 = unknown: no request has more new tokens */
    int32_t max_seq_len;            /* hint, 0 = unknown: no seq_lens[r] is larger */
} ple_kv4_batch;                    /* a wrong hint gives unspecified results, never out-of-bounds accesses */

/*
 * New keys and values into the cache, keys and (with q) queries rotated first.
 * Element pairs of the first rot_dim of each head turn by the angle
 * position * inv_freq[i] (taken in 64 bits, rounded once to fp32):
 *   (a, b) -> (a cos - b sin, b cos + a sin)
 * with pairs (i, i + rot_dim/2), or (2i, 2i+1) if interleaved.  Queries are
 * rounded to bf16.  Keys and values are quantised by blocks x of 16, with g
 * the head's fp32 scale and each quotient rounded to nearest:
 *   s = e4m3(min(448, max|x| / (6 g)));  code = e2m1(x / (s g)), ties to the even code (zero where s g = 0)
 * q, k, v: device bf16, token t and head h at t * stride + h * D elements
 * (strides multiples of 8); q_out: device bf16 [T][num_q_heads][D], not q;
 * q and q_out NULL where no query is to be rotated.  inv_freq: device fp32
 * [rot_dim/2], 4-byte aligned; rot_dim a multiple of 16, 0 <= rot_dim <= D
 * (0: nothing turns, inv_freq may be NULL).
 */
int ple_kv4_append(const ple_kv4_cache* cache, const ple_kv4_batch* batch, const uint16_t* k, int64_t k_stride,
                   const uint16_t* v, int64_t v_stride, const uint16_t* q, int64_t q_stride, int32_t num_q_heads,
                   uint16_t* q_out, const float* inv_freq, int32_t rot_dim, int32_t interleaved, void* stream);

/* The new tokens' rows as the cache holds them: k_out, v_out device bf16 [T][num_kv_heads][D]. */
int ple_kv4_read(const ple_kv4_cache* cache, const ple_kv4_batch* batch, uint16_t* k_out, uint16_t* v_out,
                 void* stream);

/*
 * Causal attention of the new tokens over the cache.  Query head h reads key
 * head h / (num_q_heads / num_kv_heads); with p the token's position it sees
 * the tokens j <= p and, with window > 0, j > p - window:
 *   out[t][h] = bf16(sum_j softmax_j(scale * <q, key_j>) value_j),  lse[t][h] = log sum_j exp(scale * <q, key_j>)
 * A row that sees nothing gives zeros and lse = -inf.  Sums, maxima and
 * partial results are fp32; the weights of the value product are rounded to
 * fp16 (relative 2^-11).  q: device bf16, token t and head h at t * q_stride +
 * h * D elements (a multiple of 8); out: device bf16 [T][num_q_heads][D]; lse:
 * device fp32 [T][num_q_heads] or NULL.  num_q_heads a multiple of
 * num_kv_heads, at most 1024.  workspace: device memory of at least
 * ple_kv4_attention_workspace_bytes(...) bytes with the same arguments,
 * 16-byte aligned (may be NULL where that is 0); written before it is read.
 */
int ple_kv4_attention(const uint16_t* q, int64_t q_stride, int32_t num_q_heads, const ple_kv4_cache* cache,
                      const ple_kv4_batch* batch, int32_t window, float scale, uint16_t* out, float* lse,
                      void* workspace, size_t workspace_bytes, void* stream);
size_t ple_kv4_attention_workspace_bytes(int32_t num_q_heads, const ple_kv4_cache* cache, const ple_kv4_batch* batch,
                                         int32_t window);

#ifdef __cplusplus
}
#endif

#endif /* PLE_FP4_H */
