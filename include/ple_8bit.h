/*
 * ple_8bit.h - C ABI of libple's 8-bit decode operators on MI355X (gfx950):
 *   ple_rms_norm8      the residual's addition and RMS norm, out in 8 bits with a scale per token
 *   ple_w8_linear      products of 8-bit integers with scales per token and output channel
 *   ple_kv8_append     keys and values, rotated by position, into a paged 8-bit cache
 *   ple_kv8_read       the rows of new tokens back out of that cache
 *   ple_kv8_attention  attention over that cache (decode, verify windows, prefill chunks)
 *
 * The conventions of ple.h hold here too: error codes and ple_error_message(),
 * checks before any HIP call, caller-owned memory, calls that only enqueue on
 * `stream`, bf16 passed as uint16_t.  Device pointers are 16-byte aligned
 * unless a field says otherwise.  e4m3 is OCP float8 e4m3fn (0x7F and 0xFF
 * are NaN, there are no infinities, the largest value is 448).
 */
#ifndef PLE_8BIT_H
#define PLE_8BIT_H

#include "ple_fp4.h"

#ifdef __cplusplus
extern "C" {
#endif

#define PLE_W8_MAX_K 131056 /* the most inputs whose products fit 32 bits, to a multiple of 16 */

/*
 * Residual, RMS norm and quantisation of a token's row:
 *   h = bf16(x + residual)  (x itself without a residual)
 *   r = 1 / sqrt(mean(h^2) + eps),  u = h * weight,  a = max |u|
 *   scales[t] = a * r / 127,  codes[t][c] = round(127 * u[c] / a)  (to nearest, ties to even; 0 where a = 0)
 * so codes * scales stands for the normalised row, as ple_w8_linear takes it.
 * Each code is the nearest one of its exact quotient.  Sums are fp32.  A row
 * whose h or u holds a NaN or an infinity, or whose sum of squares or 127 * a
 * leaves fp32's range, has scale NaN and codes of zero.
 * x: device bf16, row t at x + t * x_stride elements (x_stride >= n, a
 * multiple of 8); residual, residual_out: device bf16 [T][n], both or neither
 * (NULL), residual_out = h; it may be residual, or x where x_stride is n;
 * weight: device bf16 [n]; codes: device [T][n]; scales: device fp32 [T],
 * 4-byte aligned.  n a multiple of 16 in 16 .. PLE_W8_MAX_K, eps > 0,
 * 0 <= T <= PLE_MAX_TOKENS.
 */
int ple_rms_norm8(const uint16_t* x, int64_t x_stride, const uint16_t* residual, const uint16_t* weight,
                  int64_t num_tokens, int32_t n, float eps, int8_t* codes, float* scales, uint16_t* residual_out,
                  void* stream);

/* A weight matrix W [out_dim][k_dim], W[o][i] = codes[o][i] * scales[o].  The library only reads it. */
typedef struct ple_w8_weight {
    const int8_t* codes; /* device [out_dim][k_dim] */
    const float* scales; /* device [out_dim], 4-byte aligned */
    int32_t out_dim;     /* O, 1 .. 2^24 */
    int32_t k_dim;       /* K, a multiple of 16 in 16 .. PLE_W8_MAX_K */
} ple_w8_weight;

/*
 * out[t][o] = bf16(sum_i(x[t][i] * codes[o][i]) * scales[o] * x_scales[t]),
 * the sum exact in 32-bit integers.  x: device 8-bit integers, row t at x + t *
 * x_stride (x_stride >= K, a multiple of 16, at most 2^22); x_scales: device
 * fp32 [T], 4-byte aligned; out: device bf16 [T][O].  0 <= T <= PLE_MAX_TOKENS
 * and ceil(T/64) * ceil(O/64) <= 2^22 (else PLE_ERR_UNSUPPORTED).
 */
int ple_w8_linear(const int8_t* x, int64_t x_stride, const float* x_scales, const ple_w8_weight* w, int64_t num_tokens,
                  uint16_t* out, void* stream);

/*
 * A paged cache of 8-bit keys and values.  Token j of a request lives in page
 * page_table[r][j / page_size] at place j % page_size; 16 places make a block,
 * and a block of a head shares one scale, for keys and for values:
 *   key[d] = e4m3(code) * k_scales[page][head][place / 16]
 * Scales of blocks that hold tokens are positive, within 2^-32 .. 2^32.
 */
typedef struct ple_kv8_cache {
    uint8_t* k_codes; /* device [num_pages][num_kv_heads][page_size/16][head_dim/16][16 tokens][16] */
    float* k_scales;  /* device [num_pages][num_kv_heads][page_size/16], 4-byte aligned */
    uint8_t* v_codes; /* device [num_pages][num_kv_heads][page_size/16][head_dim][16 tokens] */
    float* v_scales;
    int64_t num_pages;    /* >= 1; num_pages * num_kv_heads * page_size / 16 < 2^31 */
    int32_t num_kv_heads; /* 1 .. 1024 */
    int32_t page_size;    /* a multiple of 16, at most 65536 */
    int32_t head_dim;     /* D: 64, 128 or 256 */
    int32_t reserved;
} ple_kv8_cache;

/* One ragged batch, as ple_kv4_batch says (positions, pages, tokens of no request, hints). */
typedef ple_kv4_batch ple_kv8_batch;

/*
 * New keys and values into the cache, keys (and with q) queries rotated first,
 * as ple_kv4_append rotates them.  Of each block and head that gets tokens,
 * keys and values each for themselves, with x the call's new elements in it:
 *   s = the least power of two with max|x| <= 448 s (finite x alone; at least 2^-32, at most 2^32),
 *   or the scale that the block has, if that is larger and tokens of the request stand in the block before the new ones;
 *   code = e4m3(x / s) to nearest, ties to even, beyond 448 to 448; NaN for infinities and NaN.
 * Where the scale grows, the codes of those earlier tokens become
 * e4m3(value / s); between powers of two that changes only values below 2^-6 s.
 * Scales that this call makes are powers of two; one that a caller brought along
 * and that is not enters as fp32 quotients, x * (1 / s) and code * (its / s).
 * Tokens of the block behind the new ones are as good as gone (their scale may
 * have changed).  A page that the batch writes to in two places, of two requests
 * or twice in one's table row, holds unspecified values.  Other arguments as for ple_kv4_append.
 * max_request_tokens sizes the launch: of a request with more new tokens than it says the last ones may not be stored.
 */
int ple_kv8_append(const ple_kv8_cache* cache, const ple_kv8_batch* batch, const uint16_t* k, int64_t k_stride,
                   const uint16_t* v, int64_t v_stride, const uint16_t* q, int64_t q_stride, int32_t num_q_heads,
                   uint16_t* q_out, const float* inv_freq, int32_t rot_dim, int32_t interleaved, void* stream);

/* The new tokens' rows as the cache holds them, rounded to bf16: k_out, v_out device bf16 [T][num_kv_heads][D]. */
int ple_kv8_read(const ple_kv8_cache* cache, const ple_kv8_batch* batch, uint16_t* k_out, uint16_t* v_out,
                 void* stream);

/*
 * Causal attention of the new tokens over the cache; definition, arguments and
 * workspace as for ple_kv4_attention.  A NaN key makes NaN the rows that see
 * it, a NaN element of a value that element of them.  Weights are rounded to
 * fp16 or better: a token's part of an output element is off by at most 2^-11
 * of itself or 2^-27 of its value, whatever the other blocks' scales are.
 * (Where the scales of a request's blocks lie more than 2^6 apart, the call
 * goes through the tiles around them twice.)  As there, a few long prefills
 * beside many single tokens take less time as two calls (1000 tokens behind
 * 1000 and 16 single ones over 6000 each 215 us as one, 107 as two; over 100000
 * 3.1 ms and 0.6).
 */
int ple_kv8_attention(const uint16_t* q, int64_t q_stride, int32_t num_q_heads, const ple_kv8_cache* cache,
                      const ple_kv8_batch* batch, int32_t window, float scale, uint16_t* out, float* lse,
                      void* workspace, size_t workspace_bytes, void* stream);
size_t ple_kv8_attention_workspace_bytes(int32_t num_q_heads, const ple_kv8_cache* cache, const ple_kv8_batch* batch,
                                         int32_t window);

#ifdef __cplusplus
}
#endif

#endif /* PLE_8BIT_H */
