// Launch interface and device helpers of the 4-bit decode operators.
#pragma once

#include "ple_device.h"
#include "ple_fp4.h"

namespace ple {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// A launch holds below 2^32 threads along x.
constexpr int64_t kMostThreads = ((int64_t)1 << 32) - 1;

// The linear kernel of a call: the many-token or the few-token one, in token and feature tiles of a block.
struct W4Shape {
    bool many;
    int mt, nt;
};
W4Shape w4_linear_shape(int64_t T, int32_t out_dim, int32_t group);
hipError_t launch_w4_linear(const uint16_t* x, int64_t x_stride, const ple_w4_weight& w, int64_t T, uint16_t* out,
                            hipStream_t s);

struct Kv4AppendArgs {
    ple_kv4_cache cache;
    ple_kv4_batch batch;
    const uint16_t* src[3];  // q, k, v
    int64_t stride[3];
    uint16_t* q_out;
    const float* inv_freq;
    int32_t num_q_heads;  // 0: no queries
    int32_t rot_dim;
    int32_t interleaved;
};
hipError_t launch_kv4_append(const Kv4AppendArgs& a, hipStream_t s);
hipError_t launch_kv4_read(const ple_kv4_cache& cache, const ple_kv4_batch& batch, uint16_t* k_out, uint16_t* v_out,
                           hipStream_t s);

struct Kv4AttentionArgs {
    ple_kv4_cache cache;
    ple_kv4_batch batch;
    const uint16_t* q;
    int64_t q_stride;
    uint16_t* out;
    float* lse;       // or NULL
    float* part;      // partial outputs and their lse: [rows][splits] (splits > 1) or [2 flat][128]
    int32_t num_q_heads;
    int32_t group;    // query heads per key head
    int32_t window;   // 0: none
    float scale;
    int32_t rows;     // rows of a block's query tile
    int32_t waves;    // of a block
    int32_t tiles;    // query tiles per request and key head (grid)
    int32_t flat;     // blocks that share the work of a few query tiles evenly (0: a block per query tile and split)
    int32_t chunk;    // tokens of the cache per split
    int32_t splits;   // most splits of any query tile (grid)
};
// The plan part of the arguments (rows, waves, tiles, flat, chunk, splits), from sizes and hints alone.
void plan_kv4_attention(Kv4AttentionArgs& a);
size_t kv4_attention_part_bytes(const Kv4AttentionArgs& a);
// Most threads along x of the call's launches.
int64_t kv4_attention_threads(const Kv4AttentionArgs& a);
hipError_t launch_kv4_attention(const Kv4AttentionArgs& a, hipStream_t s);

// One 16-token group of the cache: its number ((page * heads + head) * page_size/16 + group in page), which
// times 8 D is its byte offset in codes and times D in scales, or -1 where the table names no page.
// `g` is the token's position / 16 and lies inside the table.
__host__ __device__ __forceinline__ int kv4_group(const ple_kv4_cache& c, const int32_t* __restrict__ table_row, int head,
                                         int g) {
    const int per_page = c.page_size >> 4;
    const int p = g / per_page;
    const int page = table_row[p];
    if (page < 0 || page >= c.num_pages) return -1;
    return (page * c.num_kv_heads + head) * per_page + (g - p * per_page);
}

// Request of token t and its position; -1 if the token stands nowhere: in no request's tokens (a padded batch; the last
// request's places past its length may be another's), before position 0 or past the table.
__device__ __forceinline__ int kv4_position(const ple_kv4_cache& c, const ple_kv4_batch& b, int64_t t, int& r) {
    r = find_request(b.query_start_loc, b.num_reqs, t);
    const int64_t from = b.query_start_loc[r], to = b.query_start_loc[r + 1];
    const int64_t p = (int64_t)b.seq_lens[r] - (to - t);
    return t < from || t >= to || p < 0 || p >= (int64_t)b.table_width * c.page_size ? -1 : (int)p;
}

}  // namespace ple
