// Launch interface of the 8-bit decode operators.
#pragma once

#include "ple_8bit.h"
#include "ple_fp4_launch.h"

namespace ple {

// `blocks` blocks: along x as many as a launch takes with room to spare, the rest along y (the last ones beyond them are
// the kernel's to turn away).
constexpr int64_t kBlocksAcross = 1 << 20;
inline dim3 block_grid(int64_t blocks) {
    return dim3((unsigned)(blocks < kBlocksAcross ? blocks : kBlocksAcross),
                (unsigned)((blocks + kBlocksAcross - 1) / kBlocksAcross));
}
__device__ __forceinline__ int64_t grid_block() { return blockIdx.x + blockIdx.y * kBlocksAcross; }

struct RmsNorm8Args {
    const uint16_t* x;
    int64_t x_stride;
    const uint16_t* residual;  // or NULL
    const uint16_t* weight;
    int64_t T;
    int32_t n;
    float eps;
    int8_t* codes;
    float* scales;
    uint16_t* residual_out;  // or NULL
};
// The kernel of a call: waves a row and chunks of 8 elements a lane; 0 waves: rows that registers do not hold.
struct RmsNorm8Shape {
    int waves, chunks;
};
RmsNorm8Shape rms_norm8_shape(int32_t n);
hipError_t launch_rms_norm8(const RmsNorm8Args& a, hipStream_t s);

struct W8Args {
    const int8_t* x;
    const int8_t* w;
    const float* x_scales;
    const float* w_scales;
    int32_t M, K, O;
    int32_t x_stride;
    uint16_t* out;
};
// The kernel of a call.  block = 256: tiles of 256 x 256; 64: tiles of `rows` x `nt` blocks of 64 x 64; 0: few tokens, `rows`
// rows of x and `nt` tiles of 16 features a block, `step` bytes of K a wave at a time.
struct W8Shape {
    int block, rows, nt, step;
};
W8Shape w8_linear_shape(int64_t T, int32_t out_dim);
hipError_t launch_w8_linear(const W8Args& a, hipStream_t s);

struct Kv8AppendArgs {
    ple_kv8_cache cache;
    ple_kv8_batch batch;
    const uint16_t* src[3];  // q, k, v
    int64_t stride[3];
    uint16_t* q_out;
    const float* inv_freq;
    int32_t num_q_heads;  // 0: no queries
    int32_t rot_dim;
    int32_t interleaved;
};
// Blocks of an append's or a read's launch.
constexpr int64_t kMostBlocks = (int64_t)1 << 34;
int64_t kv8_append_blocks(const ple_kv8_cache& cache, const ple_kv8_batch& batch, int32_t num_q_heads);
int64_t kv8_read_blocks(const ple_kv8_cache& cache, const ple_kv8_batch& batch);
hipError_t launch_kv8_append(const Kv8AppendArgs& a, hipStream_t s);
hipError_t launch_kv8_read(const ple_kv8_cache& cache, const ple_kv8_batch& batch, uint16_t* k_out, uint16_t* v_out,
                           hipStream_t s);

typedef PagedAttentionArgs<ple_kv8_cache> Kv8AttentionArgs;
// (the values' scales are in the weights)
__device__ __forceinline__ float value_scale(const Kv8AttentionArgs&, int) { return 1.0f; }
void plan_kv8_attention(Kv8AttentionArgs& a);
size_t kv8_attention_part_bytes(const Kv8AttentionArgs& a);
int64_t kv8_attention_threads(const Kv8AttentionArgs& a);
hipError_t launch_kv8_attention(const Kv8AttentionArgs& a, hipStream_t s);

}  // namespace ple
