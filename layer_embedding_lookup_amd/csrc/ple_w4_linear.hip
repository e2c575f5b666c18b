// Products with 4-bit weights: out = x W^T, W dequantised on the way to the
// matrix cores and never written out.
//
// Few tokens (decode): bound by reading W once.  A wave takes 16 output
// features and a share of K.  One 16-byte load per lane brings 32 codes of
// one feature, a wave 16 features x 128 inputs, which feed four 16x16x32 bf16
// MFMAs with the tokens as the first operand and the features as the second;
// so every lane's scales belong to its own feature lane % 16.  The waves of a
// block share the features, split K between them in steps of 128 and join
// their sums through LDS.
//  NVFP4: code * block scale is exact in bf16 (6 significant bits); the
//         tensor's scale multiplies the sum.
//  INT4:  code - zero is exact in bf16.  The four lanes of a feature swap
//         their words, so that an MFMA's 32 inputs lie in one group; the
//         group's sum is formed in the accumulator and its scale applied in
//         fp32.
#include "ple_fp4_launch.h"

namespace ple {

union BFrag {
    bf16x8 v;
    uint32_t u[4];
    u32x4 q;
};

// 8 e2m1 codes times s as bf16 (exact).
__device__ __forceinline__ void nvfp4_frag(uint32_t w, float s, BFrag& f) {
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
    const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
    const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
    const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
    f.u[0] = pack_bf16x2(a[0] * s, a[1] * s);
    f.u[1] = pack_bf16x2(b[0] * s, b[1] * s);
    f.u[2] = pack_bf16x2(c[0] * s, c[1] * s);
    f.u[3] = pack_bf16x2(d[0] * s, d[1] * s);
}

// 8 unsigned codes minus z as bf16 (exact).
__device__ __forceinline__ void int4_frag(uint32_t w, float z, BFrag& f) {
    const uint32_t lo = w & 0x0F0F0F0Fu, hi = (w >> 4) & 0x0F0F0F0Fu;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f.u[i] = pack_bf16x2((float)((lo >> (8 * i)) & 0xFFu) - z, (float)((hi >> (8 * i)) & 0xFFu) - z);
}

// 4 x 4 words between the four lanes n, n+16, n+32, n+48: word j of lane group g <-> word g of lane group j.
__device__ __forceinline__ void transpose4(u32x4& w) {
    typedef unsigned int u2 __attribute__((ext_vector_type(2)));
    // swap(a, b): the upper half of a with the lower half of b, over 32 lanes and then over 16
    u2 x = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    u2 y = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    u2 p = __builtin_amdgcn_permlane16_swap(x[0], y[0], false, false);
    u2 q = __builtin_amdgcn_permlane16_swap(x[1], y[1], false, false);
    w = u32x4{p[0], p[1], q[0], q[1]};
}

struct W4Args {
    const uint16_t* x;
    int64_t x_stride;
    const uint8_t* codes;
    const void* scales;
    const uint8_t* zeros;
    const float* tensor_scale;
    int64_t T;
    int32_t O, K;
    uint16_t* out;
};

// MT tiles of 16 tokens; G: 16 for NVFP4, else the INT4 group.
template <int MT, int G, int WAVES>
__device__ __forceinline__ void w4_rows_body(const W4Args& a) {
    constexpr bool kNv = G == 16;
    __shared__ __align__(16) float join[WAVES][MT][64][4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n = lane & 15, g = lane >> 4;
    const int tiles_o = (a.O + 15) / 16, o0 = (blockIdx.x % tiles_o) * 16;
    const int o = min(o0 + n, a.O - 1);  // features past the end repeat the last and are not stored
    const int64_t t0 = (int64_t)(blockIdx.x / tiles_o) * (16 * MT);
    const uint8_t* wrow = a.codes + (int64_t)o * (a.K / 2) + g * 16;
    const uint8_t* nvs = (const uint8_t*)a.scales + (int64_t)o * (a.K / 16) + g * 2;
    const uint16_t* i4s = (const uint16_t*)a.scales + (int64_t)o * (a.K / (kNv ? 32 : G));
    const uint8_t* i4z = a.zeros == nullptr ? nullptr : a.zeros + (int64_t)o * (a.K / (kNv ? 32 : G));
    const uint16_t* xrow[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int64_t t = t0 + mt * 16 + n;  // tokens past the end repeat the last and are not stored
        xrow[mt] = a.x + (t < a.T ? t : a.T - 1) * a.x_stride;
    }
    f32x4 acc[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) acc[mt] = f32x4{0.f, 0.f, 0.f, 0.f};

    for (int k0 = wave * 128; k0 < a.K; k0 += WAVES * 128) {
        // the last step may be short: lanes past K take zeros
        const bool in = k0 + g * 32 < a.K;
        u32x4 w = in ? *(const u32x4*)(wrow + k0 / 2) : u32x4{0u, 0u, 0u, 0u};
        if constexpr (kNv) {
            const uint32_t sc = in ? *(const uint16_t*)(nvs + k0 / 16) : 0u;
            const f32x2 s = __builtin_amdgcn_cvt_pk_f32_fp8((int)sc, false);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                BFrag f;
                nvfp4_frag(w[j], s[j >> 1], f);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    BFrag xf;
                    xf.q = in ? *(const u32x4*)(xrow[mt] + k0 + g * 32 + j * 8) : u32x4{0u, 0u, 0u, 0u};
                    acc[mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf.v, f.v, acc[mt], 0, 0, 0);
                }
            }
        } else {
            transpose4(w);  // word j: inputs k0 + 32 j + 8 g ..
            f32x4 part[MT];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = k0 + 32 * j;
                const bool live = k < a.K;  // the same for the whole wave
                const int at = live ? k / G : 0;
                const float z = i4z == nullptr ? 8.f : (float)i4z[at];
                BFrag f;
                int4_frag(w[j], z, f);
                if ((j * 32) % G == 0)
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) part[mt] = f32x4{0.f, 0.f, 0.f, 0.f};
                if (live)
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        BFrag xf;
                        xf.q = *(const u32x4*)(xrow[mt] + k + g * 8);
                        part[mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf.v, f.v, part[mt], 0, 0, 0);
                    }
                if ((j * 32 + 32) % G == 0 && live) {
                    const float s = bf16_lo(i4s[at]);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[mt][e] = fmaf(part[mt][e], s, acc[mt][e]);
                }
            }
        }
    }

#pragma unroll
    for (int mt = 0; mt < MT; ++mt) *(f32x4*)join[wave][mt][lane] = acc[mt];
    __syncthreads();
    const float ts = kNv ? a.tensor_scale[0] : 1.f;
    // lane (n, g) of tile mt holds feature n of tokens 4 g ..
    for (int c = threadIdx.x; c < MT * 64; c += WAVES * kWave) {
        const int mt = c >> 6, l = c & 63;
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < WAVES; ++k) v += *(const f32x4*)join[k][mt][l];
        const int col = o0 + (l & 15);
        if (col < a.O)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int64_t t = t0 + mt * 16 + (l >> 4) * 4 + e;
                if (t < a.T) a.out[t * a.O + col] = (uint16_t)pack_bf16x2(v[e] * ts, 0.f);
            }
    }
}

#define PLE_W4_KERNEL(MT, G, WAVES)                                                                     \
    __global__ __launch_bounds__(WAVES * 64) void w4_rows_##MT##_##G##_##WAVES##_kernel(W4Args a) { \
        w4_rows_body<MT, G, WAVES>(a);                                                                  \
    }
#define PLE_W4_KERNELS(MT, WAVES) \
    PLE_W4_KERNEL(MT, 16, WAVES) PLE_W4_KERNEL(MT, 32, WAVES) PLE_W4_KERNEL(MT, 64, WAVES) PLE_W4_KERNEL(MT, 128, WAVES)
PLE_W4_KERNELS(1, 8)
PLE_W4_KERNELS(2, 8)
PLE_W4_KERNELS(4, 8)

hipError_t launch_w4_linear(const uint16_t* x, int64_t x_stride, const ple_w4_weight& w, int64_t T, uint16_t* out,
                            hipStream_t s) {
    const W4Args a = {x, x_stride, w.codes, w.scales, w.zeros, w.tensor_scale, T, w.out_dim, w.k_dim, out};
    const int MT = T <= 16 ? 1 : (T <= 32 ? 2 : 4);
    const dim3 grid((unsigned)((w.out_dim + 15) / 16 * ((T + 16 * MT - 1) / (16 * MT))));
#define PLE_W4_LAUNCH(M, GG) \
    if (MT == M && w.group == GG) hipLaunchKernelGGL(w4_rows_##M##_##GG##_8_kernel, grid, dim3(512), 0, s, a)
#define PLE_W4_LAUNCHES(M) \
    PLE_W4_LAUNCH(M, 16);  \
    PLE_W4_LAUNCH(M, 32);  \
    PLE_W4_LAUNCH(M, 64);  \
    PLE_W4_LAUNCH(M, 128)
    PLE_W4_LAUNCHES(1);
    PLE_W4_LAUNCHES(2);
    PLE_W4_LAUNCHES(4);
    return hipGetLastError();
}

}  // namespace ple
