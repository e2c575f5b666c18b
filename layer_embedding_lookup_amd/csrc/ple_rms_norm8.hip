// The residual's addition, RMS norm and quantisation to 8 bits of a token's row, in one pass over it.
//
//   h = bf16(x + residual),  u = h w,  a = max|u|,  r = 1 / sqrt(mean h^2 + eps):
//   code = round(127 u / a),  scale = a r / 127
//
// The norm's factor cancels in the quotient, so a code depends on u and a
// alone, which fp32 holds exactly (8 x 8 significant bits), and 127 u too (23
// bits): with one correction of u / a by its remainder the rounded quotient is
// never on the wrong side of a border.  (u = U 2^i, a = A 2^j, U and A below
// 2^16, d = i - j: a quotient that is not on a border is 2^d / 2A > 2^(d-17)
// from it, half a step of the quotient, which lies below 2^(8+d); the
// corrected quotient is off by 2^-22 of a step before its rounding.)  That
// takes products that fp32 does not round: where a is at least 2^-100 those
// that get a code other than 0 lie above 2^-108, with all 16 bits, and their
// remainders are multiples of 2^-139.  Rows with a smaller a (rows of zeros
// too, which have nothing to lose by it) are read again and formed in 64 bits.
//
// Bound by bytes: 7984 rows of 4096 with a residual 43.4 us, 5.3 TB/s (a copy
// reaches 6.3); a single row 2.9 us, launch and two rounds of memory latency.
// A row stays in its block's registers between the sums and the codes; sum and
// maximum of a row are joined in one exchange.
#include "ple_8bit_launch.h"

namespace ple {

__device__ __forceinline__ void unpack8(u32x4 w, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
    }
}

constexpr float kTiny = 0x1p-100f;  // largest products below it: see above

// What turns the products of a row into codes, from its sum of squares and largest product.
struct RowScale {
    float top, inv, rsqrt, scale;
    bool bad, tiny;  // tiny: not for these codes and this scale
    __device__ __forceinline__ RowScale(float sum, float largest, const RmsNorm8Args& a) {
        top = largest;
        bad = !(sum < __builtin_inff()) || !(127.f * largest < __builtin_inff());  // (or either is NaN)
        tiny = !bad && top < kTiny;
        inv = bad || tiny ? 0.f : 1.0f / top;
        rsqrt = 1.0f / sqrtf(sum / (float)a.n + a.eps);
        const float all = top * rsqrt;  // (may be beyond fp32 where its 127th part is not)
        scale = bad ? __builtin_nanf("") : all < __builtin_inff() ? all / 127.0f : top / 127.0f * rsqrt;
    }
    // the codes of four products, in a word
    __device__ __forceinline__ uint32_t codes(float u0, float u1, float u2, float u3) const {
        const uint32_t c0 = code(u0), c1 = code(u1), c2 = code(u2), c3 = code(u3);
        return (c0 & 0xFFu) | (c1 & 0xFFu) << 8 | (c2 & 0xFFu) << 16 | c3 << 24;
    }

private:
    __device__ __forceinline__ uint32_t code(float u) const {
        const float t = 127.f * u;
        float q = t * inv;
        q = fmaf(fmaf(-q, top, t), inv, q);
        return bad ? 0u : __float_as_uint(q + 12582912.0f);  // 1.5 * 2^23: the sum's last bits are the rounded quotient
    }
};

// The larger one, NaN if either is: a weight that is no number, or an infinite one over an h of 0, is not lost.
__device__ __forceinline__ float larger(float x, float y) { return __builtin_elementwise_maximum(x, y); }

// The wave's, then the block's sum and maximum.  A NaN among the values makes the sum NaN, one among the products the
// maximum.
template <int WAVES>
__device__ __forceinline__ void join_row(float& sum, float& top) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
        sum += __shfl_xor(sum, d, kWave);
        top = larger(top, __shfl_xor(top, d, kWave));
    }
    if constexpr (WAVES > 1) {
        __shared__ float sums[WAVES], tops[WAVES];
        if ((threadIdx.x & 63) == 0) {
            sums[threadIdx.x >> 6] = sum;
            tops[threadIdx.x >> 6] = top;
        }
        __syncthreads();
        sum = 0.f;
        top = 0.f;
#pragma unroll
        for (int i = 0; i < WAVES; ++i) {
            sum += sums[i];
            top = larger(top, tops[i]);
        }
    }
}

// A row whose products fp32 does not hold, by the WAVES waves that hold it: its products in 64 bits, where they and 127 of
// them are exact and a quotient is off by 2^-53, read from where h stands by now (a lane reads what it wrote itself).
template <int WAVES>
__device__ __forceinline__ void tiny_row(const RmsNorm8Args& a, int64_t t, int tid, float rsqrt) {
    constexpr int kThreads = WAVES * kWave;
    const int chunks = a.n / 8;
    const uint16_t* row = a.residual != nullptr ? a.residual_out + t * a.n : a.x + t * a.x_stride;
    double top = 0.;
    for (int c = tid; c < chunks; c += kThreads) {
        float h[8], g[8];
        unpack8(*(const u32x4*)(row + c * 8), h);
        unpack8(*(const u32x4*)(a.weight + c * 8), g);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmax(top, fabs((double)h[e] * (double)g[e]));
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) top = fmax(top, __shfl_xor(top, d, kWave));
    if constexpr (WAVES > 1) {
        __shared__ double tops[WAVES];
        if ((tid & 63) == 0) tops[tid >> 6] = top;
        __syncthreads();
        for (int i = 0; i < WAVES; ++i) top = fmax(top, tops[i]);
    }
    for (int c = tid; c < chunks; c += kThreads) {
        float h[8], g[8];
        unpack8(*(const u32x4*)(row + c * 8), h);
        unpack8(*(const u32x4*)(a.weight + c * 8), g);
        u32x2 codes = {0u, 0u};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const double q = top == 0. ? 0. : 127. * ((double)h[e] * (double)g[e]) / top;
            codes[e / 4] |= ((uint32_t)(int)rint(q) & 0xFFu) << (e % 4 * 8);
        }
        *(u32x2*)(a.codes + t * a.n + c * 8) = codes;
    }
    if (tid == 0) a.scales[t] = (float)(top * (double)rsqrt / 127.);
}

// WAVES waves a row, CH chunks of 8 elements a lane; one wave a row: four rows a block.
template <int WAVES, int CH>
__device__ __forceinline__ void norm_body(const RmsNorm8Args& a) {
    constexpr int kThreads = WAVES * kWave;
    const int tid = WAVES == 1 ? threadIdx.x & 63 : threadIdx.x;
    const int64_t block = grid_block();
    const int64_t t = WAVES == 1 ? block * 4 + (threadIdx.x >> 6) : block;
    if (t >= a.T) return;  // (the whole block, where more waves than one share a row)
    const int chunks = a.n / 8;
    u32x4 x[CH], y[CH], w[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = i * kThreads + tid;
        x[i] = y[i] = w[i] = u32x4{0u, 0u, 0u, 0u};
        if (c >= chunks) continue;
        x[i] = *(const u32x4*)(a.x + t * a.x_stride + c * 8);
        if (a.residual != nullptr) y[i] = *(const u32x4*)(a.residual + t * a.n + c * 8);
        w[i] = *(const u32x4*)(a.weight + c * 8);
    }
    float u[CH][8], sum = 0.f, top = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = i * kThreads + tid;
        float g[8];
        if (a.residual != nullptr) {
            float r[8];
            unpack8(x[i], u[i]);
            unpack8(y[i], r);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[i][e] = pack_bf16x2(u[i][2 * e] + r[2 * e], u[i][2 * e + 1] + r[2 * e + 1]);
            if (c < chunks) *(u32x4*)(a.residual_out + t * a.n + c * 8) = x[i];
        }
        unpack8(x[i], u[i]);
        unpack8(w[i], g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            sum = fmaf(u[i][e], u[i][e], sum);
            u[i][e] *= g[e];
            top = larger(top, fabsf(u[i][e]));
        }
    }
    join_row<WAVES>(sum, top);
    const RowScale s(sum, top, a);
    if (s.tiny) return tiny_row<WAVES>(a, t, tid, s.rsqrt);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = i * kThreads + tid;
        if (c < chunks)
            *(u32x2*)(a.codes + t * a.n + c * 8) =
                u32x2{s.codes(u[i][0], u[i][1], u[i][2], u[i][3]), s.codes(u[i][4], u[i][5], u[i][6], u[i][7])};
    }
    if (tid == 0) a.scales[t] = s.scale;
}

// Rows that registers do not hold: the row is read again for its codes.
constexpr int kLongThreads = 1024;
__global__ __launch_bounds__(kLongThreads) void rms_norm8_long_kernel(RmsNorm8Args a) {
    const int64_t t = grid_block();
    if (t >= a.T) return;
    const int chunks = a.n / 8;
    const uint16_t* row = a.x + t * a.x_stride;
    float sum = 0.f, top = 0.f;
    for (int c = threadIdx.x; c < chunks; c += kLongThreads) {
        float h[8], g[8];
        u32x4 x = *(const u32x4*)(row + c * 8);
        unpack8(x, h);
        if (a.residual != nullptr) {
            float r[8];
            unpack8(*(const u32x4*)(a.residual + t * a.n + c * 8), r);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = pack_bf16x2(h[2 * e] + r[2 * e], h[2 * e + 1] + r[2 * e + 1]);
            *(u32x4*)(a.residual_out + t * a.n + c * 8) = x;
            unpack8(x, h);
        }
        unpack8(*(const u32x4*)(a.weight + c * 8), g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            sum = fmaf(h[e], h[e], sum);
            top = larger(top, fabsf(h[e] * g[e]));
        }
    }
    join_row<kLongThreads / kWave>(sum, top);
    const RowScale s(sum, top, a);
    if (s.tiny) return tiny_row<kLongThreads / kWave>(a, t, threadIdx.x, s.rsqrt);
    if (a.residual != nullptr) row = a.residual_out + t * a.n;  // (a lane reads what it wrote itself)
    for (int c = threadIdx.x; c < chunks; c += kLongThreads) {
        float h[8], g[8];
        unpack8(*(const u32x4*)(row + c * 8), h);
        unpack8(*(const u32x4*)(a.weight + c * 8), g);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] *= g[e];
        *(u32x2*)(a.codes + t * a.n + c * 8) = u32x2{s.codes(h[0], h[1], h[2], h[3]), s.codes(h[4], h[5], h[6], h[7])};
    }
    if (threadIdx.x == 0) a.scales[t] = s.scale;
}

// Waves a row, chunks a lane: as many waves as leave a lane one chunk up to 4096 elements, then two (4000 rows of 8192 in
// eight waves 44.1 us, in four 48.6; 2000 of 16384 in sixteen 45.7, in eight 47.8; 7984 of 4096 in eight 43.4, four 44.5, two
// 49.2, one 54.5; one of 4096 2.9, 3.1, 3.9, 5.4; but 8000 of 2048 in four 23.9, in eight, half of whose lanes idle, 27.7; 8000
// of 512 in one 8.4, in four 11.9).  Longer rows are read again: 500 of 32000 29 us.
#define PLE_NORM_SHAPES(X) X(1, 1) X(4, 1) X(8, 1) X(8, 2) X(16, 2)
#define PLE_NORM_KERNEL(WAVES, CH)                                                                                         \
    __global__ __launch_bounds__(WAVES == 1 ? 256 : WAVES * kWave) void rms_norm8_##WAVES##x##CH##_kernel(RmsNorm8Args a) { \
        norm_body<WAVES, CH>(a);                                                                                           \
    }
PLE_NORM_SHAPES(PLE_NORM_KERNEL)
#undef PLE_NORM_KERNEL

RmsNorm8Shape rms_norm8_shape(int32_t n) {
#define PLE_NORM_FITS(WAVES, CH) \
    if (n <= WAVES * kWave * CH * 8) return {WAVES, CH};
    PLE_NORM_SHAPES(PLE_NORM_FITS)
#undef PLE_NORM_FITS
    return {0, 0};
}

hipError_t launch_rms_norm8(const RmsNorm8Args& a, hipStream_t s) {
    const RmsNorm8Shape f = rms_norm8_shape(a.n);
    const dim3 grid = block_grid(f.waves == 1 ? (a.T + 3) / 4 : a.T);
#define PLE_NORM_LAUNCH(WAVES, CH)                                                                                        \
    if (f.waves == WAVES && f.chunks == CH)                                                                               \
        hipLaunchKernelGGL(rms_norm8_##WAVES##x##CH##_kernel, grid, dim3(WAVES == 1 ? 256 : WAVES * kWave), 0, s, a);
    PLE_NORM_SHAPES(PLE_NORM_LAUNCH)
#undef PLE_NORM_LAUNCH
    if (f.waves == 0) hipLaunchKernelGGL(rms_norm8_long_kernel, grid, dim3(kLongThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace ple
