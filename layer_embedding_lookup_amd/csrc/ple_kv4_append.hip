// New keys and values, rotated by position, into the paged 4-bit cache, and
// back out of it.
//
// Bound by bytes: a token reads its q, k and v rows and writes q and 9/32 of
// the bytes of k and v.  One block per token: the token's sines and cosines
// are formed once, in 64 bits (positions of 10^5 and more lose the angle in
// 32), and shared by all heads; then each lane takes chunks of 8 elements (16
// bytes in, 4 bytes of codes out), and the two lanes of a 16-element block
// join their maxima with one exchange.  The rotation itself is 64-bit too and
// rounded once to fp32, so that a key next to a code's border falls on the
// side that the definition says.  7984 tokens of 32 + 8 + 8 heads of 128: 35 us
// (173 MB, 4.9 TB/s; with the codes found by comparisons 41.6) and 13 us to read them back (43 MB); 256 tokens: 7.3 and
// 3.8 us, of which a launch is about 3 and the rest the chain of loads that finds the request (a binary search, then its
// length and its table entry) and, for append, the angles.
#include "ple_rotate.h"

namespace ple {

constexpr int kAppendThreads = 256;

// A block per token: along x as many as a launch takes with room to spare, the rest along y.
constexpr int64_t kAppendAcross = 1 << 20;
static dim3 append_grid(int64_t T) {
    return dim3((unsigned)(T < kAppendAcross ? T : kAppendAcross), (unsigned)((T + kAppendAcross - 1) / kAppendAcross));
}

// e4m3 code of a finite or NaN value already clamped to 448, round to nearest even.
__device__ __forceinline__ uint32_t e4m3_code(float v) {
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v, 0.0f, 0, false) & 0xFFu;
}

// e2m1 codes of 8 quotients: nearest of 0 .5 1 1.5 2 3 4 6, ties to the even code, 6 beyond it.
__device__ __forceinline__ uint32_t e2m1_codes(const float (&t)[8]) {
    uint32_t c = 0;
    float u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = __builtin_amdgcn_fmed3f(t[i], -6.f, 6.f);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, u[0], u[1], 1.0f, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, u[2], u[3], 1.0f, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, u[4], u[5], 1.0f, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, u[6], u[7], 1.0f, 3);
}

// The token's 16-token group of head 0, or -1; one head on it is per_page groups on.
__device__ __forceinline__ int64_t first_group(const ple_kv4_cache& c, const int32_t* row, int pos) {
    return pos < 0 ? -1 : (int64_t)kv4_group(c, row, 0, pos >> 4);
}

__global__ __launch_bounds__(kAppendThreads) void kv4_append_kernel(Kv4AppendArgs a) {
    __shared__ double2 turn[128];  // cos, sin of the token's angles
    const int64_t t = blockIdx.x + blockIdx.y * kAppendAcross;
    if (t >= a.batch.num_tokens) return;
    const int D = a.cache.head_dim;
    const int per_head = D / 8, shift = D == 64 ? 3 : (D == 128 ? 4 : 5);  // chunks of a head
    int r;
    const int pos = kv4_position(a.cache, a.batch, t, r);
    const int rot = pos < 0 ? 0 : a.rot_dim, half = rot / 2;  // (a token that stands nowhere may hold anything, and keeps it)
    for (int i = threadIdx.x; i < half; i += kAppendThreads) {
        // (a position of 30 bits times a 24-bit frequency: rounded at most in its 54th bit, 2^-53 of the angle)
        const double angle = (double)pos * (double)a.inv_freq[i];
        double sn, cs;
        sincos(angle, &sn, &cs);
        turn[Turns<false>::place(i, half)] = make_double2(cs, sn);
    }
    __syncthreads();
    const int64_t group0 = first_group(a.cache, a.batch.page_table + (int64_t)r * a.batch.table_width, pos);
    const int per_page = a.cache.page_size >> 4, place = pos & 15;
    const int nq = a.num_q_heads * per_head, nk = a.cache.num_kv_heads * per_head;
    for (int c = threadIdx.x; c < nq + 2 * nk; c += kAppendThreads) {
        const int which = c < nq ? 0 : (c < nq + nk ? 1 : 2);
        const int at = which == 0 ? c : (which == 1 ? c - nq : c - nq - nk);
        const int head = at >> shift, d0 = (at & (per_head - 1)) * 8;
        const uint16_t* src = a.src[which] + t * a.stride[which] + head * D;
        float v[8];
        load_rotated<Turns<false>>(src, d0, which != 2 ? rot : 0, a.interleaved, turn, v);
        if (which == 0) {
            u32x4 o;
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
            *(u32x4*)(a.q_out + (t * a.num_q_heads + head) * D + d0) = o;
            continue;
        }
        // chunks 2b and 2b+1 of a head are lanes 2b and 2b+1 of a wave: nq and nk are even
        float top = 0.f;
        bool nan = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            top = fmaxf(top, fabsf(v[i]));
            nan |= v[i] != v[i];
        }
        if (nan) top = __builtin_nanf("");
        const float other = __shfl_xor(top, 1, kWave);
        top = top != top || other != other ? __builtin_nanf("") : fmaxf(top, other);
        const float g = (which == 1 ? a.cache.k_scale : a.cache.v_scale)[head];
        float s = top / (6.0f * g);
        s = s > 448.f ? 448.f : s;  // (keeps a NaN)
        const uint32_t sc = e4m3_code(s);
        float step = __builtin_amdgcn_cvt_pk_f32_fp8((int)sc, false)[0] * g;
        step = step > 0.f ? step : __builtin_inff();
        float quotient[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) quotient[i] = v[i] / step;
        const uint32_t codes = e2m1_codes(quotient);
        if (group0 < 0) continue;
        const int64_t grp = group0 + (int64_t)head * per_page;
        uint8_t* cd = (which == 1 ? a.cache.k_codes : a.cache.v_codes) + grp * (8 * D) + place * (D / 2) + d0 / 2;
        *(uint32_t*)cd = codes;
        if ((d0 & 8) == 0)
            ((which == 1 ? a.cache.k_scales : a.cache.v_scales) + grp * D)[d0 + place] = (uint8_t)sc;
    }
}

hipError_t launch_kv4_append(const Kv4AppendArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(kv4_append_kernel, append_grid(a.batch.num_tokens), dim3(kAppendThreads), 0, s, a);
    return hipGetLastError();
}

// One block per token; a lane turns 4 bytes of codes into 16 bytes of bf16.
__global__ __launch_bounds__(kAppendThreads) void kv4_read_kernel(ple_kv4_cache cache, ple_kv4_batch batch,
                                                                  uint16_t* __restrict__ k_out,
                                                                  uint16_t* __restrict__ v_out) {
    const int64_t t = blockIdx.x + blockIdx.y * kAppendAcross;
    if (t >= batch.num_tokens) return;
    const int D = cache.head_dim, per_head = D / 8, shift = D == 64 ? 3 : (D == 128 ? 4 : 5);
    int r;
    const int pos = kv4_position(cache, batch, t, r);
    const int64_t group0 = first_group(cache, batch.page_table + (int64_t)r * batch.table_width, pos);
    const int per_page = cache.page_size >> 4, place = pos & 15;
    const int nk = cache.num_kv_heads * per_head;
    for (int c = threadIdx.x; c < 2 * nk; c += kAppendThreads) {
        const bool val = c >= nk;
        const int at = val ? c - nk : c;
        const int head = at >> shift, d0 = (at & (per_head - 1)) * 8;
        u32x4 o = {0u, 0u, 0u, 0u};
        if (group0 >= 0) {
            const int64_t grp = group0 + (int64_t)head * per_page;
            const uint32_t w =
                *(const uint32_t*)((val ? cache.v_codes : cache.k_codes) + grp * (8 * D) + place * (D / 2) + d0 / 2);
            const uint8_t sc = ((val ? cache.v_scales : cache.k_scales) + grp * D)[(d0 & ~15) + place];
            const float s = __builtin_amdgcn_cvt_pk_f32_fp8((int)sc, false)[0];
            const float g = (val ? cache.v_scale : cache.k_scale)[head];
            const f32x2 e0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
            const f32x2 e1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
            const f32x2 e2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
            const f32x2 e3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
            // code * block scale is exact in fp32
            o[0] = pack_bf16x2(e0[0] * s * g, e0[1] * s * g);
            o[1] = pack_bf16x2(e1[0] * s * g, e1[1] * s * g);
            o[2] = pack_bf16x2(e2[0] * s * g, e2[1] * s * g);
            o[3] = pack_bf16x2(e3[0] * s * g, e3[1] * s * g);
        }
        *(u32x4*)((val ? v_out : k_out) + (t * cache.num_kv_heads + head) * D + d0) = o;
    }
}

hipError_t launch_kv4_read(const ple_kv4_cache& cache, const ple_kv4_batch& batch, uint16_t* k_out, uint16_t* v_out,
                           hipStream_t s) {
    hipLaunchKernelGGL(kv4_read_kernel, append_grid(batch.num_tokens), dim3(kAppendThreads), 0, s, cache, batch,
                       k_out, v_out);
    return hipGetLastError();
}

}  // namespace ple
