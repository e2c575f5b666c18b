// Products with 4-bit weights: out = x W^T, W dequantised on the way to the
// matrix cores and never written out.
//
// Few tokens (decode): bound by the latency of its rounds of loads.  A round
// is a step of 128 inputs of each of the block's eight waves, loaded, waited
// for and used; launch and join take about 3 us, a round 0.7..0.9 (one token,
// 8192 features NVFP4, kernel alone: K = 512 3.5 us, 1024 4.0, 2048 4.8, 4096
// 6.5 (18.9 MB, 2.9 TB/s), 8192 12.1; back to back no call takes less than
// the host's 5.9; 64 tokens, K = 4096 12.4).  A wave takes NT x 16 output
// features and a share of K in steps of 128.  Inputs and codes come in whole rows straight into LDS, 1 KiB
// an instruction: read as MFMA operands from memory (lane n its own row) each
// lane's 16 bytes are a cache access of their own, and those accesses, 64 an
// instruction, bound the kernel (64 tokens: 22.6 us).  Four 16x16x32 bf16
// MFMAs a step have the tokens as the first operand and the features as the
// second, so every lane's scales belong to its own feature lane % 16.  The
// waves of a block share the features, split K between them and join their
// sums through LDS, which needs no second launch and no atomics.
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

// The group scales of a step of 128 inputs.  Lane 4 r + c fetches those of row r's inputs 32 c .. (four neighbouring lanes
// in one access) and hands them to lane r + 16 c, which holds these codes (the few-token NVFP4 kernel fetches its scales
// where they are used: there the exchange costs 3% more than it saves, elsewhere it saves 2..12%).  INT4: the last
// group's past the end; nothing waits in the fetch, `group_word` puts scale and zero point together later (scale | zero
// point << 16; zero past the end), and `groups_of` gives every lane of a row all of them.
struct GroupRaw {
    uint32_t scale, zero;
};
__device__ __forceinline__ GroupRaw group_fetch(const void* scales, const uint8_t* zeros, int64_t row, int at, int groups) {
    const int64_t i = row + min(at, groups - 1);
    return {((const uint16_t*)scales)[i], zeros == nullptr ? 8u : (uint32_t)zeros[i]};
}
__device__ __forceinline__ uint32_t group_word(GroupRaw r, int at, int groups) {
    return at < groups ? r.scale | r.zero << 16 : 8u << 16;
}
template <int G>
__device__ __forceinline__ void groups_of(uint32_t mine, uint32_t (&all)[128 / G]) {
    typedef unsigned int u2 __attribute__((ext_vector_type(2)));
    if constexpr (G == 128) {
        all[0] = mine;
    } else {
        const u2 h = __builtin_amdgcn_permlane32_swap(mine, mine, false, false);  // lane groups 0 1 0 1 and 2 3 2 3
        if constexpr (G == 64) {
            all[0] = h[0];
            all[1] = h[1];
        } else {
            const u2 a = __builtin_amdgcn_permlane16_swap(h[0], h[0], false, false);
            const u2 b = __builtin_amdgcn_permlane16_swap(h[1], h[1], false, false);
            all[0] = a[0];
            all[1] = a[1];
            all[2] = b[0];
            all[3] = b[1];
        }
    }
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

// The few-token kernel's LDS: a step's inputs and codes of every wave, then the joined sums.
template <int MT, int NT, int WAVES>
struct RowsShape {
    static constexpr int CODES = MT * 4096;              // 16 MT tokens x 256 bytes, then 16 NT features x 64 bytes of codes
    static constexpr int STEP = CODES + NT * 1024;
    static constexpr int JOIN = WAVES < 4 ? WAVES : 4;   // waves whose sums are in LDS at once
    static constexpr int LDS = WAVES * STEP > JOIN * MT * NT * 1024 ? WAVES * STEP : JOIN * MT * NT * 1024;
    static_assert(LDS <= 160 * 1024, "more LDS than a CU has");
};

// MT tiles of 16 tokens, NT tiles of 16 features; G: 16 for NVFP4, else the INT4 group.
template <int MT, int NT, int G, int WAVES>
__device__ __forceinline__ void w4_rows_body(const W4Args& a) {
    constexpr bool kNv = G == 16;
    constexpr int kGroups = kNv ? 1 : 128 / G;  // groups of a step
    using Sh = RowsShape<MT, NT, WAVES>;
    constexpr int kJoin = Sh::JOIN;
    extern __shared__ __align__(16) char lds[];
    float(*const join)[MT * NT][64][4] = (float(*)[MT * NT][64][4])lds;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;
    const int tiles_o = (a.O + 16 * NT - 1) / (16 * NT), o0 = (blockIdx.x % tiles_o) * (16 * NT);
    const int64_t t0 = (int64_t)(blockIdx.x / tiles_o) * (16 * MT);
    const int groups = a.K / (kNv ? 16 : G);
    // features past the end repeat the last one, tokens past it hold anything; neither is stored
    const uint8_t* wrow[NT];
    int64_t srow[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        wrow[nt] = a.codes + (int64_t)min(o0 + nt * 16 + (lane >> 2), a.O - 1) * (a.K / 2);
        srow[nt] = (int64_t)min(o0 + nt * 16 + (kNv ? n : lane >> 2), a.O - 1) * groups;
    }
    // (codes: 16 features x 64 contiguous bytes an instruction, feature r's chunk c at place c ^ (r / 4))
    const int wchunk = ((lane & 3) ^ (lane >> 4)) * 16, wat = n * 64 + (g ^ (n >> 2)) * 16;
    // Inputs go straight to LDS, 4 tokens x 256 contiguous bytes an instruction (as fragments they would be 64 separate
    // 16-byte reads of the cache, which bound this kernel before: 8192 x 4096 NVFP4, 64 tokens, 22.7 us): token r's 16
    // chunks of 16 bytes, chunk c at place c ^ (r % 16), read back without bank conflicts.
    char* const xlds = lds + wave * Sh::STEP;
    const int live = (int)(a.T - t0 < 16 * MT ? a.T - t0 : 16 * MT);
    f32x4 acc[MT][NT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[mt][nt] = f32x4{0.f, 0.f, 0.f, 0.f};

    // NVFP4: the lane's two block scales; INT4: as fetched
    struct Step {
        GroupRaw scale[NT];
    };
    const u32x4 zero4 = {0u, 0u, 0u, 0u};
    // Lanes past K take zeros: NVFP4 products vanish, INT4 steps stop at the last group (K is a multiple of it).
    auto load = [&](int k0, Step& s) {
#pragma unroll
        for (int i = 0; i < 4 * MT; ++i) {
            if (4 * i >= live) break;
            const int r = 4 * i + g, c = n ^ (r & 15);
            const int64_t t = t0 + (r < live ? r : live - 1);
            const uint16_t* src = a.x + t * a.x_stride + (k0 + c * 8 < a.K ? k0 + c * 8 : 0);
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                             (__attribute__((address_space(3))) void*)(xlds + i * 1024), 16, 0, 0);
        }
        const bool in = k0 + g * 32 < a.K;
        const int at = k0 / 2 + wchunk < a.K / 2 ? k0 / 2 + wchunk : 0;  // (past K: anything, against zero inputs)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(wrow[nt] + at),
                                             (__attribute__((address_space(3))) void*)(xlds + Sh::CODES + nt * 1024),
                                             16, 0, 0);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if constexpr (kNv) {
                s.scale[nt].scale = in ? *(const uint16_t*)((const uint8_t*)a.scales + srow[nt] + k0 / 16 + g * 2) : 0u;
            } else {
                s.scale[nt] = group_fetch(a.scales, a.zeros, srow[nt], (k0 + 32 * (lane & 3)) / G, groups);
            }
        }
    };
    auto use = [&](int k0, Step& s) {
        u32x4 w[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) w[nt] = *(const u32x4*)(xlds + Sh::CODES + nt * 1024 + wat);
        u32x4 x[MT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = kNv ? 4 * g + j : 4 * j + g;
                x[mt][j] = *(const u32x4*)(xlds + mt * 4096 + n * 256 + (c ^ n) * 16);
                if (k0 + 128 > a.K && k0 + c * 8 >= a.K) x[mt][j] = zero4;
            }
        if constexpr (kNv) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const f32x2 sc = __builtin_amdgcn_cvt_pk_f32_fp8((int)s.scale[nt].scale, false);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    BFrag f;
                    nvfp4_frag(w[nt][j], sc[j >> 1], f);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
                        acc[mt][nt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[mt][j]), f.v,
                                                                              acc[mt][nt], 0, 0, 0);
                }
            }
        } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                transpose4(w[nt]);  // word j: inputs k0 + 32 j + 8 g ..
                uint32_t all[kGroups];
                groups_of<G>(__shfl(group_word(s.scale[nt], (k0 + 32 * (lane & 3)) / G, groups), 4 * n + g, kWave), all);
#pragma unroll
                for (int i = 0; i < kGroups; ++i) {
                    const float z = (float)(all[i] >> 16), sc = bf16_lo(all[i]);
                    f32x4 part[MT];
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) part[mt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int j = i * (G / 32); j < (i + 1) * (G / 32); ++j) {
                        BFrag f;
                        int4_frag(w[nt][j], z, f);
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
                            part[mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[mt][j]),
                                                                               f.v, part[mt], 0, 0, 0);
                    }
                    // (groups past K hold zero inputs and a zero scale)
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[mt][nt][e] = fmaf(part[mt][e], sc, acc[mt][nt][e]);
                }
            }
        }
    };
    for (int k0 = wave * 128; k0 < a.K; k0 += WAVES * 128) {
        Step st;
        load(k0, st);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        use(k0, st);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the inputs are read before the next ones come in
    }
    __syncthreads();  // the sums take the inputs' place

    // waves kJoin .. hand their sums to the first kJoin, whose sums are then added up
    for (int w0 = WAVES - kJoin; w0 > 0; w0 -= kJoin) {
        if (wave >= w0 && wave < w0 + kJoin)
#pragma unroll
            for (int i = 0; i < MT * NT; ++i) *(f32x4*)join[wave - w0][i][lane] = acc[i / NT][i % NT];
        __syncthreads();
        if (wave < kJoin)
#pragma unroll
            for (int i = 0; i < MT * NT; ++i) acc[i / NT][i % NT] += *(const f32x4*)join[wave][i][lane];
        __syncthreads();
    }
    if (wave < kJoin)
#pragma unroll
        for (int i = 0; i < MT * NT; ++i) *(f32x4*)join[wave][i][lane] = acc[i / NT][i % NT];
    __syncthreads();
    const float ts = kNv ? a.tensor_scale[0] : 1.f;
    // lane (n, g) of tile (mt, nt) holds feature n of tokens 4 g ..
    for (int c = threadIdx.x; c < MT * NT * 64; c += WAVES * kWave) {
        const int i = c >> 6, l = c & 63;
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < kJoin; ++k) v += *(const f32x4*)join[k][i][l];
        const int col = o0 + (i % NT) * 16 + (l & 15);
        if (col < a.O)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int64_t t = t0 + (i / NT) * 16 + (l >> 4) * 4 + e;
                if (t < a.T) a.out[t * a.O + col] = (uint16_t)pack_bf16x2(v[e] * ts, 0.f);
            }
    }
}

// Shapes of the few-token kernel: token tiles, feature tiles, waves, waves per SIMD that registers are kept to (up to 32
// tokens two blocks per CU and more: 8192 x 4096 INT4, one token, 14.1 us with one).
#define PLE_W4_SHAPES(X) X(1, 1, 8, 4) X(2, 1, 8, 4) X(4, 1, 8, 2) X(4, 2, 8, 2) X(4, 4, 8, 2)
#define PLE_W4_KERNEL(MT, NT, G, WAVES, OCC)                                                          \
    __global__ __launch_bounds__(WAVES * 64, OCC) void w4_rows_##MT##x##NT##_##G##_kernel(W4Args a) { \
        w4_rows_body<MT, NT, G, WAVES>(a);                                                            \
    }
#define PLE_W4_KERNELS(MT, NT, WAVES, OCC)                                              \
    PLE_W4_KERNEL(MT, NT, 16, WAVES, OCC) PLE_W4_KERNEL(MT, NT, 32, WAVES, OCC)         \
    PLE_W4_KERNEL(MT, NT, 64, WAVES, OCC) PLE_W4_KERNEL(MT, NT, 128, WAVES, OCC)
PLE_W4_SHAPES(PLE_W4_KERNELS)

// ---------------------------------------------------------------------------
// Many tokens: bound by the products and by dequantising between them (4096
// -> 8192, 1024 tokens: NVFP4 72..75 us, 0.92..0.95 PFLOP/s; INT4 in groups of
// 128 92 us, of 32, with four times the scaling of partial sums and tiles of
// 64 tokens, 164; 8192 tokens: NVFP4 618 us, INT4 in groups of 128 775).  A
// block of four waves holds MT x 16 tokens x NT x 64 features, a wave all of
// the tokens and NT x 16 features.  Inputs and codes go through LDS in slices
// of 128 (two slots), the inputs shared by the waves; each wave dequantises
// its own features in registers, once for the block's tokens.  128 features a
// block, not 256, leave room for two blocks per CU, which cover each other's
// waits (T = 1024 in 128 x 256 tiles, one block per CU: 88 us; INT4 in groups
// of 32 spilled, 1183).
//
// LDS layout of a slice: a token's 256 bytes are 16 chunks of 16 bytes, chunk
// c at place c ^ (token % 16), so the 16 lanes of a fragment read (16 tokens,
// one chunk) touch 16 different 16-byte banks.  Fragment j of lane (n, g)
// takes chunk 4 g + j (NVFP4: the lane's own 16 bytes of codes) or 4 j + g
// (INT4: words swapped, so that a fragment's inputs lie in one group).
// ---------------------------------------------------------------------------
constexpr int kGemmThreads = 256;
template <int MT, int NT>
struct GemmShape {
    static constexpr int T = 16 * MT, O = 64 * NT;
    static constexpr int SLOT = T * 256;          // bytes of a slice
    static constexpr int OUT_ROW = O * 2 + 16;    // bytes of an output row in LDS
    static constexpr int CODES = NT * 1024;       // bytes of a wave's codes of a slice
    static constexpr int CODES_AT = 2 * SLOT;
    static constexpr int LDS = CODES_AT + 8 * CODES > T * OUT_ROW ? CODES_AT + 8 * CODES : T * OUT_ROW;
};

template <int G, int MT, int NT>
__device__ __forceinline__ void w4_gemm_body(const W4Args& a) {
    using Sh = GemmShape<MT, NT>;
    constexpr bool kNv = G == 16;
    constexpr int kGroups = kNv ? 1 : 128 / G;
    extern __shared__ __align__(16) char lds[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 15, g = lane >> 4;
    const int tiles_t = (int)((a.T + Sh::T - 1) / Sh::T), tiles_o = (a.O + Sh::O - 1) / Sh::O;
    // neighbouring blocks of an XCD (block number mod 8) share features, so their codes come from its L2
    const int total = tiles_t * tiles_o;
    int lin = blockIdx.x;
    if ((total & 7) == 0) lin = (lin & 7) * (total >> 3) + (lin >> 3);
    const int to = lin / tiles_t, tt = lin - to * tiles_t;
    const int64_t t0 = (int64_t)tt * Sh::T;
    const int o0 = to * Sh::O + wave * (16 * NT);
    const int groups = a.K / (kNv ? 16 : G);
    // Codes go to LDS as 16 rows x 64 contiguous bytes an instruction, two slots per wave (read by lane (n, g) from memory
    // they would be 64 separate accesses): row r's chunk c at place c ^ (r / 4).
    const uint8_t* wrow[NT];
    int64_t srow[NT];
    const int wchunk = ((lane & 3) ^ (lane >> 4)) * 16;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        wrow[nt] = a.codes + (int64_t)min(o0 + nt * 16 + (lane >> 2), a.O - 1) * (a.K / 2);
        srow[nt] = (int64_t)min(o0 + nt * 16 + (lane >> 2), a.O - 1) * groups;
    }
    char* const wlds = lds + Sh::CODES_AT + wave * (2 * Sh::CODES);
    const int wat = n * 64 + (g ^ (n >> 2)) * 16;
    // this thread's chunks of a slice: token tid/16 + 16 i, chunk tid % 16
    const uint16_t* xsrc[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int64_t t = t0 + (tid >> 4) + 16 * i;
        xsrc[i] = a.x + (t < a.T ? t : a.T - 1) * a.x_stride + (tid & 15) * 8;
    }
    char* const xdst = lds + (tid >> 4) * 256 + ((tid & 15) ^ (tid >> 4)) * 16;

    const u32x4 zero4 = {0u, 0u, 0u, 0u};
    u32x4 xs[MT];
    GroupRaw scale[NT];
    auto load = [&](int k0) {
        const bool in = k0 + (lane & 3) * 32 < a.K;
        const int at = k0 / 2 + wchunk < a.K / 2 ? k0 / 2 + wchunk : 0;  // (past K: anything, against zero inputs)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(wrow[nt] + at),
                                             (__attribute__((address_space(3))) void*)(wlds + (k0 >> 7 & 1) * Sh::CODES + nt * 1024),
                                             16, 0, 0);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if constexpr (kNv) {
                scale[nt].scale = in ? *(const uint16_t*)((const uint8_t*)a.scales + srow[nt] + k0 / 16 + (lane & 3) * 2) : 0u;
            } else {
                scale[nt] = group_fetch(a.scales, a.zeros, srow[nt], (k0 + 32 * (lane & 3)) / G, groups);
            }
        }
        const bool xin = k0 + (tid & 15) * 8 < a.K;
#pragma unroll
        for (int i = 0; i < MT; ++i) xs[i] = xin ? *(const u32x4*)(xsrc[i] + k0) : zero4;
    };
    auto put = [&](int slot) {
#pragma unroll
        for (int i = 0; i < MT; ++i) *(u32x4*)(xdst + slot * Sh::SLOT + i * 4096) = xs[i];
    };

    f32x4 acc[MT][NT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[mt][nt] = f32x4{0.f, 0.f, 0.f, 0.f};

    load(0);
    put(0);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the codes
    const int steps = (a.K + 127) / 128;
    for (int st = 0; st < steps; ++st) {
        // this slice's codes as bf16
        u32x4 w[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) w[nt] = *(const u32x4*)(wlds + (st & 1) * Sh::CODES + nt * 1024 + wat);
        BFrag f[NT][4];
        float sc[NT][kGroups];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if constexpr (kNv) {
                const f32x2 s2 = __builtin_amdgcn_cvt_pk_f32_fp8(__shfl((int)scale[nt].scale, 4 * n + g, kWave), false);
#pragma unroll
                for (int j = 0; j < 4; ++j) nvfp4_frag(w[nt][j], s2[j >> 1], f[nt][j]);
            } else {
                u32x4 t = w[nt];
                transpose4(t);
                uint32_t all[kGroups];
                groups_of<G>(__shfl(group_word(scale[nt], (st * 128 + 32 * (lane & 3)) / G, groups), 4 * n + g, kWave), all);
#pragma unroll
                for (int j = 0; j < 4; ++j) int4_frag(t[j], (float)(all[j / (G / 32)] >> 16), f[nt][j]);
#pragma unroll
                for (int i = 0; i < kGroups; ++i) sc[nt][i] = bf16_lo(all[i]);
            }
        }
        __syncthreads();  // slice st is whole; every read of the other slot is done
        if (st + 1 < steps) load((st + 1) * 128);
        const char* slot = lds + (st & 1) * Sh::SLOT + n * 256;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            BFrag x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = kNv ? 4 * g + j : 4 * j + g;
                x[j].q = *(const u32x4*)(slot + mt * 4096 + ((c ^ n) * 16));
            }
            if constexpr (kNv) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        acc[mt][nt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[j].v, f[nt][j].v, acc[mt][nt], 0, 0, 0);
            } else {
#pragma unroll
                for (int i = 0; i < kGroups; ++i) {
                    f32x4 part[NT];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) part[nt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int j = i * (G / 32); j < (i + 1) * (G / 32); ++j)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            part[nt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[j].v, f[nt][j].v, part[nt], 0, 0, 0);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[mt][nt][e] = fmaf(part[nt][e], sc[nt][i], acc[mt][nt][e]);
                }
                // (few token tiles at a time: the partial sums of all of them would not fit the registers)
                if constexpr (G < 128)
                    if (mt % (G / 32) == G / 32 - 1) __builtin_amdgcn_sched_barrier(0);
            }
        }
        if (st + 1 < steps) put((st + 1) & 1);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the next codes
    }

    // out through LDS: lane (n, g) of tile (mt, nt) holds feature n of tokens 4 g ..
    const float ts = kNv ? a.tensor_scale[0] : 1.f;
    __syncthreads();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                *(uint16_t*)(lds + (mt * 16 + g * 4 + e) * Sh::OUT_ROW + (wave * (16 * NT) + nt * 16 + n) * 2) =
                    (uint16_t)pack_bf16x2(acc[mt][nt][e] * ts, 0.f);
    __syncthreads();
    const int ob = to * Sh::O;
    if (a.O % 8 == 0) {
        for (int c = tid; c < Sh::T * (Sh::O / 8); c += kGemmThreads) {
            const int row = c / (Sh::O / 8), col = (c % (Sh::O / 8)) * 8;
            if (t0 + row < a.T && ob + col < a.O)
                *(u32x4*)(a.out + (t0 + row) * a.O + ob + col) = *(const u32x4*)(lds + row * Sh::OUT_ROW + col * 2);
        }
    } else {
        for (int c = tid; c < Sh::T * Sh::O; c += kGemmThreads) {
            const int row = c / Sh::O, col = c % Sh::O;
            if (t0 + row < a.T && ob + col < a.O)
                a.out[(t0 + row) * a.O + ob + col] = *(const uint16_t*)(lds + row * Sh::OUT_ROW + col * 2);
        }
    }
}

#define PLE_W4_GEMM(G, MT, NT, OCC)                                                                      \
    __global__ __launch_bounds__(kGemmThreads, OCC) void w4_gemm_##MT##x##NT##_##G##_kernel(W4Args a) { \
        w4_gemm_body<G, MT, NT>(a);                                                                      \
    }
PLE_W4_GEMM(16, 4, 2, 2)
PLE_W4_GEMM(32, 4, 2, 2)
PLE_W4_GEMM(64, 4, 2, 2)
PLE_W4_GEMM(128, 4, 2, 2)
// 128 tokens; with groups of 32 or 64 their partial sums would not fit the registers of two blocks per CU
PLE_W4_GEMM(16, 8, 2, 2)
PLE_W4_GEMM(128, 8, 2, 2)
#undef PLE_W4_GEMM

template <void (*FN)(W4Args), int LDS>
static hipError_t launch_blocks(const W4Args& a, unsigned blocks, int threads, hipStream_t s) {
    static const hipError_t attr = hipFuncSetAttribute((const void*)FN, hipFuncAttributeMaxDynamicSharedMemorySize, LDS);
    if (attr != hipSuccess) return attr;
    hipLaunchKernelGGL(FN, dim3(blocks), dim3(threads), LDS, s, a);
    return hipGetLastError();
}

template <void (*FN)(W4Args), int MT, int NT>
static hipError_t launch_gemm(const W4Args& a, hipStream_t s) {
    using Sh = GemmShape<MT, NT>;
    return launch_blocks<FN, Sh::LDS>(a, (unsigned)((a.T + Sh::T - 1) / Sh::T * ((a.O + Sh::O - 1) / Sh::O)), kGemmThreads, s);
}

W4Shape w4_linear_shape(int64_t T, int32_t out_dim, int32_t group) {
    // Tiles of the many-token kernel where there are enough of them for the CUs, below that blocks that split K between
    // their waves.  Measured at K = 4096, many-token against few-token kernel: NVFP4 256 tiles 34.1 us against 32.3, 320
    // 41.0 against 45.8; INT4 320 tiles in groups of 32 81 against 68, of 64 61 against 63, of 128 62 against 59, 384 tiles
    // 83 against 71, 67 against 64 and 67 against 62; 512 tiles in groups of 32 91 against 109.  K is not looked at: with
    // K = 8192 the border lies higher (INT4 384 tiles 131..159 against 111..126), with K = 512 lower, where the few-token
    // blocks need a second round of the CUs (160 tiles NVFP4 7.4 against 12.0, INT4 9 against 12..14).
    const int64_t features = (out_dim + 127) / 128;
    if (T > 64 && (T + 63) / 64 * features > (group == 16 ? 256 : 384)) {
        // 128 tokens a block where that leaves two blocks per CU (K = 4096: 512 blocks NVFP4 75 us against 93, INT4 in
        // groups of 128 93 against 124; 256 blocks 55 against 48 and 84 against 66; 1024 blocks 144 against 180 and 181
        // against 229; just past 512 the last blocks run alone, 576 blocks 119 against 103 and 169 against 145)
        const bool tall = (group == 16 || group == 128) && (T + 127) / 128 * features >= 512;
        return {true, tall ? 8 : 4, 2};
    }
    const int mt = T <= 16 ? 1 : (T <= 32 ? 2 : 4);
    // Feature tiles of a block of 64 tokens: as few as keep one block per CU (its inputs fill the LDS; K = 4096, NVFP4: 64
    // tokens -> 4096 11.1 us in 256 blocks of one tile, 11.6 in 128 of two; -> 5120 18.0 in 320 of one, 11.5 in 160 of two;
    // 100 tokens -> 5003 24 in 626 of one, 20 in 314 of two, 16.3 in 158 of four; at K = 512 the same order).
    const int64_t rows = (T + 63) / 64;
    const int nt = mt < 4 || rows * ((out_dim + 15) / 16) <= 256 ? 1 : (rows * ((out_dim + 31) / 32) <= 256 ? 2 : 4);
    return {false, mt, nt};
}

hipError_t launch_w4_linear(const uint16_t* x, int64_t x_stride, const ple_w4_weight& w, int64_t T, uint16_t* out,
                            hipStream_t s) {
    const W4Args a = {x, x_stride, w.codes, w.scales, w.zeros, w.tensor_scale, T, w.out_dim, w.k_dim, out};
    const W4Shape shape = w4_linear_shape(T, w.out_dim, w.group);
    const int mt = shape.mt, nt = shape.nt;
    if (shape.many) switch (w.group) {
            case 16: return mt == 8 ? launch_gemm<w4_gemm_8x2_16_kernel, 8, 2>(a, s) : launch_gemm<w4_gemm_4x2_16_kernel, 4, 2>(a, s);
            case 32: return launch_gemm<w4_gemm_4x2_32_kernel, 4, 2>(a, s);
            case 64: return launch_gemm<w4_gemm_4x2_64_kernel, 4, 2>(a, s);
            default: return mt == 8 ? launch_gemm<w4_gemm_8x2_128_kernel, 8, 2>(a, s) : launch_gemm<w4_gemm_4x2_128_kernel, 4, 2>(a, s);
        }
    const unsigned blocks = (unsigned)((w.out_dim + 16 * nt - 1) / (16 * nt) * ((T + 16 * mt - 1) / (16 * mt)));
#define PLE_W4_LAUNCH(MT, NT, G, WAVES)       \
    if (mt == MT && nt == NT && w.group == G) \
        return launch_blocks<w4_rows_##MT##x##NT##_##G##_kernel, RowsShape<MT, NT, WAVES>::LDS>(a, blocks, WAVES * 64, s);
#define PLE_W4_LAUNCHES(MT, NT, WAVES, OCC)                               \
    PLE_W4_LAUNCH(MT, NT, 16, WAVES) PLE_W4_LAUNCH(MT, NT, 32, WAVES)     \
    PLE_W4_LAUNCH(MT, NT, 64, WAVES) PLE_W4_LAUNCH(MT, NT, 128, WAVES)
    PLE_W4_SHAPES(PLE_W4_LAUNCHES)
    return hipErrorInvalidValue;
}

}  // namespace ple
