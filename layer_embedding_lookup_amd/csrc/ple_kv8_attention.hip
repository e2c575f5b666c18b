// Causal attention over the paged 8-bit cache.
//
// Per query head with its rows q_i:  s_ij = scale <q_i, k_j>,  out_i = sum_j
// exp(s_ij) v_j / sum_j exp(s_ij), in one pass over the cache with a running
// maximum in fp32.  Rows, tiles of 64 tokens, page walks, splits and joins are
// those of ple_paged_attention.h; the products run on 16x16x32 MFMAs with the
// tokens (then the value elements) as the first operand, the queries as the
// second:  S^T [token][row] = K Q^T,  O^T [element][row] += V^T P^T.
//
// An e4m3 code is exact in bf16 and in fp16, so keys enter beside the bf16
// queries as codes and their block's scale multiplies the product.  The
// values' scale s_v of a block joins the exponent:
//   z_ij = s_ij log2 e + log2 s_v(j),  p_ij = 2^(z_ij - m_i),  m_i = max_j z_ij
//   out_i = sum_j p_ij code_j / sum_j p_ij / s_v(j)
// so that the weights of the value product (fp16) carry it without a product
// per element, and codes enter as they are.  Where the scales of the blocks
// that a wave goes through lie more than kFar apart, the light ones' weights
// would leave fp16 below the heavy ones': such a wave goes through its tiles
// once more with weights of two bf16 parts (FarWeights).
//
// Layouts, chosen so that nothing crosses lanes:
//  - MFMA i of a tile takes its token rows in the order row ρ <-> token
//    16 (ρ/4) + 4 i + ρ%4.  Lane (row n = lane%16, g = lane/16) of the result
//    holds rows ρ = 4g .. 4g+3, so after four MFMAs it holds tokens 16 g ..
//    16 g + 15 of its query row: one block of the cache, with one scale for
//    keys and one for values, and just what it supplies to the second product.
//  - a lane's 16 bytes of key codes are 16 elements of one token, four
//    neighbouring lanes' 64 contiguous bytes; its 16 bytes of value codes are
//    one element of 16 tokens, 16 lanes' 256 contiguous bytes.
//
// Few rows are bound by reading the cache: 256 requests of 3084 tokens on
// average 288 us, 5.6 TB/s, 89% of a copy's rate; one of 100100 tokens 43 us
// with the join of its 32 splits; 64 verify windows of four tokens 17.9, a
// chain of two to three tiles a wave.  Many rows: see there.
#include <type_traits>

#include "ple_8bit_launch.h"
#include "ple_paged_attention.h"

namespace ple {

union BFrag {
    bf16x8 v;
    uint32_t u[4];
};

// 8 codes (two words) as bf16 and as fp16.
__device__ __forceinline__ void fp8_to_bf16(uint32_t lo, uint32_t hi, BFrag& f) {
    f.u[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false));
    f.u[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true));
    f.u[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false));
    f.u[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true));
}
__device__ __forceinline__ void fp8_to_f16(uint32_t lo, uint32_t hi, Frag& f) {
    f.p[0] = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false));
    f.p[1] = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true));
    f.p[2] = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false));
    f.p[3] = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true));
}
// The queries of MT x 16 rows from row0 on: lane (n, g) holds, of row 16 mt + n, the elements that its key codes meet, and
// the tokens it sees.
template <int D, int MT>
__device__ __forceinline__ void kv8_queries(const Kv8AttentionArgs& a, const AttnTile& w, int row0, int head, int begin,
                                            int end, BFrag (&q)[MT][D / 32], int (&see_lo)[MT], int (&see_hi)[MT]) {
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int row = row0 + mt * 16 + n;
        const bool live = row < w.row1;
        const int i = row / a.group, hq = head * a.group + (row - i * a.group);
        const uint16_t* src = a.q + (w.first + i) * a.q_stride + hq * D + g * (D / 4);
#pragma unroll
        for (int ks = 0; ks < D / 32; ++ks) {
            const u32x4 x = live ? *(const u32x4*)(src + ks * 8) : u32x4{0u, 0u, 0u, 0u};
            q[mt][ks].v = __builtin_bit_cast(bf16x8, x);
        }
        const int p = w.before + i;
        // (rows past the tile's end, all zeros and never stored, see everything, which keeps the masks out of whole tiles)
        see_hi[mt] = live ? min(end, p + 1) : end;
        see_lo[mt] = live ? max(begin, a.window > 0 ? p - a.window + 1 : 0) : begin;
    }
}

// The scales of a lane's block in a tile: what turns its products into base-2 exponents, log2 of the values' scale, and
// one over it.  (A block that no token was written to may have any scale; its loaded one is looked at only here, since a
// load in a branch of its own makes the waits for those around it wait for it too.)
struct BlockScales {
    float key, log_value, per_value;
    __device__ __forceinline__ void set(float base, float k, float v, bool bad) {
        k = bad ? 1.f : k;
        v = bad ? 1.f : v;
        key = fminf(base * k, 3.4028234e38f);  // (an infinity would make NaN of products of 0)
        log_value = __builtin_amdgcn_logf(v);
        per_value = __builtin_amdgcn_rcpf(v);
    }
};

// Exponents from which on a product's rounding, as the maximum was rounded, is more than a weight's own: there the maximum
// is taken from the rounded products, not in one step with them.  `wide`: the wave has such rows.
constexpr float kWide = 4194304.0f;  // 2^22

// A lane's eight weights of a value product and the product itself.  In fp16: relative 2^-11, or 2^-24 beside weights of
// 2^8 and more (ple_paged_attention.h).
struct NearWeights {
    Frag p;
    __device__ __forceinline__ void set(int i, float x, float y) { p.p[i] = f16x2{(_Float16)x, (_Float16)y}; }
    __device__ __forceinline__ void unpack(uint32_t lo, uint32_t hi, Frag& f) const { fp8_to_f16(lo, hi, f); }
    __device__ __forceinline__ f32x4 product(const Frag& f, f32x4 c) const {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(f.v, p.v, c, 0, 0, 0);
    }
    typedef Frag Codes;
};
// As two bf16 each: relative 2^-16 down to fp32's least exponent, twice the products.
struct FarWeights {
    BFrag p, rest;
    __device__ __forceinline__ void set(int i, float x, float y) {
        p.u[i] = pack_bf16x2(x, y);
        rest.u[i] = pack_bf16x2(x - bf16_lo(p.u[i]), y - bf16_hi(p.u[i]));
    }
    __device__ __forceinline__ void unpack(uint32_t lo, uint32_t hi, BFrag& f) const { fp8_to_bf16(lo, hi, f); }
    __device__ __forceinline__ f32x4 product(const BFrag& f, f32x4 c) const {
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.v, rest.v, c, 0, 0, 0);
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.v, p.v, c, 0, 0, 0);
    }
    typedef BFrag Codes;
};

// How far apart the values' scales of a lane's blocks lie.  A block's weights are below those of equal softmax weight of the
// heaviest block by the scales' ratio r, so in fp16 a token's part of an element is off by 2^-33 r of its value beyond its
// rounding: by 2^-27 with the ratios that are left to it.  (A block has the largest of 16 tokens' values for its scale,
// which seldom differ by 2^4.)  Going through every tile twice takes 1.5 times as long for few rows (256 requests over 3084
// 495 us for 294), 2.1 times for many; watching the scales 0 to 2% (verify windows 18.5 us, 18.2 without).
constexpr float kFar = 64.0f;
struct ScaleRange {
    uint32_t low = 0x7F800000u, high = 0u;  // (as bits, which are in the order of the positive numbers)
    __device__ __forceinline__ void add(float v, bool bad) {
        low = min(low, bad ? 0x7F800000u : __float_as_uint(v));
        high = max(high, bad ? 0u : __float_as_uint(v));
    }
    // the wave's blocks (lanes n + 16 g all have those of block g)
    __device__ __forceinline__ bool far() const {
        const float least = __uint_as_float(low), most = __uint_as_float(high);
        return __ballot(quad_max(most) > -quad_max(-least) * kFar) != 0;
    }
};

// The weights of one tile: s (products, lane (n, g) holding tokens tg .. tg + 15 of MT rows) becomes the weights p;
// m, l and o (the rows' running maxima, sums and outputs) move on.  `some`: not every row sees the whole tile.
template <int NB, int MT, class Weights>
__device__ __forceinline__ void kv8_softmax(f32x4 (&s)[MT][4], const BlockScales& c, bool some, bool bad, int tg,
                                            const int (&see_lo)[MT], const int (&see_hi)[MT], float (&m)[MT], float (&l)[MT],
                                            f32x4 (&o)[MT][NB], bool& wide, Weights (&p)[MT][2]) {
    if (some) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int tok = tg + 4 * i + e;
                    if (bad || tok < see_lo[mt] || tok >= see_hi[mt]) s[mt][i][e] = -__builtin_inff();
                }
    }
    float mn[MT];
    bool up = false;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        float top = -__builtin_inff();
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) top = fmaxf(top, s[mt][i][e]);
        mn[mt] = fmaxf(m[mt], quad_max(fmaf(top, c.key, c.log_value)));  // (the scales are positive)
        up |= mn[mt] > m[mt] + kSlack;
    }
    if (__ballot(up) != 0) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            // (a row by itself, whatever the wave's others do: its result does not depend on them)
            const float next = mn[mt] > m[mt] + kSlack ? mn[mt] : m[mt];
            const float by = m[mt] == -__builtin_inff() ? 0.f : __builtin_amdgcn_exp2f(m[mt] - next);
            l[mt] *= by;
#pragma unroll
            for (int b = 0; b < NB; ++b) o[mt][b] *= by;
            m[mt] = next;
        }
        bool far = false;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) far |= fabsf(m[mt]) >= kWide && m[mt] != -__builtin_inff();
        wide |= __ballot(far) != 0;
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        float key = c.key, sub = c.log_value + (m[mt] == -__builtin_inff() ? 0.f : kWeightShift - m[mt]);
        if (wide) {
            const bool far = fabsf(m[mt]) >= kWide && m[mt] != -__builtin_inff();
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (far) s[mt][i][e] = fmaf(s[mt][i][e], key, c.log_value) - m[mt];
            if (far) {
                key = 1.f;
                sub = kWeightShift;
            }
        }
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                const float x = __builtin_amdgcn_exp2f(fmaf(s[mt][i][e], key, sub));
                const float y = __builtin_amdgcn_exp2f(fmaf(s[mt][i][e + 1], key, sub));
                sum += x + y;
                p[mt][i >> 1].set((i & 1) * 2 + e / 2, x, y);
            }
        l[mt] = fmaf(sum, c.per_value, l[mt]);
    }
}

// NaN elements of values in a tile that some row does not see as a whole would reach that row too, as 0 * NaN.  There they
// enter the product as zeros, and if there were any, the tiles are gone through once more at the end for the rows that do
// see one.

__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) >> 7 & 0x01010101u; }

// Value codes of a lane's block without those of tokens outside [lo, hi), which may be anything, and without NaN.  Returns
// whether the lane had NaN among the others.
template <int NB>
__device__ __forceinline__ bool kv8_clear(u32x4 (&v)[NB], bool bad, int tg, int lo, int hi) {
    uint32_t keep[4], found = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        keep[i] = 0u;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int tok = tg + 4 * i + e;
            if (!bad && tok >= lo && tok < hi) keep[i] |= 0xFFu << (8 * e);
        }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t x = v[b][i] & keep[i], is = nan_codes(x);
            v[b][i] = x & ~(is * 0xFFu);
            found |= is;
        }
    return found != 0u;
}

// The elements (bit 4 b + e: 16 b + 4 g + e) of the lane's rows that a NaN reaches, among the tiles at from, from + step ..
// below end: a product of ones for NaN elements and ones for seen tokens.
template <int D, int MT>
__device__ __forceinline__ void kv8_find_nans(const Kv8AttentionArgs& a, const int32_t* table_row, int head, int from, int step,
                                              int end, const int (&see_lo)[MT], const int (&see_hi)[MT], uint64_t (&nan)[MT]) {
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    for (int t0 = from; t0 < end; t0 += step) {
        const int tg = t0 + 16 * g;
        const int64_t grp = tg < end ? kv4_group(a.cache, table_row, head, tg >> 4) : -1;
#pragma unroll 1
        for (int b = 0; b < D / 16; ++b) {
            u32x4 v = {0u, 0u, 0u, 0u};
            if (grp >= 0) v = *(const u32x4*)(a.cache.v_codes + grp * (16 * D) + (b * 16 + n) * 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = nan_codes(v[i]);
            if (__ballot((v[0] | v[1] | v[2] | v[3]) != 0u) == 0) continue;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                f32x4 count = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    Frag is, sees;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int tok = tg + 8 * h + e;
                        is.v[e] = (_Float16)(v[2 * h + e / 4] >> (8 * (e % 4)) & 1u ? 1.f : 0.f);
                        sees.v[e] = (_Float16)(tok >= see_lo[mt] && tok < see_hi[mt] ? 1.f : 0.f);
                    }
                    count = __builtin_amdgcn_mfma_f32_16x16x32_f16(is.v, sees.v, count, 0, 0, 0);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (count[e] > 0.f) nan[mt] |= (uint64_t)1 << (4 * b + e);
            }
        }
    }
}

template <int NB, int MT>
__device__ __forceinline__ void kv8_give_nans(const uint64_t (&nan)[MT], f32x4 (&o)[MT][NB]) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        if (__ballot(nan[mt] != 0) == 0) continue;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (nan[mt] >> (4 * b + e) & 1u) o[mt][b][e] = __builtin_nanf("");
    }
}

// A wave's MT x 16 rows through the cache tiles at first, first + step .. below end: running maxima m, sums l and outputs o,
// NaN values found.  The next tile is on its way while this one is used, its page-table entry a tile before that, the
// queries (by `queries`) behind the first one.  Returns whether its blocks' scales are too far apart for NearWeights.
template <int D, int MT, class Weights, class Queries>
__device__ __forceinline__ bool kv8_tiles(const Kv8AttentionArgs& a, const AttnTile& w, const int32_t* table_row, int head,
                                          int first, int step, int end, BFrag (&q)[MT][D / 32], int (&see_lo)[MT],
                                          int (&see_hi)[MT], float (&m)[MT], float (&l)[MT], f32x4 (&o)[MT][D / 16],
                                          Queries queries) {
    constexpr int KS = D / 32, NB = D / 16;
    int lane = threadIdx.x & 63;
    // (the second pass's addresses are formed there, not held through the first one)
    if constexpr (std::is_same<Weights, FarWeights>::value) asm volatile("" : "+v"(lane));
    const int n = lane & 15, g = lane >> 4;
    const float base = a.scale * 1.44269504088896341f;
    bool wide = false, nans = false;
    ScaleRange range;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        m[mt] = -__builtin_inff();
        l[mt] = 0.f;
#pragma unroll
        for (int b = 0; b < NB; ++b) o[mt][b] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    bool bad_next = false;
    u32x4 kraw[4][D / 64], vraw[NB];
    float ks, vs;
    PageWalk walk(a, table_row, head, first + 16 * g, step / 16, end);
    int64_t block = 0;  // of the tile whose keys are on their way: this lane's
    auto load_keys = [&](int t0) {
        const int grp = walk.number(t0 + 16 * g, end);
        walk.fetch();
        bad_next = grp < 0;
        block = grp < 0 ? 0 : grp;
        ks = a.cache.k_scales[block];
        vs = a.cache.v_scales[block];
        // keys: block n / 4, token 4 i + n % 4
        const int64_t kg = __shfl((int)block, (n >> 2) * 16, kWave);
        const uint8_t* kc = a.cache.k_codes + kg * (16 * D) + g * (D / 64) * 256 + (n & 3) * 16;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < D / 64; ++c) kraw[i][c] = *(const u32x4*)(kc + c * 256 + i * 64);
    };
    auto load_values = [&]() {
        const uint8_t* vc = a.cache.v_codes + block * (16 * D) + n * 16;
#pragma unroll
        for (int b = 0; b < NB; ++b) vraw[b] = *(const u32x4*)(vc + b * 256);
    };
    if (first < end) {
        walk.fetch();
        load_keys(first);
        load_values();
    }
    queries();
    for (int t0 = first; t0 < end; t0 += step) {
        const int tg = t0 + 16 * g;  // this lane's block g of the tile
        const bool bad = bad_next;
        BlockScales c;
        c.set(base, ks, vs, bad);
        range.add(vs, bad);

        f32x4 s[MT][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            BFrag f[KS];
#pragma unroll
            for (int k = 0; k < KS; ++k) fp8_to_bf16(kraw[i][k / 2][2 * (k & 1)], kraw[i][k / 2][2 * (k & 1) + 1], f[k]);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                s[mt][i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < KS; ++k)
                    s[mt][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[k].v, q[mt][k].v, s[mt][i], 0, 0, 0);
            }
            __builtin_amdgcn_sched_barrier(0);  // (dequantised keys of one MFMA at a time: registers)
        }
        const bool more = t0 + step < end;
        if (more) load_keys(t0 + step);

        // a tile that not every row sees as a whole
        bool every = t0 >= w.first_seen && t0 + kTile <= end && __ballot(bad) == 0;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) every = every && t0 >= see_lo[mt] && t0 + kTile <= see_hi[mt];
        const bool some = __ballot(!every) != 0;
        Weights p[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)  // (one after the other: fewer registers than all of them together)
            kv8_softmax<NB, 1>((f32x4(&)[1][4])s[mt], c, some, bad, tg, (int(&)[1])see_lo[mt], (int(&)[1])see_hi[mt],
                               (float(&)[1])m[mt], (float(&)[1])l[mt], (f32x4(&)[1][NB])o[mt], wide, (Weights(&)[1][2])p[mt]);
        if (some) nans |= __ballot(kv8_clear<NB>(vraw, bad, tg, w.first_seen, end)) != 0;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                typename Weights::Codes f;
                p[0][h].unpack(vraw[b][2 * h], vraw[b][2 * h + 1], f);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) o[mt][b] = p[mt][h].product(f, o[mt][b]);
            }
            if (b % 2 == 1) __builtin_amdgcn_sched_barrier(0);
        }
        if (more) load_values();
    }
    if (nans) {
        uint64_t nan[MT] = {};
        kv8_find_nans<D, MT>(a, table_row, head, first, step, end, see_lo, see_hi, nan);
        kv8_give_nans<NB>(nan, o);
    }
    return range.far();
}

// The same with FarWeights, from the start, 16 rows after the other (registers).
template <int D, int MT>
__device__ __forceinline__ void kv8_far_tiles(const Kv8AttentionArgs& a, const AttnTile& w, const int32_t* table_row, int head,
                                              int first, int step, int end, BFrag (&q)[MT][D / 32], int (&see_lo)[MT],
                                              int (&see_hi)[MT], float (&m)[MT], float (&l)[MT], f32x4 (&o)[MT][D / 16]) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
        kv8_tiles<D, 1, FarWeights>(a, w, table_row, head, first, step, end, (BFrag(&)[1][D / 32])q[mt], (int(&)[1])see_lo[mt],
                                    (int(&)[1])see_hi[mt], (float(&)[1])m[mt], (float(&)[1])l[mt],
                                    (f32x4(&)[1][D / 16])o[mt], [] {});
}

// Few rows: the waves of a block take the tiles of a cache range in turn and join through LDS.
template <int D, int MT, int WAVES>
__device__ __forceinline__ void kv8_body(const Kv8AttentionArgs& a) {
    extern __shared__ __align__(16) char lds[];
    const int split = blockIdx.y;
    int r, head, tile;
    attn_block(a, r, head, tile);
    AttnTile w;
    attn_request(a, r, w);
    attn_idle_tokens(a);
    if (!attn_tile(a, tile, w)) return;
    const int splits = attn_splits(a, w);
    if (split >= splits) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int begin = w.lo + split * a.chunk;
    const int end = split == splits - 1 ? w.hi : min(w.hi, begin + a.chunk);
    const int first = begin + wave * kTile, step = WAVES * kTile;
    const int32_t* table_row = a.batch.page_table + (int64_t)r * a.batch.table_width;

    f32x4 o[MT][D / 16];
    float m[MT], l[MT];
    BFrag q[MT][D / 32];
    int see_lo[MT], see_hi[MT];
    const auto queries = [&]() { kv8_queries<D, MT>(a, w, w.row0, head, begin, end, q, see_lo, see_hi); };
    const bool far = kv8_tiles<D, MT, NearWeights>(a, w, table_row, head, first, step, end, q, see_lo, see_hi, m, l, o, queries);
    if (__builtin_expect(far, false))  // (its code out of the way)
        kv8_far_tiles<D, MT>(a, w, table_row, head, first, step, end, q, see_lo, see_hi, m, l, o);
    const uint32_t none[MT] = {};
    attn_join_waves<D, MT, WAVES>(a, w, head, split, splits, lds, m, l, o, none);
}

template <int D>
constexpr int kJoinLds = kAttnWaves * 16 * kJoinRow<D> * 4;
// D, row tiles, waves, waves per SIMD that registers allow
#define PLE_ATTN_SHAPES(X)                                                                                        \
    X(64, 1, 4, 4) X(64, 1, 8, 2) X(64, 2, 4, 2) X(64, 2, 8, 2) X(128, 1, 4, 2) X(128, 1, 8, 2) X(128, 2, 4, 2) \
    X(128, 2, 8, 2) X(256, 1, 4, 1)
#define PLE_ATTN_KERNEL(D, MT, WAVES, OCC)                                                                                  \
    __global__ __launch_bounds__(WAVES * kWave, OCC) void kv8_attention_##D##_##MT##x##WAVES##_kernel(Kv8AttentionArgs a) { \
        kv8_body<D, MT, WAVES>(a);                                                                                          \
    }
PLE_ATTN_SHAPES(PLE_ATTN_KERNEL)
#undef PLE_ATTN_KERNEL

// ---------------------------------------------------------------------------
// Many rows (a chunk of a prefill): a block's four waves hold 32 rows each and
// go through the cache tiles together; each wave dequantises a quarter of a
// tile (16 tokens of the keys, a quarter of the value elements) and leaves it
// in LDS as finished MFMA fragments, one 16-byte read per lane each, so a tile
// is dequantised once for 128 rows.
//
// A wave works on half a tile (8 tokens of each of its blocks) at a time and
// takes products and the rest in turns: beside the scores of one half stand
// the weights of the half before it, beside the value product of a half the
// next one's maxima, and the dequantising of the next tile.  The order is the
// source's, step by step (each step two MFMAs, a fragment's read three steps
// ahead, and its share of the other work): left to itself the compiler put
// every read right in front of its use, with the whole latency of LDS between
// MFMAs.  Two tiles in LDS, two barriers a tile.
//
// 1289 and 1455 tokens behind 5403 and 2004, 32 + 8 heads of 128: 237 us with
// products and the rest one after the other and reads not ahead, 217 with
// reads ahead, 209 in turns, 204 with the scales' loads out of their branch,
// 197 with row tiles that move on each by themselves and the join's loads all
// at once, 188 with the join told where cuts are, 184 with two pieces of it at a
// time, 187 with the values' scales watched (0.70 PFLOP/s, 17 us of it the join).  The SIMDs then issue vector instructions for 55% of the cycles that a
// CU is busy and their matrix cores are for 34%: two waves a SIMD, with all
// registers, overlap little more.  64 rows a wave, one wave a SIMD, halve the
// reads of LDS but take 277 us.
// ---------------------------------------------------------------------------
template <int D>
struct Kv8ChunkShape {
    static constexpr int MT = 2;
    static constexpr int KS = D / 32, NB = D / 16, WB = D / 64;  // WB: element blocks that a wave dequantises
    static constexpr int K_BYTES = 4 * KS * 1024, V_BYTES = NB * 2 * 1024;
    static constexpr int BUF = K_BYTES + V_BYTES;
    static constexpr int AHEAD = 3;             // fragments that a wave reads ahead
    static constexpr int NANS_AT = 2 * BUF;  // whether some wave has met NaN values
    static constexpr int LDS = NANS_AT + 16;
};

// Rows [w.row0, w.row1) against the cache's tokens [begin, end).  Results go to the call's outputs (at < 0), or to the
// partial results from row `at` on.
template <int D>
__device__ __forceinline__ void kv8_chunk_piece(const Kv8AttentionArgs& a, const AttnTile& w, int r, int head, int begin,
                                                int end, int at) {
    using Sh = Kv8ChunkShape<D>;
    constexpr int MT = Sh::MT, KS = Sh::KS, NB = Sh::NB, AHEAD = Sh::AHEAD;
    extern __shared__ __align__(16) char lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;
    const float base = a.scale * 1.44269504088896341f;
    // what every row of the block sees
    const int common_lo = a.window > 0 ? max(0, w.before + (w.row1 - 1) / a.group - a.window + 1) : 0;
    const int common_hi = min(end, w.before + w.row0 / a.group + 1);
    const int32_t* table_row = a.batch.page_table + (int64_t)r * a.batch.table_width;

    // a tile's quarter, as loaded, and its scales
    u32x4 kraw[D / 64], vraw[Sh::WB];
    float ks, vs;
    PageWalk walk(a, table_row, head, begin + 16 * g, kTile / 16, end);
    // of the tile to load next: the lane's block (-1: none), and block n / 4 of the tile
    int grp = -1;
    int64_t kg = 0;
    bool bad_loaded = false;
    auto aim = [&](int t0) {
        grp = walk.number(t0 + 16 * g, end);
        walk.fetch();
        kg = __shfl(max(grp, 0), (n >> 2) * 16, kWave);
    };
    auto load = [&]() {
        bad_loaded = grp < 0;
        const int64_t safe = max(grp, 0);
        ks = a.cache.k_scales[safe];
        vs = a.cache.v_scales[safe];
        // keys: token 4 wave + n % 4 of block n / 4
        const uint8_t* kc = a.cache.k_codes + kg * (16 * D) + g * (D / 64) * 256 + (4 * wave + (n & 3)) * 16;
        // values: elements 16 (wave WB + b) + n of block g
        const uint8_t* vc = a.cache.v_codes + safe * (16 * D) + (wave * Sh::WB * 16 + n) * 16;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            kraw[c] = *(const u32x4*)(kc + c * 256);
            vraw[c] = *(const u32x4*)(vc + c * 256);
        }
    };

    f32x4 o[MT][NB];
    float m[MT], l[MT];
    float limit[MT], shift[MT];  // m and the slack; what brings an exponent beside m to the weights' (without a maximum: 0)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        m[mt] = limit[mt] = -__builtin_inff();
        l[mt] = shift[mt] = 0.f;
#pragma unroll
        for (int b = 0; b < NB; ++b) o[mt][b] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    bool wide = false, nans = false;  // wide: see kWide
    ScaleRange range;
    if (threadIdx.x == 0) *(volatile int*)(lds + Sh::NANS_AT) = 0;
    // the first tile is on its way before the queries are
    if (begin < end) {
        walk.fetch();
        aim(begin);
        load();
        aim(begin + kTile);
    }
    BFrag q[MT][KS];
    int see_lo[MT], see_hi[MT];
    kv8_queries<D, MT>(a, w, w.row0 + wave * (16 * MT), head, begin, end, q, see_lo, see_hi);

    // not every row of the block sees the whole tile at t0 (the same for all its waves: `bad` is the tile's four blocks)
    auto partial = [&](int t0, bool bad) {
        return t0 < common_lo || t0 < begin || t0 + kTile > common_hi || __ballot(bad) != 0;
    };
    // the quarter that is loaded, into a buffer: group c of KS + 2 WB of 16 bytes a lane
    auto fill = [&](int buf, int c) {
        if (c < KS) {
            BFrag f;
            fp8_to_bf16(kraw[c / 2][2 * (c & 1)], kraw[c / 2][2 * (c & 1) + 1], f);
            *(bf16x8*)(lds + buf * Sh::BUF + lane * 16 + (wave * KS + c) * 1024) = f.v;
        } else {
            const int b = (c - KS) / 2, h = (c - KS) & 1;
            Frag f;
            fp8_to_f16(vraw[b][2 * h], vraw[b][2 * h + 1], f);
            *(u32x4*)(lds + buf * Sh::BUF + Sh::K_BYTES + lane * 16 + ((wave * Sh::WB + b) * 2 + h) * 1024) = f.u;
        }
    };
    constexpr int FILLS = KS + 2 * Sh::WB;
    f32x4 s[MT][2];
    // the scores of half h of a buffer's tile (fragment 4 i + k: tokens of MFMA i), with `beside(step)` beside them
    auto scores = [&](int buf, int h, f32x4 (&to)[MT][2], auto beside) {
        const char* kb = lds + buf * Sh::BUF + lane * 16 + 2 * h * KS * 1024;
        constexpr int N = 2 * KS;
        bf16x8 f[AHEAD];
#pragma unroll
        for (int c = 0; c < AHEAD; ++c) f[c] = *(const bf16x8*)(kb + c * 1024);
#pragma unroll
        for (int c = 0; c < N; ++c) {
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
                to[mt][c / KS] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    f[c % AHEAD], q[mt][c % KS].v, c % KS == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : to[mt][c / KS], 0, 0, 0);
            if (c + AHEAD < N) f[c % AHEAD] = *(const bf16x8*)(kb + (c + AHEAD) * 1024);
            beside(c, N);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    auto mask = [&](int t0, int h, bool bad, f32x4 (&x)[MT][2]) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int tok = t0 + 16 * g + 8 * h + 4 * i + e;
                    if (bad || tok < see_lo[mt] || tok >= see_hi[mt]) x[mt][i][e] = -__builtin_inff();
                }
    };
    // the maxima of scores that are here: step c of n
    auto maxima = [&](const f32x4 (&x)[MT][2], float (&top)[MT], int c, int n) {
#pragma unroll
        for (int k = 0; k < 4 * MT; ++k)
            if (k * n / (4 * MT) == c) {
                const f32x4& y = x[k / 4][k / 2 % 2];
                top[k / 4] = k % 4 == 0 ? fmaxf(y[0], y[1]) : fmaxf(fmaxf(top[k / 4], y[k % 2 * 2]), y[k % 2 * 2 + 1]);
                asm volatile("" : "+v"(top[k / 4]));  // (at its step)
            }
    };
    // Rows whose maximum passes the running one by more than the slack move on, each by itself, whatever the wave's others
    // do (their four lanes' maxima are joined only there).
    auto move_on = [&](const float (&top)[MT], const BlockScales& c) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            if (__ballot(fmaf(top[mt], c.key, c.log_value) > limit[mt]) == 0) continue;
            const float mn = quad_max(fmaf(top[mt], c.key, c.log_value));
            const float next = mn > limit[mt] ? mn : m[mt];
            const float by = m[mt] == -__builtin_inff() ? 0.f : __builtin_amdgcn_exp2f(m[mt] - next);
            l[mt] *= by;
#pragma unroll
            for (int b = 0; b < NB; ++b) o[mt][b] *= by;
            m[mt] = next;
            limit[mt] = next + kSlack;
            shift[mt] = next == -__builtin_inff() ? 0.f : kWeightShift - next;
            wide |= __ballot(fabsf(next) >= kWide && next != -__builtin_inff()) != 0;
        }
    };
    // of the half that is weighed: weights are 2^(product * key + sub)
    float key[MT], sub[MT], sum[MT];
    auto weigh = [&](f32x4 (&x)[MT][2], const BlockScales& c) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            key[mt] = c.key;
            sub[mt] = c.log_value + shift[mt];
        }
        if (wide)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                if (!(fabsf(m[mt]) >= kWide && m[mt] != -__builtin_inff())) continue;
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[mt][i][e] = fmaf(x[mt][i][e], key[mt], c.log_value) - m[mt];
                key[mt] = 1.f;
                sub[mt] = kWeightShift;
            }
    };
    // two of a lane's weights of each row tile at a time: step c of n
    auto weights = [&](const f32x4 (&x)[MT][2], Frag (&p)[MT], int c, int n) {
#pragma unroll
        for (int k = 0; k < 4 * MT; ++k)
            if (k * n / (4 * MT) == c) {
                const int mt = k / 4, i = k / 2 % 2, e = k % 2 * 2;
                const float y = __builtin_amdgcn_exp2f(fmaf(x[mt][i][e], key[mt], sub[mt]));
                const float z = __builtin_amdgcn_exp2f(fmaf(x[mt][i][e + 1], key[mt], sub[mt]));
                sum[mt] = k % 4 == 0 ? y + z : sum[mt] + (y + z);
                p[mt].p[i * 2 + e / 2] = f16x2{(_Float16)y, (_Float16)z};
                uint32_t here = p[mt].u[i * 2 + e / 2];
                asm volatile("" : "+v"(here), "+v"(sum[mt]));  // (at their step)
                p[mt].u[i * 2 + e / 2] = here;
            }
    };
    auto weighed = [&](const BlockScales& c) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) l[mt] = fmaf(sum[mt], c.per_value, l[mt]);
    };
    // the value product of half h
    auto values = [&](int buf, int h, const Frag (&p)[MT], auto beside) {
        const char* vb = lds + buf * Sh::BUF + Sh::K_BYTES + lane * 16 + h * 1024;
        f16x8 f[AHEAD];
#pragma unroll
        for (int b = 0; b < AHEAD; ++b) f[b] = *(const f16x8*)(vb + b * 2048);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
                o[mt][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f[b % AHEAD], p[mt].v, o[mt][b], 0, 0, 0);
            if (b + AHEAD < NB) f[b % AHEAD] = *(const f16x8*)(vb + (b + AHEAD) * 2048);
            beside(b, NB);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    const auto nothing = [](int, int) {};
    if (begin < end) {
        BlockScales c, c_next;
        float top[MT];
        bool bad = bad_loaded, some = partial(begin, bad), bad_next, some_next;
        const auto clear = [&](int t0) {
            int tg = t0 + 16 * g;
            asm volatile("" : "+v"(tg));  // (what follows from it is formed here, not for every tile)
            nans |= kv8_clear<Sh::WB>(vraw, bad_loaded, tg, w.first_seen, end);
        };
        c.set(base, ks, vs, bad);
        range.add(vs, bad);
        if (some) clear(begin);
#pragma unroll
        for (int i = 0; i < FILLS; ++i) fill(0, i);
        load();  // (past the last tile: the cache's first block, which nothing comes of)
        aim(begin + 2 * kTile);
        __syncthreads();
        scores(0, 0, s, nothing);
        if (some) mask(begin, 0, bad, s);
#pragma unroll
        for (int i = 0; i < 4; ++i) maxima(s, top, i, 4);
        move_on(top, c);
        int buf = 0;
        for (int t0 = begin;; t0 += kTile) {
            f32x4 x[MT][2];
            Frag p[MT];
            // first half's weights, second half's scores
            weigh(s, c);
            scores(buf, 1, x, [&](int i, int n) { weights(s, p, i, n); });
            weighed(c);
            if (some) mask(t0, 1, bad, x);
            bad_next = bad_loaded;
            some_next = partial(t0 + kTile, bad_next);
            c_next.set(base, ks, vs, bad_next);
            range.add(vs, bad_next);
            if (some_next) clear(t0 + kTile);
            __syncthreads();  // every read of the other buffer is done
            // first half's values; second half's maxima and the next tile into LDS
            values(buf, 0, p, [&](int i, int n) {
                maxima(x, top, i, n);
#pragma unroll
                for (int k = 0; k < FILLS; ++k)
                    if (k * n / FILLS == i) fill(buf ^ 1, k);
            });
            move_on(top, c);
            load();
            aim(t0 + 3 * kTile);
            __syncthreads();  // the next tile is whole
            // second half's weights, the next tile's first half's scores (where there is none: of no use)
            weigh(x, c);
            scores(buf ^ 1, 0, s, [&](int i, int n) { weights(x, p, i, n); });
            weighed(c);
            if (some_next) mask(t0 + kTile, 0, bad_next, s);
            // second half's values, the next tile's first half's maxima
            values(buf, 1, p, [&](int i, int n) { maxima(s, top, i, n); });
            if (t0 + kTile >= end) break;
            move_on(top, c_next);
            c = c_next;
            bad = bad_next;
            some = some_next;
            buf ^= 1;
        }
    }

    // (all waves agree: each has gone by the scales of all blocks)
    if (__builtin_expect(range.far(), false))
        kv8_far_tiles<D, MT>(a, w, table_row, head, begin, kTile, end, q, see_lo, see_hi, m, l, o);
    // (a wave has met its quarter of the elements alone)
    if (nans) *(volatile int*)(lds + Sh::NANS_AT) = 1;
    __syncthreads();
    nans = *(volatile int*)(lds + Sh::NANS_AT) != 0;
    if (nans) {
        uint64_t nan[MT] = {};
        kv8_find_nans<D, MT>(a, table_row, head, begin, kTile, end, see_lo, see_hi, nan);
        kv8_give_nans<NB>(nan, o);
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        float total = l[mt];
        total += __shfl_xor(total, 16, kWave);
        total += __shfl_xor(total, 32, kWave);
        const int row = w.row0 + wave * (16 * MT) + mt * 16 + n;
        if (row >= w.row1) continue;
        const float inv = total == 0.f ? 0.f : 1.f / total;
        const float lse2 = total == 0.f ? -__builtin_inff() : (m[mt] - kWeightShift) + log2f(total);
        const int i = row / a.group, hq = head * a.group + (row - i * a.group);
        const int64_t orow = (w.first + i) * a.num_q_heads + hq;
        const int64_t place = at + (row - w.row0);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const f32x4 v = o[mt][b] * inv;
            if (at < 0)
                *(u32x2*)(a.out + orow * D + b * 16 + g * 4) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
            else
                *(f32x4*)(a.part + place * D + b * 16 + g * 4) = v;
        }
        if (g == 0) {
            if (at >= 0)
                a.part[(int64_t)2 * a.flat * kChunkRows * D + place] = lse2;
            else if (a.lse != nullptr)
                a.lse[orow] = lse2 * 0.693147180559945309f;
        }
    }
}

#define PLE_ATTN_KERNEL(D, OCC)                                                                                         \
    __global__ __launch_bounds__(kAttnThreads, OCC) void kv8_attention_chunk_##D##_kernel(Kv8AttentionArgs a) {         \
        attn_chunk_body(a, [&](const AttnTile& w, int r, int head, int begin, int end, int at) {                        \
            kv8_chunk_piece<D>(a, w, r, head, begin, end, at);                                                          \
        });                                                                                                             \
    }
PLE_ATTN_KERNEL(64, 2)
PLE_ATTN_KERNEL(128, 2)
PLE_ATTN_KERNEL(256, 1)
#undef PLE_ATTN_KERNEL

#define PLE_ATTN_KERNEL(D)                                                                                  \
    __global__ __launch_bounds__(256) void kv8_attention_join_##D##_1_kernel(Kv8AttentionArgs a) {          \
        attn_join_body<D, 1>(a);                                                                            \
    }                                                                                                       \
    __global__ __launch_bounds__(256) void kv8_attention_join_##D##_4_kernel(Kv8AttentionArgs a) {          \
        attn_join_body<D, 4>(a);                                                                            \
    }                                                                                                       \
    __global__ __launch_bounds__(256) void kv8_attention_flat_join_##D##_kernel(Kv8AttentionArgs a) {       \
        attn_flat_join_body<D>(a);                                                                          \
    }
PLE_ATTN_KERNEL(64)
PLE_ATTN_KERNEL(128)
PLE_ATTN_KERNEL(256)
#undef PLE_ATTN_KERNEL

// Many rows: their query tiles are cut into equal shares where the shortest of a call go through many cache tiles, or where
// there are many.  Shares cost finding and joining, 10 to 25 us; a block a query tile leaves CUs to wait for the last ones,
// which are the shortest since the longest go first.  In shares and a block each, new tokens behind cached ones: 100 behind
// 1000 and 1400 33 and 40, 34 and 48 us; 2 x 1000 behind 1000 114 and 118; 8 x 200 behind 1200 62 and 59; 8 x 500 behind 1500
// 122 and 127; 16 x 300 behind 2000 160 and 195; 2 x 1500 behind 5000 196 and 269; 100, 1000, 2000 and 4000 behind nothing (32
// to 1000 query tiles) 28 and 14, 50 and 39, 84 and 70, 192 and 172; 8 x 1000 behind nothing and 16 x 480 behind 500 (2000
// tiles) 175 and 183, 146 and 158; 30 x 300 behind 3000 (2400) 428 and 435; 4 x 800 behind 900, D = 64, 88 and 80.  With heads
// of 256, one block per CU, shares gain from fewer on: 2000 and 4 x 1000 behind nothing (250 and 500 tiles) 101 and 111, 107
// and 122; 4 x 1000 behind 1000 156 and 244; 100 behind 600 and 1200 48 and 49, 50 and 78; 2 x 500 behind 400 55 and 54.
// How long the shortest tiles are is not known here: it is taken for what the hints (or the table and T) leave, the most
// cached tokens that a request with the most new ones can have.  Where one request has them and the others none: 4 x 500, one
// behind 6000, 118 and 220, behind 1000 67 and 64; 2 x 1000, one behind 8000 212 and 290, behind 1000 85 and 77; 8 x 100, one
// behind 2000, 49 and 64.
constexpr int kFlatPast = 896, kFlatPastWide = 384;  // cache tokens in front of the new ones
constexpr int kFlatTiles = 1536, kFlatTilesWide = 192;

// Few rows: splits of at least 1024 tokens (8 requests of up to 2500 tokens 15.9 us, with 512 15.6, 2048 16.3; one of 777
// 11.0, 15.4, 11.3; one of 10000 16.5, 16.1, 18.1; 8 x 4 windows over 9000 19.1, 19.1, 23.6).  Up to one block per CU blocks of
// eight waves (one of 100100 tokens 45.3 us, of four in more splits 49.0; verify windows 64 x 4 18.3 and 23.9; 32 over 2000
// 17.3 and 21.1; two of eight waves per CU: the windows 30.7, 4 over 20000 22.7 for 18.5).  Blocks of four waves in as many
// splits as two to four of them per CU: 16 rows and 512, 768 or 1024 slots: 33 requests over 8000 65.6, 69.7 and 61.4 us, 40
// over 4000 47.5, 41.5 and 40.3, 64 over 8000 109.4, 109.5 and 112.4.
void plan_kv8_attention(Kv8AttentionArgs& a) {
    const int64_t T = a.batch.num_tokens, R = a.batch.num_reqs;
    const int64_t cover = (int64_t)a.batch.table_width * a.cache.page_size;
    int64_t new_max = a.batch.max_request_tokens > 0 ? a.batch.max_request_tokens : T;
    new_max = new_max < T ? new_max : T;
    int64_t len = a.batch.max_seq_len > 0 && a.batch.max_seq_len < cover ? a.batch.max_seq_len : cover;
    const int64_t rows = new_max * a.group;
    a.rows = rows <= 16 || (rows <= 64 && a.cache.head_dim == 256) ? 16 : (rows <= 64 ? 32 : kChunkRows);
    a.tiles = (int)((rows + a.rows - 1) / a.rows);
    int64_t past = len - new_max;  // cache tokens in front of the new ones, by the largest of each
    if (a.window > 0) {
        const int64_t span = (int64_t)a.window + a.rows / a.group + 1 + 15;
        len = len < span ? len : span;
        past = past < len ? past : len;
    }
    const int64_t blocks = R * a.cache.num_kv_heads * a.tiles;
    // (the line's length has to fit 32 bits whatever the hints say)
    const bool wide = a.cache.head_dim == 256;
    if (a.rows == kChunkRows && R <= kWave && blocks > 0 && blocks <= kFlatUnits &&
        (past >= (wide ? kFlatPastWide : kFlatPast) || blocks >= (wide ? kFlatTilesWide : kFlatTiles)) &&
        blocks * (cover / kTile + 2 + kFlatStart) < ((int64_t)1 << 30)) {
        const int64_t most = blocks * ((len + kTile - 1) / kTile + 1 + kFlatStart), slots = a.cache.head_dim == 256 ? 256 : 512;
        const int64_t shares = (most + kFlatLeast - 1) / kFlatLeast;
        a.flat = (int)(shares < slots ? shares : slots);
        a.waves = kAttnWaves;
        a.splits = 1;
        return;
    }
    a.waves = blocks <= 256 && a.rows < kChunkRows && a.cache.head_dim < 256 ? 8 : 4;
    const int64_t slots = a.waves == 8 || a.cache.head_dim == 256 ? 256 : (a.rows == 16 ? 1024 : 512);
    int64_t splits = blocks <= 0 || a.rows == kChunkRows ? 1 : slots / blocks;
    const int64_t most_splits = (len + 1023) / 1024;
    splits = splits < most_splits ? splits : most_splits;
    splits = splits < 1 ? 1 : (splits < kMostSplits - 1 ? splits : kMostSplits - 1);
    int64_t chunk = (len + splits - 1) / splits;
    const int64_t round = a.rows == kChunkRows || a.waves == 8 ? kTile : kTile * a.waves;
    chunk = (chunk + round - 1) / round * round;
    a.chunk = (int)chunk;
    // (a range starts at a multiple of 16, up to 15 tokens before the first that is seen; the last split takes those)
    a.splits = (int)((len + chunk - 1) / chunk);
    if (a.splits < 1) a.splits = 1;
}

size_t kv8_attention_part_bytes(const Kv8AttentionArgs& a) { return attention_part_bytes(a); }
int64_t kv8_attention_threads(const Kv8AttentionArgs& a) { return attention_threads(a); }

hipError_t launch_kv8_attention(const Kv8AttentionArgs& a, hipStream_t s) {
    const int D = a.cache.head_dim, mt = a.rows / 16;
    hipError_t e = hipErrorInvalidValue;
    if (a.rows == kChunkRows)
        e = D == 64    ? launch_attention<Kv8AttentionArgs, kv8_attention_chunk_64_kernel, Kv8ChunkShape<64>::LDS>(a, kAttnThreads, s)
            : D == 128 ? launch_attention<Kv8AttentionArgs, kv8_attention_chunk_128_kernel, Kv8ChunkShape<128>::LDS>(a, kAttnThreads, s)
                       : launch_attention<Kv8AttentionArgs, kv8_attention_chunk_256_kernel, Kv8ChunkShape<256>::LDS>(a, kAttnThreads, s);
#define PLE_ATTN_LAUNCH(DD, MT, WAVES, OCC)                                                                              \
    if (D == DD && mt == MT && a.waves == WAVES)                                                                         \
        e = launch_attention<Kv8AttentionArgs, kv8_attention_##DD##_##MT##x##WAVES##_kernel, kJoinLds<DD>>(  \
            a, WAVES * kWave, s);
    PLE_ATTN_SHAPES(PLE_ATTN_LAUNCH)
#undef PLE_ATTN_LAUNCH
    if (e != hipSuccess) return e;
#define PLE_ATTN_LAUNCH(DD)                                                                                         \
    if (D == DD)                                                                                                    \
        return launch_attention_join(a, kv8_attention_join_##DD##_1_kernel, kv8_attention_join_##DD##_4_kernel,     \
                                     kv8_attention_flat_join_##DD##_kernel, s);
    PLE_ATTN_LAUNCH(64)
    PLE_ATTN_LAUNCH(128)
    PLE_ATTN_LAUNCH(256)
#undef PLE_ATTN_LAUNCH
    return hipErrorInvalidValue;
}

}  // namespace ple
