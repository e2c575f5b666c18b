// Causal attention over the paged 4-bit cache.
//
// Per query head with its rows q_i:  s_ij = scale <q_i, k_j>,  out_i = sum_j
// exp(s_ij - m_i) v_j / sum_j exp(s_ij - m_i), in one pass over the cache with
// the running maximum m_i and sum in fp32.
//
// The query heads that share a key head, times the request's new tokens, are
// the rows of one tile (row = token * group + head), so a key is read once
// for all of them.  Tokens of the cache go by in tiles of 64.  Both products
// run on 16x16x32 fp16 MFMAs with the tokens (then the value elements) as the
// first operand and the queries as the second:
//   S^T [token][row] = K Q^T,   O^T [element][row] += V^T P^T
// A 4-bit code times its block's e4m3 scale is exact in fp16 (6 significant
// bits, 2^-10 .. 2688), so dequantising costs one conversion and one packed
// multiply per two elements.  Queries are scaled by a power of two per row
// that puts the row's largest finite value at 2^14..2^15 (fp16 then holds
// them to 2^-39 of that), taken back out in fp32 together with the softmax
// scale and the head's key scale.
//
// Layouts, chosen so that nothing but the values' codes crosses lanes:
//  - MFMA i of a tile takes its token rows in the order row ρ <-> token
//    16 (ρ/4) + 4 i + ρ%4.  Lane (row n = lane%16, g = lane/16) of the result
//    holds rows ρ = 4g .. 4g+3, so after four MFMAs it holds tokens 16 g ..
//    16 g + 15 of its query row, which is just what it supplies to the second
//    product (8 consecutive k per lane and MFMA).
//  - a lane's 16 bytes of key codes are 32 elements of one token, which are
//    its operands of four MFMAs; the queries are laid out to match.
//  - value codes lie along the elements but enter along the tokens: they are
//    staged in LDS and come back through the transposing 4-bit read.
#include "ple_fp4_launch.h"

namespace ple {

constexpr int kAttnWaves = 4;
constexpr int kAttnThreads = kAttnWaves * kWave;
constexpr int kTile = 64;  // cache tokens of a tile
constexpr int kMostSplits = 1024;
// Weights are 2^(s - m + kWeightShift): fp16 keeps them above 2^-24, so tokens down to 2^-32 of the heaviest one count.
constexpr float kWeightShift = 8.0f;

// What a block's query tile sees: rows [row0, row1) of request r, cache tokens [lo, hi).
struct AttnTile {
    int64_t first;  // first new token of the request
    int n, len;     // its new tokens, its length
    int row0, row1;
    int first_seen;  // the first token that any row sees
    int lo, hi;      // lo: first_seen rounded down to a group of 16
};

__device__ __forceinline__ bool attn_tile(const Kv4AttentionArgs& a, int r, int tile, AttnTile& w) {
    int64_t q0, q1;
    carried_window(a.batch.query_start_loc, a.batch.num_tokens, r, nullptr, q0, q1);
    w.first = q0;
    w.n = (int)(q1 - q0);
    w.len = min(a.batch.seq_lens[r], a.batch.table_width * a.cache.page_size);
    w.row0 = tile * a.rows;
    w.row1 = min(w.row0 + a.rows, w.n * a.group);
    if (w.row0 >= w.row1) return false;
    const int before = w.len - w.n;  // position of new token 0
    w.hi = max(0, min(w.len, before + (w.row1 - 1) / a.group + 1));
    w.first_seen = a.window > 0 ? max(0, before + w.row0 / a.group - a.window + 1) : 0;
    w.lo = min(w.first_seen & ~15, w.hi & ~15);
    return true;
}

__device__ __forceinline__ int attn_splits(const Kv4AttentionArgs& a, const AttnTile& w) {
    const int s = (w.hi - w.lo + a.chunk - 1) / a.chunk;
    return max(1, min(s, a.splits));
}

__device__ __forceinline__ f16x2 fp4_pair(uint32_t w, int byte) {
    switch (byte) {
        case 0: return __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0));
        case 1: return __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1));
        case 2: return __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2));
        default: return __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3));
    }
}
__device__ __forceinline__ f16x2 fp8_pair(uint32_t w, bool hi) {
    return hi ? __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true))
              : __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false));
}

union Frag {
    f16x8 v;
    f16x2 p[4];
    u32x4 u;
};

template <int D>
struct AttnShape {
    static constexpr int KS = D / 32;                   // k-steps of the first product
    static constexpr int NB = D / 16;                   // element blocks
    static constexpr int NV = D / 32;                   // 16-byte loads of a lane per tile of codes
    static constexpr int VROW = D / 2 + 8;              // a token's codes in LDS: the 8 bytes spread 16 rows over the banks
    static constexpr int SROW = D * 2 + 16;             // a group's value scales in LDS, as fp16
    static constexpr int WAVE_LDS = kTile * VROW + 4 * SROW;
    static constexpr int OROW = D + 4;                  // the join's rows (fp32)
    static constexpr int JOIN_LDS = kAttnWaves * 16 * OROW * 4;
    static constexpr int LDS = WAVE_LDS * kAttnWaves > JOIN_LDS ? WAVE_LDS * kAttnWaves : JOIN_LDS;
};

template <int D, int MT>
__device__ __forceinline__ void attn_body(const Kv4AttentionArgs& a) {
    using Sh = AttnShape<D>;
    __shared__ __align__(16) char lds[Sh::LDS];
    __shared__ float join_m[kAttnWaves][16], join_l[kAttnWaves][16];
    const int heads = a.cache.num_kv_heads;
    const int pair = blockIdx.x / a.tiles, tile = blockIdx.x - pair * a.tiles;
    const int r = pair / heads, head = pair - r * heads;
    const int split = blockIdx.y;
    AttnTile w;
    if (!attn_tile(a, r, tile, w)) return;
    const int splits = attn_splits(a, w);
    if (split >= splits) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n = lane & 15, g = lane >> 4;
    const int begin = w.lo + split * a.chunk;
    const int end = split == splits - 1 ? w.hi : min(w.hi, begin + a.chunk);
    const int before = w.len - w.n;

    // queries: lane (n, g) holds, of row 16 mt + n, the elements that its key codes meet
    f16x8 q[MT][Sh::KS];
    float qs[MT];        // what turns a row's products into base-2 exponents
    int see_lo[MT], see_hi[MT];
    const float base = a.scale * 1.44269504088896341f * a.cache.k_scale[head];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int row = w.row0 + mt * 16 + n;
        const bool live = row < w.row1;
        const int i = row / a.group, hq = head * a.group + (row - i * a.group);
        const uint16_t* src = a.q + (w.first + i) * a.q_stride + hq * D;
        u32x4 raw[Sh::KS];
        float top = 0.f;
#pragma unroll
        for (int ks = 0; ks < Sh::KS; ++ks) {
            // D = 64: 16 elements a lane; else 32 elements of each 128
            const int d = D == 64 ? g * 16 + ks * 8 : (ks / 4) * 128 + g * 32 + (ks % 4) * 8;
            raw[ks] = live ? *(const u32x4*)(src + d) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x = fabsf(bf16_lo(raw[ks][e])), y = fabsf(bf16_hi(raw[ks][e]));
                if (x < __builtin_inff()) top = fmaxf(top, x);
                if (y < __builtin_inff()) top = fmaxf(top, y);
            }
        }
        top = fmaxf(top, __shfl_xor(top, 16, kWave));
        top = fmaxf(top, __shfl_xor(top, 32, kWave));
        // 2^(14 - exponent of top), within fp32 for every bf16 top
        const int e = top > 0.f ? min(max((int)(__float_as_uint(top) >> 23) - 127, -110), 127) : 14;
        const float up = __uint_as_float((uint32_t)(14 - e + 127) << 23);
        qs[mt] = base * __uint_as_float((uint32_t)(max(e - 14 + 127, 1)) << 23);
#pragma unroll
        for (int ks = 0; ks < Sh::KS; ++ks)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                q[mt][ks][2 * j] = (_Float16)(bf16_lo(raw[ks][j]) * up);
                q[mt][ks][2 * j + 1] = (_Float16)(bf16_hi(raw[ks][j]) * up);
            }
        const int p = before + i;
        // (rows past the tile's end, all zeros and never stored, see everything, which keeps the masks out of whole tiles)
        see_hi[mt] = live ? min(end, p + 1) : end;
        see_lo[mt] = live ? max(begin, a.window > 0 ? p - a.window + 1 : 0) : begin;
    }

    f32x4 o[MT][Sh::NB];
    float m[MT], l[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        m[mt] = -__builtin_inff();
        l[mt] = 0.f;
#pragma unroll
        for (int b = 0; b < Sh::NB; ++b) o[mt][b] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    char* vt = lds + wave * Sh::WAVE_LDS;
    char* vs = vt + kTile * Sh::VROW;
    const int32_t* table_row = a.batch.page_table + (int64_t)r * a.batch.table_width;
    const uint32_t pick = (uint32_t)((n & 3) | ((4 + (n & 3)) << 8));

    for (int t0 = begin + wave * kTile; t0 < end; t0 += kAttnWaves * kTile) {
        // this lane's group g of the tile
        const int tg = t0 + 16 * g;
        int grp = -1;
        if (tg < end) grp = kv4_group(a.cache, table_row, head, tg >> 4);
        const bool bad = grp < 0;
        const int safe = bad ? 0 : grp;
        // keys: group n / 4, token 4 i + n % 4
        const int64_t kg = __shfl(safe, (n >> 2) * 16, kWave);
        const uint8_t* kc = a.cache.k_codes + kg * (8 * D) + (n & 3) * (D / 2) + g * (D == 64 ? 8 : 16);
        const uint8_t* ksc = a.cache.k_scales + kg * D + (D == 64 ? g * 16 : g * 32);
        u32x4 kraw[4][D == 256 ? 2 : 1];
        u32x4 kscale[D == 64 ? 1 : D / 64];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (D == 64) {
                const u32x2 x = *(const u32x2*)(kc + i * 4 * (D / 2));
                kraw[i][0] = u32x4{x[0], x[1], 0u, 0u};
            } else {
#pragma unroll
                for (int c = 0; c < D / 128; ++c) kraw[i][c] = *(const u32x4*)(kc + i * 4 * (D / 2) + c * 64);
            }
        }
        if constexpr (D == 64) {
            kscale[0] = *(const u32x4*)ksc;
        } else {
#pragma unroll
            for (int c = 0; c < D / 128; ++c) {
                kscale[2 * c] = *(const u32x4*)(ksc + c * 128);
                kscale[2 * c + 1] = *(const u32x4*)(ksc + c * 128 + 16);
            }
        }
        // values: codes by 1 KiB a load, scales by D/16 bytes a lane
        u32x4 vraw[Sh::NV];
#pragma unroll
        for (int j = 0; j < Sh::NV; ++j) {
            const int at = j * 1024 + lane * 16;
            const int64_t vg = __shfl(safe, (at / (8 * D)) * 16, kWave);
            vraw[j] = *(const u32x4*)(a.cache.v_codes + vg * (8 * D) + at % (8 * D));
        }
        uint32_t vsc[D / 64];
        {
            const uint8_t* p = a.cache.v_scales + (int64_t)safe * D + n * (D / 16);
#pragma unroll
            for (int j = 0; j < D / 64; ++j) vsc[j] = ((const uint32_t*)p)[j];
        }

        // S^T
        f32x4 s[MT][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            Frag f[Sh::KS];
#pragma unroll
            for (int c = 0; c < (D == 256 ? 2 : 1); ++c) {
                const uint32_t two = D == 64 ? __builtin_amdgcn_perm(0u, kscale[0][i], pick)
                                             : __builtin_amdgcn_perm(kscale[D == 64 ? 0 : 2 * c + 1][i], kscale[D == 64 ? 0 : 2 * c][i], pick);
                const f16x2 sc = fp8_pair(two, false);
                const f16x2 s0 = {sc[0], sc[0]}, s1 = {sc[1], sc[1]};
#pragma unroll
                for (int k = 0; k < (D == 64 ? 2 : 4); ++k)
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                        f[c * 4 + k].p[b] = fp4_pair(kraw[i][c][k], b) * (D == 64 || k < 2 ? s0 : s1);
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                s[mt][i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < Sh::KS; ++k)
                    s[mt][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f[k].v, q[mt][k], s[mt][i], 0, 0, 0);
            }
        }

        // values into LDS; the scales of tokens that no row sees become zero (their place may hold anything)
#pragma unroll
        for (int j = 0; j < Sh::NV; ++j) {
            const int at = j * 1024 + lane * 16;
            char* dst = vt + (at / (D / 2)) * Sh::VROW + at % (D / 2);
            *(u32x2*)dst = u32x2{vraw[j][0], vraw[j][1]};
            *(u32x2*)(dst + 8) = u32x2{vraw[j][2], vraw[j][3]};
        }
        const bool whole = t0 >= w.first_seen && __ballot(bad) == 0 && t0 + kTile <= end;
        bool all[MT], every = whole;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            all[mt] = whole && t0 >= see_lo[mt] && t0 + kTile <= see_hi[mt];
            every = every && all[mt];
        }
        // A NaN value would reach, as 0 * NaN, the rows that do not see its token.  Where some row does not see the
        // whole tile, NaN scales enter as zeros and go to the rows that do see them by hand.
        uint32_t nan_scales[D / 64] = {};
        const bool some = __ballot(!every) != 0;
        {
            // bytes n * D/16 .. of the group: block by block, 16 tokens each
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
                uint32_t x = vsc[j];
                if (!whole) {
                    const int tok = tg + ((n * (D / 16) + 4 * j) & 15);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (bad || tok + e < w.first_seen || tok + e >= end) x &= ~(0xFFu << (8 * e));
                }
                if (some) {
                    nan_scales[j] = ((x & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                    x &= ~((nan_scales[j] >> 7) * 0xFFu);
                }
                f16x2* dst = (f16x2*)(vs + g * Sh::SROW + (n * (D / 16) + 4 * j) * 2);
                dst[0] = fp8_pair(x, false);
                dst[1] = fp8_pair(x, true);
            }
        }

        // softmax: lane (n, g) holds tokens 16 g .. 16 g + 15 of its row, in order
        Frag p[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            float top = -__builtin_inff();
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float x = s[mt][i][e] * qs[mt];
                    const int tok = tg + 4 * i + e;
                    if (!all[mt] && (bad || tok < see_lo[mt] || tok >= see_hi[mt])) x = -__builtin_inff();
                    s[mt][i][e] = x;
                    top = fmaxf(top, x);
                }
            top = fmaxf(top, __shfl_xor(top, 16, kWave));
            top = fmaxf(top, __shfl_xor(top, 32, kWave));
            const float mn = fmaxf(m[mt], top);
            if (__ballot(mn > m[mt]) != 0) {
                const float by = m[mt] == -__builtin_inff() ? 0.f : __builtin_amdgcn_exp2f(m[mt] - mn);
                l[mt] *= by;
#pragma unroll
                for (int b = 0; b < Sh::NB; ++b) o[mt][b] *= by;
                m[mt] = mn;
            }
            const float sub = m[mt] == -__builtin_inff() ? 0.f : m[mt] - kWeightShift;
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    const float x = __builtin_amdgcn_exp2f(s[mt][i][e] - sub);
                    const float y = __builtin_amdgcn_exp2f(s[mt][i][e + 1] - sub);
                    sum += x + y;
                    p[mt][i >> 1].p[(i & 1) * 2 + e / 2] = f16x2{(_Float16)x, (_Float16)y};
                }
            l[mt] += sum;
        }

        // O^T += V^T P^T
#pragma unroll
        for (int b = 0; b < Sh::NB; ++b) {
            typedef int i32x2 __attribute__((ext_vector_type(2)));
            const char* at = vt + lane * Sh::VROW + b * 8;
            const i32x2 c = __builtin_amdgcn_ds_read_tr4_b64_v2i32((__attribute__((address_space(3))) i32x2*)at);
            Frag sc[2];
            sc[0].u = *(const u32x4*)(vs + g * Sh::SROW + b * 32);
            sc[1].u = *(const u32x4*)(vs + g * Sh::SROW + b * 32 + 16);
            Frag v[2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) v[h].p[e] = fp4_pair((uint32_t)c[h], e) * sc[h].p[e];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                o[mt][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v[0].v, p[mt][0].v, o[mt][b], 0, 0, 0);
                o[mt][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v[1].v, p[mt][1].v, o[mt][b], 0, 0, 0);
            }
        }
        if (some) {
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
                for (uint64_t left = __ballot(nan_scales[j] != 0); left != 0; left &= left - 1) {
                    const int from = (int)__builtin_ctzll(left), at = (from & 15) * (D / 16) + 4 * j;
                    const uint32_t which = (uint32_t)__builtin_amdgcn_readlane((int)nan_scales[j], from);
                    for (int e = 0; e < 4; ++e) {
                        const int tok = t0 + 16 * (from >> 4) + (at & 15) + e;
                        if ((which >> (8 * e + 7) & 1) == 0) continue;
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                            for (int b = 0; b < Sh::NB; ++b)
                                if (b == at >> 4 && tok >= see_lo[mt] && tok < see_hi[mt]) o[mt][b] += __builtin_nanf("");
                    }
                }
        }
    }

    // join the waves, one row tile of 16 at a time
    const float vscale = a.cache.v_scale[head];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        float sum = l[mt];
        sum += __shfl_xor(sum, 16, kWave);
        sum += __shfl_xor(sum, 32, kWave);
        __syncthreads();  // the loop's LDS, or the join before this one
        if (g == 0) {
            join_m[wave][n] = m[mt];
            join_l[wave][n] = sum;
        }
        float* jo = (float*)lds + (wave * 16 + n) * Sh::OROW;
#pragma unroll
        for (int b = 0; b < Sh::NB; ++b) *(f32x4*)(jo + b * 16 + g * 4) = o[mt][b];
        __syncthreads();
        // 16 threads a row, each with D/16 elements
        const int row = threadIdx.x >> 4, part = threadIdx.x & 15;
        const int grow = w.row0 + mt * 16 + row;
        if (grow < w.row1) {
            float top = -__builtin_inff(), total = 0.f, wt[kAttnWaves];
#pragma unroll
            for (int k = 0; k < kAttnWaves; ++k) top = fmaxf(top, join_m[k][row]);
#pragma unroll
            for (int k = 0; k < kAttnWaves; ++k) {
                // a wave that saw nothing, or only NaN, still counts with its sum (0, or NaN)
                wt[k] = join_m[k][row] == -__builtin_inff() ? 1.f : __builtin_amdgcn_exp2f(join_m[k][row] - top);
                total += join_l[k][row] * wt[k];
            }
            const float inv = total == 0.f ? 0.f : 1.f / total;
            const int i = grow / a.group, hq = head * a.group + (grow - i * a.group);
            const int64_t orow = (w.first + i) * a.num_q_heads + hq;
            const float lse2 = top == -__builtin_inff() && total == 0.f ? -__builtin_inff() : (top - kWeightShift) + log2f(total);
            constexpr int E = D / 16;
            float v[E];
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = 0.f;
#pragma unroll
            for (int k = 0; k < kAttnWaves; ++k)
#pragma unroll
                for (int e = 0; e < E; e += 4) {
                    const f32x4 x = *(const f32x4*)((float*)lds + (k * 16 + row) * Sh::OROW + part * E + e);
#pragma unroll
                    for (int u = 0; u < 4; ++u) v[e + u] += x[u] * wt[k];
                }
            if (splits == 1) {
                const float f = inv * vscale;
                uint32_t* dst = (uint32_t*)(a.out + orow * D + part * E);
#pragma unroll
                for (int e = 0; e < E; e += 2) dst[e / 2] = pack_bf16x2(v[e] * f, v[e + 1] * f);
                if (a.lse != nullptr && part == 0) a.lse[orow] = lse2 * 0.693147180559945309f;
            } else {
                const int64_t slot = orow * a.splits + split;
                float* dst = a.part + slot * D + part * E;
#pragma unroll
                for (int e = 0; e < E; e += 4) *(f32x4*)(dst + e) = f32x4{v[e] * inv, v[e + 1] * inv, v[e + 2] * inv, v[e + 3] * inv};
                if (part == 0) a.part[a.batch.num_tokens * a.num_q_heads * a.splits * D + slot] = lse2;
            }
        }
    }
}

#define PLE_ATTN_KERNEL(D, MT)                                                                                  \
    __global__ __launch_bounds__(kAttnThreads) void kv4_attention_##D##_##MT##_kernel(Kv4AttentionArgs a) {     \
        attn_body<D, MT>(a);                                                                                    \
    }
PLE_ATTN_KERNEL(64, 1)
PLE_ATTN_KERNEL(64, 2)
PLE_ATTN_KERNEL(64, 4)
PLE_ATTN_KERNEL(128, 1)
PLE_ATTN_KERNEL(128, 2)
PLE_ATTN_KERNEL(128, 4)
PLE_ATTN_KERNEL(256, 1)
PLE_ATTN_KERNEL(256, 2)
#undef PLE_ATTN_KERNEL

// Joins the splits of a row: out = sum_s 2^(lse_s - top) out_s / sum_s 2^(lse_s - top).  One block a row, a wave
// taking every fourth split.
__global__ __launch_bounds__(kAttnThreads) void kv4_attention_join_kernel(Kv4AttentionArgs a) {
    __shared__ float weight[kMostSplits], sum[kAttnWaves][256];
    const int64_t orow = blockIdx.x, rows = a.batch.num_tokens * a.num_q_heads;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = orow / a.num_q_heads;
    const int hq = (int)(orow - t * a.num_q_heads), head = hq / a.group;
    const int r = find_request(a.batch.query_start_loc, a.batch.num_reqs, t);
    AttnTile w;
    int64_t q0, q1;
    carried_window(a.batch.query_start_loc, a.batch.num_tokens, r, nullptr, q0, q1);
    if (t < q0 || t >= q1) return;
    const int row = (int)(t - q0) * a.group + (hq - head * a.group);
    if (!attn_tile(a, r, row / a.rows, w)) return;
    const int splits = attn_splits(a, w);
    if (splits == 1) return;
    const int D = a.cache.head_dim;
    const float* lse = a.part + rows * a.splits * D + orow * a.splits;
    // every wave for itself: the largest lse, and the sum of the weights
    float top = -__builtin_inff(), total = 0.f;
    for (int s = lane; s < splits; s += kWave) top = fmaxf(top, lse[s]);
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor(top, d, kWave));
    for (int s = lane; s < splits; s += kWave) {
        const float x = lse[s], v = x == -__builtin_inff() ? 0.f : __builtin_amdgcn_exp2f(x - top);  // NaN stays
        total += v;
        if (wave == 0) weight[s] = v;
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) total += __shfl_xor(total, d, kWave);
    __syncthreads();
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    const float* src = a.part + orow * a.splits * D;
    const int per = D / kWave;  // elements of a lane
#pragma unroll 4
    for (int s = wave; s < splits; s += kAttnWaves) {
        const float wt = weight[s];
        const float* p = src + (int64_t)s * D + lane;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < per) v[e] = fmaf(p[e * kWave], wt, v[e]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e < per) sum[wave][e * kWave + lane] = v[e];
    __syncthreads();
    if ((int)threadIdx.x < D) {
        const int d = threadIdx.x;
        const float f = total == 0.f ? 0.f : a.cache.v_scale[head] / total;
        const float x = (sum[0][d] + sum[1][d]) + (sum[2][d] + sum[3][d]);
        a.out[orow * D + d] = (uint16_t)pack_bf16x2(x * f, 0.f);
    }
    if (a.lse != nullptr && threadIdx.x == 0)
        a.lse[orow] = total == 0.f ? -__builtin_inff() : (top + log2f(total)) * 0.693147180559945309f;
}

void plan_kv4_attention(Kv4AttentionArgs& a) {
    const int64_t T = a.batch.num_tokens, R = a.batch.num_reqs;
    const int64_t cover = (int64_t)a.batch.table_width * a.cache.page_size;
    int64_t new_max = a.batch.max_request_tokens > 0 ? a.batch.max_request_tokens : T;
    new_max = new_max < T ? new_max : T;
    int64_t len = a.batch.max_seq_len > 0 && a.batch.max_seq_len < cover ? a.batch.max_seq_len : cover;
    const int64_t rows = new_max * a.group;
    const int most = a.cache.head_dim == 256 ? 32 : 64;
    a.rows = rows <= 16 ? 16 : (rows <= 32 || most == 32 ? 32 : 64);
    a.tiles = (int)((rows + a.rows - 1) / a.rows);
    if (a.window > 0) {
        const int64_t span = (int64_t)a.window + a.rows / a.group + 1 + 15;
        len = len < span ? len : span;
    }
    // splits: about 1024 blocks (four per CU), each with at least one tile of 64 tokens per wave
    const int64_t blocks = R * a.cache.num_kv_heads * a.tiles;
    int64_t splits = blocks > 0 ? (1024 + blocks - 1) / blocks : 1;
    const int64_t most_splits = (len + kTile * kAttnWaves - 1) / (kTile * kAttnWaves);
    splits = splits < most_splits ? splits : most_splits;
    splits = splits < 1 ? 1 : (splits < kMostSplits - 1 ? splits : kMostSplits - 1);
    int64_t chunk = (len + splits - 1) / splits;
    chunk = (chunk + kTile * kAttnWaves - 1) / (kTile * kAttnWaves) * (kTile * kAttnWaves);
    // a range starts at a multiple of 16, up to 15 tokens before the first that is seen
    a.chunk = (int)chunk;
    a.splits = (int)((len + 15 + chunk - 1) / chunk);
    if (a.splits < 1) a.splits = 1;
}

size_t kv4_attention_part_bytes(const Kv4AttentionArgs& a) {
    if (a.splits <= 1) return 0;
    return (size_t)a.batch.num_tokens * a.num_q_heads * a.splits * (a.cache.head_dim + 1) * sizeof(float);
}

hipError_t launch_kv4_attention(const Kv4AttentionArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)((int64_t)a.batch.num_reqs * a.cache.num_kv_heads * a.tiles), (unsigned)a.splits);
    const int D = a.cache.head_dim, MT = a.rows / 16;
#define PLE_ATTN_LAUNCH(DD, MM) \
    if (D == DD && MT == MM) hipLaunchKernelGGL(kv4_attention_##DD##_##MM##_kernel, grid, dim3(kAttnThreads), 0, s, a)
    PLE_ATTN_LAUNCH(64, 1);
    PLE_ATTN_LAUNCH(64, 2);
    PLE_ATTN_LAUNCH(64, 4);
    PLE_ATTN_LAUNCH(128, 1);
    PLE_ATTN_LAUNCH(128, 2);
    PLE_ATTN_LAUNCH(128, 4);
    PLE_ATTN_LAUNCH(256, 1);
    PLE_ATTN_LAUNCH(256, 2);
#undef PLE_ATTN_LAUNCH
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits <= 1) return e;
    const int64_t rows = a.batch.num_tokens * a.num_q_heads;
    hipLaunchKernelGGL(kv4_attention_join_kernel, dim3((unsigned)rows), dim3(kAttnThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace ple
