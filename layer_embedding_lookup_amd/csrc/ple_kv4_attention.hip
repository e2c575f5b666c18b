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
//
// Few rows: the waves of a block take the tiles of a cache range in turn and
// join through LDS; four waves a block, eight where there is a block per CU
// at most.  The next tile is loaded while this one's weights and value
// product are formed, its page-table entry a tile before that.  Bound by
// reading the cache where there is much of it (256 requests of up to 6000
// tokens, 914 MB: 194 us, 4.7 TB/s; one of 131k tokens, 151 MB: 29 us and 5
// for the join, 38.8 with the launches), else by the chain of dependent loads
// (one of 777 tokens: 10.5 us; 64 windows of 1..4 drafts over 1024 tokens: 17).
#include "ple_fp4_launch.h"

namespace ple {

constexpr int kAttnWaves = 4;  // of a chunk block, and those whose sums a decode block joins through LDS
constexpr int kAttnThreads = kAttnWaves * kWave;
constexpr int kTile = 64;  // cache tokens of a tile
constexpr int kMostSplits = 1024;
constexpr int kFewSplits = 8;  // up to which one wave joins a row
// Weights are 2^(s - m + kWeightShift) with m a row's largest exponent but for kSlack: m only moves on, and the row's
// sums are only rescaled, when the maximum has passed it by more than that.  Weights stay below 2^15 and fp16 keeps
// them above 2^-24, so tokens down to 2^-32 of the heaviest one count.  The products take them in fp16 so that they run
// on the matrix cores beside values that fp16 holds exactly; the sums take them unrounded, which keeps the log-sum-exp
// at fp32.  That costs 1.6e-4 of an output (rms over 777 random keys; summing the rounded weights instead: the same),
// a tenth of the 1.65e-3 of its rounding to bf16: 0.00166 against 64 bits with it and 0.00165 without.
constexpr float kWeightShift = 8.0f, kSlack = 7.0f;

// What a block's query tile sees: rows [row0, row1) of request r, cache tokens [lo, hi).
struct AttnTile {
    int64_t first;  // first new token of the request
    int n, len;     // its new tokens, its length as far as the page table covers it
    int before;     // position of its first new token
    int row0, row1;
    int first_seen;  // the first token that any row sees
    int lo, hi;      // lo: first_seen rounded down to a group of 16
};

// Request r of the batch, its query tiles not yet looked at.
__device__ __forceinline__ void attn_request(const Kv4AttentionArgs& a, int r, AttnTile& w) {
    const int T = (int)a.batch.num_tokens, seq = max(a.batch.seq_lens[r], 0);
    const int q0 = min(max(a.batch.query_start_loc[r], 0), T), to = a.batch.query_start_loc[r + 1];
    w.first = q0;
    w.n = max(min(to, T), q0) - q0;
    w.len = min(seq, a.batch.table_width * a.cache.page_size);
    // As for append, by the whole length and all of the request's tokens.  Where it has new tokens, `to - q0` lies in
    // 1 .. 2^31 - 1; further before position 0 than there are new tokens is the same as that far.
    w.before = max((int)((uint32_t)seq - ((uint32_t)to - (uint32_t)q0)), -w.n);
}

// Tokens of no request (a batch padded to a graph's size): their rows of `out` are zeros and of `lse` -inf.  The blocks
// share them token by token; mostly there are none, and the two entries come with those of the block's own request.
__device__ __forceinline__ void attn_idle_tokens(const Kv4AttentionArgs& a) {
    const int64_t T = a.batch.num_tokens;
    int64_t first = a.batch.query_start_loc[0], last = a.batch.query_start_loc[a.batch.num_reqs];
    first = first < 0 ? 0 : (first > T ? T : first);
    last = last < first ? first : (last > T ? T : last);
    const int64_t idle = first + (T - last);
    if (idle == 0) return;
    const int row = a.num_q_heads * a.cache.head_dim;
    for (int64_t i = (int64_t)blockIdx.y * gridDim.x + blockIdx.x; i < idle; i += (int64_t)gridDim.x * gridDim.y) {
        const int64_t t = i < first ? i : last + (i - first);
        for (int e = threadIdx.x * 8; e < row; e += blockDim.x * 8) *(u32x4*)(a.out + t * row + e) = u32x4{0u, 0u, 0u, 0u};
        if (a.lse != nullptr)
            for (int h = threadIdx.x; h < a.num_q_heads; h += blockDim.x) a.lse[t * a.num_q_heads + h] = -__builtin_inff();
    }
}

// Its query tile; false if it has no such tile.
__device__ __forceinline__ bool attn_tile(const Kv4AttentionArgs& a, int tile, AttnTile& w) {
    w.row0 = tile * a.rows;
    w.row1 = min(w.row0 + a.rows, w.n * a.group);
    if (w.row0 >= w.row1) return false;
    w.hi = max(0, min(w.len, w.before + (w.row1 - 1) / a.group + 1));
    w.first_seen = a.window > 0 ? max(0, w.before + w.row0 / a.group - a.window + 1) : 0;
    w.lo = min(w.first_seen & ~15, w.hi & ~15);
    return true;
}

__device__ __forceinline__ int attn_splits(const Kv4AttentionArgs& a, const AttnTile& w) {
    const int s = (w.hi - w.lo + a.chunk - 1) / a.chunk;
    return max(1, min(s, a.splits));
}

// Request, key head and query tile of a block.  Blocks of one request and head are a multiple of the pairs apart, so
// with the usual 8 heads they run on one XCD and share its L2; the tiles with the most to see come first.
__device__ __forceinline__ void attn_block(const Kv4AttentionArgs& a, int& r, int& head, int& tile) {
    const int heads = a.cache.num_kv_heads, pairs = a.batch.num_reqs * heads;
    const int back = blockIdx.x / pairs, pair = blockIdx.x - back * pairs;
    tile = a.tiles - 1 - back;
    r = pair / heads;
    head = pair - r * heads;
}

// A lane's way along its request's pages: the 16-token group at token tg, then `step` groups on at a time.  Table
// entries are fetched a tile before the group's number is needed, which is a tile before its codes are.
struct PageWalk {
    const int32_t* row;
    int per_page, page, in_page, step_pages, step_in, last;  // last: the page of token end - 1
    uint32_t pages, heads, head;
    int entry;

    __device__ __forceinline__ PageWalk(const Kv4AttentionArgs& a, const int32_t* table_row, int h, int tg, int step, int end)
        : row(table_row), per_page(a.cache.page_size >> 4), pages((uint32_t)a.cache.num_pages),
          heads((uint32_t)a.cache.num_kv_heads), head((uint32_t)h) {
        page = (tg >> 4) / per_page;
        in_page = (tg >> 4) - page * per_page;
        step_pages = step / per_page;
        step_in = step - step_pages * per_page;
        last = (end - 1) / a.cache.page_size;
        entry = -1;
    }
    // the entry of the current group (in bounds even for groups past the end, which `number` turns away)
    __device__ __forceinline__ void fetch() { entry = row[min(page, last)]; }
    // the current group's number or -1, and on to the next one
    __device__ __forceinline__ int number(int tg, int end) {
        const uint32_t e = (uint32_t)entry;
        const int grp = tg < end && e < pages ? (int)((e * heads + head) * (uint32_t)per_page) + in_page : -1;
        page += step_pages;
        in_page += step_in;
        if (in_page >= per_page) {
            in_page -= per_page;
            ++page;
        }
        return grp;
    }
};

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

template <int D, int WAVES>
struct AttnShape {
    static constexpr int KS = D / 32;                   // k-steps of the first product
    static constexpr int NB = D / 16;                   // element blocks
    static constexpr int NV = D / 32;                   // 16-byte loads of a lane per tile of codes
    static constexpr int VROW = D / 2 + 8;              // a token's codes in LDS: the 8 bytes spread 16 rows over the banks
    static constexpr int SROW = D * 2 + 16;             // a group's value scales in LDS, as fp16
    static constexpr int WAVE_LDS = kTile * VROW + 4 * SROW;
    static constexpr int OROW = D + 4;                  // the join's rows (fp32)
    static constexpr int JOIN_LDS = kAttnWaves * 16 * OROW * 4;
    static constexpr int LDS = WAVE_LDS * WAVES > JOIN_LDS ? WAVE_LDS * WAVES : JOIN_LDS;
};

// The queries of MT x 16 rows from row0 on: lane (n, g) holds, of row 16 mt + n, the elements that its key codes
// meet (q), what turns the row's products into base-2 exponents (qs), and the tokens it sees.
template <int D, int MT>
__device__ __forceinline__ void attn_queries(const Kv4AttentionArgs& a, const AttnTile& w, int row0, int head, int begin,
                                             int end, f16x8 (&q)[MT][D / 32], float (&qs)[MT], int (&see_lo)[MT],
                                             int (&see_hi)[MT]) {
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    const float base = a.scale * 1.44269504088896341f * a.cache.k_scale[head];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int row = row0 + mt * 16 + n;
        const bool live = row < w.row1;
        const int i = row / a.group, hq = head * a.group + (row - i * a.group);
        const uint16_t* src = a.q + (w.first + i) * a.q_stride + hq * D;
        u32x4 raw[D / 32];
        float top = 0.f;
#pragma unroll
        for (int ks = 0; ks < D / 32; ++ks) {
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
        // (never zero: a masked product, -inf, times it has to stay -inf)
        const float back = base * __uint_as_float((uint32_t)(max(e - 14 + 127, 1)) << 23);
        qs[mt] = back < 1.17549435e-38f ? 1.17549435e-38f : back;
#pragma unroll
        for (int ks = 0; ks < D / 32; ++ks)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                q[mt][ks][2 * j] = (_Float16)(bf16_lo(raw[ks][j]) * up);
                q[mt][ks][2 * j + 1] = (_Float16)(bf16_hi(raw[ks][j]) * up);
            }
        const int p = w.before + i;
        // (rows past the tile's end, all zeros and never stored, see everything, which keeps the masks out of whole tiles)
        see_hi[mt] = live ? min(end, p + 1) : end;
        see_lo[mt] = live ? max(begin, a.window > 0 ? p - a.window + 1 : 0) : begin;
    }
}

// max over the four lanes n, n + 16, n + 32, n + 48
__device__ __forceinline__ float quad_max(float x) {
    typedef unsigned int u2 __attribute__((ext_vector_type(2)));
    u2 w = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = fmaxf(__uint_as_float(w[0]), __uint_as_float(w[1]));
    w = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(w[0]), __uint_as_float(w[1]));
}

// The weights of one tile: s (products, lane (n, g) holding tokens tg .. tg + 15 of MT rows) becomes the fp16 weights p;
// m, l and o (the rows' running maxima, sums and outputs) move on.  `some`: not every row sees the whole tile.
template <int NB, int MT>
__device__ __forceinline__ void attn_softmax(f32x4 (&s)[MT][4], const float (&qs)[MT], bool some, bool bad, int tg,
                                             const int (&see_lo)[MT], const int (&see_hi)[MT], float (&m)[MT], float (&l)[MT],
                                             f32x4 (&o)[MT][NB], Frag (&p)[MT][2]) {
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
        mn[mt] = fmaxf(m[mt], quad_max(top) * qs[mt]);  // (qs > 0)
        up |= mn[mt] > m[mt] + kSlack;
    }
    if (__ballot(up) != 0) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const float by = m[mt] == -__builtin_inff() ? 0.f : __builtin_amdgcn_exp2f(m[mt] - mn[mt]);
            l[mt] *= by;
#pragma unroll
            for (int b = 0; b < NB; ++b) o[mt][b] *= by;
            m[mt] = mn[mt];
        }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const float sub = m[mt] == -__builtin_inff() ? 0.f : kWeightShift - m[mt];
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                const float x = __builtin_amdgcn_exp2f(fmaf(s[mt][i][e], qs[mt], sub));
                const float y = __builtin_amdgcn_exp2f(fmaf(s[mt][i][e + 1], qs[mt], sub));
                sum += x + y;
                p[mt][i >> 1].p[(i & 1) * 2 + e / 2] = f16x2{(_Float16)x, (_Float16)y};
            }
        l[mt] += sum;
    }
}

template <int D, int MT, int WAVES>
__device__ __forceinline__ void attn_body(const Kv4AttentionArgs& a) {
    using Sh = AttnShape<D, WAVES>;
    extern __shared__ __align__(16) char lds[];
    __shared__ float join_m[kAttnWaves][16], join_l[kAttnWaves][16];
    const int split = blockIdx.y;
    int r, head, tile;
    attn_block(a, r, head, tile);
    AttnTile w;
    attn_request(a, r, w);
    attn_idle_tokens(a);
    if (!attn_tile(a, tile, w)) return;
    const int splits = attn_splits(a, w);
    if (split >= splits) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n = lane & 15, g = lane >> 4;
    const int begin = w.lo + split * a.chunk;
    const int end = split == splits - 1 ? w.hi : min(w.hi, begin + a.chunk);

    f16x8 q[MT][Sh::KS];
    float qs[MT];
    int see_lo[MT], see_hi[MT];
    attn_queries<D, MT>(a, w, w.row0, head, begin, end, q, qs, see_lo, see_hi);

    f32x4 o[MT][Sh::NB];
    float m[MT], l[MT];
    uint32_t nan_blocks[MT] = {};  // element blocks of the row that a NaN value makes NaN
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

    // a tile, as loaded: the next one is on its way while this one's weights and value product are formed
    bool bad_next = false;
    u32x4 kraw[4][D == 256 ? 2 : 1];
    u32x4 kscale[D == 64 ? 1 : D / 64];
    u32x4 vraw[Sh::NV];
    uint32_t vsc[D / 64];
    const int first = begin + wave * kTile;
    PageWalk walk(a, table_row, head, first + 16 * g, WAVES * kTile / 16, end);
    auto load = [&](int t0) {
        const int grp = walk.number(t0 + 16 * g, end);
        walk.fetch();
        bad_next = grp < 0;
        const int safe = grp < 0 ? 0 : grp;
        // keys: group n / 4, token 4 i + n % 4
        const int64_t kg = __shfl(safe, (n >> 2) * 16, kWave);
        const uint8_t* kc = a.cache.k_codes + kg * (8 * D) + (n & 3) * (D / 2) + g * (D == 64 ? 8 : 16);
        const uint8_t* ksc = a.cache.k_scales + kg * D + (D == 64 ? g * 16 : g * 32);
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
#pragma unroll
        for (int j = 0; j < Sh::NV; ++j) {
            const int at = j * 1024 + lane * 16;
            const int64_t vg = __shfl(safe, (at / (8 * D)) * 16, kWave);
            vraw[j] = *(const u32x4*)(a.cache.v_codes + vg * (8 * D) + at % (8 * D));
        }
        const uint8_t* p = a.cache.v_scales + (int64_t)safe * D + n * (D / 16);
#pragma unroll
        for (int j = 0; j < D / 64; ++j) vsc[j] = ((const uint32_t*)p)[j];
    };
    if (first < end) {
        walk.fetch();
        load(first);
    }
    for (int t0 = first; t0 < end; t0 += WAVES * kTile) {
        const int tg = t0 + 16 * g;  // this lane's group g of the tile
        const bool bad = bad_next;

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
        bool every = whole;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) every = every && t0 >= see_lo[mt] && t0 + kTile <= see_hi[mt];
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
        if (t0 + WAVES * kTile < end) load(t0 + WAVES * kTile);

        // lane (n, g) holds tokens 16 g .. 16 g + 15 of its row, in order
        Frag p[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)  // (one after the other: fewer registers than all of them together)
            attn_softmax<Sh::NB, 1>((f32x4(&)[1][4])s[mt], (float(&)[1])qs[mt], some, bad, tg, (int(&)[1])see_lo[mt],
                                    (int(&)[1])see_hi[mt], (float(&)[1])m[mt], (float(&)[1])l[mt],
                                    (f32x4(&)[1][Sh::NB])o[mt], (Frag(&)[1][2])p[mt]);

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
                            if (tok >= see_lo[mt] && tok < see_hi[mt]) nan_blocks[mt] |= 1u << (at >> 4);
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
        float* jo = (float*)lds + ((wave & 3) * 16 + n) * Sh::OROW;
        // the upper four waves hand theirs to the lower ones, lane by lane; then the lower ones write theirs
#pragma unroll
        for (int half = WAVES / kAttnWaves - 1; half >= 0; --half) {
            __syncthreads();  // the loop's LDS, or what was read of the join before this
            if (wave / kAttnWaves == half) {
                if (g == 0) {
                    join_m[wave & 3][n] = m[mt];
                    join_l[wave & 3][n] = sum;
                }
#pragma unroll
                for (int b = 0; b < Sh::NB; ++b) *(f32x4*)(jo + b * 16 + g * 4) = o[mt][b];
                for (uint32_t left = nan_blocks[mt]; left != 0; left &= left - 1)
                    *(f32x4*)(jo + __builtin_ctz(left) * 16 + g * 4) = f32x4{1.f, 1.f, 1.f, 1.f} * __builtin_nanf("");
            }
            __syncthreads();
            if (half > 0 && wave / kAttnWaves == half - 1) {
                const float om = join_m[wave & 3][n], top = fmaxf(m[mt], om);
                // (one that saw nothing, or only NaN, still counts with its sum: 0, or NaN)
                const float mine = m[mt] == -__builtin_inff() ? 1.f : __builtin_amdgcn_exp2f(m[mt] - top);
                const float theirs = om == -__builtin_inff() ? 1.f : __builtin_amdgcn_exp2f(om - top);
                sum = sum * mine + join_l[wave & 3][n] * theirs;
                m[mt] = top;
#pragma unroll
                for (int b = 0; b < Sh::NB; ++b) {
                    const f32x4 x = *(const f32x4*)(jo + b * 16 + g * 4);
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[mt][b][e] = o[mt][b][e] * mine + x[e] * theirs;
                }
            }
        }
        if (wave >= kAttnWaves) continue;
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

// D, row tiles, waves, waves per SIMD that registers allow
#define PLE_ATTN_SHAPES(X)                                                                                        \
    X(64, 1, 4, 3) X(64, 1, 8, 2) X(64, 2, 4, 2) X(64, 2, 8, 2) X(128, 1, 4, 3) X(128, 1, 8, 2) X(128, 2, 4, 2) \
    X(128, 2, 8, 2) X(256, 1, 4, 2) X(256, 1, 8, 2)
#define PLE_ATTN_KERNEL(D, MT, WAVES, OCC)                                                                                  \
    __global__ __launch_bounds__(WAVES * kWave, OCC) void kv4_attention_##D##_##MT##x##WAVES##_kernel(Kv4AttentionArgs a) { \
        attn_body<D, MT, WAVES>(a);                                                                                         \
    }
PLE_ATTN_SHAPES(PLE_ATTN_KERNEL)
#undef PLE_ATTN_KERNEL

// ---------------------------------------------------------------------------
// Many rows (a chunk of a prefill): bound by the products and the softmax
// between them.  A block's four waves hold 32 rows each and go through the
// cache tiles together: each wave dequantises a quarter of a tile (16 tokens
// of the keys, a quarter of the value elements) and leaves it in LDS as
// finished MFMA fragments, one 16-byte read per lane each; so a tile is
// dequantised once for 128 rows.  Two tiles in LDS: the next one is filled
// while this one is used, with one barrier a tile.  Two blocks per CU cover
// each other's softmax (D = 256: one).  1289 + 1455 tokens at 5403 and 2004,
// 32 heads of 128: 231 us, 0.57 PFLOP/s, 25 of them the join of cut tiles.  A
// CU's eight waves take about 7300 cycles for a tile each.  In those a SIMD's
// products are 2048 and its other vector instructions (softmax, dequantising)
// about 3300; LDS is busy for 1750, almost without bank conflicts.  Without
// waiting for memory, or with these hand-interleaved, it takes as long, so
// what is left is the two waves of a SIMD in the same phase.
// ---------------------------------------------------------------------------
constexpr int kChunkRows = 128;
// Measured with 32 heads of 128 over 8 where nothing else is said, and where a value other than these does better too:
//  kFlatLeast: 1289 + 1455 tokens at 5403 and 2004 232 us with 4, 8 and 16, 237 with 2; 100 behind 2000 43 (with 4 44, 2 54,
//              16 58); 1000 behind nothing 54 (4 53, 16 70); but 100 behind nothing 30 (4 21), 50 behind 500 38 (4 30).
//  kFlatStart: the first 232 us (with 0 278, 2 252, 8 242), the second 44.5 (51, 46, 43.7), the third 54 (86, 60, 56).
//  kFlatUnits: 736 query tiles 233 us in shares, 401 a block each; 4864 of 32 requests 330 and 275, which the rule keeps
//              apart; between them it takes the slower one (1920 tiles of 16 requests 165 and 155, 2560 of 32 162 and 146).
constexpr int kFlatLeast = 8;        // places of a share at least
constexpr int kFlatStart = 4;        // places that beginning a query tile counts for (queries in, results out)
constexpr int kFlatUnits = 4096;     // query tiles (of all heads and requests) up to which the work is cut into shares
constexpr int kFlatJoinRows = 32;    // rows of a block of the joining kernel

template <int D>
struct ChunkShape {
    static constexpr int KS = D / 32, NB = D / 16, WB = D / 64;  // WB: element blocks that a wave dequantises
    static constexpr int K_BYTES = 4 * KS * 1024, V_BYTES = NB * 2 * 1024;
    static constexpr int BUF = K_BYTES + V_BYTES;
    static constexpr int STAGE = kTile * WB * 8;  // a wave's value codes on their way through the transposing read
    static constexpr int NAN_AT = 2 * BUF + kAttnWaves * STAGE;
    static constexpr int LDS = NAN_AT + 2 * kAttnWaves * kTile;
};

// Few query tiles, of requests of different lengths, leave CUs idle at the end.  Then the cache tiles of all query
// tiles (at least one each), in the order request, key head, query tile, are one line that `flat` blocks cut into equal
// shares; a query tile has kFlatStart places in front of its cache tiles.  A query tile whose cache tiles a cut goes
// through is joined by a second kernel: of its pieces the one that begins it is partial result 2 * share + 1, every
// other 2 * share of its share.
// A chunk of 1289 + 1455 tokens at 5403 and 2004: 308 us with a block a query tile (CUs busy for 53% of it).
struct AttnFlat {
    // of lane r:
    int first, n, len, pos;  // request r's first new token, new tokens, length, position of the first new token
    int tiles_of;            // the places of one of its heads
    int before;              // and those of all heads of the requests before it
    int total, quota;

    __device__ __forceinline__ void request(int r, AttnTile& w) const {
        w.first = __builtin_amdgcn_readlane(first, r);
        w.n = __builtin_amdgcn_readlane(n, r);
        w.len = __builtin_amdgcn_readlane(len, r);
        w.before = __builtin_amdgcn_readlane(pos, r);
    }

    static __device__ __forceinline__ int count(const AttnTile& w) { return max(1, (w.hi - w.lo + kTile - 1) / kTile); }
    // the places of query tile t of w's request (0: it has no such tile)
    static __device__ __forceinline__ int places(const Kv4AttentionArgs& a, int t, AttnTile& w) {
        return t < a.tiles && attn_tile(a, t, w) ? kFlatStart + count(w) : 0;
    }

    __device__ __forceinline__ void lay_out(const Kv4AttentionArgs& a) {
        const int lane = threadIdx.x & 63;
        AttnTile w = {};
        if (lane < a.batch.num_reqs) attn_request(a, lane, w);
        first = (int)w.first;
        n = w.n;
        len = w.len;
        pos = w.before;
        tiles_of = 0;
        if (a.tiles < 4 * a.batch.num_reqs) {  // a lane a request, or the wave for one after the other: what is shorter
            for (int t = 0, c; (c = places(a, t, w)) > 0; ++t) tiles_of += c;
        } else {
            for (int r = 0; r < a.batch.num_reqs; ++r) {
                request(r, w);
                int sum = 0;
                for (int t = lane, c; (c = places(a, t, w)) > 0; t += kWave) sum += c;
#pragma unroll
                for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d, kWave);
                if (lane == r) tiles_of = sum;
            }
        }
        const int heads = a.cache.num_kv_heads;
        int sum = tiles_of * heads;
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
            const int x = __shfl_up(sum, d, kWave);
            if (lane >= d) sum += x;
        }
        before = sum - tiles_of * heads;
        total = __shfl(sum, kWave - 1, kWave);
        quota = max(kFlatLeast, (total + a.flat - 1) / a.flat);
    }
    // The query tile that place `at` of the line lies in, how far in (below 0: before its cache tiles), and the number
    // of its cache tiles.
    __device__ __forceinline__ void find(const Kv4AttentionArgs& a, int at, int& r, int& head, AttnTile& w, int& k0,
                                         int& cnt) const {
        const int lane = threadIdx.x & 63;
        // the last request that begins at or before it and has tiles
        r = 63 - (int)__builtin_clzll(__ballot(tiles_of > 0 && before <= at));
        const int per = __builtin_amdgcn_readlane(tiles_of, r);
        int in = at - __builtin_amdgcn_readlane(before, r);
        head = in / per;
        in -= head * per;
        request(r, w);
        for (int t0 = 0;; t0 += kWave) {
            const int c = places(a, t0 + lane, w);
            int sum = c;
#pragma unroll
            for (int d = 1; d < kWave; d <<= 1) {
                const int x = __shfl_up(sum, d, kWave);
                if (lane >= d) sum += x;
            }
            const uint64_t past = __ballot(sum > in);
            if (past != 0 || t0 + kWave >= a.tiles) {  // (always found: `in` lies below the request's sum)
                const int l = past != 0 ? (int)__builtin_ctzll(past) : 0;
                cnt = __builtin_amdgcn_readlane(c, l);
                k0 = in - (__builtin_amdgcn_readlane(sum, l) - cnt) - kFlatStart;
                cnt -= kFlatStart;
                attn_tile(a, t0 + l, w);
                return;
            }
            in -= __builtin_amdgcn_readlane(sum, kWave - 1);
        }
    }
};

// Instruction order for N fragments, each read from LDS and used by MT products: four reads go ahead of the products.
template <int N, int MT>
__device__ __forceinline__ void reads_ahead() {
    __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
#pragma unroll
    for (int i = 0; i < N - 4; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, MT, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, 4 * MT, 0);
}

// Rows [w.row0, w.row1) against the cache's tokens [begin, end).  Results go to the call's outputs (at < 0), or to the
// partial results from row `at` on.
template <int D>
__device__ __forceinline__ void attn_chunk_piece(const Kv4AttentionArgs& a, const AttnTile& w, int r, int head, int begin,
                                                 int end, int at) {
    using Sh = ChunkShape<D>;
    constexpr int MT = 2;
    extern __shared__ __align__(16) char lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;
    // what every row of the block sees
    const int common_lo = a.window > 0 ? max(0, w.before + (w.row1 - 1) / a.group - a.window + 1) : 0;
    const int common_hi = min(end, w.before + w.row0 / a.group + 1);

    const int32_t* table_row = a.batch.page_table + (int64_t)r * a.batch.table_width;
    const uint32_t pick = (uint32_t)((n & 3) | ((4 + (n & 3)) << 8));
    char* const stage = lds + 2 * Sh::BUF + wave * Sh::STAGE;

    // a tile's quarter, as loaded
    u32x4 kraw[D == 256 ? 2 : 1], vraw[D == 256 ? 2 : 1], vsc[Sh::WB];
    uint32_t ksc[D == 64 ? 1 : D / 64];
    bool bad_next = false;
    PageWalk walk(a, table_row, head, begin + 16 * g, kTile / 16, end);
    int grp = -1;
    int64_t kg = 0;  // of the tile to load next: this lane's group, and group n / 4 of the tile
    auto aim = [&](int t0) {
        grp = walk.number(t0 + 16 * g, end);
        walk.fetch();
        kg = __shfl(max(grp, 0), (n >> 2) * 16, kWave);
    };
    auto load = [&]() {
        bad_next = grp < 0;
        const int safe = max(grp, 0);
        // keys: token 4 wave + n % 4 of the group
        const uint8_t* kc = a.cache.k_codes + kg * (8 * D) + (4 * wave + (n & 3)) * (D / 2) + g * (D == 64 ? 8 : 16);
        const uint8_t* ks = a.cache.k_scales + kg * D + (D == 64 ? g * 16 : g * 32) + wave * 4;
        // values: token `lane`, this wave's 8 WB bytes of it
        const uint8_t* vc = a.cache.v_codes + (int64_t)safe * (8 * D) + n * (D / 2) + wave * (8 * Sh::WB);
        if constexpr (D == 64) {
            const u32x2 x = *(const u32x2*)kc, y = *(const u32x2*)vc;
            kraw[0] = u32x4{x[0], x[1], 0u, 0u};
            vraw[0] = u32x4{y[0], y[1], 0u, 0u};
            ksc[0] = *(const uint32_t*)ks;
        } else {
#pragma unroll
            for (int c = 0; c < D / 128; ++c) {
                kraw[c] = *(const u32x4*)(kc + c * 64);
                vraw[c] = *(const u32x4*)(vc + c * 16);
                ksc[2 * c] = *(const uint32_t*)(ks + c * 128);
                ksc[2 * c + 1] = *(const uint32_t*)(ks + c * 128 + 16);
            }
        }
#pragma unroll
        for (int b = 0; b < Sh::WB; ++b)
            vsc[b] = *(const u32x4*)(a.cache.v_scales + (int64_t)safe * D + (wave * Sh::WB + b) * 16);
    };
    // the first tile is on its way before the queries are
    if (begin < end) {
        walk.fetch();
        aim(begin);
        load();
        aim(begin + kTile);
    }
    f16x8 q[MT][Sh::KS];
    float qs[MT];
    int see_lo[MT], see_hi[MT];
    attn_queries<D, MT>(a, w, w.row0 + wave * (16 * MT), head, begin, end, q, qs, see_lo, see_hi);
    f32x4 o[MT][Sh::NB];
    float m[MT], l[MT];
    uint32_t nan_blocks[MT] = {};
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        m[mt] = -__builtin_inff();
        l[mt] = 0.f;
#pragma unroll
        for (int b = 0; b < Sh::NB; ++b) o[mt][b] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    // whether some row does not see the whole tile (the same for the block: `bad` is the tile's four groups)
    auto partial = [&](int t0, bool bad) {
        return t0 < common_lo || t0 < begin || t0 + kTile > common_hi || __ballot(bad) != 0;
    };
    auto fill = [&](int t0, int buf) {
        char* kb = lds + buf * Sh::BUF + (wave * Sh::KS) * 1024 + lane * 16;
        char* vb = lds + buf * Sh::BUF + Sh::K_BYTES + (wave * Sh::WB * 2) * 1024 + lane * 16;
        // value codes to LDS first: their way back takes a while
#pragma unroll
        for (int b = 0; b < Sh::WB; ++b)
            *(u32x2*)(stage + lane * (8 * Sh::WB) + b * 8) = u32x2{vraw[b / 2][2 * (b & 1)], vraw[b / 2][2 * (b & 1) + 1]};
        typedef int i32x2 __attribute__((ext_vector_type(2)));
        i32x2 vc[Sh::WB];
#pragma unroll
        for (int b = 0; b < Sh::WB; ++b)
            vc[b] = __builtin_amdgcn_ds_read_tr4_b64_v2i32(
                (__attribute__((address_space(3))) i32x2*)(stage + lane * (8 * Sh::WB) + b * 8));
#pragma unroll
        for (int c = 0; c < (D == 256 ? 2 : 1); ++c) {
            const uint32_t two = D == 64 ? __builtin_amdgcn_perm(0u, ksc[0], pick)
                                         : __builtin_amdgcn_perm(ksc[D == 64 ? 0 : 2 * c + 1], ksc[D == 64 ? 0 : 2 * c], pick);
            const f16x2 sc = fp8_pair(two, false);
            const f16x2 s0 = {sc[0], sc[0]}, s1 = {sc[1], sc[1]};
#pragma unroll
            for (int k = 0; k < (D == 64 ? 2 : 4); ++k) {
                Frag f;
#pragma unroll
                for (int b = 0; b < 4; ++b) f.p[b] = fp4_pair(kraw[c][k], b) * (D == 64 || k < 2 ? s0 : s1);
                *(u32x4*)(kb + (c * 4 + k) * 1024) = f.u;
            }
        }
        const bool some = partial(t0, bad_next);
        uint32_t nan_bits = 0;  // of token n of the group, this wave's blocks
        if (some) {
#pragma unroll
            for (int b = 0; b < Sh::WB; ++b)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t x = vsc[b][j];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int tok = t0 + 16 * g + 4 * j + e;
                        if (bad_next || tok < w.first_seen || tok >= end) x &= ~(0xFFu << (8 * e));
                    }
                    const uint32_t nan = ((x & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                    vsc[b][j] = x & ~((nan >> 7) * 0xFFu);
                    if ((n >> 2) == j && (nan >> (8 * (n & 3) + 7) & 1u) != 0) nan_bits |= 1u << b;
                }
            *(uint8_t*)(lds + Sh::NAN_AT + (buf * kAttnWaves + wave) * kTile + lane) = (uint8_t)nan_bits;
        }
#pragma unroll
        for (int b = 0; b < Sh::WB; ++b) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                Frag f;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    f.p[e] = fp4_pair((uint32_t)vc[b][h], e) * fp8_pair(vsc[b][2 * h + e / 2], (e & 1) != 0);
                *(u32x4*)(vb + (b * 2 + h) * 1024) = f.u;
            }
        }
    };

    bool bad = false;
    if (begin < end) {
        fill(begin, 0);
        bad = bad_next;
    }
    int buf = 0;
    for (int t0 = begin; t0 < end; t0 += kTile, buf ^= 1) {
        const bool more = t0 + kTile < end;
        __syncthreads();  // this tile is whole; every read of the other buffer is done
        if (more) load();
        const char* kb = lds + buf * Sh::BUF + lane * 16;
        const char* vb = kb + Sh::K_BYTES;
        const bool some = partial(t0, bad);
        f32x4 s[MT][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) s[mt][i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < Sh::KS; ++k) {
                const f16x8 f = *(const f16x8*)(kb + (i * Sh::KS + k) * 1024);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                    s[mt][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f, q[mt][k], s[mt][i], 0, 0, 0);
            }
        }
        reads_ahead<4 * Sh::KS, MT>();
        aim(t0 + 2 * kTile);
        Frag p[MT][2];
        attn_softmax<Sh::NB, MT>(s, qs, some, bad, t0 + 16 * g, see_lo, see_hi, m, l, o, p);
#pragma unroll
        for (int b = 0; b < Sh::NB; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const f16x8 f = *(const f16x8*)(vb + (b * 2 + h) * 1024);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                    o[mt][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f, p[mt][h].v, o[mt][b], 0, 0, 0);
            }
        reads_ahead<2 * Sh::NB, MT>();
        if (some) {
            uint32_t bits = 0;  // of token t0 + lane, all blocks
#pragma unroll
            for (int k = 0; k < kAttnWaves; ++k)
                bits |= (uint32_t)*(const uint8_t*)(lds + Sh::NAN_AT + (buf * kAttnWaves + k) * kTile + lane) << (k * Sh::WB);
            for (uint64_t left = __ballot(bits != 0); left != 0; left &= left - 1) {
                const int from = (int)__builtin_ctzll(left);
                const uint32_t blocks = (uint32_t)__builtin_amdgcn_readlane((int)bits, from);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                    if (t0 + from >= see_lo[mt] && t0 + from < see_hi[mt]) nan_blocks[mt] |= blocks;
            }
        }
        if (more) {
            fill(t0 + kTile, buf ^ 1);
            bad = bad_next;
        }
    }

    const float vscale = a.cache.v_scale[head];
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
        const float f = at < 0 ? inv * vscale : inv;
        const int64_t place = at + (row - w.row0);
#pragma unroll
        for (int b = 0; b < Sh::NB; ++b) {
            f32x4 x = o[mt][b] * f;
            if (nan_blocks[mt] >> b & 1u) x = f32x4{1.f, 1.f, 1.f, 1.f} * __builtin_nanf("");
            if (at < 0)
                *(u32x2*)(a.out + orow * D + b * 16 + g * 4) = u32x2{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
            else
                *(f32x4*)(a.part + place * D + b * 16 + g * 4) = x;
        }
        if (g == 0) {
            if (at >= 0)
                a.part[(int64_t)2 * a.flat * kChunkRows * D + place] = lse2;
            else if (a.lse != nullptr)
                a.lse[orow] = lse2 * 0.693147180559945309f;
        }
    }
}

// The pieces of share b of the line; the line without shares (flat = 0): one whole query tile.
template <int D>
__device__ __forceinline__ void attn_chunk_body(const Kv4AttentionArgs& a) {
    AttnTile w;
    int r, head, tile, count, k0 = 0, line = 0, stop = 1;
    // blocks of an XCD (block number mod 8) take neighbouring shares, which read the same heads
    const int share = (a.flat & 7) == 0 ? (int)(blockIdx.x & 7) * (a.flat >> 3) + (int)(blockIdx.x >> 3) : (int)blockIdx.x;
    AttnFlat f;
    attn_idle_tokens(a);
    if (a.flat == 0) {
        attn_block(a, r, head, tile);
        attn_request(a, r, w);
        if (!attn_tile(a, tile, w)) return;
    } else {
        f.lay_out(a);
        line = share * f.quota;
        stop = min(f.total, line + f.quota);
    }
    while (line < stop) {
        int begin = w.lo, end = w.hi, at = -1, take = 1;
        if (a.flat != 0) {
            f.find(a, line, r, head, w, k0, count);
            if (k0 < 0) {
                line -= k0;
                k0 = 0;
                if (line >= stop) break;
            }
            take = max(1, min(count - k0, stop - line));
            begin = w.lo + k0 * kTile;
            end = min(w.hi, begin + take * kTile);
            if (take != count) at = (2 * share + (k0 == 0)) * kChunkRows;
        }
        __syncthreads();  // the last piece's reads of LDS
        attn_chunk_piece<D>(a, w, r, head, begin, end, at);
        line += take;
    }
}

#define PLE_ATTN_KERNEL(D, OCC)                                                                                         \
    __global__ __launch_bounds__(kAttnThreads, OCC) void kv4_attention_chunk_##D##_kernel(Kv4AttentionArgs a) {         \
        attn_chunk_body<D>(a);                                                                                          \
    }
PLE_ATTN_KERNEL(64, 2)
PLE_ATTN_KERNEL(128, 2)
PLE_ATTN_KERNEL(256, 1)
#undef PLE_ATTN_KERNEL

// A joined row: v (E elements of each lane) over the weights' sum.
template <int D>
__device__ __forceinline__ void attn_join_store(const Kv4AttentionArgs& a, int64_t orow, float top, float total, float vscale,
                                                const float (&v)[D / 64]) {
    constexpr int E = D / 64;
    const int lane = threadIdx.x & 63;
    const float f = total == 0.f ? 0.f : vscale / total;
    uint16_t* dst = a.out + orow * D + lane * E;
    if constexpr (E == 1) {
        dst[0] = (uint16_t)pack_bf16x2(v[0] * f, 0.f);
    } else {
#pragma unroll
        for (int e = 0; e < E; e += 2) ((uint32_t*)dst)[e / 2] = pack_bf16x2(v[e] * f, v[e + 1] * f);
    }
    if (a.lse != nullptr && lane == 0)
        a.lse[orow] = total == 0.f ? -__builtin_inff() : (top + log2f(total)) * 0.693147180559945309f;
}

// Joins the splits of a row: out = sum_s 2^(lse_s - top) out_s / sum_s 2^(lse_s - top).  Few splits: a wave a row
// (WAVES = 1), four rows a block; many: four waves a row, each with a quarter of the splits, joined through LDS (30
// splits 18.0 us as a whole against 18.8, 29 of a longer cache 1 us less; 4 splits 16.0 against 15.5, between 7 and 16
// splits no difference beyond the spread).
template <int D, int WAVES>
__device__ __forceinline__ void attn_join_body(const Kv4AttentionArgs& a) {
    constexpr int E = D / 64;  // elements of a lane
    __shared__ float part[WAVES == 1 ? 1 : WAVES * D], part_l[WAVES];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t rows = a.batch.num_tokens * a.num_q_heads;
    const int64_t orow = WAVES == 1 ? (int64_t)blockIdx.x * 4 + wave : (int64_t)blockIdx.x;
    if (orow >= rows) return;
    const int64_t t = orow / a.num_q_heads;
    const int hq = (int)(orow - t * a.num_q_heads), head = hq / a.group;
    int r;
    int64_t start;
    wave_find_request(a.batch.query_start_loc, a.batch.num_reqs, t, t, 1, 0, lane, r, start);
    AttnTile w;
    attn_request(a, r, w);
    if (t < w.first || t >= w.first + w.n) return;
    const int row = (int)(t - w.first) * a.group + (hq - head * a.group);
    if (!attn_tile(a, row / a.rows, w)) return;
    const int splits = attn_splits(a, w);
    if (splits == 1) return;
    const float* lse = a.part + rows * a.splits * D + orow * a.splits;
    const float* src = a.part + orow * a.splits * D + lane * E;
    float top = -__builtin_inff();
    for (int s = lane; s < splits; s += kWave) top = fmaxf(top, lse[s]);
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor(top, d, kWave));
    float total = 0.f, v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = 0.f;
#pragma unroll 8
    for (int s = WAVES == 1 ? 0 : wave; s < splits; s += WAVES) {
        const float l = lse[s], by = l == -__builtin_inff() ? 0.f : __builtin_amdgcn_exp2f(l - top);  // NaN stays
        total += by;
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = fmaf(src[(int64_t)s * D + e], by, v[e]);
    }
    if constexpr (WAVES > 1) {
#pragma unroll
        for (int e = 0; e < E; ++e) part[wave * D + lane * E + e] = v[e];
        if (lane == 0) part_l[wave] = total;
        __syncthreads();
        if (wave != 0) return;
        total = 0.f;
#pragma unroll
        for (int k = 0; k < WAVES; ++k) total += part_l[k];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            v[e] = 0.f;
#pragma unroll
            for (int k = 0; k < WAVES; ++k) v[e] += part[k * D + lane * E + e];
        }
    }
    attn_join_store<D>(a, orow, top, total, a.cache.v_scale[head], v);
}

#define PLE_ATTN_KERNEL(D, WAVES)                                                                          \
    __global__ __launch_bounds__(256) void kv4_attention_join_##D##_##WAVES##_kernel(Kv4AttentionArgs a) { \
        attn_join_body<D, WAVES>(a);                                                                       \
    }
PLE_ATTN_KERNEL(64, 1)
PLE_ATTN_KERNEL(64, 4)
PLE_ATTN_KERNEL(128, 1)
PLE_ATTN_KERNEL(128, 4)
PLE_ATTN_KERNEL(256, 1)
PLE_ATTN_KERNEL(256, 4)
#undef PLE_ATTN_KERNEL

// Joins the pieces of the query tiles that the shares' borders cut.  Blocks: query tile, 32 of its rows; a wave a row.
template <int D>
__device__ __forceinline__ void attn_flat_join_body(const Kv4AttentionArgs& a) {
    constexpr int E = D / 64;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int r, head, tile;
    attn_block(a, r, head, tile);
    AttnTile w;
    attn_request(a, r, w);
    if (!attn_tile(a, tile, w)) return;
    if (w.row0 + (int)blockIdx.y * kFlatJoinRows >= w.row1) return;
    const int count = AttnFlat::count(w);
    AttnFlat f;
    f.lay_out(a);
    int sum = 0;
    {
        AttnTile u = w;
        for (int t = lane; t < tile; t += kWave) sum += AttnFlat::places(a, t, u);
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d, kWave);
    }
    const int at = __builtin_amdgcn_readlane(f.before, r) + head * __builtin_amdgcn_readlane(f.tiles_of, r) + sum;
    const int s0 = (at + kFlatStart) / f.quota, pieces = (at + kFlatStart + count - 1) / f.quota - s0 + 1;
    if (pieces == 1) return;
    const float* const all_lse = a.part + (int64_t)2 * a.flat * kChunkRows * D;
    const float vscale = a.cache.v_scale[head];
    // a wave takes eight rows at once, so that their loads are in flight together (rows past the tile's end repeat its last)
    constexpr int N = kFlatJoinRows / kAttnWaves;
    const int in0 = (int)blockIdx.y * kFlatJoinRows + wave * N, most = w.row1 - w.row0 - 1;
    float top[N], total[N], v[N][E];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        top[i] = -__builtin_inff();
        total[i] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) v[i][e] = 0.f;
    }
    for (int k = 0; k < pieces; ++k)
#pragma unroll
        for (int i = 0; i < N; ++i)
            top[i] = fmaxf(top[i], all_lse[(int64_t)(2 * (s0 + k) + (k == 0)) * kChunkRows + min(in0 + i, most)]);
    for (int k = 0; k < pieces; ++k)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int64_t place = (int64_t)(2 * (s0 + k) + (k == 0)) * kChunkRows + min(in0 + i, most);
            const float l = all_lse[place];
            const float by = l == -__builtin_inff() ? 0.f : __builtin_amdgcn_exp2f(l - top[i]);  // NaN stays
            total[i] += by;
#pragma unroll
            for (int e = 0; e < E; ++e) v[i][e] = fmaf(a.part[place * D + lane * E + e], by, v[i][e]);
        }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int row = w.row0 + in0 + i;
        if (row >= w.row1) break;
        const int t = row / a.group, hq = head * a.group + (row - t * a.group);
        attn_join_store<D>(a, (w.first + t) * a.num_q_heads + hq, top[i], total[i], vscale, v[i]);
    }
}

#define PLE_ATTN_KERNEL(D)                                                                            \
    __global__ __launch_bounds__(256) void kv4_attention_flat_join_##D##_kernel(Kv4AttentionArgs a) { \
        attn_flat_join_body<D>(a);                                                                    \
    }
PLE_ATTN_KERNEL(64)
PLE_ATTN_KERNEL(128)
PLE_ATTN_KERNEL(256)
#undef PLE_ATTN_KERNEL

void plan_kv4_attention(Kv4AttentionArgs& a) {
    const int64_t T = a.batch.num_tokens, R = a.batch.num_reqs;
    const int64_t cover = (int64_t)a.batch.table_width * a.cache.page_size;
    int64_t new_max = a.batch.max_request_tokens > 0 ? a.batch.max_request_tokens : T;
    new_max = new_max < T ? new_max : T;
    int64_t len = a.batch.max_seq_len > 0 && a.batch.max_seq_len < cover ? a.batch.max_seq_len : cover;
    const int64_t rows = new_max * a.group;
    // up to 64 rows in tiles whose state fits the registers of two waves per SIMD (32 windows of 8 tokens, 8 query heads a
    // key head, 3000 tokens: 27.5 us, in one tile of 128 52)
    a.rows = rows <= 16 || (rows <= 64 && a.cache.head_dim == 256) ? 16 : (rows <= 64 ? 32 : kChunkRows);
    a.tiles = (int)((rows + a.rows - 1) / a.rows);
    if (a.window > 0) {
        const int64_t span = (int64_t)a.window + a.rows / a.group + 1 + 15;
        len = len < span ? len : span;
    }
    // Splits where the query tiles alone leave CUs idle, each of at least 1024 tokens, below which a block's fixed cost
    // and the joining kernel outweigh what a shorter loop saves (8 requests of up to 2500 tokens 15.6 us, with 512 16.2,
    // 256 20.1, 2048 17.5; 4 of 20000 18.2, 18.3, 21.9 and 20.2).  Up to one block per CU: blocks of eight waves (verify
    // windows 64 x 4 17.2 us, of four in twice the splits 23.8; one of 131k tokens 34.6 against 38.5; 256 blocks over 2000
    // tokens 17.5 against 21.8; 264 blocks 21.2 against 21.1, 768 over 500 23.7 against 14.7, but 264 over 8000 44 against
    // 54).  Blocks of four waves in as many splits as two or three of them per CU (384 blocks over 4000 tokens 37.8 us
    // with 768 slots, 41.1 with 512, 39.5 with 1024; over 8000 1024 would be better, 320 blocks 49.9 against 57.6).
    const int64_t blocks = R * a.cache.num_kv_heads * a.tiles;
    // (the line's length has to fit 32 bits whatever the hints say)
    if (a.rows == kChunkRows && R <= kWave && blocks > 0 && blocks <= kFlatUnits &&
        blocks * (cover / kTile + 2 + kFlatStart) < ((int64_t)1 << 30)) {
        const int64_t most = blocks * ((len + kTile - 1) / kTile + 1 + kFlatStart), slots = a.cache.head_dim == 256 ? 256 : 512;
        const int64_t shares = (most + kFlatLeast - 1) / kFlatLeast;
        a.flat = (int)(shares < slots ? shares : slots);
        a.waves = kAttnWaves;
        a.splits = 1;
        return;
    }
    a.waves = blocks <= 256 && a.rows < kChunkRows ? 8 : 4;
    const int64_t slots = a.waves == 8 ? 256 : (a.rows == 16 && a.cache.head_dim < 256 ? 768 : 512);
    int64_t splits = blocks <= 0 || a.rows == kChunkRows ? 1 : slots / blocks;
    const int64_t most_splits = (len + 1023) / 1024;
    splits = splits < most_splits ? splits : most_splits;
    splits = splits < 1 ? 1 : (splits < kMostSplits - 1 ? splits : kMostSplits - 1);
    int64_t chunk = (len + splits - 1) / splits;
    const int64_t round = a.rows == kChunkRows ? kTile : kTile * a.waves;  // what a block goes through at a time
    chunk = (chunk + round - 1) / round * round;
    a.chunk = (int)chunk;
    // (a range starts at a multiple of 16, up to 15 tokens before the first that is seen; the last split takes those)
    a.splits = (int)((len + chunk - 1) / chunk);
    if (a.splits < 1) a.splits = 1;
}

size_t kv4_attention_part_bytes(const Kv4AttentionArgs& a) {
    if (a.flat > 0) return (size_t)2 * a.flat * kChunkRows * (a.cache.head_dim + 1) * sizeof(float);
    if (a.splits <= 1) return 0;
    return (size_t)a.batch.num_tokens * a.num_q_heads * a.splits * (a.cache.head_dim + 1) * sizeof(float);
}

// Query tiles of all requests and key heads, and blocks along x of the kernel that joins splits.
static int64_t attention_units(const Kv4AttentionArgs& a) {
    return (int64_t)a.batch.num_reqs * a.cache.num_kv_heads * a.tiles;
}
static int64_t join_blocks(const Kv4AttentionArgs& a) {
    const int64_t rows = a.batch.num_tokens * a.num_q_heads;
    return a.splits <= kFewSplits ? (rows + 3) / 4 : rows;
}

int64_t kv4_attention_threads(const Kv4AttentionArgs& a) {
    // (the shares are at most 512 blocks, their join a block per unit)
    const int64_t own = attention_units(a) * (a.flat > 0 ? 256 : a.waves * kWave);
    const int64_t join = a.splits > 1 ? join_blocks(a) * 256 : 0;
    return own > join ? own : join;
}

template <void (*FN)(Kv4AttentionArgs), int LDS>
static hipError_t launch_attention(const Kv4AttentionArgs& a, int threads, hipStream_t s) {
    static const hipError_t attr = hipFuncSetAttribute((const void*)FN, hipFuncAttributeMaxDynamicSharedMemorySize, LDS);
    if (attr != hipSuccess) return attr;
    const dim3 grid((unsigned)(a.flat > 0 ? a.flat : attention_units(a)), (unsigned)a.splits);
    hipLaunchKernelGGL(FN, grid, dim3(threads), LDS, s, a);
    return hipGetLastError();
}

hipError_t launch_kv4_attention(const Kv4AttentionArgs& a, hipStream_t s) {
    const int D = a.cache.head_dim, mt = a.rows / 16;
    hipError_t e = hipErrorInvalidValue;
    if (a.rows == kChunkRows)
        e = D == 64    ? launch_attention<kv4_attention_chunk_64_kernel, ChunkShape<64>::LDS>(a, kAttnThreads, s)
            : D == 128 ? launch_attention<kv4_attention_chunk_128_kernel, ChunkShape<128>::LDS>(a, kAttnThreads, s)
                       : launch_attention<kv4_attention_chunk_256_kernel, ChunkShape<256>::LDS>(a, kAttnThreads, s);
#define PLE_ATTN_LAUNCH(DD, MT, WAVES, OCC)                                                                             \
    if (D == DD && mt == MT && a.waves == WAVES)                                                                        \
        e = launch_attention<kv4_attention_##DD##_##MT##x##WAVES##_kernel, AttnShape<DD, WAVES>::LDS>(a, WAVES * kWave, s);
    PLE_ATTN_SHAPES(PLE_ATTN_LAUNCH)
#undef PLE_ATTN_LAUNCH
    if (e == hipSuccess && a.flat > 0) {
        const dim3 grid((unsigned)attention_units(a), kChunkRows / kFlatJoinRows);
        if (D == 64)
            hipLaunchKernelGGL(kv4_attention_flat_join_64_kernel, grid, dim3(256), 0, s, a);
        else if (D == 128)
            hipLaunchKernelGGL(kv4_attention_flat_join_128_kernel, grid, dim3(256), 0, s, a);
        else
            hipLaunchKernelGGL(kv4_attention_flat_join_256_kernel, grid, dim3(256), 0, s, a);
        return hipGetLastError();
    }
    if (e != hipSuccess || a.splits <= 1) return e;
    const bool few = a.splits <= kFewSplits;
    const dim3 grid((unsigned)join_blocks(a));
#define PLE_ATTN_LAUNCH(DD)                                                                                          \
    if (D == DD) {                                                                                                   \
        if (few)                                                                                                     \
            hipLaunchKernelGGL(kv4_attention_join_##DD##_1_kernel, grid, dim3(256), 0, s, a);                        \
        else                                                                                                         \
            hipLaunchKernelGGL(kv4_attention_join_##DD##_4_kernel, grid, dim3(256), 0, s, a);                        \
    }
    PLE_ATTN_LAUNCH(64)
    PLE_ATTN_LAUNCH(128)
    PLE_ATTN_LAUNCH(256)
#undef PLE_ATTN_LAUNCH
    return hipGetLastError();
}

}  // namespace ple
