// What attention over a paged cache does whatever its codes are: which tokens and rows a block has, the way along a
// request's pages, cutting query tiles into even shares, joining partial results.  The 4-bit and the 8-bit kernels
// (ple_kv4_attention.hip, ple_kv8_attention.hip) are written on it; A is the kernel's arguments (PagedAttentionArgs of
// its cache), value_scale(a, head) what the joined values are multiplied by.
#pragma once

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

// Measured in 4 bits with 32 heads of 128 over 8, and where a value other than these does better too:
//  kFlatLeast: 1289 + 1455 tokens at 5403 and 2004 219 us with 2, 4, 8 and 16; 100 behind 2000 40.5 (with 4 42, 2 45, 16 57);
//              1000 behind nothing 50 (4 51, 16 66); but 100 behind nothing 27 (4 18), 50 behind 500 33 (4 28).
//  kFlatStart: the first 219 us (with 0 256, 2 238, 8 228), the second 40.5 (48, 43, 40), the third 50 (82, 58, 56).
//  kFlatUnits: 736 query tiles 219 us in shares, 388 a block each; 4864 of 32 requests 419 and 388, which the rule keeps
//              apart; but it takes the slower one for 1920 tiles of 16 requests (207 and 179), 2560 of 32 (243 and 211) and
//              behind nothing (1000 tokens 50 and 47, 100 27 and 15).  The 8-bit plan has a rule of its own for those.
constexpr int kFlatLeast = 8;        // places of a share at least
constexpr int kFlatStart = 4;        // places that beginning a query tile counts for (queries in, results out)
constexpr int kFlatUnits = 4096;     // query tiles (of all heads and requests) up to which the work is cut into shares
constexpr int kFlatJoinRows = 32;    // rows of a block of the joining kernel

constexpr int kChunkRows = 128;  // rows of a query tile of the many-row kernels

union Frag {
    f16x8 v;
    f16x2 p[4];
    u32x4 u;
};

// max over the four lanes n, n + 16, n + 32, n + 48
__device__ __forceinline__ float quad_max(float x) {
    typedef unsigned int u2 __attribute__((ext_vector_type(2)));
    u2 w = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = fmaxf(__uint_as_float(w[0]), __uint_as_float(w[1]));
    w = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(w[0]), __uint_as_float(w[1]));
}

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
template <class A>
__device__ __forceinline__ void attn_request(const A& a, int r, AttnTile& w) {
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
template <class A>
__device__ __forceinline__ void attn_idle_tokens(const A& a) {
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
template <class A>
__device__ __forceinline__ bool attn_tile(const A& a, int tile, AttnTile& w) {
    w.row0 = tile * a.rows;
    w.row1 = min(w.row0 + a.rows, w.n * a.group);
    if (w.row0 >= w.row1) return false;
    w.hi = max(0, min(w.len, w.before + (w.row1 - 1) / a.group + 1));
    w.first_seen = a.window > 0 ? max(0, w.before + w.row0 / a.group - a.window + 1) : 0;
    w.lo = min(w.first_seen & ~15, w.hi & ~15);
    return true;
}

template <class A>
__device__ __forceinline__ int attn_splits(const A& a, const AttnTile& w) {
    const int s = (w.hi - w.lo + a.chunk - 1) / a.chunk;
    return max(1, min(s, a.splits));
}

// Request, key head and query tile of a block.  Blocks of one request and head are a multiple of the pairs apart, so
// with the usual 8 heads they run on one XCD and share its L2; the tiles with the most to see come first.
template <class A>
__device__ __forceinline__ void attn_block(const A& a, int& r, int& head, int& tile) {
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

    template <class A>
    __device__ __forceinline__ PageWalk(const A& a, const int32_t* table_row, int h, int tg, int step, int end)
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

// Few query tiles, of requests of different lengths, leave CUs idle at the end.  Then the cache tiles of all query
// tiles (at least one each), in the order request, key head, query tile, are one line that `flat` blocks cut into equal
// shares; a query tile has kFlatStart places in front of its cache tiles.  A query tile whose cache tiles a cut goes
// through is joined by a second kernel: of its pieces the one that begins it is partial result 2 * share + 1, every
// other 2 * share of its share.  The share that begins it leaves word of it (AttnCut) behind the partial results.
// A chunk of 1289 + 1455 tokens at 5403 and 2004: 388 us with a block a query tile, 219 in shares (in 4 bits).
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
    template <class A>
    static __device__ __forceinline__ int places(const A& a, int t, AttnTile& w) {
        return t < a.tiles && attn_tile(a, t, w) ? kFlatStart + count(w) : 0;
    }

    template <class A>
    __device__ __forceinline__ void lay_out(const A& a) {
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
    template <class A>
    __device__ __forceinline__ void find(const A& a, int at, int& r, int& head, AttnTile& w, int& k0,
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

// The join's rows of D elements in LDS (fp32).
template <int D>
constexpr int kJoinRow = D + 4;

// The end of a block's work: its waves' sums are joined, one row tile of 16 at a time, and stored (partial results where
// there are more splits).  nan_blocks: element blocks of the row that a NaN value makes NaN.
template <int D, int MT, int WAVES, class A>
__device__ __forceinline__ void attn_join_waves(const A& a, const AttnTile& w, int head, int split, int splits, char* lds,
                                                float (&m)[MT], float (&l)[MT], f32x4 (&o)[MT][D / 16],
                                                const uint32_t (&nan_blocks)[MT]) {
    constexpr int NB = D / 16, OROW = kJoinRow<D>;
    __shared__ float join_m[kAttnWaves][16], join_l[kAttnWaves][16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n = lane & 15, g = lane >> 4;
    const float vscale = value_scale(a, head);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        float sum = l[mt];
        sum += __shfl_xor(sum, 16, kWave);
        sum += __shfl_xor(sum, 32, kWave);
        float* jo = (float*)lds + ((wave & 3) * 16 + n) * OROW;
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
                for (int b = 0; b < NB; ++b) *(f32x4*)(jo + b * 16 + g * 4) = o[mt][b];
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
                for (int b = 0; b < NB; ++b) {
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
                    const f32x4 x = *(const f32x4*)((float*)lds + (k * 16 + row) * OROW + part * E + e);
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

// The query tile that a share begins and does not finish: its pieces (0: there is none), its request's first new token, its
// key head, first row and rows.
struct AttnCut {
    int pieces, first, head, row0, rows, unused[3];
};
template <class A>
__host__ __device__ __forceinline__ size_t attn_flat_floats(const A& a) {
    return (size_t)2 * a.flat * kChunkRows * (a.cache.head_dim + 1);
}
template <class A>
__device__ __forceinline__ AttnCut* attn_cuts(const A& a) {
    return (AttnCut*)(a.part + attn_flat_floats(a));
}

// The same in scalar registers: all of it is the wave's.
__device__ __forceinline__ AttnTile uniform(const AttnTile& w) {
    const auto u = [](int x) { return __builtin_amdgcn_readfirstlane(x); };
    return {u((int)w.first), u(w.n), u(w.len), u(w.before), u(w.row0), u(w.row1), u(w.first_seen), u(w.lo), u(w.hi)};
}

// The pieces (each by `piece`) of share b of the line; the line without shares (flat = 0): one whole query tile.
template <class A, class Piece>
__device__ __forceinline__ void attn_chunk_body(const A& a, Piece piece) {
    AttnTile w;
    int r, head, tile, k0 = 0, left = 1, quota = 0;
    // blocks of an XCD (block number mod 8) take neighbouring shares, which read the same heads
    const int share = (a.flat & 7) == 0 ? (int)(blockIdx.x & 7) * (a.flat >> 3) + (int)(blockIdx.x >> 3) : (int)blockIdx.x;
    attn_idle_tokens(a);
    if (a.flat == 0) {
        attn_block(a, r, head, tile);
        attn_request(a, r, w);
        if (!attn_tile(a, tile, w)) return;
    } else {
        if (threadIdx.x == 0) attn_cuts(a)[share].pieces = 0;
        AttnFlat f;
        f.lay_out(a);
        quota = __builtin_amdgcn_readfirstlane(f.quota);
        const int line = share * quota;
        left = min(f.total - line, quota);
        if (left <= 0) return;
        int count;
        f.find(a, line, r, head, w, k0, count);
        tile = w.row0 / kChunkRows;
    }
    r = __builtin_amdgcn_readfirstlane(r);
    head = __builtin_amdgcn_readfirstlane(head);
    tile = __builtin_amdgcn_readfirstlane(tile);
    k0 = __builtin_amdgcn_readfirstlane(k0);
    left = __builtin_amdgcn_readfirstlane(left);
    for (;;) {
        w = uniform(w);
        int begin = w.lo, end = w.hi, at = -1;
        if (a.flat != 0) {
            if (k0 < 0) {  // places in front of the query tile's cache tiles
                left += k0;
                k0 = 0;
                if (left <= 0) return;
            }
            const int count = AttnFlat::count(w), take = max(1, min(count - k0, left));
            begin = w.lo + k0 * kTile;
            end = min(w.hi, begin + take * kTile);
            if (take != count) at = (2 * share + (k0 == 0)) * kChunkRows;
            left -= take;
            if (k0 == 0 && take != count && threadIdx.x == 0)
                attn_cuts(a)[share] = {1 + (count - take + quota - 1) / quota, (int)w.first, head, w.row0, w.row1 - w.row0, {}};
        }
        __syncthreads();  // the last piece's reads of LDS
        piece(w, r, head, begin, end, at);
        if (a.flat == 0 || left <= 0) return;
        // the next query tile of the line
        k0 = -kFlatStart;
        ++tile;
        while (tile >= a.tiles || !attn_tile(a, tile, w)) {
            tile = 0;
            if (++head == a.cache.num_kv_heads) {
                head = 0;
                if (++r == a.batch.num_reqs) return;
                attn_request(a, r, w);
            }
        }
    }
}

// A joined row: v (E elements of each lane) over the weights' sum.
template <int D, class A>
__device__ __forceinline__ void attn_join_store(const A& a, int64_t orow, float top, float total, float vscale,
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
template <int D, int WAVES, class A>
__device__ __forceinline__ void attn_join_body(const A& a) {
    constexpr int E = D / 64;  // elements of a lane
    __shared__ float part[WAVES == 1 ? 1 : WAVES * D], part_l[WAVES];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t rows = a.batch.num_tokens * a.num_q_heads;
    const int64_t orow = WAVES == 1 ? (int64_t)blockIdx.x * 4 + wave : (int64_t)blockIdx.x;
    if (orow >= rows) return;
    const float* lse = a.part + rows * a.splits * D + orow * a.splits;
    const float* src = a.part + orow * a.splits * D + lane * E;
    // The first splits' results come in while the row's request and its number of splits are found (those past it, not
    // written by this call, are dropped again).
    constexpr int kAhead = 8;
    const float first_lse = lane < a.splits ? lse[lane] : 0.f;
    float ahead[kAhead][E];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        const int s = (WAVES == 1 ? 0 : wave) + i * WAVES;
#pragma unroll
        for (int e = 0; e < E; ++e) ahead[i][e] = s < a.splits ? src[(int64_t)s * D + e] : 0.f;
    }
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
    float top = lane < splits ? first_lse : -__builtin_inff();
    for (int s = lane + kWave; s < splits; s += kWave) top = fmaxf(top, lse[s]);
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor(top, d, kWave));
    float total = 0.f, v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = 0.f;
    const auto weight = [&](float l) { return l == -__builtin_inff() ? 0.f : __builtin_amdgcn_exp2f(l - top); };  // NaN stays
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        const int s = (WAVES == 1 ? 0 : wave) + i * WAVES;
        if (s >= splits) break;
        const float by = weight(__shfl(first_lse, s, kWave));
        total += by;
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = fmaf(ahead[i][e], by, v[e]);
    }
#pragma unroll 8
    for (int s = (WAVES == 1 ? 0 : wave) + kAhead * WAVES; s < splits; s += WAVES) {
        const float by = weight(lse[s]);
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
    attn_join_store<D>(a, orow, top, total, value_scale(a, head), v);
}

// Joins the pieces of the query tiles that the shares' borders cut.  Blocks: query tile, 32 of its rows; a wave a row.
template <int D, class A>
__device__ __forceinline__ void attn_flat_join_body(const A& a) {
    constexpr int E = D / 64;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int s0 = blockIdx.x;
    const AttnCut cut = attn_cuts(a)[s0];
    const int pieces = cut.pieces, head = cut.head;
    if (pieces == 0 || (int)blockIdx.y * kFlatJoinRows >= cut.rows) return;
    const float* const all_lse = a.part + (int64_t)2 * a.flat * kChunkRows * D;
    const float vscale = value_scale(a, head);
    // a wave takes eight rows at once, so that their loads are in flight together (rows past the tile's end repeat its last)
    constexpr int N = kFlatJoinRows / kAttnWaves;
    const int in0 = (int)blockIdx.y * kFlatJoinRows + wave * N, most = cut.rows - 1;
    float top[N], total[N], v[N][E];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        top[i] = -__builtin_inff();
        total[i] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) v[i][e] = 0.f;
    }
    const auto place = [&](int k, int i) {
        return (int64_t)(2 * (s0 + k) + (k == 0)) * kChunkRows + min(in0 + i, most);
    };
    const auto add = [&](int i, float l, const float (&x)[E]) {
        const float by = l == -__builtin_inff() ? 0.f : __builtin_amdgcn_exp2f(l - top[i]);  // NaN stays
        total[i] += by;
#pragma unroll
        for (int e = 0; e < E; ++e) v[i][e] = fmaf(x[e], by, v[i][e]);
    };
    if (pieces == 2) {  // (nearly all) everything on its way at once
        float l[2][N], x[2][N][E];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                l[k][i] = all_lse[place(k, i)];
#pragma unroll
                for (int e = 0; e < E; ++e) x[k][i][e] = a.part[place(k, i) * D + lane * E + e];
            }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            top[i] = fmaxf(fmaxf(top[i], l[0][i]), l[1][i]);
            add(i, l[0][i], x[0][i]);
            add(i, l[1][i], x[1][i]);
        }
    } else {
        // (two pieces' loads on their way at a time; past the last one it is read again, which a maximum does not mind)
        for (int k = 0; k < pieces; k += 2) {
            float l[2][N];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < N; ++i) l[u][i] = all_lse[place(min(k + u, pieces - 1), i)];
#pragma unroll
            for (int i = 0; i < N; ++i) top[i] = fmaxf(fmaxf(top[i], l[0][i]), l[1][i]);
        }
        for (int k = 0; k < pieces; k += 2) {
            float l[2][N], x[2][N][E];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int64_t at = place(min(k + u, pieces - 1), i);
                    l[u][i] = all_lse[at];
#pragma unroll
                    for (int e = 0; e < E; ++e) x[u][i][e] = a.part[at * D + lane * E + e];
                }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                add(i, l[0][i], x[0][i]);
                if (k + 1 < pieces) add(i, l[1][i], x[1][i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (in0 + i > most) break;
        const int row = cut.row0 + in0 + i, t = row / a.group, hq = head * a.group + (row - t * a.group);
        attn_join_store<D>(a, ((int64_t)cut.first + t) * a.num_q_heads + hq, top[i], total[i], vscale, v[i]);
    }
}

// Query tiles of all requests and key heads, and blocks along x of the kernel that joins splits.
template <class A>
int64_t attention_units(const A& a) {
    return (int64_t)a.batch.num_reqs * a.cache.num_kv_heads * a.tiles;
}
template <class A>
int64_t join_blocks(const A& a) {
    const int64_t rows = a.batch.num_tokens * a.num_q_heads;
    return a.splits <= kFewSplits ? (rows + 3) / 4 : rows;
}

template <class A>
size_t attention_part_bytes(const A& a) {
    if (a.flat > 0) return attn_flat_floats(a) * sizeof(float) + a.flat * sizeof(AttnCut);
    if (a.splits <= 1) return 0;
    return (size_t)a.batch.num_tokens * a.num_q_heads * a.splits * (a.cache.head_dim + 1) * sizeof(float);
}

// Most threads along x of the call's launches.
template <class A>
int64_t attention_threads(const A& a) {
    // (shares and their join are at most 512 blocks)
    const int64_t own = a.flat > 0 ? a.flat * 256 : attention_units(a) * a.waves * kWave;
    const int64_t join = a.splits > 1 ? join_blocks(a) * 256 : 0;
    return own > join ? own : join;
}

template <class A, void (*FN)(A), int LDS>
hipError_t launch_attention(const A& a, int threads, hipStream_t s) {
    static const hipError_t attr = hipFuncSetAttribute((const void*)FN, hipFuncAttributeMaxDynamicSharedMemorySize, LDS);
    if (attr != hipSuccess) return attr;
    const dim3 grid((unsigned)(a.flat > 0 ? a.flat : attention_units(a)), (unsigned)a.splits);
    hipLaunchKernelGGL(FN, grid, dim3(threads), LDS, s, a);
    return hipGetLastError();
}

// The kernel that joins partial results, if there are any: of up to kFewSplits splits or of more, or of cut query tiles.
template <class A>
hipError_t launch_attention_join(const A& a, void (*few)(A), void (*many)(A), void (*flat)(A), hipStream_t s) {
    if (a.flat > 0)
        hipLaunchKernelGGL(flat, dim3((unsigned)a.flat, kChunkRows / kFlatJoinRows), dim3(256), 0, s, a);
    else if (a.splits > 1)
        hipLaunchKernelGGL(a.splits <= kFewSplits ? few : many, dim3((unsigned)join_blocks(a)), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace ple
