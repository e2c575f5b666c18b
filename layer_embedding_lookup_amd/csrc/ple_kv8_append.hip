// New keys and values, rotated by position, into the paged 8-bit cache, and
// back out of it.
//
// A block of 16 tokens and a head share one scale, so a wave takes a whole
// block of one head's keys or values: the largest magnitude of its new tokens
// gives the scale, a power of two, by which they are coded; where tokens of
// the request stand in the block before them and its scale grows, their codes
// are read, taken to the new scale and written back.  Both layouts of the
// cache are written in 16-byte pieces where a block is filled as a whole.
// Queries go through blocks of their own, one per token.
//
// Requests' blocks are numbered one after the other without a count of them:
// request r has those from floor(start of r / 16) + 2 r on, which is enough
// for any position it begins at.
//
// Angles are formed in 64 bits (positions of 10^5 and more lose them in 32),
// in turns: position * (frequency / 2 pi), whose two roundings are 2^-52 of
// the angle, needs no reduction by pi.  A thread forms sine and cosine of its
// first new token of four and of the step from one token to the next; the
// others follow by products (2^-51 after three).
//
// Bound by bytes where tokens are many: 8178 tokens, 32 + 8 heads of 128, half
// of each rotated: 42 us for 184 MB in and out (4.4 TB/s), back out of the cache
// 13.6 us for 50 MB.  256 single tokens 10.6 and 9.6 us: a chain of loads that
// depend on each other (offsets, length, page, scale, codes), each to memory,
// and a whole 2 KiB block of a head's values where one token is read or its
// scale grows, since a lane's 16 bytes are one element of 16 tokens, as
// attention takes them.
#include "ple_8bit_launch.h"
#include "ple_rotate.h"

namespace ple {

constexpr int kAppendThreads = 256;
constexpr double kPerTurn = 0.15915494309189533577;  // 1 / (2 pi)
constexpr int kAppendWaves = kAppendThreads / kWave;

// What a unit of the launch writes or reads: new tokens of request r at places [from, to) of a block.
struct Kv8Unit {
    int r, group;     // group of head 0 (one head on: page_size / 16 groups on); -1: the table names no page
    int64_t first;    // the new token at place `from`
    int block;        // position / 16
    int from, to;     // (from > 0: earlier tokens of the request stand before it)
    bool any;
    int64_t index;    // of the request's blocks
    int64_t q0, n, lo, hi;  // its new tokens q0 .. q0 + n, of which those from lo up to hi stand on some place
};

// Blocks that the launch has for requests: with a hint as many as a request can reach, times the requests; or by their
// starts as above.
__host__ __device__ __forceinline__ int64_t kv8_units_each(const ple_kv8_batch& b) {
    return b.max_request_tokens > 0 ? ((int64_t)b.max_request_tokens + 14) / 16 + 1 : 0;
}
__host__ __device__ __forceinline__ int64_t kv8_units(const ple_kv8_batch& b, bool hint) {
    const int64_t by_start = b.num_tokens / 16 + 2 * (int64_t)b.num_reqs;
    const int64_t each = hint ? kv8_units_each(b) : 0;
    return each > 0 && each * b.num_reqs < by_start ? each * b.num_reqs : by_start;
}

__device__ __forceinline__ Kv8Unit kv8_unit(const ple_kv8_cache& c, const ple_kv8_batch& b, int64_t u, bool hint) {
    Kv8Unit w;
    const int64_t T = b.num_tokens, each = hint ? kv8_units_each(b) : 0;
    const auto start = [&](int r) { return min(max((int64_t)b.query_start_loc[r], (int64_t)0), T); };
    int64_t i;
    if (each > 0 && each * b.num_reqs == kv8_units(b, hint)) {
        w.r = (int)(u / each);
        i = u - w.r * each;
    } else {
        const auto number = [&](int64_t first, int r) { return min(max(first, (int64_t)0), T) / 16 + 2 * (int64_t)r; };
        if (b.num_reqs <= 16 * kWave) {  // the wave counts the requests that begin at or before it: one round of loads
            const int lane = threadIdx.x & 63;
            int first[16], count = 0;
#pragma unroll
            for (int c = 0; c < 16; ++c)
                if (c * kWave < b.num_reqs) first[c] = b.query_start_loc[min(c * kWave + lane, b.num_reqs)];
#pragma unroll
            for (int c = 0; c < 16; ++c)
                if (c * kWave < b.num_reqs) {
                    const int r = c * kWave + lane;
                    count += (int)__popcll(__ballot(r < b.num_reqs && number(first[c], r) <= u));
                }
            w.r = max(count - 1, 0);
        } else {
            int lo = 0, hi = b.num_reqs - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (number(b.query_start_loc[mid], mid) <= u)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            w.r = lo;
        }
        i = u - number(b.query_start_loc[w.r], w.r);
    }
    // (by the whole length and all of the request's tokens, as kv4_position)
    const int64_t q0 = start(w.r), to = b.query_start_loc[w.r + 1], n = max(min(to, T) - q0, (int64_t)0);
    const int64_t before = (int64_t)b.seq_lens[w.r] - (to - q0);
    const int64_t lo = max(before, (int64_t)0), hi = min(before + n, (int64_t)b.table_width * c.page_size);
    const int64_t block = lo / 16 + i;
    const int64_t p0 = max(lo, block * 16), p1 = min(hi, block * 16 + 16);
    w.any = i >= 0 && p0 < p1;
    w.index = i;
    w.q0 = q0;
    w.n = n;
    w.lo = min(lo - before, n);
    w.hi = max(min(hi - before, n), w.lo);
    w.block = (int)block;
    w.from = (int)(p0 - block * 16);
    w.to = (int)(p1 - block * 16);
    w.first = q0 + (p0 - before);
    w.group = w.any ? kv4_group(c, b.page_table + (int64_t)w.r * b.table_width, 0, w.block) : -1;
    return w;
}

// kv4_position with the request found by the whole wave in one round of loads.
__device__ __forceinline__ int kv8_position(const ple_kv8_cache& c, const ple_kv8_batch& b, int64_t t) {
    int r;
    int64_t start;
    wave_find_request(b.query_start_loc, b.num_reqs, t, t, 1, 0, threadIdx.x & 63, r, start);
    const int64_t from = b.query_start_loc[r], to = b.query_start_loc[r + 1];
    const int64_t p = (int64_t)b.seq_lens[r] - (to - t);
    return t < from || t >= to || p < 0 || p >= (int64_t)b.table_width * c.page_size ? -1 : (int)p;
}

// The least power of two s with top <= 448 s, within the cache's range; top >= 0 and finite.
__device__ __forceinline__ float block_scale(float top) {
    const uint32_t u = __float_as_uint(top);
    int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);  // 448 = 1.75 * 2^8
    e = min(max(e, -32), 32);
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

__device__ __forceinline__ float finite_size(float x) { return x - x == 0.f ? fabsf(x) : 0.f; }

// x / s as the cache holds it, before its rounding: at most 448, NaN for what is not finite.
__device__ __forceinline__ float coded(float x, float inv) {
    return x - x == 0.f ? __builtin_amdgcn_fmed3f(x * inv, -448.f, 448.f) : __builtin_nanf("");
}
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}
// Four codes at a larger scale (by: old over new).
__device__ __forceinline__ uint32_t rescaled4(uint32_t w, float by) {
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    return codes4(lo[0] * by, lo[1] * by, hi[0] * by, hi[1] * by);
}

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x = fmaxf(x, __shfl_xor(x, d, kWave));
    return x;
}

// The scale of a block: the one its new tokens need, or the one it has; `by`: what the earlier tokens' codes change by.
__device__ __forceinline__ float joined_scale(float old, bool earlier, float top, float& by) {
    const float s = fmaxf(block_scale(top), old);
    by = earlier ? old / s : 1.f;
    return s;
}

// What a wave's unit reads, on its way before the angles are formed.  Keys: 16 bytes a lane, whole rows (lane l of load i:
// elements 8 (l % (D/8)) .. of token i * 512/D + l / (D/8)); values: E elements of each of the 16 tokens.
template <int D>
struct AppendRows {
    static constexpr int PER = D / 8, TOKENS = kWave / PER, LOADS = 16 / TOKENS;
    static constexpr int E = D == 256 ? 4 : 2;
    union {
        u32x4 key[LOADS];
        uint32_t value[16][E / 2];
    };

    __device__ __forceinline__ void load_keys(const Kv8AppendArgs& a, const Kv8Unit& w, int head) {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int j = i * TOKENS + lane / PER;
            const uint16_t* src = a.src[1] + (w.first + (j - w.from)) * a.stride[1] + head * D + (lane % PER) * 8;
            key[i] = j >= w.from && j < w.to ? *(const u32x4*)src : u32x4{0u, 0u, 0u, 0u};
        }
    }
    __device__ __forceinline__ void load_values(const Kv8AppendArgs& a, const Kv8Unit& w, int head) {
        const int d0 = (threadIdx.x & 63) * E;
        const uint16_t* src = a.src[2] + (w.first - w.from) * a.stride[2] + head * D + d0;
#pragma unroll
        for (int j = 0; j < 16; ++j)
#pragma unroll
            for (int e = 0; e < E / 2; ++e)
                value[j][e] = d0 < D && j >= w.from && j < w.to ? ((const uint32_t*)(src + j * a.stride[2]))[e] : 0u;
    }
};

template <int D>
__device__ __forceinline__ void append_keys(const Kv8AppendArgs& a, const Kv8Unit& w, int head, const AppendRows<D>& raw,
                                            const double2 (*turn)[D / 2], char* lds) {
    using Rows = AppendRows<D>;
    constexpr int L = Rows::LOADS;
    const int lane = threadIdx.x & 63, c = lane % Rows::PER, half = a.rot_dim / 2;
    const int64_t grp = w.group + (int64_t)head * (a.cache.page_size >> 4);
    float* const scale = a.cache.k_scales + grp;
    const float held_scale = w.from > 0 ? *scale : 0.f;
    float x[L][8], top = 0.f;
#pragma unroll
    for (int i = 0; i < L; ++i) {
        const int token = i * Rows::TOKENS + lane / Rows::PER;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[i][2 * e] = bf16_lo(raw.key[i][e]);
            x[i][2 * e + 1] = bf16_hi(raw.key[i][e]);
        }
        if (half > 0) {
            u32x4 other;  // the pairs' other elements (half a rotation away), in another lane of the token
            const int from = a.interleaved ? lane : (c * 8 < half ? lane + half / 8 : (c * 8 < 2 * half ? lane - half / 8 : lane));
#pragma unroll
            for (int e = 0; e < 4; ++e) other[e] = __shfl(raw.key[i][e], from, kWave);
            if (c * 8 < a.rot_dim && token >= w.from && token < w.to) turn8<Turns<true>>(x[i], other, c * 8, half, a.interleaved, turn[token]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, finite_size(x[i][e]));
    }
    float by;
    const float s = joined_scale(held_scale, w.from > 0, wave_max(top), by), inv = 1.f / s;
    // through LDS into the cache's order: pieces of 16 elements, 16 tokens each
#pragma unroll
    for (int i = 0; i < L; ++i) {
        const int j = i * Rows::TOKENS + lane / Rows::PER;
        u32x2 codes;
#pragma unroll
        for (int e = 0; e < 2; ++e)
            codes[e] = codes4(coded(x[i][4 * e], inv), coded(x[i][4 * e + 1], inv), coded(x[i][4 * e + 2], inv),
                              coded(x[i][4 * e + 3], inv));
        *(u32x2*)(lds + (c / 2) * 256 + j * 16 + (c & 1) * 8) = codes;
    }
    __builtin_amdgcn_wave_barrier();  // (the wave's own part of LDS)
    const int j = lane & 15;
    uint8_t* const to = a.cache.k_codes + grp * (16 * D) + lane * 16;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
        u32x4* const at = (u32x4*)(to + i * 1024);
        if (j >= w.from && j < w.to) {
            *at = *(const u32x4*)(lds + i * 1024 + lane * 16);
        } else if (by != 1.f && j < w.from) {
            u32x4 held = *at;
#pragma unroll
            for (int e = 0; e < 4; ++e) held[e] = rescaled4(held[e], by);
            *at = held;
        }
    }
    if (lane == 0) *scale = s;
}

template <int D>
__device__ __forceinline__ void append_values(const Kv8AppendArgs& a, const Kv8Unit& w, int head, const AppendRows<D>& rows) {
    constexpr int E = AppendRows<D>::E;  // elements of a lane, of all 16 tokens
    const int lane = threadIdx.x & 63, d0 = lane * E;
    const bool live = d0 < D;
    const int64_t grp = w.group + (int64_t)head * (a.cache.page_size >> 4);
    float* const scale = a.cache.v_scales + grp;
    const float held_scale = w.from > 0 ? *scale : 0.f;
    const uint32_t(&raw)[16][E / 2] = rows.value;
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j)
#pragma unroll
        for (int e = 0; e < E / 2; ++e)
            top = fmaxf(top, fmaxf(finite_size(bf16_lo(raw[j][e])), finite_size(bf16_hi(raw[j][e]))));
    float by;
    const float s = joined_scale(held_scale, w.from > 0, wave_max(top), by), inv = 1.f / s;
    const bool whole = w.from == 0 && w.to == 16;
    if (live) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            uint8_t* const at = a.cache.v_codes + grp * (16 * D) + (d0 + e) * 16;
            const auto value = [&](int j) { return (e & 1) ? bf16_hi(raw[j][e / 2]) : bf16_lo(raw[j][e / 2]); };
            u32x4 c;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                c[i] = codes4(coded(value(4 * i), inv), coded(value(4 * i + 1), inv), coded(value(4 * i + 2), inv),
                              coded(value(4 * i + 3), inv));
            if (whole) {
                *(u32x4*)at = c;
                continue;
            }
            if (by != 1.f) {  // the earlier tokens' codes at the new scale (what stands behind the new tokens stays)
                const u32x4 held = *(const u32x4*)at;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t r = rescaled4(held[i], by);
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                        if (4 * i + b < w.from) at[4 * i + b] = (uint8_t)(r >> (8 * b));
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    if (4 * i + b >= w.from && 4 * i + b < w.to) at[4 * i + b] = (uint8_t)(c[i] >> (8 * b));
        }
    }
    if (lane == 0) *scale = s;
}

// Blocks [0, units * parts): a block of 16 tokens, part by part of its heads' keys and then values, a wave each; then a
// block per token for its queries.
template <int D>
__device__ __forceinline__ void append_body(const Kv8AppendArgs& a, int64_t units, int parts) {
    __shared__ double2 turn[16][D / 2];  // cos, sin of the tokens' angles
    __shared__ __align__(16) char lds[kAppendWaves * 16 * D];
    const int half = a.rot_dim / 2, heads = a.cache.num_kv_heads;
    const int64_t id = grid_block();
    const int wave = threadIdx.x >> 6;
    if (id < units * parts) {
        const int64_t u = id / parts;
        const int part = (int)(id - u * parts);
        const bool keys = part * kAppendWaves < heads && half > 0;  // some wave has keys to turn
        // (frequencies first: loads return in order, and the angles need not wait for the rows)
        constexpr int kRuns = 4, kLong = 16 / kRuns, kEach = (kRuns * (D / 2) + kAppendThreads - 1) / kAppendThreads;
        float freq[kEach];
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int i = threadIdx.x + k * kAppendThreads;
            freq[k] = keys && i < kRuns * half ? a.inv_freq[i % half] : 0.f;
        }
        const Kv8Unit w = kv8_unit(a.cache, a.batch, u, true);
        if (w.group < 0) return;
        const int unit = part * kAppendWaves + wave;
        AppendRows<D> raw;
        if (unit < heads)
            raw.load_keys(a, w, unit);
        else if (unit < 2 * heads)
            raw.load_values(a, w, unit - heads);
        if (keys) {
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                const int i = threadIdx.x + k * kAppendThreads, run = i / half, f = i - run * half;
                const int j0 = max(w.from, run * kLong), j1 = min(w.to, run * kLong + kLong);
                if (i >= kRuns * half || j0 >= j1) continue;
                const double by = (double)freq[k] * kPerTurn;
                double sn, cs, s1 = 0., c1 = 1.;
                sincospi(2. * ((double)(w.block * 16 + j0) * by), &sn, &cs);
                if (j1 > j0 + 1) sincospi(2. * by, &s1, &c1);
                for (int j = j0; j < j1; ++j) {
                    turn[j][Turns<true>::place(f, half)] = make_double2(cs, sn);
                    const double c = cs * c1 - sn * s1;
                    sn = sn * c1 + cs * s1;
                    cs = c;
                }
            }
            __syncthreads();
        }
        if (unit < heads)
            append_keys<D>(a, w, unit, raw, turn, lds + wave * (16 * D));
        else if (unit < 2 * heads)
            append_values<D>(a, w, unit - heads, raw);
        return;
    }
    const int64_t t = id - units * parts;
    if (t >= a.batch.num_tokens || a.num_q_heads == 0) return;
    const int pos = kv8_position(a.cache, a.batch, t);
    const int rot = pos < 0 ? 0 : a.rot_dim;  // (a token that stands nowhere may hold anything, and keeps it)
    for (int i = threadIdx.x; i < rot / 2; i += kAppendThreads) {
        double sn, cs;
        sincospi(2. * ((double)pos * ((double)a.inv_freq[i] * kPerTurn)), &sn, &cs);
        turn[0][Turns<true>::place(i, half)] = make_double2(cs, sn);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < a.num_q_heads * (D / 8); c += kAppendThreads) {
        const int head = c / (D / 8), d0 = c % (D / 8) * 8;
        float v[8];
        load_rotated<Turns<true>>(a.src[0] + t * a.stride[0] + head * D, d0, rot, a.interleaved, turn[0], v);
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        *(u32x4*)(a.q_out + (t * a.num_q_heads + head) * D + d0) = o;
    }
}

#define PLE_KV8_KERNEL(D)                                                                                              \
    __global__ __launch_bounds__(kAppendThreads) void kv8_append_##D##_kernel(Kv8AppendArgs a, int64_t units, int parts) { \
        append_body<D>(a, units, parts);                                                                               \
    }
PLE_KV8_KERNEL(64)
PLE_KV8_KERNEL(128)
PLE_KV8_KERNEL(256)
#undef PLE_KV8_KERNEL

// Blocks of four waves for a block of 16 tokens: a wave a head's keys or values.
static int kv8_parts(const ple_kv8_cache& c) { return (2 * c.num_kv_heads + kAppendWaves - 1) / kAppendWaves; }

int64_t kv8_append_blocks(const ple_kv8_cache& cache, const ple_kv8_batch& batch, int32_t num_q_heads) {
    return kv8_units(batch, true) * kv8_parts(cache) + (num_q_heads > 0 ? batch.num_tokens : 0);
}
int64_t kv8_read_blocks(const ple_kv8_cache& cache, const ple_kv8_batch& batch) {
    return kv8_units(batch, false) * kv8_parts(cache);
}

hipError_t launch_kv8_append(const Kv8AppendArgs& a, hipStream_t s) {
    const int64_t units = kv8_units(a.batch, true);
    const int parts = kv8_parts(a.cache);
    const dim3 grid = block_grid(kv8_append_blocks(a.cache, a.batch, a.num_q_heads));
    if (a.cache.head_dim == 64)
        hipLaunchKernelGGL(kv8_append_64_kernel, grid, dim3(kAppendThreads), 0, s, a, units, parts);
    else if (a.cache.head_dim == 128)
        hipLaunchKernelGGL(kv8_append_128_kernel, grid, dim3(kAppendThreads), 0, s, a, units, parts);
    else
        hipLaunchKernelGGL(kv8_append_256_kernel, grid, dim3(kAppendThreads), 0, s, a, units, parts);
    return hipGetLastError();
}

struct Kv8ReadArgs {
    ple_kv8_cache cache;
    ple_kv8_batch batch;
    uint16_t *k_out, *v_out;
    int64_t units;
    int32_t parts;
};

__device__ __forceinline__ void unpack4(uint32_t w, float s, float (&v)[4]) {
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    v[0] = lo[0] * s;
    v[1] = lo[1] * s;
    v[2] = hi[0] * s;
    v[3] = hi[1] * s;
}

__device__ __forceinline__ void clear_row(const Kv8ReadArgs& a, int64_t t, int row) {
    for (int e = threadIdx.x * 8; e < row; e += kAppendThreads * 8)
        *(u32x4*)(a.k_out + t * row + e) = *(u32x4*)(a.v_out + t * row + e) = u32x4{0u, 0u, 0u, 0u};
}

// A block of 16 tokens, a wave a head's keys or values, as append; tokens that stand on no page are zeros.
template <int D>
__device__ __forceinline__ void read_body(const Kv8ReadArgs& a) {
    const int64_t id = grid_block();
    if (id >= a.units * a.parts) return;
    const int64_t u = id / a.parts;
    const int lane = threadIdx.x & 63, heads = a.cache.num_kv_heads;
    const int unit = (int)(id - u * a.parts) * kAppendWaves + (threadIdx.x >> 6);
    const Kv8Unit w = kv8_unit(a.cache, a.batch, u, false);
    if (id - u * a.parts == 0) {  // tokens that stand on no place: of no request, here by the launch's units in turn, and of this one
        const int64_t T = a.batch.num_tokens, first = min(max((int64_t)a.batch.query_start_loc[0], (int64_t)0), T);
        const int64_t last = min(max((int64_t)a.batch.query_start_loc[a.batch.num_reqs], first), T);
        for (int64_t i = u; i < first + (T - last); i += a.units) clear_row(a, i < first ? i : last + (i - first), heads * D);
        if (w.index == 0) {
            for (int64_t i = 0; i < w.lo; ++i) clear_row(a, w.q0 + i, heads * D);
            for (int64_t i = w.hi; i < w.n; ++i) clear_row(a, w.q0 + i, heads * D);
        }
    }
    if (!w.any || unit >= 2 * heads) return;
    const int head = unit < heads ? unit : unit - heads;
    const int64_t grp = w.group + (int64_t)head * (a.cache.page_size >> 4), tokens = (int64_t)heads * D;
    if (unit < heads) {
        const int j = lane & 15;
        if (j < w.from || j >= w.to) return;
        uint16_t* const out = a.k_out + (w.first + (j - w.from)) * tokens + head * D + (lane >> 4) * 16;
        const float s = w.group < 0 ? 0.f : a.cache.k_scales[grp];
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
            u32x4 o[2] = {u32x4{0u, 0u, 0u, 0u}, u32x4{0u, 0u, 0u, 0u}};
            if (w.group >= 0) {
                const u32x4 c = *(const u32x4*)(a.cache.k_codes + grp * (16 * D) + i * 1024 + lane * 16);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float v[4];
                    unpack4(c[e], s, v);
                    o[e / 2][(e & 1) * 2] = pack_bf16x2(v[0], v[1]);
                    o[e / 2][(e & 1) * 2 + 1] = pack_bf16x2(v[2], v[3]);
                }
            }
            *(u32x4*)(out + i * 64) = o[0];
            *(u32x4*)(out + i * 64 + 8) = o[1];
        }
        return;
    }
    constexpr int E = D == 256 ? 4 : 2;
    const int d0 = lane * E;
    if (d0 >= D) return;
    const float s = w.group < 0 ? 0.f : a.cache.v_scales[grp];
    u32x4 c[E];
#pragma unroll
    for (int e = 0; e < E; ++e)
        c[e] = w.group < 0 ? u32x4{0u, 0u, 0u, 0u} : *(const u32x4*)(a.cache.v_codes + grp * (16 * D) + (d0 + e) * 16);
    uint16_t* const out = a.v_out + (w.first - w.from) * tokens + head * D + d0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float v[E][4];
#pragma unroll
        for (int e = 0; e < E; ++e) unpack4(c[e][i], s, v[e]);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int j = 4 * i + b;
            if (j < w.from || j >= w.to) continue;
#pragma unroll
            for (int e = 0; e < E; e += 2) ((uint32_t*)(out + j * tokens))[e / 2] = pack_bf16x2(v[e][b], v[e + 1][b]);
        }
    }
}

#define PLE_KV8_KERNEL(D) \
    __global__ __launch_bounds__(kAppendThreads) void kv8_read_##D##_kernel(Kv8ReadArgs a) { read_body<D>(a); }
PLE_KV8_KERNEL(64)
PLE_KV8_KERNEL(128)
PLE_KV8_KERNEL(256)
#undef PLE_KV8_KERNEL

hipError_t launch_kv8_read(const ple_kv8_cache& cache, const ple_kv8_batch& batch, uint16_t* k_out, uint16_t* v_out,
                           hipStream_t s) {
    const Kv8ReadArgs a = {cache, batch, k_out, v_out, kv8_units(batch, false), kv8_parts(cache)};
    const dim3 grid = block_grid(kv8_read_blocks(cache, batch));
    if (cache.head_dim == 64)
        hipLaunchKernelGGL(kv8_read_64_kernel, grid, dim3(kAppendThreads), 0, s, a);
    else if (cache.head_dim == 128)
        hipLaunchKernelGGL(kv8_read_128_kernel, grid, dim3(kAppendThreads), 0, s, a);
    else
        hipLaunchKernelGGL(kv8_read_256_kernel, grid, dim3(kAppendThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace ple
