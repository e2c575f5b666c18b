// The position rotation of keys and queries on their way into a cache.
#pragma once

#include "ple_fp4_launch.h"

namespace ple {

__device__ __forceinline__ void load8(const uint16_t* __restrict__ p, float (&v)[8]) {
    const u32x4 w = *(const u32x4*)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
    }
}

// Where angle f of a token's `half` (a multiple of 8) stands in LDS: spread, so that lanes that turn neighbouring eights of a
// head read neighbouring places, or in order, where a lane's reads are one address and the next ones (a block per token, which
// spends more on forming places than it saves: 4 bits, 7984 tokens, 42.6 us in order, 45.6 spread).
template <bool SPREAD>
struct Turns {
    static __device__ __forceinline__ int place(int f, int half) { return SPREAD ? (f & 7) * (half >> 3) + (f >> 3) : f; }
    // from an angle to the next one of the same eight, or four
    static __device__ __forceinline__ int step(int half) { return SPREAD ? half >> 3 : 1; }
};

// Elements d0 .. d0 + 7 of a head's row (v, inside its first 2 half), turned by the token's angles (turn[At::place(i)]:
// cosine and sine of angle i); other: the row's elements half a rotation away, if pairs are not neighbours.  In 64 bits and rounded once to
// fp32, so that an element next to a code's border falls on the side that the definition says.
template <class At>
__device__ __forceinline__ void turn8(float (&v)[8], u32x4 other, int d0, int half, bool interleaved, const double2* turn) {
    const int step = At::step(half);
    if (interleaved) {
        turn += At::place(d0 / 2, half);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const double2 w = turn[i * step];
            const double x = v[2 * i], y = v[2 * i + 1];
            v[2 * i] = (float)(x * w.x - y * w.y);
            v[2 * i + 1] = (float)(y * w.x + x * w.y);
        }
    } else {
        const bool upper = d0 >= half;  // half is a multiple of 8
        turn += At::place(upper ? d0 - half : d0, half);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const double2 w = turn[i * step];
            const double x = v[i], y = i % 2 ? bf16_hi(other[i / 2]) : bf16_lo(other[i / 2]);
            v[i] = (float)(upper ? x * w.x + y * w.y : x * w.x - y * w.y);
        }
    }
}

// Elements d0 .. d0 + 7 of a head's row in memory, turned where they lie in its first rot_dim.
template <class At>
__device__ __forceinline__ void load_rotated(const uint16_t* __restrict__ src, int d0, int rot_dim, bool interleaved,
                                             const double2* turn, float (&v)[8]) {
    load8(src + d0, v);
    if (d0 >= rot_dim) return;
    const int half = rot_dim / 2;
    u32x4 other = {0u, 0u, 0u, 0u};
    if (!interleaved) other = *(const u32x4*)(src + (d0 >= half ? d0 - half : d0 + half));
    turn8<At>(v, other, d0, half, interleaved, turn);
}

}  // namespace ple
