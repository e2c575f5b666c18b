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

// Elements d0 .. d0 + 7 of a head's row, turned by the token's angles (turn[i]: cosine and sine of angle i) where they lie
// in its first rot_dim.  In 64 bits and rounded once to fp32, so that an element next to a code's border falls on the side
// that the definition says.
__device__ __forceinline__ void load_rotated(const uint16_t* __restrict__ src, int d0, int rot_dim, bool interleaved,
                                             const double2* turn, float (&v)[8]) {
    load8(src + d0, v);
    if (d0 >= rot_dim) return;
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const double2 w = turn[d0 / 2 + i];
            const double x = v[2 * i], y = v[2 * i + 1];
            v[2 * i] = (float)(x * w.x - y * w.y);
            v[2 * i + 1] = (float)(y * w.x + x * w.y);
        }
    } else {
        const int half = rot_dim / 2;
        const bool upper = d0 >= half;  // half is a multiple of 8
        float o[8];
        load8(src + (upper ? d0 - half : d0 + half), o);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const double2 w = turn[(upper ? d0 - half : d0) + i];
            const double x = v[i], y = o[i];
            v[i] = (float)(upper ? x * w.x + y * w.y : x * w.x - y * w.y);
        }
    }
}

}  // namespace ple
