// Products of 8-bit integers: out = (x W^T) scaled by token and by output
// channel, sums exact in 32-bit integers.
//
// Integer MFMAs take 16 bytes of K per lane, so a row of either operand is
// read as it lies.  Three kinds of kernels, chosen in w8_linear_shape:
//  - few tokens (decode): bound by reading the weights once, and below that
//    by the latency of the rounds of loads.  A block's eight waves share its
//    features and split K between them in steps; a step's rows come straight
//    into LDS, whole rows of 128 or 256 bytes at a time, and the waves' sums
//    are joined through LDS: no second launch and no atomics.
//  - tiles of four waves for all in between, bound by the weights while 64 x
//    64 tiles do (1 token, 4096 -> 8192: 8.6 us, 3.9 TB/s; 128 tokens 9.5;
//    256 tokens 2048 -> 4096 7.2), then by LDS and the products.
//  - 256 x 256 tiles of eight waves, the pipeline of the bf16 projection
//    (ple_kv_proj.hip) on 16x16x64 products, where there are many: bound by
//    the products (8192 tokens 4096 -> 8192: 219 us, 2.5 PFLOP/s, 50% of the
//    dense peak; the library's product into 32-bit sums 238).
#include "ple_8bit_launch.h"

namespace ple {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ i32x16 mfma32(u32x4 b, u32x4 a, i32x16 c) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, b), __builtin_bit_cast(i32x4, a), c, 0, 0, 0);
}
__device__ __forceinline__ i32x4 mfma16(u32x4 b, u32x4 a, i32x4 c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, b), __builtin_bit_cast(i32x4, a), c, 0, 0, 0);
}
// Four features of a token (those past the end take the last one's scales; they are not stored).
__device__ __forceinline__ u32x2 out4(const W8Args& a, int m, int o, int v0, int v1, int v2, int v3) {
    const float s = a.x_scales[min(m, a.M - 1)];
    const float* w = a.w_scales;
    const int last = a.O - 1;
    return u32x2{pack_bf16x2((float)v0 * w[min(o, last)] * s, (float)v1 * w[min(o + 1, last)] * s),
                 pack_bf16x2((float)v2 * w[min(o + 2, last)] * s, (float)v3 * w[min(o + 3, last)] * s)};
}

// Tile order: XCD-major then grouped row-major (GROUP_M tile rows share W panels).
template <int GROUP_M>
__device__ __forceinline__ void tile_of_block(int bid, int tiles_m, int tiles_n, int& tm, int& tn) {
    const int total = tiles_m * tiles_n;
    // Blocks are dealt to the 8 XCDs round-robin; give each XCD a contiguous
    // range of tiles (when the count divides evenly).
    int lin = bid;
    if ((total & 7) == 0) {
        const int per = total >> 3;
        lin = (bid & 7) * per + (bid >> 3);
    }
    const int group = lin / (GROUP_M * tiles_n);
    const int first_m = group * GROUP_M;
    const int gm = min(tiles_m - first_m, GROUP_M);
    const int in_group = lin - group * GROUP_M * tiles_n;
    tm = first_m + in_group % gm;
    tn = in_group / gm;
}

constexpr int kSliceBytes = 128;  // of K
typedef __attribute__((address_space(3))) void* lds_ptr_t;

// The operands' rows in bytes.
struct W8Rows {
    int k, x, slices, tail;  // bytes of K and from one row of x to the next; slices; K's bytes in the last one if not all
    __device__ __forceinline__ explicit W8Rows(const W8Args& a)
        : k(a.K), x(a.x_stride), slices((k + kSliceBytes - 1) / kSliceBytes), tail(k % kSliceBytes) {}
    __device__ __forceinline__ int x_bytes(int n) const { return (n - 1) * x + k; }
};

// A block's BM x BN outputs out of LDS.
template <int BM, int BN, int THREADS>
__device__ __forceinline__ void pipe_store(const uint16_t* Cs, const W8Args& a, int m0, int n0) {
    const int M = a.M, O = a.O;
    const bool whole = O % 8 == 0;  // rows of `out` begin at 16 bytes
#pragma unroll 4
    for (int c = threadIdx.x; c < BM * BN / 8; c += THREADS) {
        const int row = c / (BN / 8);  // BN/8 chunks of 8 features per row
        const int col = (c % (BN / 8)) * 8;
        const int gr = m0 + row, gc = n0 + col;
        if (gr >= M || gc >= O) continue;
        if (whole) {
            *(u32x4*)(a.out + (int64_t)gr * O + gc) = *(const u32x4*)(Cs + row * (BN + 8) + col);
        } else {
            for (int e = 0; e < 8 && gc + e < O; ++e) a.out[(int64_t)gr * O + gc + e] = Cs[row * (BN + 8) + col + e];
        }
    }
}

// ---------------------------------------------------------------------------
// Tiles of 64 MB tokens x 64 NB features, four waves (one per SIMD) of 32 MB x
// 32 NB in 32x32x32 products.  K's slices of 128 go round a ring of NS in LDS.
// A slice's fragments are read as a whole while the last one's products run,
// so a slice costs one barrier and the reads' latency is behind the products;
// NS slices are on their way from memory.  128 tokens 4096 -> 8192 in 64 x 64
// tiles: 9.5 us (3.7 TB/s); reading each 32 of K for itself before its product
// 18.5, eight waves that share K 9.9.  512 tokens in 128 x 128 tiles: 20.6 us,
// 1.67 PFLOP/s, about 1400 cycles a slice where its products take 512 and LDS
// is busy for 770 (64 fragment reads and 32 KiB of copies).
//
// Operands go global -> LDS with buffer loads that write LDS directly: a
// scalar buffer resource per operand panel and a 32-bit per-lane offset.  Each
// copy instruction fills 1 KiB = 8 whole rows of the slice, so every request
// is a full cache line.  Row r holds 8 chunks of 16 bytes, chunk c at place
// c ^ ((r >> 1) & 7): a fragment read takes one chunk of 32 consecutive rows,
// and any 16 of them touch distinct banks.  W's fragment is the first operand,
// so each lane's sums are 4 consecutive features of one token.
//
// The LDS reads are inline assembly with explicit waits (the compiler's own
// would wait for the copies too); a wait names the registers it covers, so no
// product reading them can be scheduled above it.  The loop has no branch
// between a read and its wait but those that leave the fragments alone, so
// that nothing copies a register on its way: slices past the last one are gone
// through with x as zeros, and their copies are out of the buffer's range.
// ---------------------------------------------------------------------------
template <int MB, int NB, int NS>
struct W8Tile {
    static constexpr int BM = 64 * MB, BN = 64 * NB;
    static constexpr int X_BYTES = BM * kSliceBytes, STAGE = X_BYTES + BN * kSliceBytes;
    static constexpr int COPIES = 2 * MB + 2 * NB;  // of a wave and slice
    static constexpr int FRAGS = 4 * (MB + NB);     // of a wave and slice: x blocks, then W blocks of each 32 of K
    static constexpr int OUT = BM * (BN + 8) * 2;
    static constexpr int LDS = NS * STAGE > OUT ? NS * STAGE : OUT;
    static_assert(NS >= 2 && (NS - 1) * COPIES <= 63, "the slices on their way must fit the wait's counter");
    static_assert(LDS <= 160 * 1024, "more LDS than a CU has");
};

constexpr int kTileThreads = 256;

template <int OFFSET>
__device__ __forceinline__ void read_lds(u32x4& f, uint32_t at) {
    asm volatile("ds_read_b128 %0, %1 offset:%2" : "=v"(f) : "v"(at), "i"(OFFSET));
}
#define PLE_W8_REGS4(f, i) "+v"(f[i]), "+v"(f[i + 1]), "+v"(f[i + 2]), "+v"(f[i + 3])
// Names further fragments to a wait before it.
template <int N>
__device__ __forceinline__ void name_frags(u32x4 (&f)[N]) {
    if constexpr (N == 12) asm volatile("" : PLE_W8_REGS4(f, 8));
    if constexpr (N >= 16) asm volatile("" : PLE_W8_REGS4(f, 8), PLE_W8_REGS4(f, 12));
    if constexpr (N == 24) asm volatile("" : PLE_W8_REGS4(f, 16), PLE_W8_REGS4(f, 20));
    static_assert(N == 8 || N == 12 || N == 16 || N == 24, "fragments without a wait");
}
// Waits for these fragments and all copies but the newest V, then for the block's other waves.
template <int V, int N>
__device__ __forceinline__ void wait_slice(u32x4 (&f)[N]) {
    asm volatile("s_waitcnt vmcnt(%8) lgkmcnt(0)\n\ts_barrier" : PLE_W8_REGS4(f, 0), PLE_W8_REGS4(f, 4) : "i"(V) : "memory");
    name_frags(f);
}

template <int MB, int NB, int NS>
__device__ __forceinline__ void w8_tile(const W8Args& a) {
    using Sh = W8Tile<MB, NB, NS>;
    constexpr int BM = Sh::BM, BN = Sh::BN, N = Sh::FRAGS;
    extern __shared__ __align__(16) char lds_raw[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave >> 1, wn = wave & 1;  // 2 x 2 waves
    const int M = a.M, O = a.O;
    const W8Rows rows(a);
    int tm, tn;
    tile_of_block<8>(blockIdx.x, (M + BM - 1) / BM, (O + BN - 1) / BN, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;

    // Copy instruction i of a wave fills rows 8 (4 i + wave) .. + 7 of an operand's slice; rows past the end of x or W read
    // the last row (their outputs are never stored).
    const int x_bytes = rows.x_bytes(min(M - m0, BM)), w_bytes = min(O - n0, BN) * rows.k;
    void* const x0 = (void*)((const char*)a.x + (int64_t)m0 * rows.x);
    void* const w0 = (void*)((const char*)a.w + (int64_t)n0 * rows.k);
    uint32_t xoff[2 * MB], woff[2 * NB];
#pragma unroll
    for (int i = 0; i < 2 * MB || i < 2 * NB; ++i) {
        const int row = (i * 4 + wave) * 8 + (lane >> 3);
        const int kc = (lane & 7) ^ ((row >> 1) & 7);
        if (i < 2 * MB) xoff[i] = (uint32_t)(min(row, M - 1 - m0) * rows.x + kc * 16);
        if (i < 2 * NB) woff[i] = (uint32_t)(min(row, O - 1 - n0) * rows.k + kc * 16);
    }
    const int nk = rows.slices;
    // copy instruction c of slice s into a stage of the ring; slices past the last one copy nothing
    auto copy_one = [&](int s, int stage, int c) {
        char* base = lds_raw + stage * Sh::STAGE;
        const bool in = s < nk;
        const __amdgpu_buffer_rsrc_t r = c < 2 * MB ? __builtin_amdgcn_make_buffer_rsrc(x0, (short)0, in ? x_bytes : 0, 0x00020000)
                                                    : __builtin_amdgcn_make_buffer_rsrc(w0, (short)0, in ? w_bytes : 0, 0x00020000);
        const int i = c < 2 * MB ? c : c - 2 * MB;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)(base + (c < 2 * MB ? 0 : Sh::X_BYTES) + (i * 4 + wave) * 1024), 16,
                                                 c < 2 * MB ? xoff[i < 2 * MB ? i : 0] : woff[i < 2 * NB ? i : 0],
                                                 in ? s * kSliceBytes : 0, 0, 0);
    };

    i32x16 acc[NB][MB];
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[j][i][e] = 0;

    const int frow = lane & 31, fk = lane >> 5;
    uint32_t x_at[4], w_at[4];  // of the lane's chunk for step kk in stage 0, first 32-row block (the others 4 KiB on each)
    const uint32_t lds_base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds_raw;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
        const uint32_t col = (uint32_t)(((kk * 2 + fk) ^ ((frow >> 1) & 7)) * 16);
        x_at[kk] = lds_base + (wm * (32 * MB) + frow) * kSliceBytes + col;
        w_at[kk] = lds_base + Sh::X_BYTES + (wn * (32 * NB) + frow) * kSliceBytes + col;
    }
    // fragment q of a slice: step q / (MB + NB); x blocks, then W blocks
    auto read_one = [&](int q, uint32_t stage, u32x4 (&f)[N]) {
        const int kk = q / (MB + NB), b = q % (MB + NB);
        const uint32_t at = (b < MB ? x_at[kk] : w_at[kk]) + stage;
        switch (b < MB ? b : b - MB) {
            case 0: read_lds<0>(f[q], at); break;
            case 1: read_lds<4096>(f[q], at); break;
            case 2: read_lds<8192>(f[q], at); break;
            default: read_lds<12288>(f[q], at); break;
        }
    };
    // Slice s: cur's products; between them the reads of the next slice into nxt, and the copies of the NS-th after this one
    // into the stage that this one has left.
    auto slice = [&](int s, int stage, int next, u32x4 (&cur)[N], u32x4 (&nxt)[N]) {
        __builtin_amdgcn_sched_barrier(0);
        wait_slice<(NS - 2) * Sh::COPIES>(cur);
        __builtin_amdgcn_sched_barrier(0);
        if ((s + 1) * kSliceBytes > a.K) {  // past K x is zero (W holds the next row's there, the ring anything)
#pragma unroll
            for (int q = 0; q < N; ++q)
                if (q % (MB + NB) < MB)
                    cur[q] &= s * kSliceBytes + (q / (MB + NB) * 2 + fk) * 16 < a.K ? 0xFFFFFFFFu : 0u;
        }
        constexpr int P = 4 * MB * NB;          // products
        constexpr int R = P >= 4 ? P * 3 / 4 : P;  // the reads go behind the first of them, the copies behind all
#pragma unroll
        for (int t = 0; t < P; ++t) {
            const int kk = t / (MB * NB), j = t % (MB * NB) / MB, i = t % MB, at = kk * (MB + NB);
            acc[j][i] = mfma32(cur[at + MB + j], cur[at + i], acc[j][i]);
#pragma unroll
            for (int q = t * N / R; q < (t + 1) * N / R && q < N; ++q) read_one(q, (uint32_t)(next * Sh::STAGE), nxt);
#pragma unroll
            for (int c = t * Sh::COPIES / P; c < (t + 1) * Sh::COPIES / P; ++c) copy_one(s + NS, stage, c);
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    u32x4 f0[N], f1[N];
#pragma unroll
    for (int k = 0; k < NS; ++k)
#pragma unroll
        for (int c = 0; c < Sh::COPIES; ++c) copy_one(k, k, c);
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" : : "i"((NS - 1) * Sh::COPIES) : "memory");
#pragma unroll
    for (int q = 0; q < N; ++q) read_one(q, 0u, f0);
    int stage = 0;
    for (int s = 0; s < nk; s += 2) {
        const int s1 = stage + 1 == NS ? 0 : stage + 1, s2 = s1 + 1 == NS ? 0 : s1 + 1;
        slice(s, stage, s1, f0, f1);
        slice(s + 1, s1, s2, f1, f0);
        stage = s2;
    }
    // the last look-ahead reads (of a stage that holds anything) have landed before their registers are used again
    wait_slice<0>(f0);

    // acc[j][i][e] is feature n0 + wn*32*NB + j*32 + 8*(e/4) + 4*(lane/32) + e%4 of token m0 + wm*32*MB + i*32 + lane%32
    uint16_t* Cs = (uint16_t*)lds_raw;
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int m = wm * (32 * MB) + i * 32 + frow;
                const int o = wn * (32 * NB) + j * 32 + 8 * g + 4 * fk;
                *(u32x2*)(Cs + m * (BN + 8) + o) = out4(a, m0 + m, n0 + o, acc[j][i][4 * g], acc[j][i][4 * g + 1],
                                                        acc[j][i][4 * g + 2], acc[j][i][4 * g + 3]);
            }
    __syncthreads();
    pipe_store<BM, BN, kTileThreads>(Cs, a, m0, n0);
}

// ---------------------------------------------------------------------------
// 256-wide tiles with eight waves (two per SIMD) on 16x16x64 MFMAs: wave
// (wm, wn) holds a 128 x 64 block (x rows wm*128.., W rows wn*64..) as 8 x 4
// accumulator tiles of 16 x 16 (128 accumulation registers), so a wave
// waiting on its fragments leaves the matrix core to the other wave of its
// SIMD.  Row layout in LDS and the copy instructions as the four-wave body; a
// slice is two K-steps of 64 with 12 fragment reads each.  Instead of two
// stages of both operands, the LDS holds a ring of five operand slices, which
// gives the W copies a second slice of lead.  The tiles an XCD runs at once
// are grouped four tile rows by eight tile columns, so each W panel is shared
// by four blocks in that XCD's L2 and each x panel by eight: more of the W
// copies wait on the last-level cache.
// ---------------------------------------------------------------------------
constexpr int kWideThreads = 512;
// five operand-slice slots (160 KiB, all of the LDS), which also hold the epilogue's rows
constexpr int kWideSlot = 256 * kSliceBytes, kWideLdsBytes = 5 * kWideSlot;
static_assert(kWideLdsBytes >= 256 * (256 + 8) * 2, "the epilogue's rows fit in the ring");
struct W8WideFrag {
    u32x4 a[8], b[4];
};
#define PLE_W8_WIDE_FRAG_REGS(f)                                                                                       \
    "+v"(f.a[0]), "+v"(f.a[1]), "+v"(f.a[2]), "+v"(f.a[3]), "+v"(f.a[4]), "+v"(f.a[5]), "+v"(f.a[6]), "+v"(f.a[7]), \
        "+v"(f.b[0]), "+v"(f.b[1]), "+v"(f.b[2]), "+v"(f.b[3])

__device__ __forceinline__ void w8_pipe8w(const W8Args& a) {
    constexpr int BT = 256, NC = 4;  // copy instructions per operand, wave and slice
    extern __shared__ __align__(16) char lds_raw[];
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    const int M = a.M, O = a.O;
    const W8Rows rows(a);
    const int tiles_m = (M + BT - 1) / BT;
    const int tiles_n = (O + BT - 1) / BT;
    int tm, tn;
    tile_of_block<4>(blockIdx.x, tiles_m, tiles_n, tm, tn);
    const int m0 = tm * BT, n0 = tn * BT;
    const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(
        (void*)((const char*)a.x + (int64_t)m0 * rows.x), (short)0, rows.x_bytes(min(M - m0, BT)), 0x00020000);
    const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
        (void*)((const char*)a.w + (int64_t)n0 * rows.k), (short)0, min(O - n0, BT) * rows.k, 0x00020000);
    // copy instruction i of wave `wave` fills rows g*8 .. g*8+7, g = i*8 + wave
    uint32_t aoff[NC], boff[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int row = (i * 8 + wave) * 8 + (lane >> 3);
        const int kc = (lane & 7) ^ ((row >> 1) & 7);
        aoff[i] = (uint32_t)((min(m0 + row, M - 1) - m0) * rows.x + kc * 16);
        boff[i] = (uint32_t)((min(n0 + row, O - 1) - n0) * rows.k + kc * 16);
    }
    const int nk = rows.slices;
    // Operand ring: W slice k in slot k mod 3, x slice k in slot 3 + k mod 2
    // (slots of one operand slice, 32 KiB).  W slices are copied two slices
    // ahead of their use and x slices one ahead, each into the slot its
    // operand's slice three (W) or two (x) back has just left.
    auto copy_x = [&](int k, int i) {  // k uniform
        char* base = lds_raw + (3 + (k & 1)) * kWideSlot + (i * 8 + wave) * 1024;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_ptr_t)base, 16, aoff[i], min(k, nk - 1) * kSliceBytes, 0, 0);
    };
    auto copy_w = [&](int k, int i) {
        char* base = lds_raw + (k % 3) * kWideSlot + (i * 8 + wave) * 1024;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_ptr_t)base, 16, boff[i], min(k, nk - 1) * kSliceBytes, 0, 0);
    };

    i32x4 acc[4][8];  // [W block jb][x block ib]
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[j][i] = i32x4{0, 0, 0, 0};

    const int frow = lane & 15;
    const int fk = lane >> 4;
    const int sw = (frow >> 1) & 7;
    uint32_t a_addr[2], b_addr[2];
    const uint32_t lds_base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds_raw;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
        const uint32_t col = (uint32_t)(((ks * 4 + fk) ^ sw) * 16);
        a_addr[ks] = lds_base + (wm * 128 + frow) * 128 + col;
        b_addr[ks] = lds_base + (wn * 64 + frow) * 128 + col;
    }
    auto read_one = [&](int q, int kt, int ks, W8WideFrag& f) {
        const uint32_t pa = a_addr[ks] + (uint32_t)(3 + (kt & 1)) * kWideSlot;
        const uint32_t pb = b_addr[ks] + (uint32_t)(kt % 3) * kWideSlot;
        switch (q) {
            case 0: asm volatile("ds_read_b128 %0, %1" : "=v"(f.a[0]) : "v"(pa)); break;
            case 1: asm volatile("ds_read_b128 %0, %1 offset:2048" : "=v"(f.a[1]) : "v"(pa)); break;
            case 2: asm volatile("ds_read_b128 %0, %1 offset:4096" : "=v"(f.a[2]) : "v"(pa)); break;
            case 3: asm volatile("ds_read_b128 %0, %1 offset:6144" : "=v"(f.a[3]) : "v"(pa)); break;
            case 4: asm volatile("ds_read_b128 %0, %1 offset:8192" : "=v"(f.a[4]) : "v"(pa)); break;
            case 5: asm volatile("ds_read_b128 %0, %1 offset:10240" : "=v"(f.a[5]) : "v"(pa)); break;
            case 6: asm volatile("ds_read_b128 %0, %1 offset:12288" : "=v"(f.a[6]) : "v"(pa)); break;
            case 7: asm volatile("ds_read_b128 %0, %1 offset:14336" : "=v"(f.a[7]) : "v"(pa)); break;
            case 8: asm volatile("ds_read_b128 %0, %1" : "=v"(f.b[0]) : "v"(pb)); break;
            case 9: asm volatile("ds_read_b128 %0, %1 offset:2048" : "=v"(f.b[1]) : "v"(pb)); break;
            case 10: asm volatile("ds_read_b128 %0, %1 offset:4096" : "=v"(f.b[2]) : "v"(pb)); break;
            default: asm volatile("ds_read_b128 %0, %1 offset:6144" : "=v"(f.b[3]) : "v"(pb)); break;
        }
    };
    auto wait_frag = [&](W8WideFrag& f) { asm volatile("s_waitcnt lgkmcnt(0)" : PLE_W8_WIDE_FRAG_REGS(f)); };
    // the wait leaves the NC copies of the newest W slice in flight (copies
    // complete in issue order, so every older one has landed)
    auto wait_barrier = [&](W8WideFrag& f) {
        asm volatile("s_waitcnt vmcnt(%12) lgkmcnt(0)\n\ts_barrier" : PLE_W8_WIDE_FRAG_REGS(f) : "i"(NC) : "memory");
    };
    // one K-step of 64: 32 MFMAs on cur; after MFMA t < 12, fragment read t of
    // (rkt, rks) into nxt; with ckt >= 0, the NC copies of x slice ckt after
    // MFMAs 2 and 10, then those of W slice ckt + 1 after MFMAs 18 and 26
    auto kstep = [&](const W8WideFrag& cur, W8WideFrag& nxt, int rkt, int rks, int ckt) {
#pragma unroll
        for (int t = 0; t < 32; ++t) {
            const int j = t / 8, i = t % 8;
            acc[j][i] = mfma16(cur.b[j], cur.a[i], acc[j][i]);
            if (t < 12) read_one(t, rkt, rks, nxt);
            if (ckt >= 0 && t % 8 == 2) {
                if (t < 16) {
                    copy_x(ckt, 2 * (t / 8));
                    copy_x(ckt, 2 * (t / 8) + 1);
                } else {
                    copy_w(ckt + 1, 2 * (t / 8) - 4);
                    copy_w(ckt + 1, 2 * (t / 8) - 3);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    W8WideFrag f0, f1;
    // x0, W0, x1, W1, W2; slice 0 landed before the first reads
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int i = 0; i < NC; ++i) copy_x(k, i);
#pragma unroll
        for (int i = 0; i < NC; ++i) copy_w(k, i);
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) copy_w(2, i);
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "i"(3 * NC) : "memory");
#pragma unroll
    for (int q = 0; q < 12; ++q) read_one(q, 0, 0, f0);
    auto trim = [&](W8WideFrag& f, int kt, int ks) {  // as for the four waves
        if (kt == nk - 1 && rows.tail != 0) {
            const uint32_t keep = (ks * 4 + fk) * 16 < rows.tail ? 0xFFFFFFFFu : 0u;
#pragma unroll
            for (int i = 0; i < 8; ++i) f.a[i] &= keep;
        }
    };
    for (int kt = 0; kt < nk; ++kt) {
        wait_frag(f0);
        trim(f0, kt, 0);
        kstep(f0, f1, kt, 1, -1);
        __builtin_amdgcn_sched_barrier(0);
        wait_barrier(f1);  // slice kt+1 has landed; every read of slice kt is done
        __builtin_amdgcn_sched_barrier(0);
        trim(f1, kt, 1);
        kstep(f1, f0, kt + 1, 0, kt + 2);
    }
    // the last look-ahead reads into f0 land before its registers are reused
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" : PLE_W8_WIDE_FRAG_REGS(f0) : : "memory");
    __syncthreads();

    // acc[jb][ib][e]: feature n0 + wn*64 + jb*16 + 4*fk + e of token m0 + wm*128 + ib*16 + frow
    uint16_t* Cs = (uint16_t*)lds_raw;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int m = wm * 128 + i * 16 + frow;
            const int o = wn * 64 + j * 16 + 4 * fk;
            *(u32x2*)(Cs + m * (256 + 8) + o) =
                out4(a, m0 + m, n0 + o, acc[j][i][0], acc[j][i][1], acc[j][i][2], acc[j][i][3]);
        }
    __syncthreads();
    pipe_store<BT, BT, kWideThreads>(Cs, a, m0, n0);
}
#undef PLE_W8_WIDE_FRAG_REGS

#undef PLE_W8_REGS4

__global__ __launch_bounds__(kWideThreads, 1) void w8_gemm_256_kernel(W8Args a) { w8_pipe8w(a); }
// Tiles of four waves: 64-token blocks, 64-feature blocks, slices in LDS, what 256 of them (one per CU) take against
// others' (half us with 4096 inputs: 7.0, 11.6, 19 and 32.5 us beyond a launch; of the eight-wave kernel 54).
#define PLE_W8_TILES(X) X(1, 1, 4, 14) X(2, 1, 6, 23) X(2, 2, 4, 38) X(4, 2, 3, 65)
constexpr int kWideCost = 106;
#define PLE_W8_KERNEL(MB, NB, NS, COST)                                                                                        \
    __global__ __launch_bounds__(kTileThreads, 1) void w8_tile_##MB##x##NB##_kernel(W8Args a) { w8_tile<MB, NB, NS>(a); }
PLE_W8_TILES(PLE_W8_KERNEL)
#undef PLE_W8_KERNEL

// The few-token kernel's LDS: a step's inputs and weights of every wave, then the joined sums.  ROWS: rows of x it has room
// for (16 a token tile), STEP: bytes of K.
constexpr int kRowsWaves = 8;
template <int ROWS, int NT, int STEP>
struct W8RowsShape {
    static_assert(ROWS % 16 == 0, "whole token tiles");
    static constexpr int MT = ROWS / 16;
    static constexpr int X = ROWS * STEP;                 // bytes of a wave's inputs
    static constexpr int ALL = X + NT * 16 * STEP;        // and weights
    static constexpr int JOIN = 4;                        // waves whose sums are in LDS at once
    static constexpr int LDS = kRowsWaves * ALL > JOIN * MT * NT * 1024 ? kRowsWaves * ALL : JOIN * MT * NT * 1024;
    static_assert(LDS <= 160 * 1024, "more LDS than a CU has");
    static constexpr int CHUNKS = STEP / 16;              // of 16 bytes in a row
    static constexpr int FILL = 64 / CHUNKS;              // rows that an instruction fills
    // Row r's chunk c stands at place c ^ turn(r), so that the 16 rows of a fragment read touch different banks.
    static __device__ __forceinline__ int turn(int r) { return CHUNKS == 8 ? (r >> 1) & 7 : r & 15; }
};

template <int ROWS, int NT, int STEP>
__device__ __forceinline__ void w8_rows_body(const W8Args& a) {
    using Sh = W8RowsShape<ROWS, NT, STEP>;
    constexpr int kJoin = Sh::JOIN, MT = Sh::MT;
    extern __shared__ __align__(16) char lds[];
    int(*const join)[MT * NT][64][4] = (int(*)[MT * NT][64][4])lds;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;
    const int tiles_o = (a.O + 16 * NT - 1) / (16 * NT), o0 = (blockIdx.x % tiles_o) * (16 * NT);
    const int t0 = (int)(blockIdx.x / tiles_o) * (16 * MT);
    const int live = min(a.M - t0, ROWS);
    char* const mine = lds + wave * Sh::ALL;
    // Rows past the end repeat the last one (their sums are not stored), chunks past K the first one (zeroed in x where they
    // are used).
    const int8_t* const w0 = a.w + (int64_t)o0 * a.K;
    auto load = [&](int k0) {
#pragma unroll
        for (int i = 0; i < ROWS / Sh::FILL; ++i) {
            if (Sh::FILL * i >= live) break;
            const int r = Sh::FILL * i + lane / Sh::CHUNKS, k = k0 + ((lane % Sh::CHUNKS) ^ Sh::turn(r)) * 16;
            const int8_t* src = a.x + (int64_t)(t0 + min(r, live - 1)) * a.x_stride + (k < a.K ? k : 0);
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                             (__attribute__((address_space(3))) void*)(mine + i * 1024), 16, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 16 * NT / Sh::FILL; ++i) {
            const int r = Sh::FILL * i + lane / Sh::CHUNKS, k = k0 + ((lane % Sh::CHUNKS) ^ Sh::turn(r)) * 16;
            const int8_t* src = w0 + (int64_t)(min(o0 + r, a.O - 1) - o0) * a.K + (k < a.K ? k : 0);
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                             (__attribute__((address_space(3))) void*)(mine + Sh::X + i * 1024), 16, 0, 0);
        }
    };
    i32x4 acc[MT][NT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[mt][nt] = i32x4{0, 0, 0, 0};
    for (int k0 = wave * STEP; k0 < a.K; k0 += kRowsWaves * STEP) {
        load(k0);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
        for (int j = 0; j < STEP / 64; ++j) {
            const int c = 4 * j + g;
            u32x4 x[MT], w[NT];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const int r = mt * 16 + n;
                x[mt] = *(const u32x4*)(mine + r * STEP + (c ^ Sh::turn(r)) * 16);
                if (k0 + STEP > a.K && k0 + c * 16 >= a.K) x[mt] = u32x4{0u, 0u, 0u, 0u};
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                w[nt] = *(const u32x4*)(mine + Sh::X + (nt * 16 + n) * STEP + (c ^ Sh::turn(n)) * 16);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) acc[mt][nt] = mfma16(x[mt], w[nt], acc[mt][nt]);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the step is read before the next one comes in
    }
    __syncthreads();  // the sums take the inputs' place

    // waves kJoin .. hand their sums to the first kJoin, whose sums are then added up
    if (wave >= kJoin)
#pragma unroll
        for (int i = 0; i < MT * NT; ++i) *(i32x4*)join[wave - kJoin][i][lane] = acc[i / NT][i % NT];
    __syncthreads();
    if (wave < kJoin)
#pragma unroll
        for (int i = 0; i < MT * NT; ++i) {
            acc[i / NT][i % NT] += *(const i32x4*)join[wave][i][lane];
            *(i32x4*)join[wave][i][lane] = acc[i / NT][i % NT];
        }
    __syncthreads();
    // lane (n, g) of tile (mt, nt) holds feature n of tokens 4 g ..
    for (int c = threadIdx.x; c < MT * NT * 64; c += kRowsWaves * kWave) {
        const int i = c >> 6, l = c & 63;
        i32x4 v = {0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < kJoin; ++k) v += *(const i32x4*)join[k][i][l];
        const int col = o0 + (i % NT) * 16 + (l & 15);
        if (col < a.O) {
            const float sw = a.w_scales[col];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = t0 + (i / NT) * 16 + (l >> 4) * 4 + e;
                if (t < a.M) a.out[(int64_t)t * a.O + col] = (uint16_t)pack_bf16x2((float)v[e] * sw * a.x_scales[t], 0.f);
            }
        }
    }
}

// Rows, feature tiles, bytes of a step, waves per SIMD that registers are kept to.
#define PLE_W8_SHAPES(X) X(16, 1, 256, 4) X(32, 2, 128, 4) X(64, 2, 128, 2)
#define PLE_W8_KERNEL(ROWS, NT, STEP, OCC)                                                                             \
    __global__ __launch_bounds__(kRowsWaves * kWave, OCC) void w8_rows_##ROWS##x##NT##_##STEP##_kernel(W8Args a) {     \
        w8_rows_body<ROWS, NT, STEP>(a);                                                                               \
    }
PLE_W8_SHAPES(PLE_W8_KERNEL)
#undef PLE_W8_KERNEL

// Few 64 x 64 tiles leave CUs idle: there the waves of a block share K instead (with 4096 inputs: 37 tokens, 5003 features
// 8.9 us against 11.0, 100 and 2048 7.2 and 8.6, 4 and 4096 6.5 and 8.3; but 64 and 6400 9.7 and 9.3, 16 and 8192 10.2 and
// 8.7, 1 and 8192 8.8 and 8.6).  Of those kernels the one with the fewest rows that hold the tokens; blocks of 32 rows also
// for more tokens as long as the CUs hold them (48 tokens, 4096 features 7.6 us, in blocks of 64 rows 8.5; 37 and 5003 12.8
// and 8.9).  Otherwise the tiles whose rounds over the CUs take least: a last round that is not full still takes most of one
// (64 tiles of 128 x 128 12.5 us, 128 14.6, 256 19).
constexpr int kFewTiles = 100;
W8Shape w8_linear_shape(int64_t T, int32_t O) {
    const auto tiles = [&](int64_t m, int64_t n) { return ((T + m - 1) / m) * ((O + n - 1) / n); };
    if (tiles(64, 64) < kFewTiles) {
        if (T <= 16) return {0, 16, 1, 256};
        return T <= 32 || tiles(32, 32) <= 256 ? W8Shape{0, 32, 2, 128} : W8Shape{0, 64, 2, 128};
    }
    W8Shape best = {256, 0, 0, 0};
    const auto cost = [&](int64_t n, int64_t one) { return n / 256 * 256 * one + (n % 256 ? one * (160 + n % 256 * 3 / 8) : 0); };
    int64_t least = cost(tiles(256, 256), kWideCost);
    const auto consider = [&](int mb, int nb, int64_t one) {
        const int64_t c = cost(tiles(64 * mb, 64 * nb), one);
        if (c < least) {
            least = c;
            best = {64, mb, nb, 0};
        }
    };
#define PLE_W8_CONSIDER(MB, NB, NS, COST) consider(MB, NB, COST);
    PLE_W8_TILES(PLE_W8_CONSIDER)
#undef PLE_W8_CONSIDER
    return best;
}

template <void (*FN)(W8Args), int LDS>
static hipError_t launch_w8(const W8Args& a, int64_t blocks, int threads, hipStream_t s) {
    static const hipError_t attr = hipFuncSetAttribute((const void*)FN, hipFuncAttributeMaxDynamicSharedMemorySize, LDS);
    if (attr != hipSuccess) return attr;
    hipLaunchKernelGGL(FN, dim3((unsigned)blocks), dim3(threads), LDS, s, a);
    return hipGetLastError();
}

hipError_t launch_w8_linear(const W8Args& a, hipStream_t s) {
    const W8Shape f = w8_linear_shape(a.M, a.O);
    const auto tiles = [&](int64_t m, int64_t n) { return ((a.M + m - 1) / m) * ((a.O + n - 1) / n); };
    if (f.block == 256) return launch_w8<w8_gemm_256_kernel, kWideLdsBytes>(a, tiles(256, 256), kWideThreads, s);
#define PLE_W8_LAUNCH(MB, NB, NS, COST)                                                                               \
    if (f.block == 64 && f.rows == MB && f.nt == NB)                                                                  \
        return launch_w8<w8_tile_##MB##x##NB##_kernel, W8Tile<MB, NB, NS>::LDS>(a, tiles(64 * MB, 64 * NB), kTileThreads, s);
    PLE_W8_TILES(PLE_W8_LAUNCH)
#undef PLE_W8_LAUNCH
#define PLE_W8_LAUNCH(ROWS, NT, STEP, OCC)                                                                            \
    if (f.rows == ROWS && f.nt == NT && f.step == STEP)                                                               \
        return launch_w8<w8_rows_##ROWS##x##NT##_##STEP##_kernel, W8RowsShape<ROWS, NT, STEP>::LDS>(                   \
            a, tiles(16 * W8RowsShape<ROWS, NT, STEP>::MT, 16 * NT), kRowsWaves * kWave, s);
    PLE_W8_SHAPES(PLE_W8_LAUNCH)
#undef PLE_W8_LAUNCH
    return hipErrorInvalidValue;
}

}  // namespace ple
