// Products of 8-bit integers: out = (x W^T) scaled by token and by output
// channel, sums exact in 32-bit integers.
//
// Many tokens: the pipelines of the bf16 projection (ple_kv_proj.hip) with
// 16x16x64 and 32x32x32 integer MFMAs, whose operands are 16 bytes of K per
// lane as bf16's are: a slice of 128 bytes is 128 inputs, and tiles, copies,
// LDS layout and the order of products are as there.  What differs: rows of x
// may be strided, K may end inside a slice, O may be any number, and the
// scales multiply the sums on the way out.  Bound by the products.
//
// Few tokens (decode): bound by reading the weights once, and below that by
// the latency of the rounds of loads.  A block's eight waves share its
// features (NT x 16) and split K between them in steps of 256 bytes; a step's
// rows of inputs and weights come straight into LDS in whole rows, 1 KiB an
// instruction, and go to the matrix cores from there.  The waves' sums are
// joined through LDS: no second launch and no atomics.
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

// ---------------------------------------------------------------------------
// Pipelined kernel body for batches too small to give 256 blocks of 256 x
// 256: BT x BT block tile, 4 waves (one per SIMD), each a (BT/2) x (BT/2)
// block held in accumulator tiles of 32 x 32.  For BT = 128 that is 4 tiles
// and LDS stages of 32 KiB; for BT = 64, one tile and stages of 16 KiB.
// K-slices of 64.
//
// Why this shape: the fragment reads of the next 16-deep K-step are spread
// between the current step's MFMAs, so with one wave per SIMD the matrix core
// stays fed without a second wave to cover for it; the narrow tiles give
// blocks: a 1024-token batch gets 256 blocks of 128 x 128, a 256-token decode
// batch 256 blocks of 64 x 64 (there the W panels, read by four blocks each
// from the XCD's L2, bound the kernel, not the matrix cores).
//
// Operands go global -> LDS with buffer loads that write LDS directly
// (buffer_load_dwordx4 ... lds): a scalar buffer resource per operand panel
// and a 32-bit per-lane offset.  Each copy instruction fills 1 KiB = 8 whole
// 128-byte K-slice rows, so every request is a full cache line.  The copies
// of slice kt+2 go into the stage slice kt has just left: they start between
// the last K-step's MFMAs of slice kt (after the barrier that ends every read
// of that stage) and finish between the first K-step's MFMAs of slice kt+1,
// and the barrier at the end of slice kt+1 waits for them.
//
// LDS layout of one operand slice: row r holds 8 chunks of 16 bytes (64
// bf16 of K); chunk kc sits at position r*8 + (kc ^ ((r >> 1) & 7)).  A
// fragment read takes one k-chunk of 32 consecutive rows; the LDS serves 16
// lanes (256 bytes, 64 banks) per cycle and any 16 consecutive rows land on
// distinct 16-byte bank groups.  The MFMA operands are swapped (W fragment
// first) so each lane's accumulators are 4 consecutive output features of one
// token, which the epilogue writes to LDS as 8-byte pairs before coalesced
// 16-byte stores.
//
// The LDS fragment reads are inline assembly with explicit waits: the
// compiler's own waits would drain every read in flight before each MFMA
// group, which exposes the LDS latency on every K-step.  Each wait lists the
// fragment registers it covers as operands, so no MFMA can be scheduled
// above the wait for its inputs.
// ---------------------------------------------------------------------------
constexpr int kBigThreads = 256;
constexpr int kSliceBytes = 128;  // of K: 64 bf16, 128 bytes of 8-bit codes
constexpr int kNStage = 2;

// Block tile BT x BT (256, or 128 / 64 for problems too small to fill the
// chip with wider tiles); each of the 4 waves holds a (BT/2) x (BT/2) block
// as NB x NB accumulator tiles of 32 x 32.
template <int BT>
struct W8PipeShape {
    static constexpr int NB = BT / 64;                    // 32-row blocks per wave and operand
    static constexpr int NCOPY = BT / 32;                 // copy instructions per operand, wave and slice
    static constexpr int COPY_SPLIT = NCOPY / 2;          // of those, issued in a slice's last K-step (2 stages)
    static constexpr int OP_BYTES = BT * kSliceBytes;     // one operand's slice
    static constexpr int STAGE_BYTES = 2 * OP_BYTES;      // x + W slices
    // LDS stages: the narrower tiles run fewer MFMAs per slice, so more
    // slices are kept in flight to cover the copy latency (128 KiB each way)
    static constexpr int NS = BT == 256 ? kNStage : (128 * 1024) / STAGE_BYTES;
    static constexpr int OUT_ROW = BT + 8;                // epilogue row (elements)
    static constexpr int LDS_BYTES = (NS * STAGE_BYTES > BT * OUT_ROW * 2) ? NS * STAGE_BYTES : BT * OUT_ROW * 2;
    // copy instructions of one slice (both operands) per wave
    static constexpr int SLICE_COPIES = 2 * NCOPY;
    static_assert((NS & (NS - 1)) == 0 && (NS - 1) * SLICE_COPIES <= 63, "stages must fit the vmcnt counter");
};

typedef __attribute__((address_space(3))) void* lds_ptr_t;

// Wait for this wave's copies and LDS reads, then join the workgroup barrier.
// The "memory" clobber keeps the compiler from moving LDS or global accesses
// across it.
#define PLE_WAIT_VM_BARRIER0() asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory")

// The operands' rows in bytes.
struct W8Rows {
    int k, x, slices, tail;  // bytes of K and from one row of x to the next; slices; K's bytes in the last one if not all
    __device__ __forceinline__ explicit W8Rows(const W8Args& a)
        : k(a.K), x(a.x_stride), slices((k + kSliceBytes - 1) / kSliceBytes), tail(k % kSliceBytes) {}
    __device__ __forceinline__ int x_bytes(int n) const { return (n - 1) * x + k; }
};

// A block's BT x BT outputs out of LDS.
template <int BT, int THREADS>
__device__ __forceinline__ void pipe_store(const uint16_t* Cs, int out_row, const W8Args& a, int m0, int n0) {
    const int M = a.M, O = a.O;
    const bool whole = O % 8 == 0;  // rows of `out` begin at 16 bytes
#pragma unroll 4
    for (int c = threadIdx.x; c < BT * BT / 8; c += THREADS) {
        const int row = c / (BT / 8);  // BT/8 chunks of 8 features per row
        const int col = (c % (BT / 8)) * 8;
        const int gr = m0 + row, gc = n0 + col;
        if (gr >= M || gc >= O) continue;
        if (whole) {
            *(u32x4*)(a.out + (int64_t)gr * O + gc) = *(const u32x4*)(Cs + row * out_row + col);
        } else {
            for (int e = 0; e < 8 && gc + e < O; ++e) a.out[(int64_t)gr * O + gc + e] = Cs[row * out_row + col + e];
        }
    }
}

template <int NB>
struct W8Frag {
    u32x4 a[NB], b[NB];  // x fragments of the token blocks, W fragments of the feature blocks
};
// A wait names the fragment registers it covers, so no MFMA reading them can
// be scheduled above it.
#define PLE_W8_FRAG_REGS4(f) \
    "+v"(f.a[0]), "+v"(f.a[1]), "+v"(f.a[2]), "+v"(f.a[3]), "+v"(f.b[0]), "+v"(f.b[1]), "+v"(f.b[2]), "+v"(f.b[3])
#define PLE_W8_FRAG_REGS2(f) "+v"(f.a[0]), "+v"(f.a[1]), "+v"(f.b[0]), "+v"(f.b[1])
#define PLE_W8_FRAG_REGS1(f) "+v"(f.a[0]), "+v"(f.b[0])

template <int BT>
__device__ __forceinline__ void w8_pipe(const W8Args& a) {
    using P = W8PipeShape<BT>;
    constexpr int NB = P::NB;
    constexpr int WT = BT / 2;  // wave block
    using Frag = W8Frag<NB>;
    extern __shared__ __align__(16) char lds_raw[];
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;  // 2 x 2 waves: WT tokens x WT features each
    const int M = a.M, O = a.O;
    const W8Rows rows(a);

    const int tiles_m = (M + BT - 1) / BT;
    const int tiles_n = (O + BT - 1) / BT;
    int tm, tn;
    tile_of_block<8>(blockIdx.x, tiles_m, tiles_n, tm, tn);
    const int m0 = tm * BT, n0 = tn * BT;

    // Copy instruction i (0..NCOPY-1) of wave `wave` fills rows g*8 .. g*8+7
    // of an operand slice, g = i*4 + wave; lane L lands at position g*64 + L:
    // row g*8 + L/8, chunk kc = (L & 7) ^ ((row >> 1) & 7).  Rows past the end
    // of x or W read the last row (their outputs are never stored).
    const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(
        (void*)((const char*)a.x + (int64_t)m0 * rows.x), (short)0, rows.x_bytes(min(M - m0, BT)), 0x00020000);
    const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
        (void*)((const char*)a.w + (int64_t)n0 * rows.k), (short)0, min(O - n0, BT) * rows.k, 0x00020000);
    uint32_t aoff[P::NCOPY], boff[P::NCOPY];
#pragma unroll
    for (int i = 0; i < P::NCOPY; ++i) {
        const int row = (i * 4 + wave) * 8 + (lane >> 3);
        const int kc = (lane & 7) ^ ((row >> 1) & 7);
        aoff[i] = (uint32_t)((min(m0 + row, M - 1) - m0) * rows.x + kc * 16);
        boff[i] = (uint32_t)((min(n0 + row, O - 1) - n0) * rows.k + kc * 16);
    }
    const int nk = rows.slices;
    // copy instruction i of slice kt into stage kt % NS; slices past the end
    // (the loop below is uniform) re-read the last slice into a stage that no
    // later read uses
    auto copy_one = [&](int kt, int i) {
        char* base = lds_raw + (kt & (P::NS - 1)) * P::STAGE_BYTES;
        const int g = i * 4 + wave;
        const int ko = min(kt, nk - 1) * kSliceBytes;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_ptr_t)(base + g * 1024), 16, aoff[i], ko, 0, 0);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_ptr_t)(base + P::OP_BYTES + g * 1024), 16, boff[i], ko, 0,
                                                 0);
    };

    i32x16 acc[NB][NB];  // [W block j][x block i]
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[j][i][e] = 0;

    const int frow = lane & 31;
    const int fk = lane >> 5;
    const int sw = (frow >> 1) & 7;  // the chunk swizzle, the same for every 32-row block
    // LDS byte address of this lane's fragment chunk for K-step kk in stage 0,
    // first 32-row block (the others are +4096 bytes each)
    uint32_t a_addr[4], b_addr[4];
    const uint32_t lds_base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds_raw;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
        const uint32_t col = (uint32_t)(((kk * 2 + fk) ^ sw) * 16);
        a_addr[kk] = lds_base + (wm * WT + frow) * 128 + col;
        b_addr[kk] = lds_base + P::OP_BYTES + (wn * WT + frow) * 128 + col;
    }
    // fragment read q (0..2*NB-1) of K-step kk of slice kt: x blocks, then W blocks
    auto read_one = [&](int q, int kt, int kk, Frag& f) {
        const uint32_t so = (uint32_t)(kt & (P::NS - 1)) * P::STAGE_BYTES;
        const uint32_t pa = a_addr[kk] + so, pb = b_addr[kk] + so;
        if constexpr (NB == 4) {
            switch (q) {
                case 0: asm volatile("ds_read_b128 %0, %1" : "=v"(f.a[0]) : "v"(pa)); break;
                case 1: asm volatile("ds_read_b128 %0, %1 offset:4096" : "=v"(f.a[1]) : "v"(pa)); break;
                case 2: asm volatile("ds_read_b128 %0, %1 offset:8192" : "=v"(f.a[2]) : "v"(pa)); break;
                case 3: asm volatile("ds_read_b128 %0, %1 offset:12288" : "=v"(f.a[3]) : "v"(pa)); break;
                case 4: asm volatile("ds_read_b128 %0, %1" : "=v"(f.b[0]) : "v"(pb)); break;
                case 5: asm volatile("ds_read_b128 %0, %1 offset:4096" : "=v"(f.b[1]) : "v"(pb)); break;
                case 6: asm volatile("ds_read_b128 %0, %1 offset:8192" : "=v"(f.b[2]) : "v"(pb)); break;
                default: asm volatile("ds_read_b128 %0, %1 offset:12288" : "=v"(f.b[3]) : "v"(pb)); break;
            }
        } else if constexpr (NB == 2) {
            switch (q) {
                case 0: asm volatile("ds_read_b128 %0, %1" : "=v"(f.a[0]) : "v"(pa)); break;
                case 1: asm volatile("ds_read_b128 %0, %1 offset:4096" : "=v"(f.a[1]) : "v"(pa)); break;
                case 2: asm volatile("ds_read_b128 %0, %1" : "=v"(f.b[0]) : "v"(pb)); break;
                default: asm volatile("ds_read_b128 %0, %1 offset:4096" : "=v"(f.b[1]) : "v"(pb)); break;
            }
        } else {
            if (q == 0)
                asm volatile("ds_read_b128 %0, %1" : "=v"(f.a[0]) : "v"(pa));
            else
                asm volatile("ds_read_b128 %0, %1" : "=v"(f.b[0]) : "v"(pb));
        }
    };
    auto wait_frag = [&](Frag& f) {
        if constexpr (NB == 4)
            asm volatile("s_waitcnt lgkmcnt(0)" : PLE_W8_FRAG_REGS4(f));
        else if constexpr (NB == 2)
            asm volatile("s_waitcnt lgkmcnt(0)" : PLE_W8_FRAG_REGS2(f));
        else
            asm volatile("s_waitcnt lgkmcnt(0)" : PLE_W8_FRAG_REGS1(f));
    };
    // the barrier of an NS-stage slice: this wave's copies of every slice but
    // the next NS-2 have landed
    auto wait_barrier_vm = [&](Frag& f) {
        constexpr int V = (P::NS - 2) * P::SLICE_COPIES;
        if constexpr (NB == 2)
            asm volatile("s_waitcnt vmcnt(%4) lgkmcnt(0)\n\ts_barrier" : PLE_W8_FRAG_REGS2(f) : "i"(V) : "memory");
        else
            asm volatile("s_waitcnt vmcnt(%2) lgkmcnt(0)\n\ts_barrier" : PLE_W8_FRAG_REGS1(f) : "i"(V) : "memory");
    };
    auto wait_barrier = [&](Frag& f) {
        if constexpr (NB == 4)
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" : PLE_W8_FRAG_REGS4(f) : : "memory");
        else if constexpr (NB == 2)
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" : PLE_W8_FRAG_REGS2(f) : : "memory");
        else
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" : PLE_W8_FRAG_REGS1(f) : : "memory");
    };
    // One K-step: NB*NB MFMAs on `cur`.  After MFMA t < 2*NB comes fragment
    // read t of (rkt, rkk) into `nxt`, and copy instructions [c0, c1) of slice
    // ckt are spread over the MFMAs.  The order is pinned.
    auto kstep = [&](const Frag& cur, Frag& nxt, int rkt, int rkk, int ckt, int c0, int c1) {
        constexpr int NT = NB * NB;
        const int nc = c1 - c0;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int j = t / NB, i = t % NB;
            acc[j][i] = mfma32(cur.b[j], cur.a[i], acc[j][i]);
            if (rkk >= 0) {
                if constexpr (2 * NB <= NT) {
                    if (t < 2 * NB) read_one(t, rkt, rkk, nxt);
                } else {
#pragma unroll
                    for (int q = 0; q < 2 * NB; ++q) read_one(q, rkt, rkk, nxt);  // NT == 1
                }
            }
            if (nc > 0 && nc <= NT && (t * nc) % NT < nc) copy_one(ckt, c0 + (t * nc) / NT);
            if (nc > NT)
#pragma unroll
                for (int c = (t * nc) / NT; c < ((t + 1) * nc) / NT; ++c) copy_one(ckt, c0 + c);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // a last slice that K ends in: x past K becomes zero (W holds the next row's there)
    auto trim = [&](Frag& f, int kt, int kk) {
        if (kt == nk - 1 && rows.tail != 0) {
            const uint32_t keep = (kk * 2 + fk) * 16 < rows.tail ? 0xFFFFFFFFu : 0u;
#pragma unroll
            for (int i = 0; i < NB; ++i) f.a[i] &= keep;
        }
    };
    // One slice.  On entry f0 is receiving K-step 0 of slice kt.  LDS reads
    // return in order, so when a K-step starts, the reads issued during the
    // previous one are the only ones in flight and waiting for all of them
    // covers its fragments.  The first K-step finishes the copies of slice
    // kt+1 that slice kt-1 began; the last begins those of slice kt+2, into
    // the stage this slice has just left.  The last slice's look-ahead reads
    // and copies land in the other stage and are never used.
    auto slice = [&](int kt, Frag& f0, Frag& f1) {
        if constexpr (P::NS == 2) {
            wait_frag(f0);
            trim(f0, kt, 0);
            kstep(f0, f1, kt, 1, kt + 1, P::COPY_SPLIT, P::NCOPY);
            wait_frag(f1);
            trim(f1, kt, 1);
            kstep(f1, f0, kt, 2, 0, 0, 0);
            wait_frag(f0);
            trim(f0, kt, 2);
            kstep(f0, f1, kt, 3, 0, 0, 0);
            // every read of this stage is complete (all waves) and slice kt+1 has landed
            __builtin_amdgcn_sched_barrier(0);
            wait_barrier(f1);
            __builtin_amdgcn_sched_barrier(0);
            trim(f1, kt, 3);
            kstep(f1, f0, kt + 1, 0, kt + 2, 0, P::COPY_SPLIT);
        } else {
            // NS stages: slices kt+1 .. kt+NS-1 are in flight or landed; after
            // the barrier (this wave's copies of slice kt+1 done, every read of
            // slice kt done) the last K-step refills slice kt's stage with
            // slice kt+NS
            wait_frag(f0);
            trim(f0, kt, 0);
            kstep(f0, f1, kt, 1, 0, 0, 0);
            wait_frag(f1);
            trim(f1, kt, 1);
            kstep(f1, f0, kt, 2, 0, 0, 0);
            wait_frag(f0);
            trim(f0, kt, 2);
            kstep(f0, f1, kt, 3, 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
            wait_barrier_vm(f1);
            __builtin_amdgcn_sched_barrier(0);
            trim(f1, kt, 3);
            kstep(f1, f0, kt + 1, 0, kt + P::NS, 0, P::NCOPY);
        }
    };

    Frag f0, f1;
    if constexpr (P::NS == 2) {
        // slice 0 whole, then the first part of slice 1
#pragma unroll
        for (int i = 0; i < P::NCOPY; ++i) copy_one(0, i);
        PLE_WAIT_VM_BARRIER0();
#pragma unroll
        for (int i = 0; i < P::COPY_SPLIT; ++i) copy_one(1, i);
    } else {
        // slices 0 .. NS-1, then wait for slice 0
#pragma unroll
        for (int k = 0; k < P::NS; ++k)
#pragma unroll
            for (int i = 0; i < P::NCOPY; ++i) copy_one(k, i);
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "i"((P::NS - 1) * P::SLICE_COPIES) : "memory");
    }
#pragma unroll
    for (int q = 0; q < 2 * NB; ++q) read_one(q, 0, 0, f0);
    for (int kt = 0; kt < nk; ++kt) slice(kt, f0, f1);
    // The last slice's look-ahead reads into f0 are still in flight and
    // opaque to the compiler's own waits: this wait names f0's registers, so
    // no epilogue value is placed in them before the reads have landed.
    if constexpr (NB == 4)
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" : PLE_W8_FRAG_REGS4(f0) : : "memory");
    else if constexpr (NB == 2)
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" : PLE_W8_FRAG_REGS2(f0) : : "memory");
    else
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" : PLE_W8_FRAG_REGS1(f0) : : "memory");
    __syncthreads();  // every wave is done with the stages before the epilogue reuses LDS

    // epilogue: acc[j][i][e] is feature n0 + wn*WT + j*32 + 8*(e/4) + 4*(lane/32) + e%4
    // of token m0 + wm*WT + i*32 + lane%32
    uint16_t* Cs = (uint16_t*)lds_raw;
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int m = wm * WT + i * 32 + frow;
                const int o = wn * WT + j * 32 + 8 * g + 4 * fk;
                *(u32x2*)(Cs + m * P::OUT_ROW + o) = out4(a, m0 + m, n0 + o, acc[j][i][4 * g], acc[j][i][4 * g + 1],
                                                              acc[j][i][4 * g + 2], acc[j][i][4 * g + 3]);
            }
    __syncthreads();
    pipe_store<BT, kBigThreads>(Cs, P::OUT_ROW, a, m0, n0);
}

// ---------------------------------------------------------------------------
// 256-wide tiles with eight waves (two per SIMD) on 16x16x32 MFMAs: wave
// (wm, wn) holds a 128 x 64 block (x rows wm*128.., W rows wn*64..) as 8 x 4
// accumulator tiles of 16 x 16 (128 accumulation registers), so a wave
// waiting on its fragments leaves the matrix core to the other wave of its
// SIMD.  Row layout in LDS and the copy instructions as the four-wave body; a
// slice is two K-steps of 32 with 12 fragment reads each.  Instead of two
// stages of both operands, the LDS holds a ring of five operand slices, which
// gives the W copies a second slice of lead.  The tiles an XCD runs at once
// are grouped four tile rows by eight tile columns, so each W panel is shared
// by four blocks in that XCD's L2 and each x panel by eight: more of the W
// copies wait on the last-level cache.
// ---------------------------------------------------------------------------
constexpr int kWideThreads = 512;
// five operand-slice slots (160 KiB, all of the LDS), which also hold the epilogue's rows
constexpr int kWideLdsBytes = 5 * W8PipeShape<256>::OP_BYTES;
static_assert(kWideLdsBytes >= W8PipeShape<256>::LDS_BYTES, "the epilogue's rows fit in the ring");
struct W8WideFrag {
    u32x4 a[8], b[4];
};
#define PLE_W8_WIDE_FRAG_REGS(f)                                                                                       \
    "+v"(f.a[0]), "+v"(f.a[1]), "+v"(f.a[2]), "+v"(f.a[3]), "+v"(f.a[4]), "+v"(f.a[5]), "+v"(f.a[6]), "+v"(f.a[7]), \
        "+v"(f.b[0]), "+v"(f.b[1]), "+v"(f.b[2]), "+v"(f.b[3])

__device__ __forceinline__ void w8_pipe8w(const W8Args& a) {
    using P = W8PipeShape<256>;
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
        char* base = lds_raw + (3 + (k & 1)) * P::OP_BYTES + (i * 8 + wave) * 1024;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_ptr_t)base, 16, aoff[i], min(k, nk - 1) * kSliceBytes, 0, 0);
    };
    auto copy_w = [&](int k, int i) {
        char* base = lds_raw + (k % 3) * P::OP_BYTES + (i * 8 + wave) * 1024;
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
        const uint32_t pa = a_addr[ks] + (uint32_t)(3 + (kt & 1)) * P::OP_BYTES;
        const uint32_t pb = b_addr[ks] + (uint32_t)(kt % 3) * P::OP_BYTES;
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
    // one K-step of 32: 32 MFMAs on cur; after MFMA t < 12, fragment read t of
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
            *(u32x2*)(Cs + m * P::OUT_ROW + o) =
                out4(a, m0 + m, n0 + o, acc[j][i][0], acc[j][i][1], acc[j][i][2], acc[j][i][3]);
        }
    __syncthreads();
    pipe_store<BT, kWideThreads>(Cs, P::OUT_ROW, a, m0, n0);
}
#undef PLE_W8_WIDE_FRAG_REGS

#undef PLE_W8_FRAG_REGS4
#undef PLE_W8_FRAG_REGS2
#undef PLE_W8_FRAG_REGS1

__global__ __launch_bounds__(kWideThreads, 1) void w8_gemm_256_kernel(W8Args a) { w8_pipe8w(a); }
__global__ __launch_bounds__(kBigThreads, 1) void w8_gemm_128_kernel(W8Args a) { w8_pipe<128>(a); }
__global__ __launch_bounds__(kBigThreads, 1) void w8_gemm_64_kernel(W8Args a) { w8_pipe<64>(a); }

// The few-token kernel's LDS: a step's inputs and weights of every wave, then the joined sums.
constexpr int kStep = 256;  // bytes of K
constexpr int kRowsWaves = 8;
template <int MT, int NT>
struct W8RowsShape {
    static constexpr int X = MT * 16 * kStep;             // bytes of a wave's inputs
    static constexpr int STEP = X + NT * 16 * kStep;
    static constexpr int JOIN = 4;                        // waves whose sums are in LDS at once
    static constexpr int LDS = kRowsWaves * STEP > JOIN * MT * NT * 1024 ? kRowsWaves * STEP : JOIN * MT * NT * 1024;
    static_assert(LDS <= 160 * 1024, "more LDS than a CU has");
};

template <int MT, int NT>
__device__ __forceinline__ void w8_rows_body(const W8Args& a) {
    using Sh = W8RowsShape<MT, NT>;
    constexpr int kJoin = Sh::JOIN;
    extern __shared__ __align__(16) char lds[];
    int(*const join)[MT * NT][64][4] = (int(*)[MT * NT][64][4])lds;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;
    const int tiles_o = (a.O + 16 * NT - 1) / (16 * NT), o0 = (blockIdx.x % tiles_o) * (16 * NT);
    const int t0 = (int)(blockIdx.x / tiles_o) * (16 * MT);
    const int live = min(a.M - t0, 16 * MT);
    char* const mine = lds + wave * Sh::STEP;
    // An instruction fills four rows of 256 bytes: row r's 16 chunks of 16 bytes, chunk c at place c ^ (r % 16), so that
    // the 16 rows of a fragment read touch different banks.  Rows past the end repeat the last one (their sums are not
    // stored), chunks past K the first one (zeroed in x where they are used).
    const int64_t wrow = (int64_t)o0 * a.K;
    auto load = [&](int k0) {
#pragma unroll
        for (int i = 0; i < 4 * MT; ++i) {
            if (4 * i >= live) break;
            const int r = 4 * i + g, k = k0 + (n ^ (r & 15)) * 16;
            const int8_t* src = a.x + (int64_t)(t0 + min(r, live - 1)) * a.x_stride + (k < a.K ? k : 0);
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                             (__attribute__((address_space(3))) void*)(mine + i * 1024), 16, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 4 * NT; ++i) {
            const int r = 4 * i + g, k = k0 + (n ^ (r & 15)) * 16;
            const int8_t* src = a.w + wrow + (int64_t)(min(o0 + r, a.O - 1) - o0) * a.K + (k < a.K ? k : 0);
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                             (__attribute__((address_space(3))) void*)(mine + Sh::X + i * 1024), 16, 0, 0);
        }
    };
    i32x4 acc[MT][NT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[mt][nt] = i32x4{0, 0, 0, 0};
    for (int k0 = wave * kStep; k0 < a.K; k0 += kRowsWaves * kStep) {
        load(k0);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
        for (int j = 0; j < kStep / 64; ++j) {
            const int at = n * kStep + ((4 * j + g) ^ n) * 16;
            u32x4 x[MT], w[NT];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                x[mt] = *(const u32x4*)(mine + mt * (16 * kStep) + at);
                if (k0 + kStep > a.K && k0 + (4 * j + g) * 16 >= a.K) x[mt] = u32x4{0u, 0u, 0u, 0u};
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) w[nt] = *(const u32x4*)(mine + Sh::X + nt * (16 * kStep) + at);
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

// Token tiles, feature tiles, waves per SIMD that registers are kept to.
#define PLE_W8_SHAPES(X) X(1, 1, 4) X(2, 1, 4) X(4, 1, 2)
#define PLE_W8_KERNEL(MT, NT, OCC) \
    __global__ __launch_bounds__(kRowsWaves * kWave, OCC) void w8_rows_##MT##x##NT##_kernel(W8Args a) { w8_rows_body<MT, NT>(a); }
PLE_W8_SHAPES(PLE_W8_KERNEL)
#undef PLE_W8_KERNEL

W8Shape w8_linear_shape(int64_t T, int32_t O) {
    if (T <= 64) return {0, T <= 16 ? 1 : (T <= 32 ? 2 : 4), 1};
    // the widest tile that still gives 256 blocks, one per CU (64-wide tiles take 128 KiB of LDS, so only while one block
    // per CU covers them)
    const auto tiles = [&](int64_t b) { return ((T + b - 1) / b) * ((O + b - 1) / b); };
    if (tiles(256) >= 256) return {256, 0, 0};
    if (tiles(128) >= 256 || tiles(64) > 256) return {128, 0, 0};
    return {64, 0, 0};
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
    if (f.block == 128) return launch_w8<w8_gemm_128_kernel, W8PipeShape<128>::LDS_BYTES>(a, tiles(128, 128), kBigThreads, s);
    if (f.block == 64) return launch_w8<w8_gemm_64_kernel, W8PipeShape<64>::LDS_BYTES>(a, tiles(64, 64), kBigThreads, s);
#define PLE_W8_LAUNCH(MT, NT, OCC)                                                                                     \
    if (f.mt == MT && f.nt == NT)                                                                                      \
        return launch_w8<w8_rows_##MT##x##NT##_kernel, W8RowsShape<MT, NT>::LDS>(a, tiles(16 * MT, 16 * NT),           \
                                                                                kRowsWaves * kWave, s);
    PLE_W8_SHAPES(PLE_W8_LAUNCH)
#undef PLE_W8_LAUNCH
    return hipErrorInvalidValue;
}

}  // namespace ple
