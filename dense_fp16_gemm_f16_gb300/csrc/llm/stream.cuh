// stream.cuh -- weight rows times a few columns, the weights streamed once
// through shared memory: the part that the 4-bit product and both products of
// the mixture-of-experts layer have in common.
//
// out[row, col] = sum_k W[row, k] X[col, k] with W 16-bit or 4-bit rows and at
// most 64 columns X.  Each weight byte meets few columns, so the rate is set by
// reading W from HBM; everything here serves keeping that stream unbroken:
//  - the work is a list of stages: a few 128-byte atoms of every row in hand
//    (64 k of 16-bit weights, 256 k of 4-bit ones each), their scales and zero
//    points, and the same k of the columns.  Rows come by TMA; the columns, which
//    for an expert are scattered rows of the activations, come in 16-byte pieces
//    per thread (one bulk copy per column held its warp for some 150 clocks each);
//  - 8 or 16 warps take the stages in turn: stage i belongs to the MW warps
//    with warp / MW == i % KW, each of which owns up to MT 16-row tiles in a row.
//    Every group of MW warps has slots of its own and its first warp refills
//    them itself, so many warps issue copies side by side (one producer warp for
//    all took 0.3 us per stage whatever its size, and bound the kernels at
//    0.4-2 TB/s); groups never meet until the rows' sums do.
// The products run on mma.sync m16n8k16 with the weights as the 16-row operand.
// 4-bit weights have to pass through registers to become 16-bit numbers, and
// mma.sync takes them from there; tcgen05 would need them written back to
// shared memory or TMEM first, and at these column counts the tensor pipe is
// idle most of the time either way.  The 16-bit weights use the same path so
// that experts of both kinds share one kernel: at 23 bytes per clock and SM
// (HBM's share) a stage of 64 rows x 64 k with 8 columns keeps the legacy
// tensor path busy under a tenth of the time.
//
// 4-bit codes.  ldmatrix hands thread (g, t) of a tile the 8 codes of k = 8t..8t+7
// of rows g and g + 8 of a 32-k chunk.  A mask of one nibble leaves the codes i
// and i + 4 in the low bits of two 16-bit numbers; the k order of an MMA is free,
// so the columns are paired (i, i + 4) the same way.
//   fp16: the bits are the subnormal numbers code * 2^-24, or * 2^-20 one nibble
//         up, exact; even and odd places have sums of their own, so half the
//         shifts go, and the scale takes the power of two with it.
//   bf16: or 0x4300 makes them 128 + code, exact.
// Over one group  sum (code - z) x = sum (code + o) x - (z + o) sum x,  o the
// offset 0 or 128; sum x comes from one more MMA with a matrix of ones, shared
// by a warp's tiles, and the group's scale multiplies the fp32 sums.  Nothing
// is rounded below fp32 between the codes and the output.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

#include "epilogue.cuh"
#include "ptx.cuh"
#include "wait.cuh"

namespace gemm_gb300 {

constexpr int kMaxRing = 48;                        // slots of all groups together
constexpr int kMaxAtoms = 4;                        // atoms per stage

constexpr int kConsumers = 8;                       // warps
constexpr int kStreamThreads = 32 * kConsumers;
// CTAs per SM for NT groups of 8 columns.  With few columns the sums take few
// registers and two CTAs fit: 16 warps to cover the chains of short latencies,
// and one CTA's start and end beside the other's middle.  For 4-bit experts with
// more than 8 columns, registers for 4 tiles a warp and shared memory for the
// columns (as many bytes per K as 4 times the weights) are worth more; for the
// plain product, which has exactly its columns, they are not (13 rows of A,
// 11000 x 4128: 21 us against 24).
template <bool W4, int NT, bool MOE>
constexpr int kCtasPerSm = NT == 1 || (NT == 2 && !(W4 && MOE)) ? 2 : 1;
constexpr int kSmemPerSm = 226 * 1024;              // 228 KB less what the CTAs' static parts take

// arrivals on a slot's full barrier: the byte count, and the columns of every
// lane of the mw warps that share the slot
__device__ __forceinline__ uint32_t full_arrivals(int mw) { return 1u + 32u * mw; }

constexpr uint32_t kSiteStreamEmpty = 9, kSiteStreamFull = 10, kSiteStreamDrain = 11;

// elements of k per atom: 128 bytes of a row
template <bool W4>
constexpr int kAtomElems = W4 ? 256 : 64;
// bytes between columns in a stage of ka atoms.  16-bit weights: ldmatrix reads
// 8 columns at the same 16-byte chunk; 4-bit: 16-byte loads read 64 bytes of 2
// columns at a time.  Both pitches spread those over all banks.
__host__ __device__ constexpr int col_pitch(bool w4, int ka) { return w4 ? ka * 512 + 64 : ka * 128 + 16; }
// 16-row tiles per warp: the fp32 sums of tiles x columns stay in registers
template <bool W4, int NT, bool MOE>
constexpr int kTilesPerWarp = NT == 8 || (W4 && NT == 4) || (W4 && NT == 2 && !MOE) ? 2 : 4;

namespace ptx {

// Reads of a stage and MMAs are free to move, so that independent chains
// overlap.  What holds them between the stage's arrival and its refill: their
// addresses depend on stage_token(), read after the wait, and keep() needs the
// sums before anything behind it.
template <int OFF>
__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4+%5];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr), "n"(OFF));
}

template <int OFF>
__device__ __forceinline__ void ldmatrix_x2(uint32_t addr, uint32_t (&r)[2]) {
    asm("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0, %1}, [%2+%3];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr), "n"(OFF));
}

template <int OFF>
__device__ __forceinline__ void ld_shared_u4(uint32_t addr, uint32_t (&r)[4]) {
    asm("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4+%5];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr), "n"(OFF));
}

template <int OFF>
__device__ __forceinline__ uint32_t ld_shared_u16(uint32_t addr) {
    uint16_t v;
    asm("ld.shared.u16 %0, [%1+%2];" : "=h"(v) : "r"(addr), "n"(OFF));
    return v;
}

// A zero that is not known before this point.
__device__ __forceinline__ uint32_t stage_token() {
    uint32_t z;
    asm volatile("mov.u32 %0, 0;" : "=r"(z) :: "memory");
    return z;
}

// (x & mask) | offset in one instruction: with both as immediates the compiler
// makes it two, and the ALU is what decoding bf16 is short of (207 against 145
// clocks per scheduler for a 16 x 128 tile, one group of columns).
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t offset) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(x), "r"(mask), "r"(offset));
    return r;
}

// A constant that the compiler does not know to be one.
__device__ __forceinline__ uint32_t opaque(uint32_t v) {
    uint32_t r;
    asm volatile("mov.u32 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ void keep(float (&v)[4]) {
    asm volatile("" : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]) :: "memory");
}

// 16 bytes from global to shared memory by this thread
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// An arrival on `bar` once this thread's copies so far have landed (one of the
// arrivals that the barrier was set up for).
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(bar) : "memory");
}

// d += a (16 x 16) * b (16 x 8), fp32 sums
template <class T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same<T, __half>::value)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
                     " {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
                     " {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// d = a * b
template <class T>
__device__ __forceinline__ void mma16816_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same<T, __half>::value)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
                     " {%10, %10, %10, %10};"
                     : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
                     " {%10, %10, %10, %10};"
                     : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

}  // namespace ptx

// How one launch lays its ring out.  Offsets are from the 1024-byte aligned
// base of dynamic shared memory.
struct RingLayout {
    int32_t atoms;       // atoms per stage
    int32_t slots;       // of all groups; group kg owns slots / KW of them, and one more if kg < slots % KW
    int32_t w_bytes;     // a slot's weights: atoms * atom_bytes
    int32_t atom_bytes;  // the rows of one atom, a multiple of 2048
    int32_t side_bytes;  // a slot's scales and zero points, a multiple of 256; 0 for 16-bit weights
    int32_t x_bytes;     // a slot's columns
    int32_t side_off, x_off, end;   // end: first byte behind the ring
};

// The slots [first, first + depth) of one group.
struct GroupSlots {
    int first, depth;
    __device__ __forceinline__ GroupSlots(int slots, int kw, int kg) {
        const int each = slots / kw, more = slots - each * kw;
        first = kg * each + min(kg, more);
        depth = each + (kg < more ? 1 : 0);
    }
};

// Where the rows of a tile lie.  In an atom: rows 0-7 of tile i at i * TILE
// bytes (a multiple of 1024, the swizzle's period), rows 8-15 `half` bytes behind
// them.  In the scales of one group: row 0 of tile i at i * SIDE bytes, row 8
// side_half bytes behind it, the next group `pitch` bytes on.
struct SideView {
    uint32_t scales, zeros;   // of row 0 of tile 0 in the first group
    uint32_t half, pitch;
};

// f(0) ... f(N - 1), each argument a compile-time constant
template <int I, int N, class F>
__device__ __forceinline__ void unrolled(F&& f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        unrolled<I + 1, N>(f);
    }
}

// The consumer's state for one warp: fp32 sums of its tiles.
template <class T, bool W4, int NT, bool MOE>
struct StreamWarp {
    static constexpr int MT = kTilesPerWarp<W4, NT, MOE>;
    float acc[MT][NT][4];

    __device__ __forceinline__ void hold() {
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
            for (int n = 0; n < NT; ++n) ptx::keep(acc[j][n]);
    }

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[j][n][i] = 0.0f;
    }

    // One atom of 16-bit weights: `w` the rows of this warp's first tile
    // (128-byte swizzle), `x` the columns, `k` valid elements (a multiple of 8),
    // `tiles` tiles and `nt` groups of 8 columns in use.
    template <int TILE>
    __device__ __forceinline__ void atom16(uint32_t w, uint32_t half, uint32_t x, int pitch, int k, int tiles, int nt,
                                           int lane) {
        const int i = lane >> 3, r = lane & 7;
        const uint32_t w_row = w + (i & 1) * half + static_cast<uint32_t>(r * 128);
        const uint32_t x_row = x + static_cast<uint32_t>(r * pitch + i * 16);
        const uint32_t x_step = static_cast<uint32_t>(8 * pitch);
        unrolled<0, 2>([&](auto step) {   // two steps of 16 k each
            constexpr int S = decltype(step)::value;
            if (S * 32 < k) {
                uint32_t b[NT][4];      // (b0, b1) of steps 2 S and 2 S + 1
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (n == 0 || n < nt) {
                        ptx::ldmatrix_x4<S * 64>(x_row + n * x_step, b[n]);
                        // a stage that ends early holds older data behind its end, which may not be numbers
                        if (S * 32 + 32 > k) {
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                if (S * 32 + q * 8 >= k) b[n][q] = 0u;
                        }
                    }
                }
                const uint32_t w0 = w_row + static_cast<uint32_t>(((4 * S + (i >> 1)) ^ r) << 4);
                const uint32_t w1 = w_row + static_cast<uint32_t>(((4 * S + 2 + (i >> 1)) ^ r) << 4);
                unrolled<0, MT>([&](auto tile) {
                    constexpr int J = decltype(tile)::value;
                    if (J < tiles) {
                        uint32_t a0[4], a1[4];
                        ptx::ldmatrix_x4<J * TILE>(w0, a0);
                        ptx::ldmatrix_x4<J * TILE>(w1, a1);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            if (n == 0 || n < nt) {
                                ptx::mma16816<T>(acc[J][n], a0, b[n][0], b[n][1]);
                                ptx::mma16816<T>(acc[J][n], a1, b[n][2], b[n][3]);
                            }
                        }
                    }
                });
            }
        });
    }

    // One atom of 4-bit weights: k a multiple of the group of 32 CPG; `side` the
    // scales of its first group.  A group's column registers serve all tiles.
    template <int CPG, int TILE, int SIDE>
    __device__ __forceinline__ void atom4(uint32_t w, uint32_t half, uint32_t x, int pitch, const SideView& side,
                                          bool has_zeros, int k, int tiles, int nt, int lane) {
        constexpr bool kF16 = std::is_same<T, __half>::value;
        constexpr float kOffset = kF16 ? 0.0f : 128.0f;
        // what a code of 1 counts in the even and in the odd places
        constexpr float kUnit = kF16 ? 16777216.0f : 1.0f, kUnitOdd = kF16 ? 1048576.0f : 1.0f;
        // Even and odd places added up in one chain of MMAs leave a third less to do to
        // the sums.  It costs fp16 its saved shifts, so there only groups of one chunk do
        // it (13 rows of A, 11000 x 4128, groups of 32: 21.5 -> 20.7 us); bf16 does in the
        // plain product (16 rows, 8192 x 8192, groups of 128: 21.1 -> 20.2 us).  Experts
        // often have 8 columns or fewer in use, and then the longer chain is what counts
        // (16 tokens, 8 of 64 experts, groups of 128: 123 us, merged 126).
        constexpr bool kMerge = NT >= 2 && (CPG == 1 || (!kF16 && !MOE));
        constexpr uint32_t kOne = kF16 ? 0x3C003C00u : 0x3F803F80u;
        const uint32_t ones[4] = {kOne, kOne, kOne, kOne};
        const uint32_t mask = ptx::opaque(0x000f000fu), offset = ptx::opaque(0x43004300u);
        const int i = lane >> 3, r = lane & 7, g = lane >> 2, t = lane & 3;
        const uint32_t w_row = w + (i & 1) * half + static_cast<uint32_t>(r * 128);
        const uint32_t x_step = static_cast<uint32_t>(8 * pitch);
        uint32_t xp = x + static_cast<uint32_t>(g * pitch + t * 16);
        uint32_t sp = side.scales + 2u * g, zp = side.zeros + 2u * g;
        const int groups = k / (32 * CPG);
#pragma unroll 1
        for (int grp = 0; grp < groups; ++grp, xp += CPG * 64, sp += side.pitch, zp += side.pitch) {
            uint32_t b[CPG][NT][4];
            float xs[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (n == 0 || n < nt) {
                    unrolled<0, CPG>([&](auto chunk) {
                        constexpr int C = decltype(chunk)::value;
                        uint32_t v[4];
                        ptx::ld_shared_u4<C * 64>(xp + n * x_step, v);
                        b[C][n][0] = __byte_perm(v[0], v[2], 0x5410);   // k 0, 4
                        b[C][n][1] = __byte_perm(v[1], v[3], 0x5410);   // k 2, 6
                        b[C][n][2] = __byte_perm(v[0], v[2], 0x7632);   // k 1, 5
                        b[C][n][3] = __byte_perm(v[1], v[3], 0x7632);   // k 3, 7
                    });
                }
            }
            // sum of the columns: two chains, even and odd places
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (n == 0 || n < nt) {
                    float odd[4];
                    ptx::mma16816_first<T>(xs[n], ones, b[0][n][0], b[0][n][1]);
                    ptx::mma16816_first<T>(odd, ones, b[0][n][2], b[0][n][3]);
#pragma unroll
                    for (int c = 1; c < CPG; ++c) {
                        ptx::mma16816<T>(xs[n], ones, b[c][n][0], b[c][n][1]);
                        ptx::mma16816<T>(odd, ones, b[c][n][2], b[c][n][3]);
                    }
                    xs[n][0] += odd[0];
                    xs[n][1] += odd[1];
                }
            }
            uint32_t w_at[CPG];   // this lane's row of chunk c
#pragma unroll
            for (int c = 0; c < CPG; ++c) w_at[c] = w_row + static_cast<uint32_t>(((grp * CPG + c) ^ r) << 4);
            unrolled<0, MT>([&](auto tile) {
                constexpr int J = decltype(tile)::value;
                if (J < tiles) {
                    uint32_t m[CPG][2];   // codes of rows g and g + 8
#pragma unroll
                    for (int c = 0; c < CPG; ++c) ptx::ldmatrix_x2<J * TILE>(w_at[c], m[c]);
                    const float s0 = Elem<T>::lo(ptx::ld_shared_u16<J * SIDE>(sp));
                    const float s1 = Elem<T>::lo(ptx::ld_shared_u16<J * SIDE>(sp + side.half));
                    float z0 = 8.0f + kOffset, z1 = z0;
                    if (has_zeros) {
                        z0 = Elem<T>::lo(ptx::ld_shared_u16<J * SIDE>(zp)) + kOffset;
                        z1 = Elem<T>::lo(ptx::ld_shared_u16<J * SIDE>(zp + side.half)) + kOffset;
                    }
                    float p[NT][4];   // even places (kMerge: both)
                    [[maybe_unused]] float q[NT][4];   // odd places
#pragma unroll
                    for (int c = 0; c < CPG; ++c) {
                        uint32_t even[4], odd[4];
                        if constexpr (kF16) {
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const uint32_t u = m[c][h] >> 8;
                                even[h] = m[c][h] & 0x000f000fu;
                                odd[h] = kMerge ? (m[c][h] >> 4) & 0x000f000fu : m[c][h] & 0x00f000f0u;
                                even[h + 2] = u & 0x000f000fu;
                                odd[h + 2] = kMerge ? (m[c][h] >> 12) & 0x000f000fu : u & 0x00f000f0u;
                            }
                        } else {
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                even[h] = ptx::and_or(m[c][h], mask, offset);
                                odd[h] = ptx::and_or(m[c][h] >> 4, mask, offset);
                                even[h + 2] = ptx::and_or(m[c][h] >> 8, mask, offset);
                                odd[h + 2] = ptx::and_or(m[c][h] >> 12, mask, offset);
                            }
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            if (n == 0 || n < nt) {
                                if constexpr (kMerge) {
                                    if (c == 0) ptx::mma16816_first<T>(p[n], even, b[c][n][0], b[c][n][1]);
                                    else ptx::mma16816<T>(p[n], even, b[c][n][0], b[c][n][1]);
                                    ptx::mma16816<T>(p[n], odd, b[c][n][2], b[c][n][3]);
                                } else if (c == 0) {
                                    ptx::mma16816_first<T>(p[n], even, b[c][n][0], b[c][n][1]);
                                    ptx::mma16816_first<T>(q[n], odd, b[c][n][2], b[c][n][3]);
                                } else {
                                    ptx::mma16816<T>(p[n], even, b[c][n][0], b[c][n][1]);
                                    ptx::mma16816<T>(q[n], odd, b[c][n][2], b[c][n][3]);
                                }
                            }
                        }
                    }
                    const float o0 = -s0 * z0, o1 = -s1 * z1;
                    const float e0 = s0 * kUnit, e1 = s1 * kUnit, d0 = s0 * kUnitOdd, d1 = s1 * kUnitOdd;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        if (n == 0 || n < nt) {
#pragma unroll
                            for (int v = 0; v < 4; ++v) {
                                const float o = v < 2 ? o0 : o1, e = v < 2 ? e0 : e1;
                                [[maybe_unused]] const float d = v < 2 ? d0 : d1;
                                float sum = fmaf(o, xs[n][v & 1], acc[J][n][v]);
                                if constexpr (!kMerge) sum = fmaf(d, q[n][v], sum);
                                acc[J][n][v] = fmaf(e, p[n][v], sum);
                            }
                        }
                    }
                }
            });
        }
    }
};

}  // namespace gemm_gb300
