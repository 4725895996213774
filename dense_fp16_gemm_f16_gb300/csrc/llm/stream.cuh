// stream.cuh -- weight rows times a few columns, the weights streamed once
// through shared memory: the part that the 4-bit product and both products of
// the mixture-of-experts layer have in common.
//
// out[row, col] = sum_k W[row, k] X[col, k] with W 16-bit or 4-bit rows and at
// most 64 columns X.  Each weight byte meets few columns, so the rate is set by
// reading W from HBM; everything here serves keeping that stream unbroken:
//  - one producer warp fills a ring of stages with TMA, each stage 128 bytes of
//    every row in hand (64 k of 16-bit weights, 256 k of 4-bit ones), their
//    scales and zero points, and the same k of the columns, one bulk copy per
//    column (the columns of an expert are scattered rows of the activations);
//  - kConsumers warps share the stages in turn: stage i belongs to the MW
//    warps with warp / MW == i % KW, each of which owns every MW-th 16-row
//    tile.  Warps of different stages never meet until the rows' sums do.
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
// of rows g and g + 8 of a 32-k chunk.  (w >> 4i) & 0x000f000f are the codes i
// and i + 4 in the low bits of two 16-bit numbers; the k order of an MMA is free,
// so the columns are paired (i, i + 4) the same way.
//   fp16: the bits are the subnormal numbers code * 2^-24, exact; the scale
//         takes 2^24 with it.
//   bf16: or 0x4300 makes them 128 + code, exact.
// Over one group  sum (code - z) x = sum (code + o) x - (z + o) sum x,  o the
// offset 0 or 128; sum x comes from one more MMA with a matrix of ones, and
// the group's scale multiplies the fp32 difference.  Nothing is rounded below
// fp32 between the codes and the output.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

#include "epilogue.cuh"
#include "ptx.cuh"
#include "wait.cuh"

namespace gemm_gb300 {

constexpr int kConsumers = 8;                       // consumer warps
constexpr int kStreamThreads = 32 * (kConsumers + 1);
constexpr int kMaxRing = 32;                        // stages

constexpr uint32_t kSiteStreamEmpty = 9, kSiteStreamFull = 10, kSiteStreamDrain = 11;

// elements of k per stage: 128 bytes of a row
template <bool W4>
constexpr int kStageElems = W4 ? 256 : 64;
// bytes between columns in a stage.  16-bit weights: ldmatrix reads 8 columns
// at the same 16-byte chunk; 4-bit: 16-byte loads read 64 bytes of 2 columns
// at a time.  Both pitches spread those over all banks.
template <bool W4>
constexpr int kColPitch = W4 ? 512 + 64 : 128 + 16;
// 16-row tiles per warp: the fp32 sums of tiles x columns stay in registers
template <int NT>
constexpr int kTilesPerWarp = NT <= 2 ? 4 : (NT <= 4 ? 2 : 1);

namespace ptx {

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

__device__ __forceinline__ void ldmatrix_x2(uint32_t addr, uint32_t (&r)[2]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr) : "memory");
}

__device__ __forceinline__ void ld_shared_u4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

__device__ __forceinline__ uint32_t ld_shared_u16(uint32_t addr) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
    return v;
}

// d += a (16 x 16) * b (16 x 8), fp32 sums
template <class T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same<T, __half>::value)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
                     " {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
                     " {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// `bytes` (a multiple of 16) from global to this CTA's shared memory, both
// 16-byte aligned; completion counted on `bar`
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 :: "r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

}  // namespace ptx

// How one launch lays its ring out.  Offsets are from the 1024-byte aligned
// base of dynamic shared memory.
struct RingLayout {
    // Ring stages: a multiple of KW, so that a slot is always read by the same
    // warps.  They have then seen the slot's last use complete before they wait
    // for the next one; a wait by parity cannot tell uses two apart.
    int32_t stages;
    int32_t w_bytes;     // a stage's weight rows, whole tiles: a multiple of 2048
    int32_t side_bytes;  // a stage's scales (as many again for zero points), a multiple of 128; 0 for 16-bit weights
    int32_t x_bytes;     // a stage's columns
    int32_t side_off, x_off, end;   // end: first byte behind the ring
};

// Scales of one stage in shared memory: [groups][cap] of T for each of two
// row halves (the same one unless they are different matrices' rows).
struct SideView {
    uint32_t scales[2], zeros[2];   // address of the first row of half 0 / 1 of tile 0
    int32_t cap;                    // rows per group
    int32_t tile_step;              // rows from one tile to the next
};

// The consumer's state for one warp: fp32 sums of its tiles.
template <class T, bool W4, int NT>
struct StreamWarp {
    static constexpr int MT = kTilesPerWarp<NT>;
    float acc[MT][NT][4];

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[j][n][i] = 0.0f;
    }

    // One stage of 16-bit weights: `w` the rows (128-byte swizzle), `x` the
    // columns, `k` valid elements (a multiple of 8), `tiles` tiles of which
    // this warp takes mg, mg + mw, ..., `nt` groups of 8 columns in use.
    __device__ __forceinline__ void stage16(uint32_t w, uint32_t x, int k, int tiles, int mg, int mw, int nt, int lane) {
        const int i = lane >> 3, r = lane & 7;
        const uint32_t w_row = w + static_cast<uint32_t>(((i & 1) * 8 + r) * 128);
        const uint32_t x_row = x + static_cast<uint32_t>(r * kColPitch<false>);
#pragma unroll
        for (int s = 0; s < 4; s += 2) {   // two steps of 16 k
            if (s * 16 >= k) break;
            uint32_t b[NT][4];             // (b0, b1) of steps s and s + 1
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (n < nt) {
                    ptx::ldmatrix_x4(x_row + static_cast<uint32_t>(n * 8 * kColPitch<false> + (2 * s + i) * 16), b[n]);
                    // a stage that ends early holds older data behind its end, which may not be numbers
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if ((2 * s + q) * 8 >= k) b[n][q] = 0u;
                }
            }
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                const int tile = mg + j * mw;
                if (tile < tiles) {
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint32_t a[4];
                        ptx::ldmatrix_x4(w_row + static_cast<uint32_t>(tile * 2048 + (((2 * (s + q) + (i >> 1)) ^ r) << 4)), a);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            if (n < nt) ptx::mma16816<T>(acc[j][n], a, b[n][2 * q], b[n][2 * q + 1]);
                    }
                }
            }
        }
    }

    // One stage of 4-bit weights: k a multiple of the group; chunks_per_group = group / 32.
    __device__ __forceinline__ void stage4(uint32_t w, uint32_t x, const SideView& side, bool has_zeros, int k,
                                           int chunks_per_group, int tiles, int mg, int mw, int nt, int lane) {
        constexpr bool kHalf = std::is_same<T, __half>::value;
        constexpr uint32_t kOr = kHalf ? 0u : 0x43004300u;
        constexpr float kOffset = kHalf ? 0.0f : 128.0f;
        constexpr float kUnit = kHalf ? 16777216.0f : 1.0f;
        constexpr uint32_t kOne = kHalf ? 0x3C003C00u : 0x3F803F80u;
        const uint32_t ones[4] = {kOne, kOne, kOne, kOne};
        const int i = lane >> 3, r = lane & 7, g = lane >> 2, t = lane & 3;
        const uint32_t w_row = w + static_cast<uint32_t>(((i & 1) * 8 + r) * 128);
        const uint32_t x_row = x + static_cast<uint32_t>(g * kColPitch<true> + t * 16);
        const int chunks = k >> 5;
        float p[MT][NT][4], xs[NT][4];
        for (int c = 0; c < chunks; c += chunks_per_group) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    xs[n][q] = 0.0f;
#pragma unroll
                    for (int j = 0; j < MT; ++j) p[j][n][q] = 0.0f;
                }
            }
            for (int cc = c; cc < c + chunks_per_group; ++cc) {
                uint32_t b[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (n < nt) {
                        uint32_t v[4];
                        ptx::ld_shared_u4(x_row + static_cast<uint32_t>(n * 8 * kColPitch<true> + cc * 64), v);
                        b[n][0] = __byte_perm(v[0], v[2], 0x5410);   // k 0, 4
                        b[n][1] = __byte_perm(v[0], v[2], 0x7632);   // k 1, 5
                        b[n][2] = __byte_perm(v[1], v[3], 0x5410);   // k 2, 6
                        b[n][3] = __byte_perm(v[1], v[3], 0x7632);   // k 3, 7
                        ptx::mma16816<T>(xs[n], ones, b[n][0], b[n][1]);
                        ptx::mma16816<T>(xs[n], ones, b[n][2], b[n][3]);
                    }
                }
#pragma unroll
                for (int j = 0; j < MT; ++j) {
                    const int tile = mg + j * mw;
                    if (tile < tiles) {
                        uint32_t m[2];   // codes of rows g and g + 8
                        ptx::ldmatrix_x2(w_row + static_cast<uint32_t>(tile * 2048 + ((cc ^ r) << 4)), m);
                        uint32_t a[4];
                        a[0] = (m[0] & 0x000f000fu) | kOr;
                        a[1] = (m[1] & 0x000f000fu) | kOr;
                        a[2] = ((m[0] >> 4) & 0x000f000fu) | kOr;
                        a[3] = ((m[1] >> 4) & 0x000f000fu) | kOr;
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            if (n < nt) ptx::mma16816<T>(p[j][n], a, b[n][0], b[n][1]);
                        a[0] = ((m[0] >> 8) & 0x000f000fu) | kOr;
                        a[1] = ((m[1] >> 8) & 0x000f000fu) | kOr;
                        a[2] = ((m[0] >> 12) & 0x000f000fu) | kOr;
                        a[3] = ((m[1] >> 12) & 0x000f000fu) | kOr;
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            if (n < nt) ptx::mma16816<T>(p[j][n], a, b[n][2], b[n][3]);
                    }
                }
            }
            const int grp = c / chunks_per_group;
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                const int tile = mg + j * mw;
                if (tile < tiles) {
                    const uint32_t at = static_cast<uint32_t>((grp * side.cap + tile * side.tile_step + g) * 2);
                    float s[2], o[2];
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        s[q] = Elem<T>::lo(ptx::ld_shared_u16(side.scales[q] + at));
                        const float z = has_zeros ? Elem<T>::lo(ptx::ld_shared_u16(side.zeros[q] + at)) : 8.0f;
                        o[q] = -s[q] * (z + kOffset);
                        s[q] *= kUnit;
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        if (n < nt) {
                            acc[j][n][0] += fmaf(s[0], p[j][n][0], o[0] * xs[n][0]);
                            acc[j][n][1] += fmaf(s[0], p[j][n][1], o[0] * xs[n][1]);
                            acc[j][n][2] += fmaf(s[1], p[j][n][2], o[1] * xs[n][0]);
                            acc[j][n][3] += fmaf(s[1], p[j][n][3], o[1] * xs[n][1]);
                        }
                    }
                }
            }
        }
    }
};

}  // namespace gemm_gb300
