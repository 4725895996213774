// w4_tiles.cuh -- D = A·Bᵀ with B in 4 bits and more than a few rows of A, on
// tcgen05: 128 rows of weights x up to 256 rows of A per CTA.
//
// The operands swap roles (D^T = B A^T), so that decoded weights are the MMA's
// left operand, which tcgen05 takes from TMEM: codes go smem -> registers ->
// TMEM and never back through shared memory, whose bandwidth the right
// operand needs (A rows, staged by TMA, K-major, 128-byte swizzle).  TMEM lane
// = weight row, so a decoding thread owns one row: its codes are 32
// contiguous bytes per K block of 64, its scale one number per group.
// The K loop runs in steps of KB blocks of 64 k.  A step costs the issuing warp
// some 330 clocks beside its MMAs, so with few of these it takes two blocks: 65 to
// 128 rows.  With more rows the MMAs are longer and shared memory holds four
// single blocks (M = 512: 46 us; two double ones 60); with PAIRS a block is two
// operands, and TMEM holds four single blocks.
//   warps 0-15  four warpgroups: group g decodes every fourth step, in registers
//               while the MMAs catch up, then into TMEM (tcgen05.st); later they
//               read the accumulator out
//   warp 16     TMA: A
//   warp 18     TMA: codes and scales in atoms of 256 k, as far ahead as their
//               slots allow (behind the A loads of one producer they came too late:
//               512 x 8192 x 8192 57 us)
//   warp 17     issues tcgen05.mma (M = 128, N = A rows, K = 16): the whole warp
//               walks the loop and one elected lane issues, so that descriptors stay
//               in uniform registers (from a loop in one thread's branch an MMA took
//               57 clocks to issue: M = 48, 8192 x 8192 35 us instead of 24)
// A weight is s * (code - z): code - z and the product each one rounded step in
// the activations' type (the first exact for whole and half zero points).
// For M > 64 that product is the operand.  For fewer rows, where the MMA is not
// what bounds, PAIRS makes the products exact: what the rounding left (one fma)
// is a second operand beside the first, and both are multiplied with the same A
// (with the two parts in lanes 0-63 and 64-127 of one operand every weight was
// decoded twice: 40 us).
// Split K.  With fewer tiles than SMs a cluster of S CTAs shares a tile's K
// loop; the fp32 partial sums meet in distributed shared memory and are added
// in ascending order, so results are reproducible.
// Measured, 8192 x 8192 weights, bf16: M = 17 22 us, 48 24 us, 96 19 us, 512 46 us
// (1.5 PFLOP/s; the MMAs alone would take 36).  Up to 128 rows the chain of a step
// bounds it -- decoded weights into TMEM, MMAs, the stage handed back -- with the
// MMA pipe and HBM both under a third of their rates.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "epilogue.cuh"
#include "llm/stream.cuh"
#include "ptx.cuh"
#include "wait.cuh"

namespace gemm_gb300 {

constexpr int kTileGroups = 4;          // decoding warpgroups
constexpr int kDecodeWarps = 4 * kTileGroups;
constexpr int kTileThreads = 32 * (kDecodeWarps + 3);
// Steps in flight: weights in TMEM, A in shared memory, one stage per group.  Every
// wait here is by parity, which tells a slot's uses apart only for a waiter that
// has seen each of them complete, so a slot's uses always belong to the same
// waiters; the code slots are even in number because with KB = 2 a group reads
// every second atom.
constexpr int kTileStages = kTileGroups;
constexpr int kTileRows = 128;          // weight rows per tile, one per TMEM lane
constexpr int kTileCodes = 8;           // code atoms in flight, at most
constexpr int kTileTmemCols = 512;      // accumulator: columns 0-255; weights of stage s: 32 KB columns at 256 + 32 KB s
constexpr uint32_t kSiteTileCodes = 13, kSiteTileMma = 14, kSiteTileDone = 15, kSiteTileEmpty = 16;

struct TileParams {
    int32_t M, N, K;
    int32_t rows_a;          // rows of A per tile: MMA N, a multiple of 16, <= 256
    int32_t codes;           // code atoms in flight
    int32_t m_tiles, split;
    int32_t atoms;           // code atoms over K
    int32_t atom_groups;     // 256 / group
    int32_t group;
    int32_t has_zeros, stream_w;
    int32_t side_bytes;      // scales of one atom (zero points behind them)
    int32_t codes_off, side_off, end;   // shared memory, A slots first
    uint32_t ab_format;
    void* D;
    EpiParams epi;
    uint32_t* status;
    uint64_t timeout_ns;
};

namespace ptx {

// D(tmem) (+)= A(tmem) * B(smem desc)^T, 16-bit inputs, fp32 accumulator
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        :: "r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}

// Each thread writes 32 consecutive 32-bit TMEM columns of its lane.
__device__ __forceinline__ void tmem_st_x32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0],"
        " {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
        :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
           "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
           "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]),
           "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

}  // namespace ptx

// Two numbers of T at once.
template <class T>
struct Pair;
template <>
struct Pair<__half> {
    static constexpr uint32_t kBase = 0x64006400u;     // 1024 + code in the low bits
    static constexpr uint32_t kMinusBase = 0xE400E400u, kMinusBase8 = 0xE408E408u;   // -1024, -1032
    __device__ __forceinline__ static uint32_t add(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    __device__ __forceinline__ static uint32_t mul(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    __device__ __forceinline__ static uint32_t fma(uint32_t a, uint32_t b, uint32_t c) {
        uint32_t r;
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
        return r;
    }
    __device__ __forceinline__ static uint32_t neg(uint32_t a) {
        uint32_t r;
        asm("neg.f16x2 %0, %1;" : "=r"(r) : "r"(a));
        return r;
    }
};
template <>
struct Pair<__nv_bfloat16> {
    static constexpr uint32_t kBase = 0x43004300u;     // 128 + code
    static constexpr uint32_t kMinusBase = 0xC300C300u, kMinusBase8 = 0xC308C308u;   // -128, -136
    __device__ __forceinline__ static uint32_t add(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    __device__ __forceinline__ static uint32_t mul(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    __device__ __forceinline__ static uint32_t fma(uint32_t a, uint32_t b, uint32_t c) {
        uint32_t r;
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
        return r;
    }
    __device__ __forceinline__ static uint32_t neg(uint32_t a) {
        uint32_t r;
        asm("neg.bf16x2 %0, %1;" : "=r"(r) : "r"(a));
        return r;
    }
};

template <class T, bool PAIRS, int KB>
__global__ void __launch_bounds__(kTileThreads, 1)
w4_tiles_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmS,
                const __grid_constant__ CUtensorMap tmZ, const __grid_constant__ CUtensorMap tmA, const TileParams p) {
    static_assert(!PAIRS || KB == 1, "a stage has 64 columns of TMEM at most");
    constexpr uint32_t kStageCols = PAIRS ? 64 : 32 * KB;   // PAIRS: the remainders behind the products
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    const uint32_t base = ptx::smem_u32(smem);
    // per stage: A landed and weights decoded, MMAs done; per code atom: landed, read; all MMAs done
    __shared__ __align__(8) uint64_t bars[2 * kTileStages + 2 * kTileCodes + 1];
    __shared__ uint32_t tmem_slot;
    const uint32_t bar0 = ptx::smem_u32(bars);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (kTileStages + s); };
    auto c_full = [&](int c) { return bar0 + 8u * (2 * kTileStages + c); };
    auto c_empty = [&](int c) { return bar0 + 8u * (2 * kTileStages + kTileCodes + c); };
    const uint32_t done = bar0 + 8u * (2 * kTileStages + 2 * kTileCodes);
    if (warp == kDecodeWarps && lane == 0) {
        ptx::prefetch_tensormap(&tmW);
        ptx::prefetch_tensormap(&tmA);
        for (int s = 0; s < kTileStages; ++s) {
            ptx::mbar_init(full(s), 5);   // the group's warps, and the byte count of A
            ptx::mbar_init(empty(s), 1);
        }
        for (int c = 0; c < kTileCodes; ++c) {
            ptx::mbar_init(c_full(c), 1);
            ptx::mbar_init(c_empty(c), 16 / KB);   // an atom is 4 / KB steps of 4 warps each
        }
        ptx::mbar_init(done, 1);
        ptx::fence_mbar_init();
    }
    if (warp == kDecodeWarps + 1) {
        ptx::tmem_alloc<1>(ptx::smem_u32(&tmem_slot), kTileTmemCols);
        ptx::tmem_relinquish<1>();
    }
    const int S = p.split;
    const int j = static_cast<int>(blockIdx.x % S);
    const int64_t tile = blockIdx.x / S;
    const int m0 = static_cast<int>(tile % p.m_tiles) * p.rows_a;
    const int n0 = static_cast<int>(tile / p.m_tiles) * kTileRows;
    const int at0 = static_cast<int>(static_cast<int64_t>(j) * p.atoms / S);
    const int at1 = static_cast<int>(static_cast<int64_t>(j + 1) * p.atoms / S);
    // this CTA's K blocks, KB to a step (the last atom's end may pass 2^31)
    const int blocks = at1 < p.atoms ? (at1 - at0) * 4 : (p.K - at0 * 256 - 1) / 64 + 1;
    const int steps = (blocks + KB - 1) / KB;
    ptx::tc_fence_before();
    if (S > 1) ptx::cluster_sync(); else __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&tmem_slot);
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const uint32_t a_bytes = static_cast<uint32_t>(p.rows_a) * 128u;
    bool ok = true;

    if (warp == kDecodeWarps) {
        // ------------------------------------------------------------ producer (one thread)
        if (lane == 0) {
            const uint64_t pol_a = ptx::policy_evict_last();
            int s = 0;
            uint32_t ph = 1;   // a slot's first use waits for nothing
            for (int b = 0; b < blocks; b += KB) {
                if (!wait_phase(empty(s), ph, p.status, kSiteTileEmpty, p.timeout_ns)) {
                    ok = false;
                    break;
                }
                const int n = min(KB, blocks - b);
                ptx::mbar_arrive_expect_tx(full(s), n * a_bytes);
                for (int i = 0; i < n; ++i)
                    ptx::tma_load_2d_hint(base + (KB * s + i) * a_bytes, &tmA, full(s), at0 * 256 + (b + i) * 64, m0, pol_a);
                if (++s == kTileStages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            if (!ok) {   // leave no copy in flight behind
                for (uint32_t q = 0; q < 2; ++q)
                    for (int i = 0; i < kTileStages; ++i) wait_phase(full(i), q, p.status, kSiteStreamDrain, 1000000);
            }
        }
        __syncwarp();
    } else if (warp == kDecodeWarps + 2) {
        // ------------------------------------------------------------ codes and scales (one thread)
        if (lane == 0) {
            const uint64_t pol_w = p.stream_w ? ptx::policy_evict_first() : ptx::policy_evict_normal();
            const uint32_t tx = static_cast<uint32_t>(kTileRows) * 128u +
                                static_cast<uint32_t>(kTileRows * p.atom_groups * 2) * (p.has_zeros ? 2u : 1u);
            int c = 0;
            uint32_t ph = 1;
            for (int at = at0; at < at1; ++at) {
                if (!wait_phase(c_empty(c), ph, p.status, kSiteTileCodes, p.timeout_ns)) {
                    ok = false;
                    break;
                }
                const uint32_t side = base + static_cast<uint32_t>(p.side_off + c * 2 * p.side_bytes);
                ptx::mbar_arrive_expect_tx(c_full(c), tx);
                ptx::tma_load_2d_hint(base + static_cast<uint32_t>(p.codes_off + c * kTileRows * 128), &tmW, c_full(c), at * 128, n0, pol_w);
                ptx::tma_load_2d(side, &tmS, c_full(c), n0, at * p.atom_groups);
                if (p.has_zeros) ptx::tma_load_2d(side + static_cast<uint32_t>(p.side_bytes), &tmZ, c_full(c), n0, at * p.atom_groups);
                if (++c == p.codes) {
                    c = 0;
                    ph ^= 1u;
                }
            }
            if (!ok) {
                for (uint32_t q = 0; q < 2; ++q)
                    for (int i = 0; i < p.codes; ++i) wait_phase(c_full(i), q, p.status, kSiteStreamDrain, 1000000);
            }
        }
        __syncwarp();
    } else if (warp == kDecodeWarps + 1) {
        // ------------------------------------------------------------ MMA issue
        // (whole warp, one elected lane issues: with the loop in one thread's branch
        // the descriptors go through vector registers)
        const uint32_t idesc = ptx::instr_desc(128, p.rows_a, p.ab_format);
        int s = 0;
        uint32_t ph = 0;
        for (int b = 0; b < blocks; b += KB) {
            if (!wait_phase_warp(full(s), ph, p.status, kSiteTileMma, p.timeout_ns)) {
                ok = false;
                break;
            }
            ptx::tc_fence_after();
            const uint32_t a = base + KB * s * a_bytes, w = tmem + 256u + kStageCols * s;
            if (ptx::elect_one()) {
#pragma unroll
                for (int i = 0; i < KB; ++i) {
                    if (b + i < blocks) {
                        const uint64_t x = ptx::sw128_kmajor_desc(a + i * a_bytes);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            ptx::mma_f16_ts(tmem, w + 32u * i + 8u * k, x + 2u * k, idesc, (b != 0 || i != 0 || k != 0) ? 1u : 0u);
                        if constexpr (PAIRS) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) ptx::mma_f16_ts(tmem, w + 32u + 8u * k, x + 2u * k, idesc, 1u);
                        }
                    }
                }
                ptx::mma_commit(empty(s));
            }
            __syncwarp();
            if (++s == kTileStages) {
                s = 0;
                ph ^= 1u;
            }
        }
        // also after a wait that gave up: the MMAs issued so far
        if (ptx::elect_one()) ptx::mma_commit(done);
        __syncwarp();
        wait_phase_warp(done, 0, p.status, kSiteTileDone, p.timeout_ns);
    } else {
        // ------------------------------------------------------------ decode
        const int wg = warp >> 2, q = warp & 3;
        const int row = q * 32 + lane;                      // weight row within the tile, and TMEM lane
        const uint32_t lane_addr = tmem + (static_cast<uint32_t>(q * 32) << 16);
        const uint32_t mask = ptx::opaque(0x000f000fu), kb = ptx::opaque(Pair<T>::kBase);
        const int g_shift = p.group == 32 ? 5 : (p.group == 64 ? 6 : 7);
        for (int t = wg; t < steps; t += kTileGroups) {
            const int i = t / (4 / KB), c_use = i / p.codes, c = i - c_use * p.codes, use = t / kTileStages, s = wg;
            const int part = t % (4 / KB);   // of the atom
            if (!wait_phase_warp(c_full(c), c_use & 1, p.status, kSiteTileCodes, p.timeout_ns)) {
                ok = false;
                break;
            }
            const uint32_t there = base + ptx::stage_token();
            const uint32_t codes = there + static_cast<uint32_t>(p.codes_off + (c * kTileRows + row) * 128);
            uint32_t w[8 * KB];
#pragma unroll
            for (int v = 0; v < 2 * KB; ++v) {
                uint32_t x[4];
                ptx::ld_shared_u4<0>(codes + static_cast<uint32_t>(((part * 2 * KB + v) ^ (row & 7)) << 4), x);
#pragma unroll
                for (int u = 0; u < 4; ++u) w[4 * v + u] = x[u];
            }
            // scale and minus zero point of each 32 k, in both halves of a register
            uint32_t sc[2 * KB], zr[2 * KB];
#pragma unroll
            for (int h = 0; h < 2 * KB; ++h) {
                const int grp = (part * 64 * KB + h * 32) >> g_shift;
                const uint32_t at = there + static_cast<uint32_t>(p.side_off + c * 2 * p.side_bytes + (grp * kTileRows + row) * 2);
                sc[h] = ptx::ld_shared_u16<0>(at) * 0x10001u;
                zr[h] = p.has_zeros ? ((ptx::ld_shared_u16<0>(at + static_cast<uint32_t>(p.side_bytes)) * 0x10001u) ^ 0x80008000u) : 0u;
            }
            // code words and scales are in registers: the atom may be refilled
#pragma unroll
            for (int v = 0; v < 8 * KB; ++v) asm volatile("" : "+r"(w[v]) :: "memory");
#pragma unroll
            for (int h = 0; h < 2 * KB; ++h) asm volatile("" : "+r"(sc[h]), "+r"(zr[h]) :: "memory");
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(c_empty(c));
#pragma unroll
            for (int blk = 0; blk < KB; ++blk) {
                if (KB * t + blk >= blocks) break;
                uint32_t r[32];
                [[maybe_unused]] uint32_t rest[PAIRS ? 32 : 1];   // what rounding the products left
#pragma unroll
                for (int v = 0; v < 8; ++v) {
                    const uint32_t word = w[8 * blk + v], odd = word >> 4, sv = sc[2 * blk + (v >> 2)];
                    // codes 2 u and 2 u + 1 in the low bits of each half
                    const uint32_t x[4] = {__byte_perm(word, odd, 0x0400), __byte_perm(word, odd, 0x0501),
                                           __byte_perm(word, odd, 0x0602), __byte_perm(word, odd, 0x0703)};
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        uint32_t d = ptx::and_or(x[u], mask, kb);
                        if (p.has_zeros) d = Pair<T>::add(Pair<T>::add(d, Pair<T>::kMinusBase), zr[2 * blk + (v >> 2)]);
                        else d = Pair<T>::add(d, Pair<T>::kMinusBase8);
                        const uint32_t prod = Pair<T>::mul(d, sv);
                        r[4 * v + u] = prod;
                        if constexpr (PAIRS) rest[4 * v + u] = Pair<T>::fma(d, sv, Pair<T>::neg(prod));
                    }
                }
                if (blk == 0) {
                    if (use > 0 && !wait_phase_warp(empty(s), (use & 1) ^ 1u, p.status, kSiteTileEmpty, p.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                }
                const uint32_t to = lane_addr + 256u + kStageCols * s + 32u * blk;
                ptx::tmem_st_x32(to, r);
                if constexpr (PAIRS) ptx::tmem_st_x32(to + 32u, rest);
            }
            if (!ok) break;
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(full(s));
        }
    }

    // ---------------------------------------------------------------- output
    T* D = static_cast<T*>(p.D);
    const int cols = p.rows_a;
    if (warp < kDecodeWarps) {
        if (!wait_phase_warp(done, 0, p.status, kSiteTileDone, p.timeout_ns)) ok = false;
        ptx::tc_fence_after();
    }
    const int wg = warp >> 2, q = warp & 3, l = q * 32 + lane;
    const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16);
    if (S == 1) {
        if (warp < kDecodeWarps) {
            const int64_t n = n0 + l;
            const bool in = n < p.N;
            EpiColumnFactors<T> cf;
            if (p.epi.on && in) cf.load(p.epi, n);
            // the warpgroups share the columns, 16 at a time
            for (int c0 = wg * 16; c0 < cols; c0 += 16 * kTileGroups) {
                uint32_t v[16];
                ptx::tmem_ld_x16(acc + static_cast<uint32_t>(c0), v);
                ptx::tmem_wait_ld();
                if (in) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int64_t m = m0 + c0 + i;
                        if (m < p.M) {
                            float x = __uint_as_float(v[i]);
                            if (p.epi.on) x = cf.apply(p.epi, x, m, n, p.N);
                            D[m * p.N + n] = Elem<T>::from_float(x);
                        }
                    }
                }
            }
        }
    } else {
        // CTA d of the cluster finishes columns [d per, (d + 1) per); its receive
        // buffer, over the operand slots that nobody needs any more, is
        // [S][per / 4][128 lanes][4 columns].
        const int per = (cols / 16 + S - 1) / S * 16;
        __syncwarp();
        ptx::cluster_sync();   // every MMA and copy of the cluster is done
        if (warp < kDecodeWarps) {
            for (int c0 = wg * 16; c0 < cols; c0 += 16 * kTileGroups) {
                uint32_t v[16];
                ptx::tmem_ld_x16(acc + static_cast<uint32_t>(c0), v);
                ptx::tmem_wait_ld();
                const int d = c0 / per;
                const uint32_t to = base + static_cast<uint32_t>((((j * per + c0 - d * per) >> 2) * 128 + l) * 16);
                const uint32_t peer = ptx::mapa(to, static_cast<uint32_t>(d));
#pragma unroll
                for (int i = 0; i < 16; i += 4) ptx::st_cluster_v4(peer + static_cast<uint32_t>(i * 512), v[i], v[i + 1], v[i + 2], v[i + 3]);
            }
        }
        ptx::cluster_sync();
        const int mine = min(per, cols - j * per);
        for (int e = threadIdx.x; e < (mine >> 2) * kTileRows; e += kTileThreads) {
            const int c = e / kTileRows * 4, r = e % kTileRows;
            const int64_t m = m0 + j * per + c, n = n0 + r;
            if (n >= p.N) continue;
            float x[4] = {};
            for (int i = 0; i < S; ++i) {
                float t[4];
                const uint32_t at = base + static_cast<uint32_t>((((i * per + c) >> 2) * 128 + r) * 16);
                ptx::ld_shared_v4(at, t);
#pragma unroll
                for (int q2 = 0; q2 < 4; ++q2) x[q2] += t[q2];
            }
#pragma unroll
            for (int q2 = 0; q2 < 4; ++q2) {
                if (m + q2 < p.M) {
                    if (p.epi.on) x[q2] = epi_apply1<T>(p.epi, x[q2], m + q2, n, p.N);
                    D[(m + q2) * p.N + n] = Elem<T>::from_float(x[q2]);
                }
            }
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == kDecodeWarps + 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc<1>(tmem, kTileTmemCols);
    }
}

}  // namespace gemm_gb300
