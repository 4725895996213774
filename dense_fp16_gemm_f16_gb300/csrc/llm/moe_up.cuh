// moe_up.cuh -- the first products of the chosen experts and what follows
// them: h = silu(G x) * (U x) for every (token, expert) pair.
//
// Work split.  The gate rows of all segments, in granules of 8, form one list
// that the CTAs (one per SM or two) share evenly; each granule brings the 8 up rows that
// belong to it, as the other half of a 16-row MMA tile, so both sums of an h
// lie in one thread.  A CTA takes its granules in pieces of up to 4 of one
// expert, each piece over all of K: no sums cross CTAs.  The stage groups' sums
// of a piece meet in shared memory, where the gated product is formed in fp32,
// while the copies of the next pieces are in flight.
// h goes to the second product as the sum of two numbers of the activations'
// type, rows 2 s and 2 s + 1 for slot s: one rounding to 16 bits here would cost
// as much accuracy as the output's own, and two columns instead of one are
// nearly free where weights set the pace.
// Measured: 8 experts of 2 x 8200 x 4096 in 16 bits (1.07 GB), 16 tokens: 167 us,
// 6.4 TB/s, bound by HBM.  64 experts of 2 x 1408 x 2048 in 4 bits (185 MB), 64
// tokens: 96 us, bound by the eight warps' chains from codes to sums (1.5 of 4
// instructions per clock; 16 warps with half the registers: 107 us).
#pragma once

#include "llm/lists.cuh"
#include "llm/llm.h"
#include "llm/rows.cuh"
#include "llm/stream.cuh"

namespace gemm_gb300 {

constexpr int kUpGranules = 4;                    // granules per piece
constexpr int kUpRows = kUpGranules * 16;         // rows of gate and up together
constexpr int kUpPitch = kUpRows + 8;

struct UpParams {
    CUtensorMap tm_piece;         // the weights in boxes of kUpGranules granules (tmW: of one)
    RingLayout ring;
    int32_t list_off, sums_off;
    int32_t x_resident, x_off, x_pitch;   // 4-bit weights: a segment's columns, all K
    int32_t H, I, k_stages, mw;
    int32_t groups_k, atom_groups, has_zeros;
    int32_t stream_w;
    const void* X;                // [T][H]
    void* h;                      // [2 T k][I]
    const int32_t* ids;
    const float* weights;
    int32_t T, k, E;
    uint32_t* status;
    uint64_t timeout_ns;
};

// A CTA's pieces, one after the other: granules [at, at + count) of segment seg.
struct UpPieces {
    int64_t pos, end;
    int per_seg;   // granules of one segment
    __device__ __forceinline__ bool next(int& seg, int& at, int& count) {
        if (pos >= end) return false;
        seg = static_cast<int>(pos / per_seg);
        at = static_cast<int>(pos - static_cast<int64_t>(seg) * per_seg);
        const int run = static_cast<int>(min(static_cast<int64_t>(per_seg - at), end - pos));
        const int pieces = (run + kUpGranules - 1) / kUpGranules;
        count = (run + pieces - 1) / pieces;
        pos += count;
        return true;
    }
};

template <class T, int CPG, int NT>
__global__ void __launch_bounds__(kStreamThreads, kCtasPerSm<(CPG != 0), NT, true>)
moe_up_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmS,
              const __grid_constant__ CUtensorMap tmZ, const __grid_constant__ UpParams p) {
    constexpr bool W4 = CPG != 0;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    const uint32_t base = ptx::smem_u32(smem);
    __shared__ __align__(8) uint64_t bars[2 * kMaxRing];
    const uint32_t bar0 = ptx::smem_u32(bars);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int KW = kConsumers / p.mw;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (kMaxRing + s); };
    if (warp == 0 && lane == 0) {
        ptx::prefetch_tensormap(&tmW);
        ptx::prefetch_tensormap(&p.tm_piece);
    }
    if (static_cast<int>(threadIdx.x) < p.ring.slots) {
        ptx::mbar_init(full_bar(threadIdx.x), p.x_resident ? 1u : full_arrivals(p.mw));
        ptx::mbar_init(empty_bar(threadIdx.x), static_cast<uint32_t>(p.mw));
        ptx::fence_mbar_init();
    }
    ptx::griddep_wait();
    // from here on everything before this kernel is complete, which is what the
    // second product's early reads rely on
    ptx::griddep_launch_dependents();
    const SlotLists lists = build_lists(p.ids, p.weights, p.T, p.k, p.E, NT * 8, smem + p.list_off);
    const int per_seg = p.I / 8;
    const int64_t total = static_cast<int64_t>(lists.nseg) * per_seg;
    const UpPieces all{total * blockIdx.x / gridDim.x, total * (blockIdx.x + 1) / gridDim.x, per_seg};

    constexpr int KE = kAtomElems<W4>;
    const int pitch = p.x_resident ? p.x_pitch : col_pitch(W4, 1);
    const int mg = warp % p.mw, kg = warp / p.mw;
    const GroupSlots own(p.ring.slots, KW, kg);
    const uint64_t pol_w = p.stream_w ? ptx::policy_evict_first() : ptx::policy_evict_normal();
    const uint32_t side_half = static_cast<uint32_t>(kUpGranules * 8 * p.atom_groups * 2);
    constexpr uint32_t kHalf = kUpGranules * 1024;   // up rows behind the gate rows

    // The copies of one stage (K atom kb of a piece) into slot s.
    auto issue = [&](int seg, int at, int count, int kb, int s) {
        const int first = lists.seg_begin[seg], n = lists.seg_begin[seg + 1] - first;
        const int e = lists.seg_e[seg];
        const int kv = min(KE, p.H - kb * KE);
        if (mg == 0) {
            if (lane == 0)
                ptx::mbar_arrive_expect_tx(full_bar(s), static_cast<uint32_t>(count) * 2048u +
                                                            (W4 ? 2u * side_half * (p.has_zeros ? 2u : 1u) : 0u));
            __syncwarp();
            const int32_t y = e * 2 * p.I + at * 8 + ((lane & 1) ? p.I : 0);   // even lanes: gate rows, odd lanes: up rows
            const uint32_t dst = base + static_cast<uint32_t>(s * p.ring.w_bytes) + (lane & 1) * kHalf;
            if (count == kUpGranules) {
                if (lane < 2) ptx::tma_load_2d_hint(dst, &p.tm_piece, full_bar(s), kb * (W4 ? 128 : 64), y, pol_w);
            } else if (lane < 2 * count) {
                ptx::tma_load_2d_hint(dst + (lane >> 1) * 1024u, &tmW, full_bar(s), kb * (W4 ? 128 : 64),
                                      y + (lane >> 1) * 8, pol_w);
            }
            if constexpr (W4) {
                // [scales | zero points] x [gate | up] x [groups][32 rows]
                const int q = lane - 8;
                if (q >= 0 && q < (p.has_zeros ? 4 : 2)) {
                    const int side = p.ring.side_off + s * p.ring.side_bytes + (q >> 1) * (p.ring.side_bytes / 2);
                    ptx::tma_load_2d(base + static_cast<uint32_t>(side) + (q & 1) * side_half, (q >> 1) ? &tmZ : &tmS,
                                     full_bar(s), at * 8 + ((q & 1) ? p.I : 0), e * p.groups_k + kb * p.atom_groups);
                }
            }
        }
        if (p.x_resident) return;
        const uint32_t x = base + static_cast<uint32_t>(p.ring.x_off + s * p.ring.x_bytes);
        constexpr int kShift = W4 ? 5 : 3;   // 32 or 8 pieces of 16 bytes per column
        for (int i = mg * 32 + lane; i < (n << kShift); i += 32 * p.mw) {   // the group's warps share them
            const int c = i >> kShift, o = (i - (c << kShift)) * 8;
            if (o < kv) {
                const int64_t token = lists.slot[first + c] / p.k;
                ptx::cp_async16(x + static_cast<uint32_t>(c * pitch + o * 2),
                                static_cast<const T*>(p.X) + token * p.H + static_cast<int64_t>(kb) * KE + o);
            }
        }
        ptx::cp_async_arrive(full_bar(s));
    };
    // The group's next stage to fetch: it walks the pieces ahead of the sums.
    UpPieces ahead = all;
    int f_seg = 0, f_at = 0, f_count = 0, f_kb = kg - KW;
    bool f_more = ahead.next(f_seg, f_at, f_count);
    auto fetch_next = [&](int s) {
        f_kb += KW;
        while (f_more && f_kb >= p.k_stages) {
            f_kb -= p.k_stages;
            f_more = ahead.next(f_seg, f_at, f_count);
        }
        if (f_more) issue(f_seg, f_at, f_count, f_kb, s);
        return f_more;
    };

    {
        const int g = lane >> 2, t = lane & 3;
        constexpr int kCols = 8 * NT;
        const int tile0 = mg * StreamWarp<T, W4, NT, true>::MT;   // this warp's tiles
        float* sums = reinterpret_cast<float*>(smem + p.sums_off);
        T* h = static_cast<T*>(p.h);
        for (int d = 0; d < own.depth; ++d)
            if (!fetch_next(own.first + d)) break;
        StreamWarp<T, W4, NT, true> sw;
        bool ok = true;
        int d = 0, kb = kg;
        uint32_t phase = 0;
        UpPieces pieces = all;
        int seg, at, count, x_seg = -1;
        while (pieces.next(seg, at, count)) {
            const int first = lists.seg_begin[seg], n = lists.seg_begin[seg + 1] - first;
            const int nt = (n + 7) >> 3;
            if (p.x_resident && seg != x_seg) {
                // nobody reads the last segment's columns any more: the sums'
                // barriers are behind every warp
                x_seg = seg;
                const int pieces16 = p.H >> 3;
                for (int c = warp; c < n; c += kConsumers) {
                    const T* src = static_cast<const T*>(p.X) + static_cast<int64_t>(lists.slot[first + c] / p.k) * p.H;
                    const uint32_t dst = base + static_cast<uint32_t>(p.x_off + c * p.x_pitch);
                    for (int o = lane; o < pieces16; o += 32) ptx::cp_async16(dst + o * 16u, src + o * 8);
                }
                ptx::cp_async_wait_all();
                __syncthreads();
            }
            sw.clear();
            for (; ok && kb < p.k_stages; kb += KW) {
                const int s = own.first + d;
                if (!wait_phase_warp(full_bar(s), phase, p.status, kSiteStreamFull, p.timeout_ns)) {
                    ok = false;
                    break;
                }
                const int kv = min(KE, p.H - kb * KE);
                const uint32_t there = base + ptx::stage_token();
                const uint32_t w = there + static_cast<uint32_t>(s * p.ring.w_bytes + tile0 * 1024);
                const uint32_t x = there + static_cast<uint32_t>(p.x_resident ? p.x_off + kb * KE * 2 : p.ring.x_off + s * p.ring.x_bytes);
                if constexpr (W4) {
                    const uint32_t sc = there + static_cast<uint32_t>(p.ring.side_off + s * p.ring.side_bytes + tile0 * 16);
                    const SideView side{sc, sc + static_cast<uint32_t>(p.ring.side_bytes / 2), side_half, kUpGranules * 16u};
                    sw.template atom4<CPG, 1024, 16>(w, kHalf, x, pitch, side, p.has_zeros != 0, kv, count - tile0, nt, lane);
                } else {
                    sw.template atom16<1024>(w, kHalf, x, pitch, kv, count - tile0, nt, lane);
                }
                sw.hold();
                __syncwarp();
                if (p.mw > 1) {
                    if (lane == 0) ptx::mbar_arrive(empty_bar(s));
                    if (f_more && !wait_phase_warp(empty_bar(s), phase, p.status, kSiteStreamEmpty, p.timeout_ns)) {
                        ok = false;
                        break;
                    }
                }
                if (f_more) fetch_next(s);
                if (++d == own.depth) {
                    d = 0;
                    phase ^= 1u;
                }
            }
            kb -= p.k_stages;   // where this group's stages go on in the next piece
            // [stage group][column][tile * 16 + (gate: g, up: 8 + g)]
            float* mine = sums + kg * kCols * kUpPitch;
#pragma unroll
            for (int jt = 0; jt < sw.MT; ++jt) {
                const int tile = tile0 + jt;
                if (tile < count) {
#pragma unroll
                    for (int q = 0; q < NT; ++q) {
                        if (q < nt) {
                            float* to = mine + (q * 8 + 2 * t) * kUpPitch + tile * 16 + g;
                            to[0] = sw.acc[jt][q][0];
                            to[kUpPitch] = sw.acc[jt][q][1];
                            to[8] = sw.acc[jt][q][2];
                            to[kUpPitch + 8] = sw.acc[jt][q][3];
                        }
                    }
                }
            }
            __syncthreads();
            const int rows = count * 8;
            for (int e = threadIdx.x; e < n * rows; e += kConsumers * 32) {
                const int c = e / rows, r = e - c * rows;
                const float* a = sums + c * kUpPitch + (r >> 3) * 16 + (r & 7);
                float gate = a[0], up = a[8];
                for (int q = 1; q < KW; ++q) {
                    gate += a[q * kCols * kUpPitch];
                    up += a[q * kCols * kUpPitch + 8];
                }
                const float v = gate / (1.0f + expf(-gate)) * up;
                const T hi = Elem<T>::from_float(v);
                const float back = Elem<T>::to_float(hi);
                const int64_t to = 2 * static_cast<int64_t>(lists.slot[first + c]) * p.I + at * 8 + r;
                h[to] = hi;
                // past the type's largest number the first part is infinite and stays the value
                h[to + p.I] = Elem<T>::from_float(isfinite(back) ? v - back : 0.0f);
            }
            __syncthreads();   // the next piece's sums go to the same place
        }
        if (!ok && mg == 0) {   // leave no copy in flight behind
            for (int q = 0; q < own.depth; ++q)
                for (uint32_t ph = 0; ph < 2; ++ph)
                    wait_phase(full_bar(own.first + q), ph, p.status, kSiteStreamDrain, 1000000);
        }
    }
}

}  // namespace gemm_gb300
