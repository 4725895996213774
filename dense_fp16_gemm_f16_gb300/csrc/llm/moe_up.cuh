// moe_up.cuh -- the first products of the chosen experts and what follows
// them: h = silu(G x) * (U x) for every (token, expert) pair.
//
// Work split.  The gate rows of all segments, in granules of 8, form one list
// that the CTAs (one per SM) share evenly; each granule brings the 8 up rows that
// belong to it, as the other half of a 16-row MMA tile, so both sums of an h
// lie in one thread.  A CTA takes its granules in pieces of up to 4 of one
// expert, each piece over all of K: no sums cross CTAs.  The stage groups' sums
// of a piece meet in shared memory (two buffers in turn), where the gated
// product is formed in fp32.
// h goes to the second product as the sum of two numbers of the activations'
// type, rows 2 s and 2 s + 1 for slot s: one rounding to 16 bits here would cost
// as much accuracy as the output's own, and two columns instead of one are
// nearly free where weights set the pace.
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
    RingLayout ring;
    int32_t list_off, sums_off;
    int32_t H, I, k_stages, mw;
    int32_t groups_k, stage_groups, chunks_per_group, has_zeros;
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

template <class T, bool W4, int NT>
__global__ void __launch_bounds__(kStreamThreads, 1)
moe_up_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmS,
              const __grid_constant__ CUtensorMap tmZ, const UpParams p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    const uint32_t base = ptx::smem_u32(smem);
    __shared__ __align__(8) uint64_t bars[2 * kMaxRing];
    const uint32_t bar0 = ptx::smem_u32(bars);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int NS = p.ring.stages;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (kMaxRing + s); };
    if (warp == 0 && lane == 0) {
        ptx::prefetch_tensormap(&tmW);
        for (int s = 0; s < NS; ++s) {
            ptx::mbar_init(full_bar(s), 1);
            ptx::mbar_init(empty_bar(s), static_cast<uint32_t>(p.mw));
        }
        ptx::fence_mbar_init();
    }
    ptx::griddep_wait();
    // from here on everything before this kernel is complete, which is what the
    // second product's early reads rely on
    ptx::griddep_launch_dependents();
    const SlotLists lists = build_lists(p.ids, p.weights, p.T, p.k, p.E, NT * 8, smem + p.list_off);
    const int per_seg = p.I / 8;
    const int64_t total = static_cast<int64_t>(lists.nseg) * per_seg;
    UpPieces pieces{total * blockIdx.x / gridDim.x, total * (blockIdx.x + 1) / gridDim.x, per_seg};
    int seg, at, count;

    if (warp == kConsumers) {
        // ------------------------------------------------------------ producer
        const uint64_t pol_w = p.stream_w ? ptx::policy_evict_first() : ptx::policy_evict_normal();
        const T* X = static_cast<const T*>(p.X);
        bool ok = true;
        int i = 0;
        while (ok && pieces.next(seg, at, count)) {
            const int first = lists.seg_begin[seg], n = lists.seg_begin[seg + 1] - first;
            const int32_t gate = lists.seg_e[seg] * 2 * p.I + at * 8, up = gate + p.I;   // rows of the stack
            const uint32_t side_tx = W4 ? static_cast<uint32_t>(2 * kUpGranules * 8 * p.stage_groups * 2) * (p.has_zeros ? 2u : 1u) : 0u;
            for (int kb = 0; kb < p.k_stages; ++kb, ++i) {
                const int s = i % NS;
                if (i >= NS && !wait_phase_warp(empty_bar(s), ((i / NS) & 1) ^ 1u, p.status, kSiteStreamEmpty, p.timeout_ns)) {
                    ok = false;
                    break;
                }
                const int kv = min(kStageElems<W4>, p.H - kb * kStageElems<W4>);
                if (lane == 0)
                    ptx::mbar_arrive_expect_tx(full_bar(s), static_cast<uint32_t>(count) * 2048u + side_tx + static_cast<uint32_t>(n * kv * 2));
                __syncwarp();
                // granule i: 8 gate rows, then its 8 up rows
                if (lane < 2 * count) {
                    const int32_t y = ((lane & 1) ? up : gate) + (lane >> 1) * 8;
                    ptx::tma_load_2d_hint(base + static_cast<uint32_t>(s * p.ring.w_bytes + lane * 1024), &tmW, full_bar(s),
                                          kb * (W4 ? 128 : 64), y, pol_w);
                }
                if constexpr (W4) {
                    // [gate | up] x [groups][32 rows] of scales, then of zero points
                    const uint32_t side = base + static_cast<uint32_t>(p.ring.side_off + s * p.ring.side_bytes);
                    if (lane < (p.has_zeros ? 4 : 2)) {
                        const int x = at * 8 + ((lane & 1) ? p.I : 0);
                        ptx::tma_load_2d(side + static_cast<uint32_t>((lane >> 1) * (p.ring.side_bytes / 2) + (lane & 1) * kUpGranules * 8 * p.stage_groups * 2),
                                         (lane >> 1) ? &tmZ : &tmS, full_bar(s), x, lists.seg_e[seg] * p.groups_k + kb * p.stage_groups);
                    }
                }
                const uint32_t dst = base + static_cast<uint32_t>(p.ring.x_off + s * p.ring.x_bytes);
                for (int c = lane; c < n; c += 32)
                    ptx::bulk_load(dst + static_cast<uint32_t>(c * kColPitch<W4>),
                                   X + static_cast<int64_t>(lists.slot[first + c] / p.k) * p.H + static_cast<int64_t>(kb) * kStageElems<W4>,
                                   static_cast<uint32_t>(kv * 2), full_bar(s));
            }
        }
        if (!ok) {   // leave no copy in flight behind
            for (int s = 0; s < NS; ++s)
                for (uint32_t ph = 0; ph < 2; ++ph) wait_phase(full_bar(s), ph, p.status, kSiteStreamDrain, 1000000);
        }
    } else {
        // ------------------------------------------------------------ consumers
        const int KW = kConsumers / p.mw;
        const int mg = warp % p.mw, kg = warp / p.mw;
        const int g = lane >> 2, t = lane & 3;
        constexpr int kCols = 8 * NT;
        float* sums = reinterpret_cast<float*>(smem + p.sums_off);
        T* h = static_cast<T*>(p.h);
        StreamWarp<T, W4, NT> sw;
        bool ok = true;
        int i = 0;   // stages before this piece
        for (int buf = 0; pieces.next(seg, at, count); buf ^= 1) {
            const int first = lists.seg_begin[seg], n = lists.seg_begin[seg + 1] - first;
            const int nt = (n + 7) >> 3;
            sw.clear();
            for (int kb = (kg - i % KW + KW) % KW; ok && kb < p.k_stages; kb += KW) {
                const int s = (i + kb) % NS;
                if (!wait_phase_warp(full_bar(s), ((i + kb) / NS) & 1, p.status, kSiteStreamFull, p.timeout_ns)) {
                    ok = false;
                    break;
                }
                const int kv = min(kStageElems<W4>, p.H - kb * kStageElems<W4>);
                const uint32_t w = base + static_cast<uint32_t>(s * p.ring.w_bytes);
                const uint32_t x = base + static_cast<uint32_t>(p.ring.x_off + s * p.ring.x_bytes);
                if constexpr (W4) {
                    const uint32_t sc = base + static_cast<uint32_t>(p.ring.side_off + s * p.ring.side_bytes);
                    const uint32_t zr = sc + static_cast<uint32_t>(p.ring.side_bytes / 2);
                    const uint32_t half = static_cast<uint32_t>(kUpGranules * 8 * p.stage_groups * 2);
                    const SideView side{{sc, sc + half}, {zr, zr + half}, kUpGranules * 8, 8};
                    sw.stage4(w, x, side, p.has_zeros != 0, kv, p.chunks_per_group, count, mg, p.mw, nt, lane);
                } else {
                    sw.stage16(w, x, kv, count, mg, p.mw, nt, lane);
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(empty_bar(s));
            }
            i += p.k_stages;
            // [stage group][column][tile * 16 + (gate: g, up: 8 + g)]
            float* mine = sums + (buf * KW + kg) * kCols * kUpPitch;
#pragma unroll
            for (int jt = 0; jt < sw.MT; ++jt) {
                const int tile = mg + jt * p.mw;
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
            ptx::named_bar_sync(1, kConsumers * 32);
            // a buffer is written again only after the barrier of the piece in between
            const float* from = sums + buf * KW * kCols * kUpPitch;
            const int rows = count * 8;
            for (int e = threadIdx.x; e < n * rows; e += kConsumers * 32) {
                const int c = e / rows, r = e - c * rows;
                const float* a = from + c * kUpPitch + (r >> 3) * 16 + (r & 7);
                float gate = a[0], up = a[8];
                for (int q = 1; q < KW; ++q) {
                    gate += a[q * kCols * kUpPitch];
                    up += a[q * kCols * kUpPitch + 8];
                }
                const float v = gate / (1.0f + __expf(-gate)) * up;
                const T hi = Elem<T>::from_float(v);
                const float back = Elem<T>::to_float(hi);
                const int64_t to = 2 * static_cast<int64_t>(lists.slot[first + c]) * p.I + at * 8 + r;
                h[to] = hi;
                // past the type's largest number the first part is infinite and stays the value
                h[to + p.I] = Elem<T>::from_float(isfinite(back) ? v - back : 0.0f);
            }
        }
    }
}

}  // namespace gemm_gb300
