// rows.cuh -- out[col][row] over every row of a matrix, or of the chosen
// experts' matrices added up by token: the 4-bit product D = A·Bᵀ for few rows
// of A, and the second product of the mixture-of-experts layer.
//
// Work split.  The rows are cut into ranges of `width` (a multiple of 8), one
// per cluster of P CTAs.  All the stages of a range -- segment after segment (one
// segment in the plain product), K block after K block -- form one list, and
// CTA j of the cluster takes the j-th of P even shares of it.  Nearly all
// ranges are equally wide, so every SM streams nearly the same bytes.
// Sums.  A warp adds its registers to its own fp32 table [column or token][row]
// in shared memory whenever it moves to another segment; warps that own the
// same rows (the KW stage groups) have tables of their own, so no two threads
// ever add to one number.  At the end the tables are added in a fixed order,
// across the cluster through distributed shared memory, and each output is
// rounded once.  Results are bitwise reproducible.
#pragma once

#include "llm/lists.cuh"
#include "llm/llm.h"
#include "llm/stream.cuh"

namespace gemm_gb300 {

struct RowsParams {
    RingLayout ring;
    int32_t list_off, table_off, recv_off;   // shared-memory offsets (list only for experts)
    int32_t table_pitch;                     // floats from one column to the next
    int32_t N, K, k_stages;                  // rows of one matrix; K; stages over K
    int32_t width, ranges, pieces;           // pieces = P
    int32_t mw;                              // warps that share a stage's tiles
    int32_t groups_k;                        // K / group (4-bit)
    int32_t stage_groups, chunks_per_group;  // 256 / group, group / 32
    int32_t has_zeros;
    int32_t stream_w;                        // weights larger than L2 should hold: evict first
    int32_t cols;                            // plain: rows of A in this launch; experts: tokens T
    const void* X;                           // plain: A's rows; experts: h, rows 2 s and 2 s + 1 for slot s
    void* D;
    EpiParams epi;                           // plain
    int64_t row0;                            // plain: first row of A in this launch (for C)
    const int32_t* ids;                      // experts
    const float* weights;
    int32_t k, E;
    uint32_t* status;
    uint64_t timeout_ns;
};

template <class T, bool W4, int NT, bool MOE>
__global__ void __launch_bounds__(kStreamThreads, 1)
weight_rows_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmS,
                   const __grid_constant__ CUtensorMap tmZ, const RowsParams p) {
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
    const int KW = kConsumers / p.mw;
    float* table = reinterpret_cast<float*>(smem + p.table_off);
    const int tokens = MOE ? p.cols : 8 * NT;
    const int table_size = tokens * p.table_pitch;   // one stage group's
    for (int i = threadIdx.x; i < KW * table_size; i += kStreamThreads) table[i] = 0.0f;

    const int P = p.pieces;
    const int64_t cid = blockIdx.x / P;
    const int j = static_cast<int>(blockIdx.x % P);
    const int32_t row0 = static_cast<int32_t>(cid * p.width);
    const int rows = min(p.width, p.N - row0);
    // Experts: the kernel before this one in the layer has waited for whatever
    // wrote the choices before it let this one start, so they are read early.
    SlotLists lists{};
    if constexpr (MOE) {
        lists = build_lists(p.ids, p.weights, p.cols, p.k, p.E, NT * 4, smem + p.list_off);
    }
    if (P > 1) ptx::cluster_sync(); else __syncthreads();
    const int total = (MOE ? lists.nseg : 1) * p.k_stages;
    const int i0 = static_cast<int>(static_cast<int64_t>(j) * total / P);
    const int i1 = static_cast<int>(static_cast<int64_t>(j + 1) * total / P);

    if (warp == kConsumers) {
        // ------------------------------------------------------------ producer
        const uint64_t pol_w = p.stream_w ? ptx::policy_evict_first() : ptx::policy_evict_normal();
        const uint32_t w_tx = static_cast<uint32_t>(p.width) * 128u;
        const uint32_t side_tx = W4 ? static_cast<uint32_t>(p.width * p.stage_groups * 2) : 0u;
        const T* X = static_cast<const T*>(p.X);
        bool ok = true;
        // weights and scales of list entry i
        auto issue_w = [&](int i, int s) {
            const int seg = MOE ? i / p.k_stages : 0;
            const int kb = i - seg * p.k_stages;
            const int matrix = MOE ? lists.seg_e[seg] : 0;
            const uint32_t dst = base + static_cast<uint32_t>(s * p.ring.w_bytes);
            ptx::tma_load_2d_hint(dst, &tmW, full_bar(s), kb * (W4 ? 128 : 64), matrix * p.N + row0, pol_w);
            if constexpr (W4) {
                const uint32_t side = base + static_cast<uint32_t>(p.ring.side_off + s * p.ring.side_bytes);
                const int y = matrix * p.groups_k + kb * p.stage_groups;
                ptx::tma_load_2d(side, &tmS, full_bar(s), row0, y);
                if (p.has_zeros) ptx::tma_load_2d(side + static_cast<uint32_t>(p.ring.side_bytes / 2), &tmZ, full_bar(s), row0, y);
            }
        };
        auto columns = [&](int i, int& first, int& n, int& kb) {
            const int seg = MOE ? i / p.k_stages : 0;
            kb = i - seg * p.k_stages;
            first = MOE ? lists.seg_begin[seg] : 0;
            n = MOE ? 2 * (lists.seg_begin[seg + 1] - first) : p.cols;
        };
        auto arm = [&](int i, int s) {
            int first, n, kb;
            columns(i, first, n, kb);
            const int kv = min(kStageElems<W4>, p.K - kb * kStageElems<W4>);
            ptx::mbar_arrive_expect_tx(full_bar(s), w_tx + side_tx * (p.has_zeros ? 2u : 1u) + static_cast<uint32_t>(n * kv * 2));
        };
        auto issue_x = [&](int i, int s) {
            int first, n, kb;
            columns(i, first, n, kb);
            const int kv = min(kStageElems<W4>, p.K - kb * kStageElems<W4>);
            const uint32_t dst = base + static_cast<uint32_t>(p.ring.x_off + s * p.ring.x_bytes);
            for (int c = lane; c < n; c += 32) {
                const int64_t row = MOE ? 2 * static_cast<int64_t>(lists.slot[first + (c >> 1)]) + (c & 1) : c;
                ptx::bulk_load(dst + static_cast<uint32_t>(c * kColPitch<W4>),
                               X + row * p.K + static_cast<int64_t>(kb) * kStageElems<W4>, static_cast<uint32_t>(kv * 2), full_bar(s));
            }
        };
        // Before the wait for the kernel before this one: with experts the first
        // ring of weights (they were complete before that kernel began); in the
        // plain product only a prefetch into L2, which cannot expose stale data.
        const int pre = min(NS, i1 - i0);
        if (lane == 0) {
            for (int i = 0; i < pre; ++i) {
                if constexpr (MOE) {
                    arm(i0 + i, i);
                    issue_w(i0 + i, i);
                } else {
                    ptx::tma_prefetch_2d(&tmW, (i0 + i) * (W4 ? 128 : 64), row0);
                }
            }
        }
        __syncwarp();
        ptx::griddep_wait();
        ptx::griddep_launch_dependents();
        for (int i = 0; i < i1 - i0; ++i) {
            const int s = i % NS;
            if (i >= pre || !MOE) {
                if (i >= NS && !wait_phase_warp(empty_bar(s), ((i / NS) & 1) ^ 1u, p.status, kSiteStreamEmpty, p.timeout_ns)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    arm(i0 + i, s);
                    issue_w(i0 + i, s);
                }
                __syncwarp();
            }
            issue_x(i0 + i, s);
        }
        if (!ok) {   // leave no copy in flight behind
            for (int s = 0; s < NS; ++s)
                for (uint32_t ph = 0; ph < 2; ++ph) wait_phase(full_bar(s), ph, p.status, kSiteStreamDrain, 1000000);
        }
    } else {
        // ------------------------------------------------------------ consumers
        ptx::griddep_wait();
        const int mg = warp % p.mw, kg = warp / p.mw;
        const int tiles = (rows + 15) >> 4;
        const int g = lane >> 2, t = lane & 3;
        float* mine = table + kg * table_size;
        StreamWarp<T, W4, NT> sw;
        sw.clear();
        int seg = -1, nt = 0, first = 0, n = 0;
        bool ok = true;
        // the sums of the segment in hand into this warp's table
        auto flush = [&]() {
#pragma unroll
            for (int jt = 0; jt < sw.MT; ++jt) {
                const int tile = mg + jt * p.mw;
                if (tile < tiles) {
                    float* to = mine + tile * 16 + g;
#pragma unroll
                    for (int q = 0; q < NT; ++q) {
                        if (q < nt) {
                            if constexpr (MOE) {
                                // columns 2t and 2t + 1 are the two parts of one slot's h
                                const int c = q * 4 + t;
                                if (c < n) {
                                    const float w = lists.weight[first + c];
                                    float* at = to + (lists.slot[first + c] / p.k) * p.table_pitch;
                                    at[0] += w * (sw.acc[jt][q][0] + sw.acc[jt][q][1]);
                                    at[8] += w * (sw.acc[jt][q][2] + sw.acc[jt][q][3]);
                                }
                            } else {
                                float* at = to + (q * 8 + 2 * t) * p.table_pitch;
                                at[0] += sw.acc[jt][q][0];
                                at[p.table_pitch] += sw.acc[jt][q][1];
                                at[8] += sw.acc[jt][q][2];
                                at[p.table_pitch + 8] += sw.acc[jt][q][3];
                            }
                        }
                    }
                }
            }
            sw.clear();
            __syncwarp();
        };
        for (int i = kg; i < i1 - i0; i += KW) {
            const int s = i % NS;
            const int sg = MOE ? (i0 + i) / p.k_stages : 0;
            const int kb = i0 + i - sg * p.k_stages;
            if (sg != seg) {
                if (seg >= 0) flush();
                seg = sg;
                first = MOE ? lists.seg_begin[sg] : 0;
                n = MOE ? lists.seg_begin[sg + 1] - first : p.cols;
                nt = MOE ? (n + 3) >> 2 : (n + 7) >> 3;
            }
            if (!wait_phase_warp(full_bar(s), (i / NS) & 1, p.status, kSiteStreamFull, p.timeout_ns)) {
                ok = false;
                break;
            }
            const int kv = min(kStageElems<W4>, p.K - kb * kStageElems<W4>);
            const uint32_t w = base + static_cast<uint32_t>(s * p.ring.w_bytes);
            const uint32_t x = base + static_cast<uint32_t>(p.ring.x_off + s * p.ring.x_bytes);
            if constexpr (W4) {
                const uint32_t sc = base + static_cast<uint32_t>(p.ring.side_off + s * p.ring.side_bytes);
                const uint32_t zr = sc + static_cast<uint32_t>(p.ring.side_bytes / 2);
                const SideView side{{sc, sc + 16u}, {zr, zr + 16u}, p.width, 16};
                sw.stage4(w, x, side, p.has_zeros != 0, kv, p.chunks_per_group, tiles, mg, p.mw, nt, lane);
            } else {
                sw.stage16(w, x, kv, tiles, mg, p.mw, nt, lane);
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(empty_bar(s));
        }
        if (seg >= 0 && ok) flush();
    }

    // ------------------------------------------------ the tables into the output
    __syncthreads();
    T* D = static_cast<T*>(p.D);
    const int out_cols = p.cols;
    const int total_out = out_cols * p.width;
    auto store = [&](int e, float v) {
        const int col = e / p.width, row = e - col * p.width;
        if (row >= rows) return;
        const int64_t n = row0 + row;
        if constexpr (!MOE) {
            if (p.epi.on) v = epi_apply1<T>(p.epi, v, p.row0 + col, n, p.N);
        }
        D[(MOE ? col : p.row0 + col) * static_cast<int64_t>(p.N) + n] = Elem<T>::from_float(v);
    };
    auto own_sum = [&](int e) {
        const int col = e / p.width, row = e - col * p.width;
        const float* at = table + col * p.table_pitch + row;
        float v = at[0];
        for (int q = 1; q < KW; ++q) v += at[q * table_size];
        return v;
    };
    if (P == 1) {
        for (int e = threadIdx.x; e < total_out; e += kStreamThreads) store(e, own_sum(e));
    } else {
        // CTA d of the cluster finishes outputs [d per, (d + 1) per); its receive
        // buffer is [P][per].
        const int per = (total_out + P - 1) / P;
        const uint32_t recv = base + static_cast<uint32_t>(p.recv_off);
        for (int e = threadIdx.x; e < total_out; e += kStreamThreads) {
            const int d = e / per;
            ptx::st_cluster_f32(ptx::mapa(recv + static_cast<uint32_t>((j * per + e - d * per) * 4), static_cast<uint32_t>(d)),
                                own_sum(e));
        }
        ptx::cluster_sync();
        const float* got = reinterpret_cast<const float*>(smem + p.recv_off);
        for (int e = threadIdx.x; e < per; e += kStreamThreads) {
            if (j * per + e >= total_out) break;
            float v = got[e];
            for (int q = 1; q < P; ++q) v += got[q * per + e];
            store(j * per + e, v);
        }
    }
}

// ------------------------------------------------------------------- host side
struct RowsShape {
    int width, ranges, pieces, mw, smem;
    RingLayout ring;
    int list_off, table_off, recv_off, table_pitch;
};

inline int up_to(int a, int b) { return (a + b - 1) / b * b; }

// The ring for `rows` rows and `cols` columns a stage, as deep as `budget`
// bytes allow in multiples of `kw` stages (at least kw).
inline RingLayout ring_layout(bool w4, int rows, int side_rows, int stage_groups, int cols, int budget, int kw) {
    RingLayout r;
    r.w_bytes = up_to(rows, 16) * 128;
    r.side_bytes = w4 ? 2 * up_to(side_rows * stage_groups * 2, 128) : 0;
    const int pitch = w4 ? kColPitch<true> : kColPitch<false>;
    r.x_bytes = up_to(cols * pitch, 128);
    const int one = r.w_bytes + r.side_bytes + r.x_bytes;
    // columns are read 8 at a time: the last stage's end in room of their own
    const int pad = up_to(cols, 8) * pitch - cols * pitch;
    r.stages = std::max(kw, std::min(std::max(budget - pad, 0) / one, kMaxRing) / kw * kw);
    r.side_off = r.stages * r.w_bytes;
    r.x_off = r.side_off + r.stages * r.side_bytes;
    r.end = up_to(r.x_off + r.stages * r.x_bytes + pad, 128);
    return r;
}

}  // namespace gemm_gb300
