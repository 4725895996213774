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
// in shared memory whenever it moves to another segment (the plain product has
// one and just stores); warps that own the
// same rows (the KW stage groups) have tables of their own, so no two threads
// ever add to one number.  At the end the tables are added in a fixed order,
// across the cluster through distributed shared memory, and each output is
// rounded once.  Results are bitwise reproducible.
// Measured: 8192 x 8192 4-bit weights (34.6 MB), M = 1 12.5 us, M = 8 13 us, M = 16
// 20 us; 11000 x 4128 with zero points in groups of 32, M = 13 21 us, of which the
// warps' instructions for decoding and scaling (2.2 of 4 issued per clock) are most;
// 2 of 8 experts of 4096 x 8200 per token, 16 tokens (all 8 read, 537 MB): 105 us,
// 5.2 TB/s.
#pragma once

#include "llm/lists.cuh"
#include "llm/llm.h"
#include "llm/stream.cuh"

namespace gemm_gb300 {

struct RowsParams {
    RingLayout ring;
    int32_t list_off, table_off, recv_off;   // shared-memory offsets (list only for experts)
    int32_t table_pitch;                     // floats from one column to the next
    int32_t N, K, k_stages;                  // rows of one matrix; K; stages over K (of ring.atoms atoms)
    int32_t width, ranges, pieces;           // pieces = P
    int32_t mw;                              // warps that share a stage's tiles
    int32_t groups_k;                        // K / group (4-bit)
    int32_t atom_groups;                     // 256 / group
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

// CPG: 32-k chunks per group of 4-bit weights, 0 for 16-bit weights
template <class T, int CPG, int NT, bool MOE>
__global__ void __launch_bounds__(kStreamThreads, kCtasPerSm<(CPG != 0), NT, MOE>)
weight_rows_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmS,
                   const __grid_constant__ CUtensorMap tmZ, const RowsParams p) {
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
    }
    if (static_cast<int>(threadIdx.x) < p.ring.slots) {
        ptx::mbar_init(full_bar(threadIdx.x), full_arrivals(p.mw));
        ptx::mbar_init(empty_bar(threadIdx.x), static_cast<uint32_t>(p.mw));
        ptx::fence_mbar_init();
    }
    float* table = reinterpret_cast<float*>(smem + p.table_off);
    const int tokens = MOE ? p.cols : 8 * NT;
    const int table_size = tokens * p.table_pitch;   // one stage group's
    if constexpr (MOE)   // the plain product stores whole tables
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
    const int mine_n = static_cast<int>(static_cast<int64_t>(j + 1) * total / P) - i0;   // this CTA's stages

    constexpr int KE = kAtomElems<W4>;
    const int stage_elems = p.ring.atoms * KE;
    const int pitch = col_pitch(W4, p.ring.atoms);
    const int mg = warp % p.mw, kg = warp / p.mw;
    const GroupSlots own(p.ring.slots, KW, kg);
    const uint64_t pol_w = p.stream_w ? ptx::policy_evict_first() : ptx::policy_evict_normal();

    // The weights and scales of K stage kb of segment seg into slot s, with the byte count ...
    auto issue_w = [&](int seg, int kb, int s) {
        const int kv = min(stage_elems, p.K - kb * stage_elems);
        const int na = (kv + KE - 1) / KE;
        const int matrix = MOE ? lists.seg_e[seg] : 0;
        const uint32_t w_tx = static_cast<uint32_t>(na * p.width * 128);
        const uint32_t side_tx = W4 ? static_cast<uint32_t>(p.width * p.ring.atoms * p.atom_groups * 2) : 0u;
        if (lane == 0) ptx::mbar_arrive_expect_tx(full_bar(s), w_tx + side_tx * (p.has_zeros ? 2u : 1u));
        __syncwarp();
        if (lane < na)
            ptx::tma_load_2d_hint(base + static_cast<uint32_t>(s * p.ring.w_bytes + lane * p.ring.atom_bytes), &tmW,
                                  full_bar(s), (kb * p.ring.atoms + lane) * (W4 ? 128 : 64), matrix * p.N + row0, pol_w);
        if constexpr (W4) {
            const uint32_t side = base + static_cast<uint32_t>(p.ring.side_off + s * p.ring.side_bytes);
            const int y = matrix * p.groups_k + kb * p.ring.atoms * p.atom_groups;
            if (lane == 8) ptx::tma_load_2d(side, &tmS, full_bar(s), row0, y);
            if (lane == 9 && p.has_zeros)
                ptx::tma_load_2d(side + static_cast<uint32_t>(p.ring.side_bytes / 2), &tmZ, full_bar(s), row0, y);
        }
    };
    // ... and the columns
    const int row_shift = 31 - __clz(stage_elems / 8);   // 16-byte pieces of a column in a whole stage
    auto issue_x = [&](int seg, int kb, int s) {
        const int kv = min(stage_elems, p.K - kb * stage_elems);
        const int first = MOE ? lists.seg_begin[seg] : 0;
        const int n = MOE ? 2 * (lists.seg_begin[seg + 1] - first) : p.cols;
        const uint32_t dst = base + static_cast<uint32_t>(p.ring.x_off + s * p.ring.x_bytes);
        const T* X = static_cast<const T*>(p.X) + static_cast<int64_t>(kb) * stage_elems;
        for (int i = mg * 32 + lane; i < (n << row_shift); i += 32 * p.mw) {   // the group's warps share them
            const int c = i >> row_shift, o = (i - (c << row_shift)) * 8;
            if (o < kv) {
                const int64_t row = MOE ? 2 * static_cast<int64_t>(lists.slot[first + (c >> 1)]) + (c & 1) : c;
                ptx::cp_async16(dst + static_cast<uint32_t>(c * pitch + o * 2), X + row * p.K + o);
            }
        }
        ptx::cp_async_arrive(full_bar(s));
    };
    // The group's stages, kg, kg + KW, ... of the CTA's list.
    struct Place {
        int left, seg, kb;
    };
    auto start = [&]() {
        const int i = i0 + kg;
        const int seg = MOE ? i / p.k_stages : 0;
        return Place{mine_n - kg, seg, i - seg * p.k_stages};
    };
    auto advance = [&](Place& at) {
        at.left -= KW;
        at.kb += KW;
        if constexpr (MOE) {
            while (at.kb >= p.k_stages) {
                at.kb -= p.k_stages;
                ++at.seg;
            }
        }
    };

    // Before the wait for the kernel before this one: with experts the first
    // slots' weights (they were complete before that kernel began); in the plain
    // product only a prefetch into L2, which cannot expose stale data.
    if (mg == 0) {
        Place at = start();
        for (int d = 0; d < own.depth && at.left > 0; ++d, advance(at)) {
            if constexpr (MOE) {
                issue_w(at.seg, at.kb, own.first + d);
            } else {
                if (lane < p.ring.atoms && static_cast<int64_t>(at.kb * p.ring.atoms + lane) * KE < p.K)
                    ptx::tma_prefetch_2d(&tmW, (at.kb * p.ring.atoms + lane) * (W4 ? 128 : 64), row0);
            }
        }
    }
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    Place ahead = start();   // the next stage to fetch: the first warp its rows, all of the group its columns
    for (int d = 0; d < own.depth && ahead.left > 0; ++d, advance(ahead)) {
        if constexpr (!MOE) {
            if (mg == 0) issue_w(ahead.seg, ahead.kb, own.first + d);
        }
        issue_x(ahead.seg, ahead.kb, own.first + d);
    }

    {
        const int g = lane >> 2, t = lane & 3;
        const int tile0 = mg * StreamWarp<T, W4, NT, MOE>::MT;               // this warp's tiles
        const int tiles = max(0, ((rows + 15) >> 4) - tile0);
        float* mine = table + kg * table_size;
        StreamWarp<T, W4, NT, MOE> sw;
        sw.clear();
        int seg = -1, nt = 0, first = 0, n = 0;
        bool ok = true;
        // the sums of the segment in hand into this warp's table
        auto flush = [&]() {
#pragma unroll
            for (int jt = 0; jt < sw.MT; ++jt) {
                if (jt < tiles) {
                    float* to = mine + (tile0 + jt) * 16 + g;
#pragma unroll
                    for (int q = 0; q < NT; ++q) {
                        if (q == 0 || q < nt) {
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
                                at[0] = sw.acc[jt][q][0];
                                at[p.table_pitch] = sw.acc[jt][q][1];
                                at[8] = sw.acc[jt][q][2];
                                at[p.table_pitch + 8] = sw.acc[jt][q][3];
                            }
                        }
                    }
                }
            }
            sw.clear();
            __syncwarp();
        };
        int d = 0;
        uint32_t phase = 0;
        for (Place now = start(); now.left > 0; advance(now)) {
            const int s = own.first + d;
            if (now.seg != seg) {
                if (seg >= 0) flush();
                seg = now.seg;
                first = MOE ? lists.seg_begin[seg] : 0;
                n = MOE ? lists.seg_begin[seg + 1] - first : p.cols;
                nt = MOE ? (n + 3) >> 2 : (n + 7) >> 3;
            }
            if (!wait_phase_warp(full_bar(s), phase, p.status, kSiteStreamFull, p.timeout_ns)) {
                ok = false;
                break;
            }
            const uint32_t there = base + ptx::stage_token();
            const int kv = min(stage_elems, p.K - now.kb * stage_elems);
            for (int a = 0; a * KE < kv; ++a) {
                const uint32_t w = there + static_cast<uint32_t>(s * p.ring.w_bytes + a * p.ring.atom_bytes + tile0 * 2048);
                const uint32_t x = there + static_cast<uint32_t>(p.ring.x_off + s * p.ring.x_bytes + a * KE * 2);
                const int k = min(KE, kv - a * KE);
                if constexpr (W4) {
                    const int first_scale = a * p.atom_groups * p.width + tile0 * 16;
                    const uint32_t sc = there + static_cast<uint32_t>(p.ring.side_off + s * p.ring.side_bytes + first_scale * 2);
                    const SideView side{sc, sc + static_cast<uint32_t>(p.ring.side_bytes / 2), 16u,
                                        static_cast<uint32_t>(p.width * 2)};
                    sw.template atom4<CPG, 2048, 32>(w, 1024u, x, pitch, side, p.has_zeros != 0, k, tiles, nt, lane);
                } else {
                    sw.template atom16<2048>(w, 1024u, x, pitch, k, tiles, nt, lane);
                }
            }
            sw.hold();
            __syncwarp();
            if (now.left > own.depth * KW) {   // another stage takes this slot
                if (p.mw > 1) {
                    if (lane == 0) ptx::mbar_arrive(empty_bar(s));
                    if (!wait_phase_warp(empty_bar(s), phase, p.status, kSiteStreamEmpty, p.timeout_ns)) {
                        ok = false;
                        break;
                    }
                }
                if (mg == 0) issue_w(ahead.seg, ahead.kb, s);
                issue_x(ahead.seg, ahead.kb, s);
                advance(ahead);
            }
            if (++d == own.depth) {
                d = 0;
                phase ^= 1u;
            }
        }
        if (seg >= 0 && ok) flush();
        if (!ok && mg == 0) {   // leave no copy in flight behind
            for (int q = 0; q < own.depth; ++q)
                for (uint32_t ph = 0; ph < 2; ++ph)
                    wait_phase(full_bar(own.first + q), ph, p.status, kSiteStreamDrain, 1000000);
        }
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
    const int used = MOE ? KW : min(KW, mine_n);   // groups that had a stage
    auto own_sum = [&](int e) {
        if (used == 0) return 0.0f;
        const int col = e / p.width, row = e - col * p.width;
        const float* at = table + col * p.table_pitch + row;
        float v = at[0];
        for (int q = 1; q < used; ++q) v += at[q * table_size];
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
inline int up_to(int a, int b) { return (a + b - 1) / b * b; }

// A ring for kw groups with `rows` rows and `cols` columns a stage, with as many
// slots as `budget` bytes allow (at least one a group; the caller checks `end`).
inline RingLayout ring_layout(bool w4, int atoms, int rows, int side_rows, int atom_groups, int cols, int budget,
                              int kw) {
    RingLayout r;
    r.atoms = atoms;
    r.atom_bytes = up_to(rows, 16) * 128;
    r.w_bytes = atoms * r.atom_bytes;
    r.side_bytes = w4 ? 2 * up_to(side_rows * atom_groups * atoms * 2, 128) : 0;
    const int pitch = col_pitch(w4, atoms);
    r.x_bytes = up_to(cols * pitch, 128);
    const int one = r.w_bytes + r.side_bytes + r.x_bytes;
    // columns are read 8 at a time: the last slot's end in room of their own
    const int pad = up_to(cols, 8) * pitch - cols * pitch;
    r.slots = std::max(kw, std::min(std::max(budget - pad, 0) / one, kMaxRing));
    r.side_off = r.slots * r.w_bytes;
    r.x_off = r.side_off + r.slots * r.side_bytes;
    r.end = up_to(r.x_off + r.slots * r.x_bytes + pad, 128);
    return r;
}

}  // namespace gemm_gb300
