// lists.cuh -- which columns each expert gets: the tokens' choices sorted by
// expert, in shared memory, by every CTA for itself.
#pragma once

#include <cstdint>

#include "llm/llm.h"
#include "llm/stream.cuh"

namespace gemm_gb300 {

// A choice is a slot s = token * k + j.  A segment is up to `cap` slots of one
// expert; an expert with more gets several segments, one behind the other.
struct SlotLists {
    int nseg;
    const uint16_t* seg_e;       // [nseg]
    const uint16_t* seg_begin;   // [nseg + 1] into slot / weight
    const uint16_t* slot;
    const float* weight;
};

struct ListOffsets {
    int head, ids, wt, base, seg_e, seg_begin, slot, cnt, end;
};

__host__ __device__ inline ListOffsets list_offsets(int S, int E) {
    const int chunks = (S + 31) / 32;
    ListOffsets o;
    o.head = 0;
    o.ids = 16;
    o.wt = o.ids + 4 * S;
    o.base = o.wt + 4 * S;
    o.seg_e = o.base + 4 * E;
    o.seg_begin = o.seg_e + 2 * S;
    o.slot = o.seg_begin + 2 * (S + 2);
    o.cnt = (o.slot + 2 * S + 15) / 16 * 16;
    o.end = (o.cnt + (S > 32 ? chunks * ((E + 15) / 16 * 16) : 0) + 127) / 128 * 128;
    return o;
}

// All threads of the CTA call this; it ends with a barrier.  Ids outside
// [0, E) are left out; an expert that a token lists twice becomes one slot (its
// first) with the weights added, so no two columns of a segment share a token.
// An expert's slots keep their order: CTAs that share a segment's work build
// the same lists.  Up to 32 slots are sorted by one warp in registers; more by
// counting, 32 slots to a warp.
__device__ inline SlotLists build_lists(const int32_t* ids, const float* weights, int T, int k, int E, int cap,
                                        uint8_t* mem) {
    const int S = T * k;
    const ListOffsets o = list_offsets(S, E);
    float* l_wt = reinterpret_cast<float*>(mem + o.wt);
    uint16_t* seg_e = reinterpret_cast<uint16_t*>(mem + o.seg_e);
    uint16_t* seg_begin = reinterpret_cast<uint16_t*>(mem + o.seg_begin);
    uint16_t* slot = reinterpret_cast<uint16_t*>(mem + o.slot);
    const int lane = threadIdx.x & 31;
    if (S <= 32) {
        if (threadIdx.x < 32) {
            const int e = lane < S ? ids[lane] : -1;
            const float own = lane < S ? weights[lane] : 0.0f;
            const int token = lane / k;
            bool keep = e >= 0 && e < E;
            float w = own;
            int at = 0, same_before = 0, same = 0;
            for (int q = 0; q < S; ++q) {   // drop repeats within a token, add their weights
                const int eq = __shfl_sync(0xffffffffu, e, q);
                const float wq = __shfl_sync(0xffffffffu, own, q);
                if (q / k == token && eq == e) {
                    if (q < lane) keep = false;
                    if (q > lane) w += wq;
                }
            }
            const uint32_t kept = __ballot_sync(0xffffffffu, keep);
            for (int q = 0; q < S; ++q) {
                const int eq = __shfl_sync(0xffffffffu, e, q);
                if ((kept >> q) & 1u) {
                    at += eq < e || (eq == e && q < lane);
                    same += eq == e;
                    same_before += eq == e && q < lane;
                }
            }
            // the first slot of each `cap` of an expert opens a segment
            const bool opens = keep && same_before % cap == 0;
            const uint32_t open = __ballot_sync(0xffffffffu, opens);
            int seg = 0;
            for (int q = 0; q < S; ++q) {
                const int aq = __shfl_sync(0xffffffffu, at, q);
                if ((open >> q) & 1u) seg += aq < at;
            }
            if (keep) {
                slot[at] = static_cast<uint16_t>(lane);
                l_wt[at] = w;
            }
            if (opens) {
                seg_e[seg] = static_cast<uint16_t>(e);
                seg_begin[seg] = static_cast<uint16_t>(at);
            }
            if (lane == 0) {
                const int n = __popc(open);
                seg_begin[n] = static_cast<uint16_t>(__popc(kept));
                *reinterpret_cast<int32_t*>(mem + o.head) = n;
            }
        }
        __syncthreads();
        return SlotLists{*reinterpret_cast<const int32_t*>(mem + o.head), seg_e, seg_begin, slot, l_wt};
    }

    int32_t* l_ids = reinterpret_cast<int32_t*>(mem + o.ids);
    int32_t* base = reinterpret_cast<int32_t*>(mem + o.base);
    uint8_t* cnt = mem + o.cnt;   // [chunk][expert]: kept slots, then kept slots before the chunk (at most T)
    const int pitch = (E + 15) / 16 * 16, chunks = (S + 31) / 32;
    for (int i = threadIdx.x; i < chunks * pitch / 16; i += blockDim.x)
        reinterpret_cast<uint4*>(cnt)[i] = make_uint4(0u, 0u, 0u, 0u);
    for (int s = threadIdx.x; s < S; s += blockDim.x) {
        l_ids[s] = ids[s];
        l_wt[s] = weights[s];
    }
    __syncthreads();
    // a slot belongs to the warp and lane of its chunk; at most 4 per thread (1024 slots, 8 warps)
    constexpr int kMost = 4;
    int e_of[kMost], rank[kMost];   // rank < 0: left out
    float w_of[kMost];
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
        const int c = (threadIdx.x >> 5) + i * (blockDim.x >> 5), s = c * 32 + lane;
        e_of[i] = -1;
        rank[i] = -1;
        w_of[i] = 0.0f;
        if (c < chunks) {
            const int e = s < S ? l_ids[s] : -1;
            bool keep = e >= 0 && e < E;
            if (keep) {
                const int first = s - s % k;
                float w = l_wt[s];
                for (int q = first; q < first + k; ++q) {
                    if (q != s && l_ids[q] == e) {
                        if (q < s) keep = false;
                        else w += l_wt[q];
                    }
                }
                w_of[i] = w;
            }
            const uint32_t same = __match_any_sync(0xffffffffu, keep ? e : -1 - lane);
            if (keep) {
                e_of[i] = e;
                rank[i] = __popc(same & ((1u << lane) - 1u));
                if (rank[i] == 0) cnt[c * pitch + e] = static_cast<uint8_t>(__popc(same));
            }
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        int run = 0;
        for (int c = 0; c < chunks; ++c) {
            const int v = cnt[c * pitch + e];
            cnt[c * pitch + e] = static_cast<uint8_t>(run);
            run += v;
        }
        base[e] = run;   // the expert's slots, for now
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        // lane l takes experts [l per, (l + 1) per)
        const int per = (E + 31) / 32, e0 = lane * per, e1 = min(E, e0 + per);
        int slots = 0, segs = 0;
        for (int e = e0; e < e1; ++e) {
            slots += base[e];
            segs += (base[e] + cap - 1) / cap;
        }
        int ic = slots, ig = segs;   // inclusive sums over the lanes
        for (int d = 1; d < 32; d <<= 1) {
            const int uc = __shfl_up_sync(0xffffffffu, ic, d), ug = __shfl_up_sync(0xffffffffu, ig, d);
            if (lane >= d) {
                ic += uc;
                ig += ug;
            }
        }
        if (lane == 31) {
            seg_begin[ig] = static_cast<uint16_t>(ic);
            *reinterpret_cast<int32_t*>(mem + o.head) = ig;
        }
        int at = ic - slots, seg = ig - segs;
        for (int e = e0; e < e1; ++e) {
            const int n = base[e];
            base[e] = at;
            for (int i = 0; i < n; i += cap, ++seg) {
                seg_e[seg] = static_cast<uint16_t>(e);
                seg_begin[seg] = static_cast<uint16_t>(at + i);
            }
            at += n;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
        const int c = (threadIdx.x >> 5) + i * (blockDim.x >> 5);
        if (rank[i] >= 0) {
            const int at = base[e_of[i]] + cnt[c * pitch + e_of[i]] + rank[i];
            slot[at] = static_cast<uint16_t>(c * 32 + lane);
            l_wt[at] = w_of[i];
        }
    }
    __syncthreads();
    return SlotLists{*reinterpret_cast<const int32_t*>(mem + o.head), seg_e, seg_begin, slot, l_wt};
}

}  // namespace gemm_gb300
