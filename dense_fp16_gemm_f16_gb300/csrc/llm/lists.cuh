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
    int head, ids, wt, cnt, base, seg_e, seg_begin, slot, pos, end;
};

__host__ __device__ inline ListOffsets list_offsets(int S, int E) {
    ListOffsets o;
    o.head = 0;
    o.ids = 16;
    o.wt = o.ids + 4 * S;
    o.cnt = o.wt + 4 * S;
    o.base = o.cnt + 4 * E;
    o.seg_e = o.base + 4 * E;
    o.seg_begin = o.seg_e + 2 * S;
    o.slot = o.seg_begin + 2 * (S + 2);
    o.pos = o.slot + 2 * S;
    o.end = (o.pos + 2 * S + 127) / 128 * 128;
    return o;
}

// All threads of the CTA call this; it ends with a barrier.  Ids outside
// [0, E) are left out; an expert that a token lists twice becomes one slot (its
// first) with the weights added, so no two columns of a segment share a token.
// An expert's slots keep their order: CTAs that share a segment's work build
// the same lists.
__device__ inline SlotLists build_lists(const int32_t* ids, const float* weights, int T, int k, int E, int cap,
                                        uint8_t* mem) {
    const int S = T * k;
    const ListOffsets o = list_offsets(S, E);
    int32_t* l_ids = reinterpret_cast<int32_t*>(mem + o.ids);
    float* l_wt = reinterpret_cast<float*>(mem + o.wt);
    int32_t* cnt = reinterpret_cast<int32_t*>(mem + o.cnt);
    int32_t* base = reinterpret_cast<int32_t*>(mem + o.base);
    uint16_t* seg_e = reinterpret_cast<uint16_t*>(mem + o.seg_e);
    uint16_t* seg_begin = reinterpret_cast<uint16_t*>(mem + o.seg_begin);
    uint16_t* slot = reinterpret_cast<uint16_t*>(mem + o.slot);
    uint16_t* pos = reinterpret_cast<uint16_t*>(mem + o.pos);
    for (int e = threadIdx.x; e < E; e += blockDim.x) cnt[e] = 0;
    for (int s = threadIdx.x; s < S; s += blockDim.x) l_ids[s] = ids[s];
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        // a slot's place: the slots of its expert before it, 32 slots at a time
        for (int s0 = 0; s0 < S; s0 += 32) {
            const int s = s0 + lane;
            const int e = s < S ? l_ids[s] : -1;
            bool keep = e >= 0 && e < E;
            for (int q = s - s % k; q < s; ++q) keep = keep && l_ids[q] != e;
            const uint32_t same = __match_any_sync(0xffffffffu, keep ? e : -1 - lane);
            const int before = keep ? cnt[e] : 0;
            __syncwarp();
            if (keep && (same >> lane) == 1u) cnt[e] = before + __popc(same);   // the last of them
            if (s < S) pos[s] = keep ? static_cast<uint16_t>(before + __popc(same & ((1u << lane) - 1u))) : 0xFFFFu;
            __syncwarp();
        }
        int slots = 0, segs = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            const int c = e < E ? cnt[e] : 0;
            const int g = (c + cap - 1) / cap;
            int ic = c, ig = g;   // inclusive sums over the lanes
            for (int d = 1; d < 32; d <<= 1) {
                const int uc = __shfl_up_sync(0xffffffffu, ic, d), ug = __shfl_up_sync(0xffffffffu, ig, d);
                if (lane >= d) {
                    ic += uc;
                    ig += ug;
                }
            }
            if (e < E) base[e] = slots + ic - c;
            for (int i = 0; i < g; ++i) {
                seg_e[segs + ig - g + i] = static_cast<uint16_t>(e);
                seg_begin[segs + ig - g + i] = static_cast<uint16_t>(slots + ic - c + i * cap);
            }
            slots += __shfl_sync(0xffffffffu, ic, 31);
            segs += __shfl_sync(0xffffffffu, ig, 31);
        }
        if (lane == 0) {
            seg_begin[segs] = static_cast<uint16_t>(slots);
            *reinterpret_cast<int32_t*>(mem + o.head) = segs;
        }
    }
    __syncthreads();
    for (int s = threadIdx.x; s < S; s += blockDim.x) {
        if (pos[s] == 0xFFFFu) continue;
        const int e = l_ids[s], last = s - s % k + k;
        float w = weights[s];
        for (int q = s + 1; q < last; ++q)
            if (l_ids[q] == e) w += weights[q];
        const int at = base[e] + pos[s];
        slot[at] = static_cast<uint16_t>(s);
        l_wt[at] = w;
    }
    __syncthreads();
    return SlotLists{*reinterpret_cast<const int32_t*>(mem + o.head), seg_e, seg_begin, slot, l_wt};
}

}  // namespace gemm_gb300
