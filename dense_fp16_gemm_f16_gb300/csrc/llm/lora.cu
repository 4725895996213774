// lora.cu -- low-rank adapters of many requests:
//   U[m] = beta C[m] + c_a (X[m] A_aᵀ) B_aᵀ,  a = ids[m].
//
// Rows are put in order of their adapters: up to 256 by every CTA for itself, so that one
// kernel does everything, more by a kernel before (lora_list_kernel), which also cuts an
// adapter's rows into units.  A cluster of up to eight CTAs takes one adapter's rows, or one
// unit: each CTA forms V = X Aᵀ over its share of K, the partial sums meet in distributed shared
// memory in a fixed order, and each CTA multiplies V by its share of B's rows.
// Up to 16 rows beside a 16-bit projection, V alone is made (lora_v_kernel), while that
// product already streams its weights, and the product's epilogue does the rest.
//
// What bounds it.  A few rows: bytes (A and B of the adapters in use) and a chain of
// latencies; 250 rows, 62 adapters of rank 32 beside 5000 x 4104: 15.7 us for 39 MB, of
// which 1.5 put the rows in order, 5 form V, 2 exchange it, 4 to 5 multiply it.  Many rows: X, C and U up
// to rank 16 (4096 rows of 8192, runs of 8 adapters: 48 us for 140 MB: 14 us a unit for V, at
// 5 TB/s, and 12 for U), the rate of mma.sync above (rank 64: 82 us; hi and lo below double the
// second product).  Each byte meets few others in the first two cases, so the operands go to mma.sync by
// way of copies that every thread makes for itself; the k order within an MMA is free, so a
// thread's 16 (or 8) consecutive bytes of a row are its slots of two steps (or one).
//
// V is a sum in fp32.  For the second product it is cut into two numbers of the
// operands' type, hi + lo (for fp16 after scaling each row by a power of two to about 1, so
// that its range does not matter): the product then has twice the type's precision.
// U is rounded once; where U is the C of a product that follows, its rounding adds
// u |U| to that product's own u |D|.  The other way, U in fp32, would cost a
// prompt twice the bytes for a part that is small beside the projection's.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "config.h"
#include "llm/llm.h"
#include "llm/rows_host.cuh"
#include "llm/stream.cuh"

namespace gemm_gb300 {
namespace {

constexpr int kLoraThreads = 256;
constexpr int kLoraWarps = kLoraThreads / 32;
constexpr int kLoraTile = 256;           // most rows that a CTA puts in order: one per thread
constexpr int kLoraStepK = 32;           // k per warp and step of `down`: 16 bytes per thread and row
constexpr int kLoraColumns = 32;         // columns per warp and step of `up`
constexpr int kLoraMaxCluster = 8;

struct LoraParams {
    const void* X;           // [M][K]
    const void* A;           // [count][R][K]
    const void* B;           // [count][N][R]
    const float* factors;    // [count] or nullptr
    const int32_t* ids;      // [M], or nullptr: no row has an adapter
    const struct LoraList* list;   // the rows in order, or nullptr: every CTA makes that itself
    const void* C;           // [M][N] or nullptr
    void* U;                 // [M][N]
    float* V;                // [M][R]: factors X Aᵀ is all that is wanted, or nullptr
    uint32_t* ready;         // with V: for the product behind, which starts early
    int32_t M, N, K, R, count;
    int32_t k_steps, width;  // width: columns per CTA of a cluster
    int32_t unit_rows;       // with a list: most rows of a unit, 32, 64 or 128
    int32_t most_rows;       // rows of V in hand at one time
    int32_t cluster;         // its CTAs
    float beta;
};

// Up to 256 rows in order of their adapters.
struct Groups {
    int32_t order[kLoraTile];         // rows, group by group, each in row order
    int32_t start[kLoraTile + 1];     // group i is order[start[i]] .. order[start[i + 1] - 1]
    int32_t adapter[kLoraTile];       // of each group, in the order of their first rows
    int32_t n;                        // groups with an adapter; rows without one lie behind them
};
constexpr int kGroupsBytes = (sizeof(Groups) + 127) / 128 * 128;

// The same for more rows, made by a kernel of its own: units of up to unit_rows rows of one
// adapter, rows order[start] .. order[start + rows - 1].
constexpr int kListRows = 8192;
struct LoraUnit {
    int32_t adapter, start, rows, unused;
};
struct LoraList {
    int32_t n, with;     // units; rows that have an adapter, behind which the others lie
    int32_t unused[2];
    LoraUnit units[kListRows];
    int32_t order[kListRows];
};

// The table that finds them.
constexpr int kLoraSlots = 2 * kLoraTile;
struct GroupTable {
    uint8_t rows[kLoraSlots][kLoraWarps];   // an adapter's rows in each warp
    int32_t key[kLoraSlots];          // the adapter that has this slot, -1 free
    int32_t first[kLoraSlots];        // its first row, then its group
    int32_t leaders[kLoraWarps];
    int32_t none[kLoraWarps];         // rows without an adapter in each warp
};
static_assert(kLoraWarps == 8, "a slot's row counts are cleared as 8 bytes");

// Rows of warps before `warp` in a slot's counts.
__device__ __forceinline__ int rows_before(const uint8_t (&rows)[kLoraWarps], int warp) {
    int n = 0;
#pragma unroll
    for (int w = 0; w < kLoraWarps; ++w) n += w < warp ? rows[w] : 0;
    return n;
}

// Called by the whole CTA, one row per thread.  Which slot an adapter gets depends on
// timing, groups and their order do not.  Ids are read past L1: a kernel launched early may
// share an SM with one that read older ids there.
__device__ void group_rows(const LoraParams& p, int rows, Groups& s, GroupTable& table) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int id = -2;   // no row
    if (tid < rows) {
        id = p.ids != nullptr ? __ldcg(p.ids + tid) : -1;
        if (id < 0 || id >= p.count) id = -1;
    }
#pragma unroll
    for (int i = tid; i < kLoraSlots; i += kLoraThreads) {
        table.key[i] = -1;
        table.first[i] = kLoraTile;
        *reinterpret_cast<uint2*>(table.rows[i]) = make_uint2(0u, 0u);
    }
    s.start[tid] = 0;
    __syncthreads();
    const uint32_t mine = __match_any_sync(0xffffffffu, id);
    const int in_warp = __popc(mine & ((1u << lane) - 1u));
    const int lead_lane = __ffs(mine) - 1;
    int slot = 0;
    if (id >= 0 && in_warp == 0) {
        slot = static_cast<int>((static_cast<uint32_t>(id) * 2654435761u) >> 23);   // of 512
        while (true) {   // at most 256 adapters in 512 slots
            const int other = atomicCAS(&table.key[slot], -1, id);
            if (other == -1 || other == id) break;
            slot = (slot + 1) & (kLoraSlots - 1);
        }
        table.rows[slot][warp] = static_cast<uint8_t>(__popc(mine));
        atomicMin(&table.first[slot], tid);
    }
    slot = __shfl_sync(0xffffffffu, slot, lead_lane);
    const uint32_t none = __ballot_sync(0xffffffffu, id == -1);
    if (lane == 0) table.none[warp] = __popc(none);
    __syncthreads();
    const bool leads = id >= 0 && table.first[slot] == tid;
    const uint32_t mask = __ballot_sync(0xffffffffu, leads);
    if (lane == 0) table.leaders[warp] = __popc(mask);
    __syncthreads();
    int number = __popc(mask & ((1u << lane) - 1u)), n = 0, before = 0;
#pragma unroll
    for (int w = 0; w < kLoraWarps; ++w) {
        if (w < warp) {
            number += table.leaders[w];
            before += table.none[w];
        }
        n += table.leaders[w];
    }
    if (leads) {
        table.first[slot] = number;
        s.adapter[number] = id;
        s.start[number] = rows_before(table.rows[slot], kLoraWarps);   // sizes first
    }
    __syncthreads();
    if (warp == 0) {   // sizes to starts, 8 groups per lane
        int size[8], sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            size[i] = s.start[lane * 8 + i];
            sum += size[i];
        }
        int at = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, at, d);
            if (lane >= d) at += o;
        }
        if (lane == 31) s.start[kLoraTile] = at;
        at -= sum;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            s.start[lane * 8 + i] = at;
            at += size[i];
        }
        if (lane == 0) s.n = n;
    }
    __syncthreads();
    // behind the last group, start holds the number of rows that have an adapter
    if (id >= 0) s.order[s.start[table.first[slot]] + rows_before(table.rows[slot], warp) + in_warp] = tid;
    else if (id == -1) s.order[s.start[n] + before + in_warp] = tid;
    __syncthreads();
}

// The same for up to 32 rows: one warp does it, without a table.
__device__ void group_few_rows(const LoraParams& p, int rows, Groups& s) {
    const int lane = threadIdx.x & 31;
    if (threadIdx.x < 32) {
        int id = -2;
        if (lane < rows) {
            id = p.ids != nullptr ? __ldcg(p.ids + lane) : -1;
            if (id < 0 || id >= p.count) id = -1;
        }
        const uint32_t mine = __match_any_sync(0xffffffffu, id), before = (1u << lane) - 1u;
        const int lead = __ffs(mine) - 1;
        const uint32_t leads = __ballot_sync(0xffffffffu, id >= 0 && lead == lane);
        const uint32_t none = __ballot_sync(0xffffffffu, id == -1);
        const int number = __popc(leads & ((1u << lead) - 1u));
        // rows of the groups whose first row comes earlier
        int start = 0;
        for (uint32_t l = leads; l != 0; l &= l - 1) {
            const int at = __ffs(l) - 1, size = __popc(__shfl_sync(0xffffffffu, mine, at));
            start += at < lead ? size : 0;
        }
        if (id >= 0) {
            s.order[start + __popc(mine & before)] = lane;
            if (lead == lane) {
                s.adapter[number] = id;
                s.start[number] = start;
            }
        } else if (id == -1) {
            s.order[rows - __popc(none) + __popc(none & before)] = lane;
        }
        if (lane == 0) {
            s.n = __popc(leads);
            s.start[s.n] = rows - __popc(none);
        }
    }
    __syncthreads();
}

// The list of up to kListRows rows, by one CTA: a table in shared memory counts the rows
// of every adapter, the counts become places.  Which of an adapter's rows share a unit depends on
// timing; the sums of a row do not depend on what shares its unit.  4 us for 300 rows, 5 for 4096.
constexpr int kListThreads = 1024;
constexpr int kListEach = kListRows / kListThreads;
// Slots of the table: a power of two, twice the rows at least, one per thread at least.
int list_bits(int M) {
    int bits = 10;
    while ((1 << bits) < 2 * M) ++bits;
    return bits;
}

__global__ void __launch_bounds__(kListThreads) lora_list_kernel(const LoraParams p, LoraList* list, int bits) {
    extern __shared__ __align__(16) uint8_t smem[];
    const int slots = 1 << bits;
    int32_t* key = reinterpret_cast<int32_t*>(smem);
    int32_t* count = key + slots;   // the last is of rows without an adapter
    __shared__ int2 totals[32];
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int i = tid; i < slots; i += kListThreads) {
        key[i] = -1;
        count[i] = 0;
    }
    if (tid == 0) count[slots] = 0;
    int id[kListEach], slot[kListEach], rank[kListEach];
#pragma unroll
    for (int i = 0; i < kListEach; ++i) {
        const int row = i * kListThreads + tid;
        id[i] = -2;   // no row
        if (row < p.M) {
            id[i] = p.ids != nullptr ? __ldcg(p.ids + row) : -1;
            if (id[i] < 0 || id[i] >= p.count) id[i] = -1;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kListEach; ++i) {
        if (i * kListThreads >= p.M) break;
        const uint32_t mine = __match_any_sync(0xffffffffu, id[i]);
        const int lead = __ffs(mine) - 1;
        int at = slots, before = 0;
        if (lane == lead && id[i] >= -1) {
            if (id[i] >= 0) {
                at = static_cast<int>((static_cast<uint32_t>(id[i]) * 2654435761u) >> (32 - bits));
                while (true) {   // at most half of the slots are taken
                    const int other = atomicCAS(&key[at], -1, id[i]);
                    if (other == -1 || other == id[i]) break;
                    at = (at + 1) & (slots - 1);
                }
            }
            before = atomicAdd(&count[at], __popc(mine));
        }
        slot[i] = __shfl_sync(0xffffffffu, at, lead);
        rank[i] = __shfl_sync(0xffffffffu, before, lead) + __popc(mine & ((1u << lane) - 1u));
    }
    __syncthreads();
    // places: each thread sums up its slots, then all threads
    int2 sum = make_int2(0, 0);   // rows, units
    for (int i = tid; i < slots; i += kListThreads) {
        const int c = count[i];
        sum.x += c;
        sum.y += (c + p.unit_rows - 1) / p.unit_rows;
    }
    int2 at = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, at.x, d), y = __shfl_up_sync(0xffffffffu, at.y, d);
        if (lane >= d) {
            at.x += x;
            at.y += y;
        }
    }
    if (lane == 31) totals[warp] = at;
    __syncthreads();
    at.x -= sum.x;
    at.y -= sum.y;
    for (int w = 0; w < warp; ++w) {
        at.x += totals[w].x;
        at.y += totals[w].y;
    }
    for (int i = tid; i < slots; i += kListThreads) {
        const int c = count[i];
        count[i] = at.x;   // where the adapter's rows begin
        for (int r = 0; r < c; r += p.unit_rows) list->units[at.y++] = LoraUnit{key[i], at.x + r, min(p.unit_rows, c - r), 0};
        at.x += c;
    }
    if (tid == kListThreads - 1) {
        list->n = at.y;
        list->with = at.x;
        count[slots] = at.x;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kListEach; ++i)
        if (id[i] >= -1) list->order[count[slot[i]] + rank[i]] = i * kListThreads + tid;
}

// -------------------------------------------------------------------------- down
// Every thread copies the pieces of its own fragments to places of its own in shared
// memory (cp.async), some steps ahead, and reads them back: many bytes under way without
// registers for them, and nobody to wait for.
//
// How a launch is built.  MT: 16-row tiles of ranks of the first product in hand, TILE:
// ranks in hand with many rows; SLOTS: 16-byte places per thread for its copies; S: steps of 16
// ranks per chunk of the second product, LONG: R has more than one chunk; AHEAD: chunks
// under way.  SLOTS and AHEAD leave room for two CTAs per SM up to 32 ranks; with more, a CTA has
// enough to copy to be alone (61 rows, 48 adapters of rank 64 beside 4-bit 8192 x 4096, the whole
// call: 36 -> 33 us).
struct Ranks16 {
    static constexpr int MT = 1, TILE = 16, SLOTS = 18, WARPS = kLoraWarps, S = 1, AHEAD = 2;
    static constexpr bool LONG = false;
};
struct Ranks32 {
    static constexpr int MT = 2, TILE = 32, SLOTS = 16, WARPS = kLoraWarps, S = 2, AHEAD = 1;
    static constexpr bool LONG = false;
};
struct RanksMore {
    static constexpr int MT = 2, TILE = 64, SLOTS = 24, WARPS = kLoraWarps, S = 2, AHEAD = 3;
    static constexpr bool LONG = true;
};
struct RanksOnlyV {   // V alone, by fewer warps with little memory
    static constexpr int SLOTS = 8, WARPS = 4;
};

// Floats between the sums of two rows in the warps' exchange, which takes the same
// space: the two columns of a fragment fall into different banks.
__host__ __device__ constexpr int down_pitch(int MT) { return 16 * MT + 4; }
template <class Sh>
constexpr int kDownBytes = Sh::SLOTS * 16 * 32 * Sh::WARPS;

// part = V of m <= 8 NT rows (`rows`) and 16 MT ranks from r0 on over the k steps
// [s0, s1), which are dealt out to the warps.
template <class T, class Sh, int MT, int NT>
__device__ __forceinline__ void down_rows(const LoraParams& p, const T* A, int r0, const int32_t* rows, int m, int s0, int s1,
                                          uint8_t* space, float* part) {
    constexpr int W = Sh::WARPS, NF = 2 * MT + NT, D = Sh::SLOTS / NF, P = down_pitch(MT);
    constexpr int PLACE = 16 * 32 * W;
    static_assert(D >= 2, "a step ahead at least");
    static_assert(W * 8 * NT * P * 4 <= kDownBytes<Sh>, "the exchange fits the places");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t places = ptx::smem_u32(space) + threadIdx.x * 16;   // f of stage d: (d * NF + f) * PLACE behind
    const T* a_ptr = A + static_cast<int64_t>(r0 + g) * p.K + 8 * t;
    const T* x_ptr[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const bool in = 8 * j + g < m;
        x_ptr[j] = in ? static_cast<const T*>(p.X) + static_cast<int64_t>(rows[8 * j + g]) * p.K + 8 * t : nullptr;
    }
    // copies of one step into stage d; what lies outside becomes zeros
    auto fetch = [&](int s, int d) {
        const int64_t k = static_cast<int64_t>(s) * kLoraStepK;
        const bool in = s < s1 && k + 8 * t < p.K;   // K % 8 == 0: all eight or none
        const uint32_t to = places + d * (NF * PLACE);
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) {
            const bool take = in && r0 + 8 * i + g < p.R;
            ptx::cp_async16_or_zero(to + i * PLACE, take ? a_ptr + static_cast<int64_t>(8 * i) * p.K + k : A, take);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const bool take = in && x_ptr[j] != nullptr;
            ptx::cp_async16_or_zero(to + (2 * MT + j) * PLACE, take ? x_ptr[j] + k : A, take);
        }
    };
    float acc[MT][NT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.0f;
    int s = s0 + warp;
#pragma unroll
    for (int d = 0; d < D - 1; ++d) {
        fetch(s + d * W, d);
        ptx::cp_async_commit();
    }
    int d = 0;
    for (; s < s1; s += W) {
        ptx::cp_async_wait_group<D - 2>();   // this step's copies, by this thread, are done
        uint32_t a[2 * MT][4], x[NT][4];
        const uint32_t from = places + d * (NF * PLACE);
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) ptx::ld_shared_v4_u32(from + i * PLACE, a[i]);
#pragma unroll
        for (int j = 0; j < NT; ++j) ptx::ld_shared_v4_u32(from + (2 * MT + j) * PLACE, x[j]);
        const int back = d == 0 ? D - 1 : d - 1;   // the stage read in the step before
        fetch(s + (D - 1) * W, back);
        ptx::cp_async_commit();
        if (++d == D) d = 0;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const uint32_t lo[4] = {a[2 * i][0], a[2 * i + 1][0], a[2 * i][1], a[2 * i + 1][1]};
            const uint32_t hi[4] = {a[2 * i][2], a[2 * i + 1][2], a[2 * i][3], a[2 * i + 1][3]};
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                ptx::mma16816<T>(acc[i][j], lo, x[j][0], x[j][1]);
                ptx::mma16816<T>(acc[i][j], hi, x[j][2], x[j][3]);
            }
        }
    }
    ptx::cp_async_wait_group<0>();
    __syncthreads();   // nobody's copies are under way
    // the warps' sums meet in shared memory and are added in their order
    float* red = reinterpret_cast<float*>(space);
    float* mine = red + warp * 8 * NT * P;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) mine[(8 * j + 2 * t + (e & 1)) * P + 16 * i + g + 8 * (e >> 1)] = acc[i][j][e];
    __syncthreads();
    for (int i = threadIdx.x; i < m * 16 * MT; i += 32 * W) {
        const int n = i / (16 * MT), r = i % (16 * MT);
        if (r0 + r >= p.R) continue;
        const float* from = red + n * P + r;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) v += from[w * 8 * NT * P];
        part[n * p.R + r0 + r] = v;
    }
    __syncthreads();
}

// The same for units of ROWS = 64 or 128 rows and TILE ranks from r0 on: rows and ranks meet
// so often that they are copied once for the whole CTA, 64 k at a time, in 128-byte rows whose
// 16-byte pieces are swapped by the row's number, and read by ldmatrix; 32 rows per warp, the steps
// of 16 k dealt out to the warps of the same rows.  (The form above, where every warp copies the
// ranks for itself, took 117 us where this takes 108: 4096 rows of 8192, rank 64.)
template <class T, class Sh, int ROWS>
__device__ __forceinline__ void down_tile(const LoraParams& p, const T* A, int r0, const int32_t* rows, int m, int s0, int s1,
                                          uint8_t* space, float* part) {
    constexpr int RT = Sh::TILE, STAGE = (ROWS + RT) * 128, D = kDownBytes<Sh> / STAGE < 6 ? kDownBytes<Sh> / STAGE : 6;
    constexpr int PARTS = ROWS / 32, KW = kLoraWarps / PARTS, P = RT + 2;
    static_assert(D >= 3 && kLoraWarps * 32 * P * 4 <= kDownBytes<Sh>, "two stages ahead; the exchange fits");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const uint32_t base = ptx::smem_u32(space);
    // this thread's pieces: column c of rows tid / 8 + 32 i
    const int c = tid & 7, row = tid >> 3;
    const int64_t k_first = static_cast<int64_t>(s0) * kLoraStepK;
    const int64_t k_last = min(static_cast<int64_t>(s1) * kLoraStepK, static_cast<int64_t>(p.K));
    const int chunks = static_cast<int>((k_last - k_first + 63) / 64);
    const uint32_t place = base + row * 128 + ((c ^ (row & 7)) << 4);
    const T* x_ptr[ROWS / 32];
#pragma unroll
    for (int i = 0; i < ROWS / 32; ++i)
        x_ptr[i] = row + 32 * i < m ? static_cast<const T*>(p.X) + static_cast<int64_t>(rows[row + 32 * i]) * p.K + k_first + 8 * c
                                    : nullptr;
    const T* a_ptr = A + static_cast<int64_t>(r0 + row) * p.K + k_first + 8 * c;
    auto fetch = [&](int chunk, int d) {
        const int64_t k = static_cast<int64_t>(chunk) * 64;
        const bool in = k_first + k + 8 * c < k_last;
#pragma unroll
        for (int i = 0; i < ROWS / 32; ++i) {
            const bool take = in && x_ptr[i] != nullptr;
            ptx::cp_async16_or_zero(place + d * STAGE + i * 4096, take ? x_ptr[i] + k : A, take);
        }
#pragma unroll
        for (int i = 0; i < (RT + 31) / 32; ++i) {
            if (RT < 32 && row >= RT) break;
            const bool take = in && r0 + row + 32 * i < p.R;
            ptx::cp_async16_or_zero(place + d * STAGE + ROWS * 128 + i * 4096,
                                    take ? a_ptr + static_cast<int64_t>(32 * i) * p.K + k : A, take);
        }
        ptx::cp_async_commit();
    };
    float acc[2][RT / 8][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < RT / 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.0f;
#pragma unroll
    for (int d = 0; d < D - 1; ++d) fetch(d, d);
    // ldmatrix: lane l gives the address of row l % 8 of matrix l / 8.  Rows: matrices are
    // (rows, k) = (lo, lo), (hi, lo), (lo, hi), (hi, hi); ranks: (lo, lo), (lo, hi), (hi, lo), (hi, hi).
    const int x_row = warp % PARTS * 32 + (lane & 15), x_half = lane >> 4;
    const int a_row = (lane & 7) + ((lane >> 4) << 3), a_half = (lane >> 3) & 1;
    int d = 0;
    for (int i = 0; i < chunks; ++i) {
        ptx::cp_async_wait_group<D - 2>();
        __syncthreads();   // everybody's copies of this chunk are there, the stage before has been read
        fetch(i + D - 1, d == 0 ? D - 1 : d - 1);
        const uint32_t x_at = base + d * STAGE + x_row * 128, a_at = base + d * STAGE + (ROWS + a_row) * 128;
        for (int k = warp / PARTS; k < 4; k += KW) {
            uint32_t x[2][4];
#pragma unroll
            for (int q = 0; q < 2; ++q)
                ptx::ldmatrix_x4_now(x_at + q * 2048 + (((2 * k + x_half) ^ (x_row & 7)) << 4), x[q]);
#pragma unroll
            for (int j = 0; j < RT / 16; ++j) {
                uint32_t a[4];
                ptx::ldmatrix_x4_now(a_at + j * 2048 + (((2 * k + a_half) ^ (a_row & 7)) << 4), a);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    ptx::mma16816<T>(acc[q][2 * j], x[q], a[0], a[1]);
                    ptx::mma16816<T>(acc[q][2 * j + 1], x[q], a[2], a[3]);
                }
            }
        }
        if (++d == D) d = 0;
    }
    ptx::cp_async_wait_group<0>();
    __syncthreads();
    float* red = reinterpret_cast<float*>(space);
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int j = 0; j < RT / 8; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                *reinterpret_cast<float2*>(red + (warp * 32 + 16 * q + 8 * h + g) * P + 8 * j + 2 * t) =
                    make_float2(acc[q][j][2 * h], acc[q][j][2 * h + 1]);
    __syncthreads();
    for (int i = tid; i < m * RT; i += kLoraThreads) {
        const int n = i / RT, r = i % RT;
        if (r0 + r >= p.R) continue;
        const float* from = red + n * P + r;   // row n of part n / 32, of the first warp that has it
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < KW; ++w) v += from[w * PARTS * 32 * P];
        part[n * p.R + r0 + r] = v;
    }
    __syncthreads();
}

// `like`: how many rows decide how the warps share the work, and so the order of a row's sums.
template <class T, class Sh>
__device__ __forceinline__ void down(const LoraParams& p, const T* A, const int32_t* rows, int m, int like, int s0, int s1,
                                     uint8_t* space, float* part) {
    if (like > 32) {
        for (int r0 = 0; r0 < p.R; r0 += Sh::TILE) {
            if constexpr (Sh::TILE == 32) {   // never more than 64 rows
                down_tile<T, Sh, 64>(p, A, r0, rows, m, s0, s1, space, part);
            } else {
                if (like <= 64) down_tile<T, Sh, 64>(p, A, r0, rows, m, s0, s1, space, part);
                else down_tile<T, Sh, 128>(p, A, r0, rows, m, s0, s1, space, part);
            }
        }
        return;
    }
    for (int r0 = 0; r0 < p.R; r0 += 16 * Sh::MT) {
        if (like <= 8) down_rows<T, Sh, Sh::MT, 1>(p, A, r0, rows, m, s0, s1, space, part);
        else if (like <= 16) down_rows<T, Sh, Sh::MT, 2>(p, A, r0, rows, m, s0, s1, space, part);
        else down_rows<T, Sh, Sh::MT, 4>(p, A, r0, rows, m, s0, s1, space, part);
    }
}

// ---------------------------------------------------------------------------- up
// Ranks of a chunk: the MMA steps whose part of B a thread reads with one load, 8
// bytes a row for up to 16 ranks, else 16.  V is kept with zeros up to a whole chunk.
__host__ __device__ constexpr int up_chunk(int R) { return R <= 16 ? 16 : 32; }
__host__ __device__ constexpr int up_ranks(int R) { return (R + up_chunk(R) - 1) / up_chunk(R) * up_chunk(R); }
// Bytes of a row of V in shared memory: groups of four fp32 sums become four hi and four
// lo numbers in the same 16 bytes.  A thread reads one group (or two) of its chunk's; the
// rows' distance keeps eight threads' reads in different banks.
__host__ __device__ constexpr int up_pitch(int R) {
    return up_ranks(R) * 4 + (((R <= 16 ? 64 : 16) - up_ranks(R) * 4) & 127);
}
// rows of V in shared memory at one time
int up_rows(int R) { return R <= 16 ? 128 : (R <= 32 ? 64 : (R <= 64 ? 128 : (R <= 128 ? 64 : 32))); }

// The two numbers of type T that v is the sum of.
template <class T>
__device__ __forceinline__ void cut(float v, float& hi, float& lo) {
    hi = Elem<T>::to_float(Elem<T>::from_float(v));
    lo = fabsf(hi) <= 0x1.fffffep+127f ? v - hi : 0.0f;   // an infinity or NaN goes with hi alone
}

// Biased exponent of the power of two that is taken out of a row whose largest
// magnitude has these bits; it and its reciprocal are normal numbers.
__device__ __forceinline__ uint32_t row_exponent(uint32_t bits) { return min(max(bits >> 23, 1u), 253u); }

// The m rows of V of one group: the cluster's partial sums added in its CTAs' order, times
// the factor, cut.
template <class T>
__device__ __forceinline__ void take_rows(const LoraParams& p, int m, float factor, uint32_t part, uint8_t* v,
                                          uint32_t* row_max) {
    constexpr bool kScaled = std::is_same<T, __half>::value;   // bf16 has fp32's exponents
    const int quads = p.R / 4, items = m * quads, pitch = up_pitch(p.R);
    const int pad = up_ranks(p.R) / 4 - quads;   // at most 6
    for (int i = threadIdx.x; i < m * pad; i += kLoraThreads)
        *reinterpret_cast<uint4*>(v + i / pad * pitch + 16 * (quads + i % pad)) = make_uint4(0u, 0u, 0u, 0u);
    if (kScaled && threadIdx.x < 128) row_max[threadIdx.x] = 0u;
    if (kScaled) __syncthreads();
    for (int i = threadIdx.x; i < items; i += kLoraThreads) {
        const int r = i / quads, q = i - r * quads;
        float o[kLoraMaxCluster][4], a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < kLoraMaxCluster; ++c)
            if (c < p.cluster) ptx::ld_cluster_v4(ptx::mapa(part + 16 * i, c), o[c]);
#pragma unroll
        for (int c = 0; c < kLoraMaxCluster; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) a[e] += c < p.cluster ? o[c][e] : 0.0f;
        uint8_t* at = v + r * pitch + 16 * q;
        float top = 0.0f, h[4], l[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            a[e] *= factor;
            top = fmaxf(top, fabsf(a[e]));
        }
        if constexpr (kScaled) {
            *reinterpret_cast<float4*>(at) = make_float4(a[0], a[1], a[2], a[3]);
            if (top <= 0x1.fffffep+127f) atomicMax(&row_max[r], __float_as_uint(top));   // finite
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) cut<T>(a[e], h[e], l[e]);
            *reinterpret_cast<uint4*>(at) = make_uint4(Elem<T>::pack2(h[0], h[1]), Elem<T>::pack2(h[2], h[3]),
                                                       Elem<T>::pack2(l[0], l[1]), Elem<T>::pack2(l[2], l[3]));
        }
    }
    __syncthreads();
    if constexpr (kScaled) {
        for (int i = threadIdx.x; i < items; i += kLoraThreads) {
            const int r = i / quads, q = i - r * quads;
            uint8_t* at = v + r * pitch + 16 * q;
            const float4 a = *reinterpret_cast<const float4*>(at);
            const float down = __uint_as_float((254u - row_exponent(row_max[r])) << 23);
            float h[4], l[4];
            cut<T>(a.x * down, h[0], l[0]);
            cut<T>(a.y * down, h[1], l[1]);
            cut<T>(a.z * down, h[2], l[2]);
            cut<T>(a.w * down, h[3], l[3]);
            *reinterpret_cast<uint4*>(at) = make_uint4(Elem<T>::pack2(h[0], h[1]), Elem<T>::pack2(h[2], h[3]),
                                                       Elem<T>::pack2(l[0], l[1]), Elem<T>::pack2(l[2], l[3]));
        }
        __syncthreads();
    }
}

// The same rows, not cut, to V: every CTA of the cluster writes a part.
__device__ __forceinline__ void give_rows(const LoraParams& p, int m, float factor, uint32_t part, int rank, const int32_t* order) {
    const int quads = p.R / 4;
    for (int i = rank * blockDim.x + threadIdx.x; i < m * quads; i += p.cluster * blockDim.x) {
        const int r = i / quads, q = i - r * quads;
        float a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < kLoraMaxCluster; ++c) {
            float o[4];
            if (c >= p.cluster) break;
            ptx::ld_cluster_v4(ptx::mapa(part + 16 * i, c), o);
#pragma unroll
            for (int e = 0; e < 4; ++e) a[e] += o[e];
        }
        *reinterpret_cast<float4*>(p.V + static_cast<int64_t>(order[r]) * p.R + 4 * q) =
            make_float4(a[0] * factor, a[1] * factor, a[2] * factor, a[3] * factor);
    }
}

// Fragments of B for 32 columns and one chunk of ranks (S steps of 16).  Column c of
// MMA tile j is column 8 (c / 2) + 2 j + c % 2 of the 32, so that a thread's two of every tile are
// eight in a row of the output; rank 4 S t + 4 k + e of the chunk is thread t's e-th of step k.
// As in the first product, every thread copies its own to places of its own, AHEAD chunks ahead.
template <class T, int S>
struct BFragments {
    uint32_t b[4][2 * S];
    __device__ __forceinline__ void read(uint32_t from) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (S == 1) ptx::ld_shared_v2_u32(from + j * (8 * kLoraThreads), b[j]);
            else ptx::ld_shared_v4_u32(from + j * (16 * kLoraThreads), b[j]);
        }
    }
};
__host__ __device__ constexpr int up_stage_bytes(int S) { return 4 * 8 * S * kLoraThreads; }
template <class Sh>
constexpr int kUpBytes = (Sh::AHEAD + 1) * up_stage_bytes(Sh::S);

// Row blocks of 16 that share a chunk of B in hand.
template <class Sh>
constexpr int kRowBlocks = Sh::LONG ? 4 : 1;

// The chunks of B that a warp multiplies, in order: its 32-column blocks, for LONG every
// chunk of ranks for each kRowBlocks row blocks.  Fetches what comes next, zeros outside.
template <class T, class Sh>
struct BStream {
    static constexpr int S = Sh::S, AHEAD = Sh::AHEAD;
    static constexpr bool LONG = Sh::LONG;
    const T* rows;     // B's rows of this CTA's columns
    uint32_t places;   // this thread's, of stage 0
    int R, columns, row_blocks;
    int nb, rb, k0;    // of the next chunk to fetch
    int in, out;       // stages
    __device__ __forceinline__ void start(const T* b_rows, int R_, int columns_, int m, uint32_t space) {
        rows = b_rows;
        places = space + threadIdx.x * 8 * S;
        R = R_;
        columns = columns_;
        row_blocks = LONG ? (m + 16 * kRowBlocks<Sh> - 1) / (16 * kRowBlocks<Sh>) : 1;
        nb = (threadIdx.x >> 5) * kLoraColumns;
        rb = k0 = in = out = 0;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) fetch();
    }
    __device__ __forceinline__ void fetch() {
        const int lane = threadIdx.x & 31, gr = lane >> 2, t = lane & 3;
        const int r = k0 + 4 * S * t, c0 = nb + 8 * (gr >> 1) + (gr & 1);
        const T* at = rows + static_cast<int64_t>(c0) * R + r;
        const uint32_t to = places + in * up_stage_bytes(S);
        if (nb < columns) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool take = r < R && c0 + 2 * j < columns;
                if constexpr (S == 1) ptx::cp_async8_or_zero(to + j * (8 * kLoraThreads), take ? at + 2 * j * R : rows, take);
                else ptx::cp_async16_or_zero(to + j * (16 * kLoraThreads), take ? at + 2 * j * R : rows, take);
            }
        }
        ptx::cp_async_commit();
        if (++in == AHEAD + 1) in = 0;
        if (LONG) {
            k0 += 16 * S;
            if (k0 < R) return;
            k0 = 0;
            if (++rb < row_blocks) return;
            rb = 0;
        }
        nb += kLoraWarps * kLoraColumns;
    }
    __device__ __forceinline__ void next(BFragments<T, S>& f) {
        ptx::cp_async_wait_group<AHEAD - 1>();
        f.read(places + out * up_stage_bytes(S));
        if (++out == AHEAD + 1) out = 0;
        fetch();
    }
};

// acc (FIRST: =, else +=) V's 16 rows times the fragments of a chunk; v: this thread's
// place in the rows and the chunk.
template <class T, int S, bool FIRST>
__device__ __forceinline__ void up_mma(float (&acc)[4][4], const uint8_t* v, int pitch, const BFragments<T, S>& f) {
#pragma unroll
    for (int k = 0; k < S; ++k) {
        const uint4 f0 = *reinterpret_cast<const uint4*>(v + 16 * k);
        const uint4 f1 = *reinterpret_cast<const uint4*>(v + 8 * pitch + 16 * k);
        const uint32_t hi[4] = {f0.x, f1.x, f0.y, f1.y}, lo[4] = {f0.z, f1.z, f0.w, f1.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (FIRST && k == 0) ptx::mma16816_first<T>(acc[j], hi, f.b[j][2 * k], f.b[j][2 * k + 1]);
            else ptx::mma16816<T>(acc[j], hi, f.b[j][2 * k], f.b[j][2 * k + 1]);
            ptx::mma16816<T>(acc[j], lo, f.b[j][2 * k], f.b[j][2 * k + 1]);
        }
    }
}

// Writes a thread's eight columns of one row: y (times `back` for fp16) + beta C.
template <class T>
__device__ __forceinline__ void up_store(const LoraParams& p, const float (&acc)[4][4], int h, int64_t at, float back) {
    float y[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        y[2 * j] = acc[j][2 * h];
        y[2 * j + 1] = acc[j][2 * h + 1];
    }
    if constexpr (std::is_same<T, __half>::value) {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] *= back;
    }
    if (p.C != nullptr) {
        const uint4 cv = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.C) + at);
        const uint32_t w[4] = {cv.x, cv.y, cv.z, cv.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            y[2 * j] += p.beta * Elem<T>::lo(w[j]);
            y[2 * j + 1] += p.beta * Elem<T>::hi(w[j]);
        }
    }
    *reinterpret_cast<uint4*>(static_cast<T*>(p.U) + at) =
        make_uint4(Elem<T>::pack2(y[0], y[1]), Elem<T>::pack2(y[2], y[3]), Elem<T>::pack2(y[4], y[5]), Elem<T>::pack2(y[6], y[7]));
}

// U of m rows of one group and `columns` columns from n0 on; b: their part of B, on its
// way.  With one chunk (!LONG) its fragments serve all rows.
template <class T, class Sh, int RB>
__device__ __forceinline__ void up(const LoraParams& p, BStream<T, Sh>& b, const int32_t* order, int m, int64_t n0,
                                   int columns, const uint8_t* v_rows, const uint32_t* row_max) {
    constexpr int S = Sh::S;
    constexpr bool LONG = Sh::LONG;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, t = lane & 3, pitch = up_pitch(p.R);
    for (int nb = warp * kLoraColumns; nb < columns; nb += kLoraWarps * kLoraColumns) {
        BFragments<T, S> f;
        if constexpr (!LONG) b.next(f);
        const int64_t n = n0 + nb + 8 * t;   // this thread's 8 columns of the output
        const bool n_in = nb + 8 * t < columns;
        for (int r0 = 0; r0 < m; r0 += 16 * RB) {
            // rows beyond m read what lies there: only outputs that are not written come of it
            const uint8_t* v = v_rows + (r0 + gr) * pitch + 16 * S * t;
            float acc[RB][4][4];
            if constexpr (!LONG) {
                up_mma<T, S, true>(acc[0], v, pitch, f);
            } else {
#pragma unroll
                for (int q = 0; q < RB; ++q)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[q][j][e] = 0.0f;
                for (int k0 = 0; k0 < p.R; k0 += 16 * S) {
                    b.next(f);
#pragma unroll
                    for (int q = 0; q < RB; ++q)
                        if (r0 + 16 * q < m) up_mma<T, S, false>(acc[q], v + 4 * k0 + 16 * q * pitch, pitch, f);
                }
            }
#pragma unroll
            for (int q = 0; q < 2 * RB; ++q) {
                const int r = r0 + gr + 8 * q;
                if (r >= m || !n_in) continue;
                float back = 1.0f;
                if constexpr (std::is_same<T, __half>::value) back = __uint_as_float(row_exponent(row_max[r]) << 23);
                up_store<T>(p, acc[q / 2], q & 1, static_cast<int64_t>(order[r]) * p.N + n, back);
            }
        }
    }
    ptx::cp_async_wait_group<0>();
}

// U = beta C (or zero) of the m rows without an adapter, shared out over all warps in
// parts of up to 1024 columns.
template <class T>
__device__ __forceinline__ void up_none(const LoraParams& p, const int32_t* order, int m) {
    const int lane = threadIdx.x & 31;
    const int64_t parts = (static_cast<int64_t>(p.N) + 1023) / 1024, total = m * parts;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * kLoraWarps;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kLoraWarps + (threadIdx.x >> 5); i < total; i += warps) {
        const int64_t r = div_nonneg(i, parts), n0 = (i - r * parts) * 1024;
        const int64_t row = p.list != nullptr ? __ldcg(order + r) : order[r];
        const float zero[4][4] = {};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t n = n0 + 256 * j + 8 * lane;
            if (n < p.N) up_store<T>(p, zero, 0, row * p.N + n, 1.0f);
        }
    }
}

// Shared memory: the groups; the first product's copies and exchange, then V; the
// second product's copies; the partial sums.
template <class Sh>
__host__ __device__ constexpr int lora_space_bytes(int R, int rows) {
    const int v = rows * up_pitch(R), e = kDownBytes<Sh>;
    return ((v > e ? v : e) + 127) / 128 * 128;
}

// Clusters that share a unit's columns at most.
constexpr int kLoraMaxShare = 8;

// Grid: clusters, which take groups (or units of the list) in turn.  Where the last round leaves
// two clusters or more per unit, they share its columns, each forming V for itself (61 rows
// beside 4-bit 8192 x 4096, rank 64, the whole call: 3 adapters in use 39 -> 29 us, 8 31.5 -> 28,
// 38, two more than the GPU holds at one time, 45 -> 40; where nothing is left to share, 0.2 to 0.7 us
// more.  As code of its own behind the loop: 30.5, 28.3, 46 and 0 to 0.4).
// Two CTAs per SM leave 128 registers: Ranks32 spills 80 bytes there.
template <class T, class Sh>
__global__ void __launch_bounds__(kLoraThreads, Sh::LONG ? 1 : 2) lora_kernel(const LoraParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ uint32_t row_max[128];
    Groups& s = *reinterpret_cast<Groups*>(smem);
    uint8_t* space = smem + kGroupsBytes;
    uint8_t* b_places = space + lora_space_bytes<Sh>(p.R, p.most_rows);
    float* part = reinterpret_cast<float*>(b_places + kUpBytes<Sh>);
    ptx::griddep_wait();
    const int rank = static_cast<int>(ptx::cluster_ctarank());
    int groups;
    if (p.list != nullptr) {
        groups = __ldcg(&p.list->n);
    } else {
        if (p.M <= 32) group_few_rows(p, p.M, s);
        else group_rows(p, p.M, s, *reinterpret_cast<GroupTable*>(space));
        groups = s.n;
    }
    const int s0 = static_cast<int>(static_cast<int64_t>(p.k_steps) * rank / p.cluster);
    const int s1 = static_cast<int>(static_cast<int64_t>(p.k_steps) * (rank + 1) / p.cluster);
    const int most = p.most_rows, clusters = static_cast<int>(ptx::cluster_count());
    // turns: one per unit, or several for each of the last round's; the divisions for these are kept
    // out of the others' way
    int turns = groups;
    if (const int left = groups < clusters ? groups : groups % clusters; left > 0 && 2 * left <= clusters)
        turns += left * (min(clusters / left, kLoraMaxShare) - 1);
    for (int turn = static_cast<int>(ptx::cluster_id()); turn < turns; turn += clusters) {
        int g = turn, from = 0, width = p.width;   // `width` of this CTA's columns, from `from` on
        if (turns > groups) {
            const int whole = groups - groups % clusters;
            if (turn >= whole) {
                const int share = (turns - whole) / (groups - whole);
                width = (p.width / kLoraColumns + share - 1) / share * kLoraColumns;
                g = whole + (turn - whole) / share;
                from = (turn - whole) % share * width;
                width = min(width, p.width - from);
            }
        }
        const int64_t n0 = static_cast<int64_t>(rank) * p.width + from;
        const int columns = static_cast<int>(max(int64_t{0}, min(static_cast<int64_t>(width), p.N - n0)));
        int64_t adapter;
        int begin, end;
        if (p.list != nullptr) {
            const int4 unit = __ldcg(reinterpret_cast<const int4*>(&p.list->units[g]));
            adapter = unit.x;
            begin = 0;
            end = unit.z;   // at most unit_rows <= most
            if (static_cast<int>(threadIdx.x) < end) s.order[threadIdx.x] = __ldcg(&p.list->order[unit.y + threadIdx.x]);
            __syncthreads();
        } else {
            adapter = s.adapter[g];
            begin = s.start[g];
            end = s.start[g + 1];
        }
        const T* A = static_cast<const T*>(p.A) + adapter * p.R * p.K;
        const T* B = static_cast<const T*>(p.B) + (adapter * p.N + n0) * p.R;
        const float factor = p.factors != nullptr ? p.factors[adapter] : 1.0f;
        for (int i = begin; i < end; i += most) {
            const int m = min(most, end - i);
            BStream<T, Sh> b;
            b.start(B, p.R, columns, m, ptx::smem_u32(b_places));   // on its way while V is formed
            down<T, Sh>(p, A, s.order + i, m, p.list != nullptr ? p.unit_rows : m, s0, s1, space, part);
            ptx::cluster_sync();   // every CTA's partial sums are there
            take_rows<T>(p, m, factor, ptx::smem_u32(part), space, row_max);
            ptx::cluster_arrive();   // this CTA has read them
            // The product behind starts only now: from the beginning on, its CTAs took SMs as they came
            // and its prefetches the adapters' bandwidth (64 rows, 8192 x 8192 E4M3, rank 16: the two 39.4 -> 37.0 us;
            // 61 rows beside 4 bits 34.4 -> 34.1, 300 rows 80.7 -> 79.1; 32 rows beside bf16 37.0 -> 38.3).
            ptx::griddep_launch_dependents();
            if (m > 16) up<T, Sh, kRowBlocks<Sh>>(p, b, s.order + i, m, n0, columns, space, row_max);
            else up<T, Sh, 1>(p, b, s.order + i, m, n0, columns, space, row_max);
            ptx::cluster_wait();   // nobody reads this CTA's partial sums any more
            __syncthreads();       // nor V, nor the order
        }
    }
    if (p.list != nullptr) {
        const int with = __ldcg(&p.list->with);
        up_none<T>(p, p.list->order + with, p.M - with);
    } else if (s.start[s.n] < p.M) {
        up_none<T>(p, s.order + s.start[s.n], p.M - s.start[s.n]);
    }
}

// V alone, of up to 16 rows with M R <= kLoraEpiFloats, for the product of a few rows.  That
// runs beside this kernel and hides it, so it takes little of an SM rather than little time.
constexpr int kLoraOnlyThreads = 32 * RanksOnlyV::WARPS;
constexpr int kLoraOnlyBytes = kGroupsBytes + kDownBytes<RanksOnlyV> + kLoraEpiFloats * 4;
static_assert(kLoraOnlyBytes + 2048 <= kLoraBesideBytes, "fits beside the product, with what either CTA has reserved");

template <class T>
__global__ void __launch_bounds__(kLoraOnlyThreads) lora_v_kernel(const LoraParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    Groups& s = *reinterpret_cast<Groups*>(smem);
    uint8_t* space = smem + kGroupsBytes;
    float* part = reinterpret_cast<float*>(space + kDownBytes<RanksOnlyV>);
    ptx::griddep_wait();
    // only now: the product that starts early reads what is written before this kernel, and finds the
    // flag that says so
    if (blockIdx.x == 0 && threadIdx.x == 0) ptx::st_release_gpu(p.ready, 1u);
    __syncthreads();
    ptx::griddep_launch_dependents();
    const int rank = static_cast<int>(ptx::cluster_ctarank());
    group_few_rows(p, p.M, s);
    const int s0 = static_cast<int>(static_cast<int64_t>(p.k_steps) * rank / p.cluster);
    const int s1 = static_cast<int>(static_cast<int64_t>(p.k_steps) * (rank + 1) / p.cluster);
    for (int g = static_cast<int>(ptx::cluster_id()); g < s.n; g += static_cast<int>(ptx::cluster_count())) {
        const int64_t adapter = s.adapter[g];
        const float factor = p.factors != nullptr ? p.factors[adapter] : 1.0f;
        const int m = s.start[g + 1] - s.start[g];
        const int32_t* order = s.order + s.start[g];
        const T* A = static_cast<const T*>(p.A) + adapter * p.R * p.K;
        for (int r0 = 0; r0 < p.R; r0 += 16) {
            if (m <= 8) down_rows<T, RanksOnlyV, 1, 1>(p, A, r0, order, m, s0, s1, space, part);
            else down_rows<T, RanksOnlyV, 1, 2>(p, A, r0, order, m, s0, s1, space, part);
        }
        ptx::cluster_sync();   // every CTA's partial sums are there
        give_rows(p, m, factor, ptx::smem_u32(part), rank, order);
        ptx::cluster_sync();   // and have been read
    }
}

// -------------------------------------------------------------------------- host

// Sets a kernel's preference for shared memory over L1, once per kernel and device.
bool keep_smem(const void* kernel, int dev) {
    static std::mutex mu;
    static std::map<LaunchKey, bool> done;
    std::lock_guard<std::mutex> lock(mu);
    bool& ready = done[LaunchKey{kernel, dev, 0, 0}];
    if (!ready) {
        ready = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) ==
                cudaSuccess;
        if (!ready) cudaGetLastError();
    }
    return ready;
}

// Clusters of 1 .. kLoraMaxCluster CTAs that run at one time.
struct Slots {
    int of[kLoraMaxCluster + 1];
};
Slots cluster_slots(const void* kernel, const DeviceView& dev, int smem) {
    static std::mutex mu;
    static std::map<LaunchKey, Slots> known;
    std::lock_guard<std::mutex> lock(mu);
    const LaunchKey key{kernel, dev.dev, smem, 0};
    const auto at = known.find(key);
    if (at != known.end()) return at->second;
    Slots s{};
    for (int c = 1; c <= kLoraMaxCluster; ++c) s.of[c] = std::max(1, active_clusters(kernel, dev, kLoraThreads, smem, c));
    return known[key] = s;
}

// Work of a launch, as far as the host knows: `units` pieces, within about `spread`, of `rows` rows.
struct Work {
    double units, spread, rows;
};

// How it is shared out: clusters of which size, and with a list units of how many rows.  A
// unit takes 8 us and what its CTAs share, 24 us and one more per row, once for every round of units
// that the GPU cannot hold at one time.  That is 8192 x 4096, rank 64.  The 8, which are order, barriers and
// exchange, do not shrink with K, N and R, but the rule takes them to: small projections get clusters that
// are too large by up to 0.8 us (20, 64 and 200 rows of 4 to 64 adapters: 256 x 256, rank 8, 5.2 to 6.2 us,
// with one CTA each 4.7 to 5.6; 2048 x 2048, rank 16, 5.4 to 7.2, the best sizes 5.3 to 7.1; 4096 x
// 4096, rank 32, no size is better by more than 0.1).
// Adapters are taken to be chosen evenly, from all or from half of them.
// Measured, adapters alone in a graph:
//   61 rows, rank 64, clusters of 8, 6, 4, 3, 2: 16 adapters in use 17.8, 12.3, 14.6, 17.1, 21.8 us
//   (the GPU holds 15, 23, 36, 46, 76 of them), 36 adapters 28.7, 24.0, 17.2, 19.1, 23.4, 40 adapters
//   29.2, 24.4, 28.6, 19.4, 23.5;  4096 rows of 30 adapters, 4096 x 1024, rank 128, units of 64
//   rows, clusters of 4, 2, 1: 78, 64, 100;  four of rank 256, units of 32: 204, 166, 155.
//   Five and seven gain nothing on their neighbours (rank 16: 9.6 us with five, 8.3 with four).
struct Share {
    int cluster = 0, rows = 0;
    double cost = 0.0;
};
void weigh(Share& best, const Slots& slots, const Work (&work)[2], int unit_rows) {
    for (int c : {8, 6, 4, 3, 2, 1}) {
        const double s = slots.of[c];
        double cost = 0.0;
        for (const Work& w : work) {
            const double rounds = 0.5 * std::ceil(w.units / s) + 0.25 * std::ceil(std::max(w.units - w.spread, 1.0) / s) +
                                  0.25 * std::ceil((w.units + w.spread) / s);
            cost += rounds * (8.0 + (24.0 + w.rows) / c);
        }
        if (best.cluster == 0 || cost < best.cost) best = Share{c, unit_rows, cost};
    }
}

// Fills the split of `p` and launches.
//  - Up to 256 rows, a batch of requests, make as many groups as adapters are in use.  Where
//    all clusters fit the GPU with one CTA per SM, they get one each (by asking for
//    more than half of its shared memory): started while the kernel before drains, two would go
//    to the SMs that are free first (61 rows, 48 adapters of rank 64 beside 4-bit
//    8192 x 4096, the whole call: 39 -> 36 us).
//    An adapter's rows are not cut: one with most of them is taken by one cluster, up_rows at a time,
//    and by the clusters that share its columns, which each form V again.  256 rows of one adapter of
//    8192 x 8192, rank 16, 64, 256: 23, 52, 278 us, and 257 rows, in units, 13, 20, 54; of four adapters 11, 20,
//    82 and 14, 20, 55.
//  - More rows are cut into units of 32, 64 or 128 rows; an adapter's last one is half full.
template <class T, class Sh>
gemm_status_t launch(LoraParams p, const DeviceView& dev, cudaStream_t s) {
    const auto kernel = lora_kernel<T, Sh>;
    p.most_rows = up_rows(p.R);
    int smem = kGroupsBytes + lora_space_bytes<Sh>(p.R, p.most_rows) + kUpBytes<Sh> + p.most_rows * p.R * 4;
    const Slots slots = cluster_slots(reinterpret_cast<const void*>(kernel), dev, smem);
    const double M = p.M, all = std::max(1, p.count), half = std::max(1.0, all / 2);
    Share share;
    int clusters;
    if (p.list == nullptr) {
        auto groups = [&](double count) {   // adapters in use, their standard deviation
            const double empty = std::exp(-M / count), n = std::max(1.0, count * (1.0 - std::pow(1.0 - 1.0 / count, M)));
            return Work{n, 1.2 * std::sqrt(std::max(0.0, count * empty * (1.0 - (1.0 + M / count) * empty))), M / n};
        };
        const Work work[2] = {groups(all), groups(half)};
        weigh(share, slots, work, 0);
        const int alone = std::max(smem, kMaxDynamicSmem / 2 + 2048);
        const Slots slots_alone = cluster_slots(reinterpret_cast<const void*>(kernel), dev, alone);
        clusters = slots.of[share.cluster];
        if (work[0].units <= slots_alone.of[share.cluster]) {
            smem = alone;
            clusters = slots_alone.of[share.cluster];
        }
        // one CTA per SM; more only where there may be as many groups
        const int most = static_cast<int>(std::min<int64_t>(p.M, std::max(1, p.count)));
        clusters = std::min(clusters, std::max(most, dev.sms / share.cluster));
    } else {
        for (int rows = 32; rows <= p.most_rows; rows *= 2) {
            auto units = [&](double count) {
                const double used = count * (1.0 - std::exp(-M / count));
                return Work{used * std::max(1.0, M / count / rows + 0.5), 0.6 * std::sqrt(used), static_cast<double>(rows)};
            };
            weigh(share, slots, {units(all), units(half)}, rows);
        }
        p.unit_rows = share.rows;
        clusters = slots.of[share.cluster];
        const int bits = list_bits(p.M);
        const gemm_status_t st = launch_clusters(lora_list_kernel, dev.dev, dim3(1, 1, 1), kListThreads, 1,
                                                 (2 << bits) * 4 + 16, true, s, p, const_cast<LoraList*>(p.list), bits);
        if (st != GEMM_OK) return st;
    }
    p.cluster = share.cluster;
    const int64_t per = p.cluster * kLoraColumns;
    p.width = static_cast<int32_t>((p.N + per - 1) / per * kLoraColumns);
    return launch_clusters(kernel, dev.dev, dim3(static_cast<unsigned>(clusters * p.cluster), 1, 1), kLoraThreads, p.cluster,
                           smem, true, s, p);
}

// Eight CTAs per adapter in use, on as many SMs as there are.  The SMs keep all of their
// shared memory as such, or the product's CTAs would wait for them to change over.
template <class T>
gemm_status_t launch_v(LoraParams p, const DeviceView& dev, cudaStream_t s) {
    const auto kernel = lora_v_kernel<T>;
    if (!keep_smem(reinterpret_cast<const void*>(kernel), dev.dev)) return GEMM_ERR_CUDA;
    p.cluster = 8;
    const int clusters = std::min(std::max(1, dev.sms / p.cluster), std::min(p.M, p.count));
    return launch_clusters(kernel, dev.dev, dim3(static_cast<unsigned>(clusters * p.cluster), 1, 1), kLoraOnlyThreads,
                           p.cluster, kLoraOnlyBytes, true, s, p);
}

template <class T>
gemm_status_t run(const LoraParams& p, const DeviceView& dev, cudaStream_t s) {
    if (p.V != nullptr) return launch_v<T>(p, dev, s);
    if (p.R <= 16) return launch<T, Ranks16>(p, dev, s);
    if (p.R <= 32) return launch<T, Ranks32>(p, dev, s);
    return launch<T, RanksMore>(p, dev, s);
}

}  // namespace

size_t lora_scratch_bytes(int64_t M) { return M > kLoraTile ? sizeof(LoraList) : 0; }

gemm_status_t run_lora(bool bf16, const LoraArgs& a, uint8_t* data, const DeviceView& dev, cudaStream_t s) {
    for (int64_t m0 = 0; m0 < a.M; m0 += kListRows) {
        const int64_t M = std::min<int64_t>(kListRows, a.M - m0);
        LoraParams p{};
        p.X = static_cast<const uint16_t*>(a.X) + m0 * a.K;
        p.A = a.A;
        p.B = a.B;
        p.factors = a.factors;
        p.ids = a.K > 0 && a.count > 0 ? a.ids + m0 : nullptr;
        p.list = M > kLoraTile ? reinterpret_cast<const LoraList*>(data) : nullptr;
        p.C = a.C != nullptr ? static_cast<const uint16_t*>(a.C) + m0 * a.N : nullptr;
        p.U = static_cast<uint16_t*>(a.U) + m0 * a.N;
        p.V = a.V;
        p.ready = a.ready;
        p.M = static_cast<int32_t>(M);
        p.N = static_cast<int32_t>(a.N);
        p.K = static_cast<int32_t>(a.K);
        p.R = static_cast<int32_t>(a.R);
        p.count = static_cast<int32_t>(a.count);
        p.k_steps = static_cast<int32_t>((a.K + kLoraStepK - 1) / kLoraStepK);
        p.beta = a.beta;
        const gemm_status_t st = bf16 ? run<__nv_bfloat16>(p, dev, s) : run<__half>(p, dev, s);
        if (st != GEMM_OK) return st;
    }
    return GEMM_OK;
}

}  // namespace gemm_gb300
