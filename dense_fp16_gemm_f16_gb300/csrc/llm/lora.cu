// lora.cu -- low-rank adapters of many requests:
//   U[m] = beta C[m] + c_a (X[m] A_aᵀ) B_aᵀ,  a = ids[m].
//
// One kernel.  Rows are taken in tiles of up to 256; a CTA puts the rows of a tile in
// order of their adapters itself, so no list has to be made by a kernel before, and every
// adapter's matrices are read once per tile.  A cluster of eight CTAs takes one
// adapter's rows: each CTA forms V = X Aᵀ over an eighth of K, the partial sums meet in
// distributed shared memory in a fixed order, and each CTA multiplies V by an
// eighth of B's rows.
// Each byte meets few others (R is small): the operands go straight from global
// memory to mma.sync fragments.  The k order within an MMA is free, so a thread's
// 16 (or 8) consecutive bytes of a row are its slots of two steps (or one).
// Bound by bytes: A and B of the adapters in use for a few rows, X, C and U for many.
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

#include "llm/llm.h"
#include "llm/rows_host.cuh"
#include "llm/stream.cuh"

namespace gemm_gb300 {
namespace {

constexpr int kLoraThreads = 256;
constexpr int kLoraWarps = kLoraThreads / 32;
constexpr int kLoraTile = 256;           // most rows per tile: one per thread
constexpr int kLoraStepK = 32;           // k per warp and step of `down`: 16 bytes per thread and row
constexpr int kLoraColumns = 32;         // columns per warp and step of `up`
constexpr int kLoraCluster = 8;

struct LoraParams {
    const void* X;           // [M][K]
    const void* A;           // [count][R][K]
    const void* B;           // [count][N][R]
    const float* factors;    // [count] or nullptr
    const int32_t* ids;      // [M], or nullptr: no row has an adapter
    const void* C;           // [M][N] or nullptr
    void* U;                 // [M][N]
    int32_t M, N, K, R, count;
    int32_t tile_rows, k_steps, width;   // width: columns per CTA of a cluster
    float beta;
};

// The rows of one tile in order of their adapters, and the table that finds them.
constexpr int kLoraSlots = 2 * kLoraTile;
struct Groups {
    int32_t order[kLoraTile];         // rows of the tile, group by group, each in row order
    int32_t start[kLoraTile + 1];     // group i is order[start[i]] .. order[start[i + 1] - 1]
    int32_t adapter[kLoraTile];       // of each group, in the order of their first rows
    int32_t key[kLoraSlots];          // the adapter that has this slot, -1 free
    int32_t first[kLoraSlots];        // its first row, then its group
    alignas(16) uint8_t rows[kLoraSlots][kLoraWarps];   // its rows in each warp
    int32_t leaders[kLoraWarps];
    int32_t none[kLoraWarps];         // rows without an adapter in each warp
    int32_t n;                        // groups with an adapter; rows without one lie behind them
};
static_assert(kLoraWarps == 8, "a slot's row counts are read as 8 bytes");
constexpr int kGroupsBytes = (sizeof(Groups) + 127) / 128 * 128;

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
__device__ void group_rows(const LoraParams& p, int row0, int rows, Groups& s) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int id = -2;   // no row
    if (tid < rows) {
        id = p.ids != nullptr ? __ldcg(p.ids + row0 + tid) : -1;
        if (id < 0 || id >= p.count) id = -1;
    }
#pragma unroll
    for (int i = tid; i < kLoraSlots; i += kLoraThreads) {
        s.key[i] = -1;
        s.first[i] = kLoraTile;
        *reinterpret_cast<uint2*>(s.rows[i]) = make_uint2(0u, 0u);
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
            const int other = atomicCAS(&s.key[slot], -1, id);
            if (other == -1 || other == id) break;
            slot = (slot + 1) & (kLoraSlots - 1);
        }
        s.rows[slot][warp] = static_cast<uint8_t>(__popc(mine));
        atomicMin(&s.first[slot], tid);
    }
    slot = __shfl_sync(0xffffffffu, slot, lead_lane);
    const uint32_t none = __ballot_sync(0xffffffffu, id == -1);
    if (lane == 0) s.none[warp] = __popc(none);
    __syncthreads();
    const bool leads = id >= 0 && s.first[slot] == tid;
    const uint32_t mask = __ballot_sync(0xffffffffu, leads);
    if (lane == 0) s.leaders[warp] = __popc(mask);
    __syncthreads();
    int number = __popc(mask & ((1u << lane) - 1u)), n = 0, before = 0;
#pragma unroll
    for (int w = 0; w < kLoraWarps; ++w) {
        if (w < warp) {
            number += s.leaders[w];
            before += s.none[w];
        }
        n += s.leaders[w];
    }
    if (leads) {
        s.first[slot] = number;
        s.adapter[number] = id;
        s.start[number] = rows_before(s.rows[slot], kLoraWarps);   // sizes first
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
    if (id >= 0) s.order[s.start[s.first[slot]] + rows_before(s.rows[slot], warp) + in_warp] = tid;
    else if (id == -1) s.order[s.start[n] + before + in_warp] = tid;
    __syncthreads();
}

// -------------------------------------------------------------------------- down
// 16-byte loads of a thread that are under way at one time, and how many steps make them.
template <int MT, int NT>
constexpr int kDownUnroll = 12 / (2 * MT + NT);
// Floats between the sums of two rows in the warps' exchange: the two columns of
// a fragment fall into different banks.
__host__ __device__ constexpr int down_pitch(int MT) { return 16 * MT + 4; }
__host__ __device__ constexpr int down_bytes(int MT) { return kLoraWarps * 32 * down_pitch(MT) * 4; }

// part = V of m <= 8 NT WR rows (`rows`) and 16 MT ranks from r0 on over the k steps
// [s0, s1): WR parts of 8 NT rows, the steps of each dealt out to 8 / WR warps.
template <class T, int MT, int NT, int WR>
__device__ __forceinline__ void down_rows(const LoraParams& p, const T* A, int r0, const int32_t* rows, int m, int row0,
                                          int s0, int s1, float* red, float* part) {
    constexpr int KW = kLoraWarps / WR, UN = kDownUnroll<MT, NT>, P = down_pitch(MT);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int first = warp / KW * 8 * NT;   // this warp's rows
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    const T* a_ptr = A + static_cast<int64_t>(r0 + g) * p.K + 8 * t;
    const T* x_ptr[NT];
    bool x_in[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        x_in[j] = first + 8 * j + g < m;
        x_ptr[j] = static_cast<const T*>(p.X) + static_cast<int64_t>(row0 + (x_in[j] ? rows[first + 8 * j + g] : 0)) * p.K + 8 * t;
    }
    float acc[MT][NT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.0f;
    if (first < m) {
        for (int s = s0 + warp % KW; s < s1; s += KW * UN) {
            uint4 a[UN][MT][2], x[UN][NT];
#pragma unroll
            for (int u = 0; u < UN; ++u) {
                const int64_t k = static_cast<int64_t>(s + u * KW) * kLoraStepK;
                const bool in = s + u * KW < s1 && k + 8 * t < p.K;   // K % 8 == 0: all eight or none
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        a[u][i][h] = in && r0 + 16 * i + 8 * h + g < p.R
                                         ? *reinterpret_cast<const uint4*>(a_ptr + (16 * i + 8 * h) * static_cast<int64_t>(p.K) + k)
                                         : none;
#pragma unroll
                for (int j = 0; j < NT; ++j) x[u][j] = in && x_in[j] ? *reinterpret_cast<const uint4*>(x_ptr[j] + k) : none;
            }
#pragma unroll
            for (int u = 0; u < UN; ++u)
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const uint32_t lo[4] = {a[u][i][0].x, a[u][i][1].x, a[u][i][0].y, a[u][i][1].y};
                    const uint32_t hi[4] = {a[u][i][0].z, a[u][i][1].z, a[u][i][0].w, a[u][i][1].w};
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        ptx::mma16816<T>(acc[i][j], lo, x[u][j].x, x[u][j].y);
                        ptx::mma16816<T>(acc[i][j], hi, x[u][j].z, x[u][j].w);
                    }
                }
        }
    }
    // the sums of a part's warps meet in shared memory and are added in their order
    float* mine = red + warp * 8 * NT * P;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) mine[(8 * j + 2 * t + (e & 1)) * P + 16 * i + g + 8 * (e >> 1)] = acc[i][j][e];
    __syncthreads();
    for (int i = threadIdx.x; i < m * 16 * MT; i += kLoraThreads) {
        const int n = i / (16 * MT), r = i % (16 * MT);
        if (r0 + r >= p.R) continue;
        const float* from = red + (n / (8 * NT) * KW * 8 * NT + n % (8 * NT)) * P + r;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < KW; ++w) v += from[w * 8 * NT * P];
        part[n * p.R + r0 + r] = v;
    }
    __syncthreads();
}

template <class T, int MT>
__device__ __forceinline__ void down(const LoraParams& p, const T* A, const int32_t* rows, int m, int row0, int s0, int s1,
                                     float* red, float* part) {
    for (int r0 = 0; r0 < p.R; r0 += 16 * MT) {
        if (m <= 8) down_rows<T, MT, 1, 1>(p, A, r0, rows, m, row0, s0, s1, red, part);
        else if (m <= 16) down_rows<T, MT, 2, 1>(p, A, r0, rows, m, row0, s0, s1, red, part);
        else if (m <= 32) down_rows<T, MT, 4, 1>(p, A, r0, rows, m, row0, s0, s1, red, part);
        else if (m <= 64) down_rows<T, MT, 4, 2>(p, A, r0, rows, m, row0, s0, s1, red, part);
        else down_rows<T, MT, 4, 4>(p, A, r0, rows, m, row0, s0, s1, red, part);
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
__host__ __device__ constexpr int up_rows(int R) { return R <= 64 ? 128 : (R <= 128 ? 64 : 32); }

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
        float o[kLoraCluster][4], a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < kLoraCluster; ++c) ptx::ld_cluster_v4(ptx::mapa(part + 16 * i, c), o[c]);
#pragma unroll
        for (int c = 0; c < kLoraCluster; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) a[e] += o[c][e];
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

// Fragments of B for 32 columns and one chunk of ranks (S steps of 16).  Column c of
// MMA tile j is column 8 (c / 2) + 2 j + c % 2 of the 32, so that a thread's two of every tile are
// eight in a row of the output; rank 4 S t + 4 k + e of the chunk is thread t's e-th of step k.
template <class T, int S>
struct BFragments {
    uint32_t b[4][2 * S];
    __device__ __forceinline__ void load(const T* rows, int R, int k0, int nb, int columns, int gr, int t) {
        const int r = k0 + 4 * S * t, c0 = nb + 8 * (gr >> 1) + (gr & 1);
        const T* at = rows + static_cast<int64_t>(c0) * R + r;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool in = r < R && c0 + 2 * j < columns;
            if constexpr (S == 1) {
                const uint2 v = in ? *reinterpret_cast<const uint2*>(at + 2 * j * R) : make_uint2(0u, 0u);
                b[j][0] = v.x;
                b[j][1] = v.y;
            } else {
                const uint4 v = in ? *reinterpret_cast<const uint4*>(at + 2 * j * R) : make_uint4(0u, 0u, 0u, 0u);
                b[j][0] = v.x;
                b[j][1] = v.y;
                b[j][2] = v.z;
                b[j][3] = v.w;
            }
        }
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

// U of m rows of one group and `columns` columns from n0 on; b_rows: their part of B.
// The next fragments are on their way while a chunk is multiplied; with one chunk
// (!LONG) they serve all rows.
template <class T, int S, bool LONG>
__device__ __forceinline__ void up(const LoraParams& p, const T* b_rows, const int32_t* order, int m, int row0, int64_t n0,
                                   int columns, const uint8_t* v_rows, const uint32_t* row_max) {
    constexpr int kStride = kLoraWarps * kLoraColumns;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, t = lane & 3, pitch = up_pitch(p.R);
    BFragments<T, S> next;
    if (warp * kLoraColumns < columns) next.load(b_rows, p.R, 0, warp * kLoraColumns, columns, gr, t);
    for (int nb = warp * kLoraColumns; nb < columns; nb += kStride) {
        BFragments<T, S> b = next;
        if (!LONG && nb + kStride < columns) next.load(b_rows, p.R, 0, nb + kStride, columns, gr, t);
        const int64_t n = n0 + nb + 8 * t;   // this thread's 8 columns of the output
        const bool n_in = nb + 8 * t < columns;
        for (int rb = 0; rb < m; rb += 16) {
            // rows beyond m read what lies there: only outputs that are not written come of it
            const uint8_t* v = v_rows + (rb + gr) * pitch + 16 * S * t;
            float acc[4][4];
            if constexpr (!LONG) {
                up_mma<T, S, true>(acc, v, pitch, b);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[j][e] = 0.0f;
                for (int k0 = 0; k0 < p.R; k0 += 16 * S) {
                    b = next;
                    if (k0 + 16 * S < p.R) next.load(b_rows, p.R, k0 + 16 * S, nb, columns, gr, t);
                    else if (rb + 16 < m) next.load(b_rows, p.R, 0, nb, columns, gr, t);
                    else if (nb + kStride < columns) next.load(b_rows, p.R, 0, nb + kStride, columns, gr, t);
                    up_mma<T, S, false>(acc, v + 4 * k0, pitch, b);
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = rb + gr + 8 * h;
                if (r >= m || !n_in) continue;
                float back = 1.0f;
                if constexpr (std::is_same<T, __half>::value) back = __uint_as_float(row_exponent(row_max[r]) << 23);
                up_store<T>(p, acc, h, static_cast<int64_t>(row0 + order[r]) * p.N + n, back);
            }
        }
    }
}

// U = beta C (or zero) of rows without an adapter.
template <class T>
__device__ void up_none(const LoraParams& p, const int32_t* order, int m, int row0, int64_t n0, int columns) {
    const int vecs = columns / 8;
    for (int i = threadIdx.x; i < m * vecs; i += kLoraThreads) {
        const int r = i / vecs;
        const float zero[4][4] = {};
        up_store<T>(p, zero, 0, static_cast<int64_t>(row0 + order[r]) * p.N + n0 + 8 * (i - r * vecs), 1.0f);
    }
}

// Shared memory: the groups, the warps' exchange and later V, the partial sums.
__host__ __device__ constexpr int lora_exchange_bytes(int MT, int R) {
    const int v = up_rows(R) * up_pitch(R), e = down_bytes(MT);
    return ((v > e ? v : e) + 127) / 128 * 128;
}

// Grid: clusters that share a tile, tiles; a cluster takes groups in turn, the last
// of which is the rows without an adapter.  MT: 16-row tiles of ranks of the first
// product in hand; S: steps of 16 ranks per chunk, LONG: R has more than one chunk.
template <class T, int MT, int S, bool LONG>
__global__ void __launch_bounds__(kLoraThreads, 2) lora_kernel(const LoraParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ uint32_t row_max[128];
    Groups& s = *reinterpret_cast<Groups*>(smem);
    uint8_t* exchange = smem + kGroupsBytes;
    float* part = reinterpret_cast<float*>(exchange + lora_exchange_bytes(MT, p.R));
    ptx::griddep_wait();
    // only now: what starts early may then rely on everything before this kernel
    ptx::griddep_launch_dependents();
    const int rank = static_cast<int>(ptx::cluster_ctarank());
    const int row0 = static_cast<int>(blockIdx.y) * p.tile_rows;
    const int rows = min(p.tile_rows, p.M - row0);
    group_rows(p, row0, rows, s);
    const int groups = s.n + (s.start[s.n] < rows ? 1 : 0);
    const int64_t n0 = static_cast<int64_t>(rank) * p.width;
    const int columns = static_cast<int>(max(int64_t{0}, min(static_cast<int64_t>(p.width), p.N - n0)));
    const int s0 = static_cast<int>(static_cast<int64_t>(p.k_steps) * rank / kLoraCluster);
    const int s1 = static_cast<int>(static_cast<int64_t>(p.k_steps) * (rank + 1) / kLoraCluster);
    const int most = up_rows(p.R);
    for (int g = blockIdx.x / kLoraCluster; g < groups; g += gridDim.x / kLoraCluster) {
        const bool has = g < s.n;
        const int end = has ? s.start[g + 1] : rows;
        const int64_t adapter = has ? s.adapter[g] : 0;
        const T* A = static_cast<const T*>(p.A) + adapter * p.R * p.K;
        const T* B = static_cast<const T*>(p.B) + (adapter * p.N + n0) * p.R;
        const float factor = has && p.factors != nullptr ? p.factors[adapter] : 1.0f;
        if (has && threadIdx.x == 0 && columns > 0)   // on its way while V is formed
            ptx::bulk_prefetch_l2(B, static_cast<uint32_t>(min(static_cast<int64_t>(columns) * p.R * 2, int64_t{1} << 20)));
        for (int i = s.start[g]; i < end; i += most) {
            const int m = min(most, end - i);
            if (!has) {
                up_none<T>(p, s.order + i, m, row0, n0, columns);
                continue;
            }
            down<T, MT>(p, A, s.order + i, m, row0, s0, s1, reinterpret_cast<float*>(exchange), part);
            ptx::cluster_sync();   // every CTA's partial sums are there
            take_rows<T>(p, m, factor, ptx::smem_u32(part), exchange, row_max);
            ptx::cluster_arrive();   // this CTA has read them
            up<T, S, LONG>(p, B, s.order + i, m, row0, n0, columns, exchange, row_max);
            ptx::cluster_wait();   // nobody reads this CTA's partial sums any more
            __syncthreads();       // nor V
        }
    }
}

// -------------------------------------------------------------------------- host
constexpr int64_t kLoraRows = 1 << 20;   // rows per launch: tiles are the grid's second dimension

template <class T, int MT, int S, bool LONG>
gemm_status_t launch(const LoraParams& p, dim3 grid, const DeviceView& dev, cudaStream_t s) {
    const int smem = kGroupsBytes + lora_exchange_bytes(MT, p.R) + up_rows(p.R) * p.R * 4;
    return launch_clusters(lora_kernel<T, MT, S, LONG>, dev.dev, grid, kLoraThreads, kLoraCluster, smem, true, s, p);
}

template <class T>
gemm_status_t run(const LoraParams& p, dim3 grid, const DeviceView& dev, cudaStream_t s) {
    if (p.R <= 16) return launch<T, 1, 1, false>(p, grid, dev, s);
    if (p.R <= 32) return launch<T, 2, 2, false>(p, grid, dev, s);
    return launch<T, 2, 2, true>(p, grid, dev, s);
}

}  // namespace

gemm_status_t run_lora(bool bf16, const LoraArgs& a, const DeviceView& dev, cudaStream_t s) {
    for (int64_t m0 = 0; m0 < a.M; m0 += kLoraRows) {
        const int64_t M = std::min(kLoraRows, a.M - m0);
        LoraParams p{};
        p.X = static_cast<const uint16_t*>(a.X) + m0 * a.K;
        p.A = a.A;
        p.B = a.B;
        p.factors = a.factors;
        p.ids = a.K > 0 && a.count > 0 ? a.ids + m0 : nullptr;
        p.C = a.C != nullptr ? static_cast<const uint16_t*>(a.C) + m0 * a.N : nullptr;
        p.U = static_cast<uint16_t*>(a.U) + m0 * a.N;
        p.M = static_cast<int32_t>(M);
        p.N = static_cast<int32_t>(a.N);
        p.K = static_cast<int32_t>(a.K);
        p.R = static_cast<int32_t>(a.R);
        p.count = static_cast<int32_t>(a.count);
        p.k_steps = static_cast<int32_t>((a.K + kLoraStepK - 1) / kLoraStepK);
        p.beta = a.beta;
        const int64_t per = kLoraCluster * kLoraColumns;
        p.width = static_cast<int32_t>((a.N + per - 1) / per * kLoraColumns);
        // Two CTAs per SM, shared out over the tiles.  A batch of requests is one tile with
        // many groups, a prompt's tiles have one or two each.
        const int64_t most = 2 * dev.sms / kLoraCluster;
        const int64_t even = ((M + most - 1) / most + 15) / 16 * 16;
        p.tile_rows = M <= kLoraTile ? kLoraTile : static_cast<int32_t>(std::min<int64_t>(kLoraTile, std::max<int64_t>(96, even)));
        const int64_t tiles = (M + p.tile_rows - 1) / p.tile_rows;
        int64_t clusters = std::max<int64_t>(1, most / tiles);
        if (tiles == 1) clusters = std::min({clusters, M, a.count + 1});
        const dim3 grid(static_cast<unsigned>(clusters * kLoraCluster), static_cast<unsigned>(tiles), 1);
        const gemm_status_t st = bf16 ? run<__nv_bfloat16>(p, grid, dev, s) : run<__half>(p, grid, dev, s);
        if (st != GEMM_OK) return st;
    }
    return GEMM_OK;
}

}  // namespace gemm_gb300
