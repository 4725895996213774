// lora.cu -- low-rank adapters of many requests:
//   U[m] = beta C[m] + c_a (X[m] A_aᵀ) B_aᵀ,  a = ids[m],
// in two kernels.  `down` forms the rows V = X A_aᵀ (K split over CTAs, partial sums
// in scratch), `up` adds the partial sums and multiplies by B_aᵀ.
//
// Rows are taken in tiles of up to 256; a CTA puts the rows of a tile in order of
// their adapters itself (one comparison of every pair of ids), so no list has to be
// made by a kernel before, and every adapter's matrices are read once per tile.
// Each byte meets few others (R is small): the operands go straight from global
// memory to mma.sync fragments.  The k order within an MMA is free, so a thread's
// 16 (or 8) consecutive bytes of a row are its slots of two steps (or one).
// Bound by bytes: A and B of the adapters in use for a few rows, X, C and U for many.
//
// V is a sum in fp32.  For the second product it is cut into two numbers of the
// operands' type, hi + lo, after scaling each row by a power of two to about 1: the
// product then has twice the type's precision, and fp16's range does not matter.
// U is rounded once; where U is the C of a product that follows, its rounding adds
// u |U| to that product's own u |D|.  The other way, U in fp32, would cost a
// prompt twice the bytes for a part that is small beside the projection's.
#include <algorithm>

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
constexpr int kLoraMaxPieces = 32;

struct LoraParams {
    const void* X;           // [M][K]
    const void* A;           // [count][R][K]
    const void* B;           // [count][N][R]
    const float* factors;    // [count] or nullptr
    const int32_t* ids;      // [M], or nullptr: no row has an adapter
    const void* C;           // [M][N] or nullptr
    void* U;                 // [M][N]
    float* part;             // [pieces][M][R]
    int32_t M, N, K, R, count;
    int32_t tile_rows, pieces, k_steps, width;
    float beta;
};

// The rows of one tile in order of their adapters.
struct Groups {
    int32_t id[kLoraTile];            // adapter of each row, -1 none, -2 no row
    int32_t order[kLoraTile];         // rows of the tile, group by group
    int32_t start[kLoraTile + 1];     // group i is order[start[i]] .. order[start[i + 1] - 1]
    int32_t adapter[kLoraTile];       // of each group
    int32_t number[kLoraTile];        // of the group that a row leads
    int32_t leaders[kLoraWarps];
    int32_t n;                        // groups with an adapter; rows without one lie behind them
};

constexpr int kGroupsBytes = (sizeof(Groups) + 127) / 128 * 128;

// Called by the whole CTA.  Ids are read past L1: a kernel launched early may share
// an SM with one that read older ids there.
__device__ void group_rows(const LoraParams& p, int row0, int rows, Groups& s) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int id = -2;
    if (tid < rows) {
        id = p.ids != nullptr ? __ldcg(p.ids + row0 + tid) : -1;
        if (id < 0 || id >= p.count) id = -1;
    }
    s.id[tid] = id;
    __syncthreads();
    int first = tid, before = 0, all = 0;
    for (int j = 0; j < rows; j += 4) {
        const int4 v = *reinterpret_cast<const int4*>(&s.id[j]);
        const int o[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (o[e] == id) {
                first = min(first, j + e);
                before += j + e < tid ? 1 : 0;
                ++all;
            }
        }
    }
    const bool leads = id >= 0 && before == 0;
    const uint32_t mask = __ballot_sync(0xffffffffu, leads);
    if (lane == 0) s.leaders[warp] = __popc(mask);
    s.start[tid] = 0;
    __syncthreads();
    int number = __popc(mask & ((1u << lane) - 1u)), n = 0;
    for (int w = 0; w < kLoraWarps; ++w) {
        if (w < warp) number += s.leaders[w];
        n += s.leaders[w];
    }
    if (leads) {
        s.number[tid] = number;
        s.adapter[number] = id;
        s.start[number] = all;   // sizes first
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
    if (id >= 0) s.order[s.start[s.number[first]] + before] = tid;
    else if (id == -1) s.order[s.start[n] + before] = tid;
    __syncthreads();
}

// -------------------------------------------------------------------------- down
// Bytes between the sums of two rows in the warps' exchange: the two columns of
// a fragment fall into different banks.
__host__ __device__ constexpr int down_pitch(int MT) { return 16 * MT + 4; }
constexpr int down_smem(int MT, int NT) { return kGroupsBytes + kLoraWarps * 8 * NT * down_pitch(MT) * 4; }

// V of up to 8 NT rows (`rows`, m of them) and 16 MT ranks from r0 on over the k
// steps [s0, s1), which the warps take in turn.
template <class T, int MT, int NT>
__device__ __forceinline__ void down_rows(const LoraParams& p, const T* A, int r0, const int32_t* rows, int m, int row0,
                                          int s0, int s1, int piece, float* red) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    const T* a_ptr[MT][2];
    const T* x_ptr[NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = r0 + 16 * i + 8 * h + g;
            a_ptr[i][h] = r < p.R ? A + static_cast<int64_t>(r) * p.K : nullptr;
        }
#pragma unroll
    for (int j = 0; j < NT; ++j)
        x_ptr[j] = 8 * j + g < m ? static_cast<const T*>(p.X) + static_cast<int64_t>(row0 + rows[8 * j + g]) * p.K : nullptr;
    float acc[MT][NT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.0f;
    for (int s = s0 + warp; s < s1; s += kLoraWarps) {
        const int64_t k = static_cast<int64_t>(s) * kLoraStepK + 8 * t;
        const bool in = k < p.K;   // K % 8 == 0: all eight or none
        uint4 a[MT][2], x[NT];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                a[i][h] = in && a_ptr[i][h] != nullptr ? *reinterpret_cast<const uint4*>(a_ptr[i][h] + k) : none;
#pragma unroll
        for (int j = 0; j < NT; ++j)
            x[j] = in && x_ptr[j] != nullptr ? *reinterpret_cast<const uint4*>(x_ptr[j] + k) : none;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const uint32_t lo[4] = {a[i][0].x, a[i][1].x, a[i][0].y, a[i][1].y};
            const uint32_t hi[4] = {a[i][0].z, a[i][1].z, a[i][0].w, a[i][1].w};
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                ptx::mma16816<T>(acc[i][j], lo, x[j].x, x[j].y);
                ptx::mma16816<T>(acc[i][j], hi, x[j].z, x[j].w);
            }
        }
    }
    // the warps' sums meet in shared memory and are added in their order
    constexpr int P = down_pitch(MT);
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
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kLoraWarps; ++w) v += red[(w * 8 * NT + n) * P + r];
        p.part[(static_cast<int64_t>(piece) * p.M + row0 + rows[n]) * p.R + r0 + r] = v;
    }
    __syncthreads();
}

// Grid: pieces of K, groups in turn, tiles.  MT: 16-row tiles of ranks in hand,
// NT: most tiles of 8 rows in hand.
template <class T, int MT, int NT>
__global__ void __launch_bounds__(kLoraThreads, 2) lora_down_kernel(const LoraParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    Groups& s = *reinterpret_cast<Groups*>(smem);
    float* red = reinterpret_cast<float*>(smem + kGroupsBytes);
    ptx::griddep_wait();
    // only now: what starts early may then rely on everything before this kernel
    ptx::griddep_launch_dependents();
    const int piece = blockIdx.x, row0 = static_cast<int>(blockIdx.z) * p.tile_rows;
    const int rows = min(p.tile_rows, p.M - row0);
    group_rows(p, row0, rows, s);
    const int s0 = static_cast<int>(static_cast<int64_t>(p.k_steps) * piece / p.pieces);
    const int s1 = static_cast<int>(static_cast<int64_t>(p.k_steps) * (piece + 1) / p.pieces);
    for (int g = blockIdx.y; g < s.n; g += gridDim.y) {
        const T* A = static_cast<const T*>(p.A) + static_cast<int64_t>(s.adapter[g]) * p.R * p.K;
        const int begin = s.start[g], end = s.start[g + 1];
        for (int r0 = 0; r0 < p.R; r0 += 16 * MT) {
            for (int i = begin; i < end; i += 8 * NT) {
                const int m = min(8 * NT, end - i);
                if (m <= 8) down_rows<T, MT, 1>(p, A, r0, s.order + i, m, row0, s0, s1, piece, red);
                else if (m <= 16) down_rows<T, MT, 2>(p, A, r0, s.order + i, m, row0, s0, s1, piece, red);
                else if (NT <= 4 || m <= 32) down_rows<T, MT, 4>(p, A, r0, s.order + i, m, row0, s0, s1, piece, red);
                else down_rows<T, MT, NT>(p, A, r0, s.order + i, m, row0, s0, s1, piece, red);
            }
        }
    }
}

// ---------------------------------------------------------------------------- up
// Bytes of a row of V in shared memory: groups of four fp32 sums become four hi and
// four lo numbers in the same 16 bytes; 64 more than a multiple of 128 keeps the rows' reads
// in different banks.
__host__ __device__ inline int up_pitch(int R) { return R * 4 + ((64 - R * 4) & 127); }
// rows of V in shared memory at one time
__host__ __device__ inline int up_rows(int R) { return R <= 64 ? 128 : (R <= 128 ? 64 : 32); }

// The two numbers of type T that v is the sum of.
template <class T>
__device__ __forceinline__ void cut(float v, float& hi, float& lo) {
    hi = Elem<T>::to_float(Elem<T>::from_float(v));
    lo = fabsf(hi) <= 0x1.fffffep+127f ? v - hi : 0.0f;   // an infinity or NaN goes with hi alone
}

// Biased exponent of the power of two that is taken out of a row whose largest
// magnitude has these bits; it and its reciprocal are normal numbers.
__device__ __forceinline__ uint32_t row_exponent(uint32_t bits) { return min(max(bits >> 23, 1u), 253u); }

// Grid: ranges of `width` columns, groups in turn, tiles.
template <class T>
__global__ void __launch_bounds__(kLoraThreads, 2) lora_up_kernel(const LoraParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    Groups& s = *reinterpret_cast<Groups*>(smem);
    uint8_t* v_raw = smem + kGroupsBytes;
    __shared__ uint32_t row_max[128];
    // This kernel runs once every CTA of `down` has seen the kernels before it end, so
    // ids and B may be read here, and a product launched early may read its operands.
    ptx::griddep_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gr = lane >> 2, t = lane & 3;
    const int n0 = blockIdx.x * p.width, row0 = static_cast<int>(blockIdx.z) * p.tile_rows;
    const int rows = min(p.tile_rows, p.M - row0), columns = min(p.width, p.N - n0);
    group_rows(p, row0, rows, s);
    const T* B = static_cast<const T*>(p.B);
    if (tid == 0 && static_cast<int>(blockIdx.y) < s.n) {
        const T* b = B + (static_cast<int64_t>(s.adapter[blockIdx.y]) * p.N + n0) * p.R;
        const uint32_t bytes = min(static_cast<int64_t>(columns) * p.R * 2, int64_t{1} << 20);
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" :: "l"(b), "r"(bytes) : "memory");
    }
    ptx::griddep_wait();
    const int pitch = up_pitch(p.R), most = up_rows(p.R), steps = (p.R + 15) / 16;
    // groups, and behind them the rows without an adapter
    for (int g = blockIdx.y; g <= s.n; g += gridDim.y) {
        const bool has = g < s.n;
        const int begin = s.start[g], end = has ? s.start[g + 1] : rows;
        const int64_t adapter = has ? s.adapter[g] : 0;
        const float factor = has && p.factors != nullptr ? p.factors[adapter] : 1.0f;
        const T* b_rows = B + adapter * p.N * p.R;
        for (int i0 = begin; i0 < end; i0 += most) {
            const int m = min(most, end - i0);
            if (has) {
                __syncthreads();   // V of the rows before has been used
                if (tid < 128) row_max[tid] = 0u;
                __syncthreads();
                const int quads = p.R / 4;
                for (int i = tid; i < m * quads; i += kLoraThreads) {
                    const int r = i / quads, q = i - r * quads;
                    const float4* src = reinterpret_cast<const float4*>(
                        p.part + static_cast<int64_t>(row0 + s.order[i0 + r]) * p.R + 4 * q);
                    const int64_t step = static_cast<int64_t>(p.M) * p.R / 4;
                    float4 v = *src;
                    for (int c = 1; c < p.pieces; ++c) {
                        const float4 o = src[c * step];
                        v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
                    }
                    *reinterpret_cast<float4*>(v_raw + r * pitch + 16 * q) = v;
                    const float top = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
                    if (top <= 0x1.fffffep+127f) atomicMax(&row_max[r], __float_as_uint(top));   // finite
                }
                __syncthreads();
                for (int i = tid; i < m * quads; i += kLoraThreads) {
                    const int r = i / quads, q = i - r * quads;
                    uint4* at = reinterpret_cast<uint4*>(v_raw + r * pitch + 16 * q);
                    const float4 v = *reinterpret_cast<const float4*>(at);
                    const float down = __uint_as_float((254u - row_exponent(row_max[r])) << 23);
                    float h[4], l[4];
                    cut<T>(v.x * down, h[0], l[0]);
                    cut<T>(v.y * down, h[1], l[1]);
                    cut<T>(v.z * down, h[2], l[2]);
                    cut<T>(v.w * down, h[3], l[3]);
                    *at = make_uint4(Elem<T>::pack2(h[0], h[1]), Elem<T>::pack2(h[2], h[3]), Elem<T>::pack2(l[0], l[1]),
                                     Elem<T>::pack2(l[2], l[3]));
                }
                __syncthreads();
            }
            for (int nb = warp * kLoraColumns; nb < columns; nb += kLoraWarps * kLoraColumns) {
                const int64_t n = static_cast<int64_t>(n0) + nb + 8 * t;   // this thread's 8 columns of the output
                const bool n_in = nb + 8 * t < columns;
                for (int rb = 0; rb < m; rb += 16) {
                    float acc[4][4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[j][e] = 0.0f;
                    if (has) {
                        // rows beyond m read what lies there: only outputs that are not written come of it
                        const uint8_t* v0 = v_raw + (rb + gr) * pitch + 16 * t;
#pragma unroll 2
                        for (int k = 0; k < steps; ++k) {
                            const bool k_in = 16 * k + 4 * t < p.R;
                            uint4 f0 = make_uint4(0u, 0u, 0u, 0u), f1 = f0;
                            if (k_in) {
                                f0 = *reinterpret_cast<const uint4*>(v0 + 64 * k);
                                f1 = *reinterpret_cast<const uint4*>(v0 + 8 * pitch + 64 * k);
                            }
                            const uint32_t hi[4] = {f0.x, f1.x, f0.y, f1.y}, lo[4] = {f0.z, f1.z, f0.w, f1.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                // column c of tile j is column 8 (c / 2) + 2 j + c % 2 of the 32, so that a
                                // thread's two of every tile are eight in a row
                                const int c = nb + 8 * (gr >> 1) + 2 * j + (gr & 1);
                                uint2 b = make_uint2(0u, 0u);
                                if (k_in && c < columns)
                                    b = *reinterpret_cast<const uint2*>(b_rows + static_cast<int64_t>(n0 + c) * p.R + 16 * k + 4 * t);
                                ptx::mma16816<T>(acc[j], hi, b.x, b.y);
                                ptx::mma16816<T>(acc[j], lo, b.x, b.y);
                            }
                        }
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int r = rb + gr + 8 * h;
                        if (r >= m || !n_in) continue;
                        const int64_t at = static_cast<int64_t>(row0 + s.order[i0 + r]) * p.N + n;
                        float y[8];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            y[2 * j] = acc[j][2 * h];
                            y[2 * j + 1] = acc[j][2 * h + 1];
                        }
                        if (has) {
                            const float up = __uint_as_float(row_exponent(row_max[r]) << 23);
#pragma unroll
                            for (int j = 0; j < 8; ++j) y[j] = y[j] * up * factor;
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
                            make_uint4(Elem<T>::pack2(y[0], y[1]), Elem<T>::pack2(y[2], y[3]), Elem<T>::pack2(y[4], y[5]),
                                       Elem<T>::pack2(y[6], y[7]));
                    }
                }
            }
        }
    }
}

// -------------------------------------------------------------------------- host
constexpr int64_t kLoraRows = 8192;      // rows whose partial sums are in scratch at one time
constexpr int kLoraMaxWidth = 65536;

struct LoraPlan {
    int tile_rows, tiles, groups, pieces, ranges, width;
};

// Two CTAs per SM: over the tiles, over the groups of a single tile (a batch of
// requests has many, a prompt's tile one or two), and then over K or N.
LoraPlan lora_plan(int64_t M, int64_t N, int64_t K, int64_t count, int sms) {
    LoraPlan pl;
    pl.tile_rows = M <= kLoraTile ? kLoraTile : kLoraTile / 2;
    pl.tiles = static_cast<int>((M + pl.tile_rows - 1) / pl.tile_rows);
    pl.groups = pl.tiles == 1 ? static_cast<int>(std::min<int64_t>(std::min<int64_t>(M, count + 1), 64)) : 1;
    const int64_t each = std::max(1, 2 * sms / (pl.tiles * pl.groups));
    const int64_t steps = (K + kLoraStepK - 1) / kLoraStepK;
    pl.pieces = static_cast<int>(
        std::max<int64_t>(1, std::min({each, static_cast<int64_t>(kLoraMaxPieces), steps / kLoraWarps})));
    const int64_t ranges = std::max(std::min(each, (N + 255) / 256), (N + kLoraMaxWidth - 1) / kLoraMaxWidth);
    pl.width = static_cast<int>(((N + ranges - 1) / ranges + kLoraColumns - 1) / kLoraColumns * kLoraColumns);
    pl.ranges = static_cast<int>((N + pl.width - 1) / pl.width);
    return pl;
}

template <class T>
gemm_status_t run(LoraParams p, const LoraPlan& pl, const DeviceView& dev, cudaStream_t s) {
    const unsigned groups = static_cast<unsigned>(pl.groups), tiles = static_cast<unsigned>(pl.tiles);
    if (p.ids != nullptr) {
        const dim3 grid(static_cast<unsigned>(pl.pieces), groups, tiles);
        gemm_status_t st;
        if (p.R <= 16)
            st = launch_clusters(lora_down_kernel<T, 1, 8>, dev.dev, grid, kLoraThreads, 1, down_smem(1, 8), true, s, p);
        else if (p.R <= 32)
            st = launch_clusters(lora_down_kernel<T, 2, 4>, dev.dev, grid, kLoraThreads, 1, down_smem(2, 4), true, s, p);
        else
            st = launch_clusters(lora_down_kernel<T, 4, 4>, dev.dev, grid, kLoraThreads, 1, down_smem(4, 4), true, s, p);
        if (st != GEMM_OK) return st;
    }
    return launch_clusters(lora_up_kernel<T>, dev.dev, dim3(static_cast<unsigned>(pl.ranges), groups, tiles), kLoraThreads, 1,
                           kGroupsBytes + up_rows(p.R) * up_pitch(p.R), true, s, p);
}

}  // namespace

size_t lora_scratch_bytes(const LoraArgs& a, const DeviceView& dev) {
    // fewer rows are cut into more pieces: the last, shorter block may need more than a whole one
    int64_t most = 0;
    for (const int64_t rows : {std::min(a.M, kLoraRows), a.M % kLoraRows})
        if (rows > 0) most = std::max(most, rows * lora_plan(rows, a.N, a.K, a.count, dev.sms).pieces);
    return static_cast<size_t>(most) * static_cast<size_t>(a.R) * 4;
}

gemm_status_t run_lora(bool bf16, const LoraArgs& a, uint8_t* data, const DeviceView& dev, cudaStream_t s) {
    for (int64_t m0 = 0; m0 < a.M; m0 += kLoraRows) {
        const int64_t M = std::min(kLoraRows, a.M - m0);
        const LoraPlan pl = lora_plan(M, a.N, a.K, a.count, dev.sms);
        LoraParams p{};
        p.X = static_cast<const uint16_t*>(a.X) + m0 * a.K;
        p.A = a.A;
        p.B = a.B;
        p.factors = a.factors;
        p.ids = a.K > 0 && a.count > 0 ? a.ids + m0 : nullptr;
        p.C = a.C != nullptr ? static_cast<const uint16_t*>(a.C) + m0 * a.N : nullptr;
        p.U = static_cast<uint16_t*>(a.U) + m0 * a.N;
        p.part = reinterpret_cast<float*>(data);
        p.M = static_cast<int32_t>(M);
        p.N = static_cast<int32_t>(a.N);
        p.K = static_cast<int32_t>(a.K);
        p.R = static_cast<int32_t>(a.R);
        p.count = static_cast<int32_t>(a.count);
        p.tile_rows = pl.tile_rows;
        p.pieces = pl.pieces;
        p.k_steps = static_cast<int32_t>((a.K + kLoraStepK - 1) / kLoraStepK);
        p.width = pl.width;
        p.beta = a.beta;
        const gemm_status_t st = bf16 ? run<__nv_bfloat16>(p, pl, dev, s) : run<__half>(p, pl, dev, s);
        if (st != GEMM_OK) return st;
    }
    return GEMM_OK;
}

}  // namespace gemm_gb300
