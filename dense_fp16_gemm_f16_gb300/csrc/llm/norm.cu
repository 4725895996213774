// norm.cu -- RMS norm with the residual's addition, its output in 16 bits, in 8
// bits with a scale per row, or both:
//   h = x + r,  y = h / sqrt(mean(h^2) + eps) * w,  scale = max|y| / F,  y8 = y / scale
// A row stays in its threads' registers between the one pass that reads it and
// the one that writes it, so x, r, w, the stored sum and y each cross memory once
// and many rows are bound by those bytes: 4096 x 8192 bf16 with residual, sum and E4M3
// rows 39 us for 235 MB, 6.0 TB/s, 0.88 of the measured copy rate (in 16 bits without a residual 30 us
// for 134 MB: the registers that would hold the residual's pieces fetch nothing); 4096 x 11000 63 us
// where the bytes take 46.
// A few rows are bound by the launch and one round of sums (37 x 5128: 3 us in a graph).
// One round serves both the mean and the scale: max|h w| is taken beside the sum of
// squares, and the root's factor multiplies it afterwards.
// Copies by cp.async some rows ahead in place of the registers took 42 us where these
// take 39 (28 against 30 without residual); two elements per instruction (f32x2) 40.
#include <cuda_fp8.h>

#include <algorithm>
#include <cfloat>

#include "llm/llm.h"
#include "llm/rows_host.cuh"

namespace gemm_gb300 {
namespace {

constexpr int kNormVec = 8;            // elements per 16-byte access
constexpr int kNormMaxThreads = 1024;  // per row
constexpr int kNormMaxVecs = 4;        // 16-byte pieces of a row per thread
constexpr int kStayThreads = 512;      // per SM where CTAs stay

struct NormParams {
    const void* X;
    const void* R;        // or nullptr
    const void* W;        // or nullptr
    void* Y;              // or nullptr
    uint8_t* Y8;          // or nullptr
    float* scales;        // nullptr: `scale` for every row
    void* total;          // or nullptr
    int64_t T;
    int32_t H;
    int32_t row_threads;  // the whole CTA, or a power of two from 4 on of it
    float eps, scale, top;
    int32_t e5m2;
};

template <class T>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = Elem<T>::lo(w[i]);
        f[2 * i + 1] = Elem<T>::hi(w[i]);
    }
}

template <class T>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(Elem<T>::pack2(f[0], f[1]), Elem<T>::pack2(f[2], f[3]), Elem<T>::pack2(f[4], f[5]),
                      Elem<T>::pack2(f[6], f[7]));
}

template <class T>
__device__ __forceinline__ uint4 load8(const void* base, int64_t vec) {
    return static_cast<const uint4*>(base)[vec];
}

// Magnitudes are compared as bits, where NaN is above infinity: it stays.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Sum and maximum over the row's threads, in a fixed order; every thread gets them.
__device__ __forceinline__ void reduce_row(float& sum, uint32_t& top, int row_threads) {
    __shared__ float part_sum[kNormMaxThreads / 32];
    __shared__ uint32_t part_top[kNormMaxThreads / 32];
    for (int d = row_threads < 32 ? row_threads / 2 : 16; d > 0; d >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, d);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
    }
    const int warps = row_threads >> 5;
    if (warps <= 1) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) {
        part_sum[warp] = sum;
        part_top[warp] = top;
    }
    __syncthreads();
    const int first = warp / warps * warps;
    sum = lane < warps ? part_sum[first + lane] : 0.0f;
    top = lane < warps ? part_top[first + lane] : 0u;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    top = __reduce_max_sync(0xffffffffu, top);
}

// What turns a row's h into its outputs.
struct RowFactors {
    float root;         // 1 / sqrt(mean(h^2) + eps)
    float scale, inv;   // y8 = y / scale
    float lift;         // a power of two that keeps 1 / scale finite
};

__device__ __forceinline__ RowFactors row_factors(const NormParams& p, float sum, uint32_t top, int64_t row, bool first) {
    RowFactors f;
    f.root = __frsqrt_rn(sum / static_cast<float>(p.H) + p.eps);
    f.scale = p.scale;
    f.lift = 1.0f;
    if (p.scales != nullptr) {
        f.scale = __uint_as_float(top) * f.root / p.top;
        if (first) p.scales[row] = f.scale;
    }
    if (f.scale < 0x1p-100f) {
        f.lift = 0x1p+64f;
        f.scale *= 0x1p+64f;
    }
    f.inv = f.scale == 0.0f ? 0.0f : 1.0f / f.scale;
    return f;
}

// The quotient y / scale from its reciprocal, put right by its remainder.  A given scale may be so
// small that it passes fp32's numbers: rounded towards zero it is the largest of them and not
// infinite, so that it has a remainder, and becomes the largest code.  (A comparison that leaves out the
// remainder there cost 0.45 us of 39.4 at 4096 x 8192, limits on y or q up to 1.4.)
__device__ __forceinline__ float divided(float y, const RowFactors& f) {
    y = __fmul_rz(y, f.lift);
    const float q = __fmul_rz(y, f.inv);
    return fmaf(fmaf(-q, f.scale, y), f.inv, q);
}

__device__ __forceinline__ uint32_t pack4_8bit(float a, float b, float c, float d, bool e5m2) {
    const auto kind = e5m2 ? __NV_E5M2 : __NV_E4M3;
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, kind);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, kind);
    return lo | hi << 16;
}

// Writes y (and its 8-bit form) of one 16-byte piece from h.
template <class T>
__device__ __forceinline__ void write_piece(const NormParams& p, const RowFactors& f, const float (&h)[8], const uint4& wv,
                                            int64_t vec) {
    float y[8], w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = h[e] * f.root;
    if (p.W != nullptr) {
        unpack8<T>(wv, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] *= w[e];
    }
    if (p.Y != nullptr) static_cast<uint4*>(p.Y)[vec] = pack8<T>(y);
    if (p.Y8 != nullptr) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = divided(y[e], f);
        uint2 v;
        if (p.e5m2) {
            v.x = pack4_8bit(y[0], y[1], y[2], y[3], true);
            v.y = pack4_8bit(y[4], y[5], y[6], y[7], true);
        } else {
            v.x = pack4_8bit(y[0], y[1], y[2], y[3], false);
            v.y = pack4_8bit(y[4], y[5], y[6], y[7], false);
        }
        reinterpret_cast<uint2*>(p.Y8)[vec] = v;
    }
}

// h of one piece, stored where `total` is asked for; adds it to the row's sums.
template <class T>
__device__ __forceinline__ void take_piece(const NormParams& p, const uint4& xv, const uint4& rv, const uint4& wv,
                                           float (&h)[8], float& sum, uint32_t& top) {
    unpack8<T>(xv, h);
    if (p.R != nullptr) {
        float r[8];
        unpack8<T>(rv, r);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] += r[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(h[e], h[e], sum);
    if (p.scales != nullptr) {
        float w[8] = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
        if (p.W != nullptr) unpack8<T>(wv, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, magnitude(h[e] * w[e]));
    }
}

// Rows of up to row_threads * NV pieces, blockDim / row_threads of them per CTA.
template <class T, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_kernel(const NormParams p) {
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int row_threads = p.row_threads;
    const int in_row = threadIdx.x % row_threads;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / row_threads) + threadIdx.x / row_threads;
    const int vecs = p.H / kNormVec;
    const int64_t base = row * vecs;
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    uint4 x[NV], r[NV], w[NV];
    float h[NV][8], sum = 0.0f;
    uint32_t top = 0u;
    bool in[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = in_row + i * row_threads;
        in[i] = row < p.T && v < vecs;
        x[i] = in[i] ? load8<T>(p.X, base + v) : none;
        r[i] = in[i] && p.R != nullptr ? load8<T>(p.R, base + v) : none;
        w[i] = in[i] && p.W != nullptr ? load8<T>(p.W, v) : none;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) take_piece<T>(p, x[i], r[i], w[i], h[i], sum, top);
    if (p.total != nullptr) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (in[i]) static_cast<uint4*>(p.total)[base + in_row + i * row_threads] = pack8<T>(h[i]);
    }
    reduce_row(sum, top, row_threads);
    if (row >= p.T) return;
    const RowFactors f = row_factors(p, sum, top, row, in_row == 0);
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (in[i]) write_piece<T>(p, f, h[i], w[i], base + in_row + i * row_threads);
}

// The same for many rows: CTAs stay and fetch the next rows while they work on these; the
// weight stays in registers.  NV pieces of each of x, r and w per thread.
template <class T, int NV>
__global__ void __launch_bounds__(kStayThreads) norm_stay_kernel(const NormParams p) {
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int row_threads = p.row_threads, rows = blockDim.x / row_threads;
    const int in_row = threadIdx.x % row_threads;
    const int vecs = p.H / kNormVec;
    const int64_t step = static_cast<int64_t>(gridDim.x) * rows;
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    uint4 w[NV], xn[NV], rn[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = in_row + i * row_threads;
        w[i] = v < vecs && p.W != nullptr ? load8<T>(p.W, v) : none;
    }
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = in_row + i * row_threads;
            const bool in = row < p.T && v < vecs;
            xn[i] = in ? load8<T>(p.X, row * vecs + v) : none;
            rn[i] = in && p.R != nullptr ? load8<T>(p.R, row * vecs + v) : none;
        }
    };
    int64_t row = static_cast<int64_t>(blockIdx.x) * rows + threadIdx.x / row_threads;
    fetch(row);
    // whole CTAs go round: the sums meet at a barrier
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * rows; first < p.T; first += step, row += step) {
        float h[NV][8], sum = 0.0f;
        uint32_t top = 0u;
#pragma unroll
        for (int i = 0; i < NV; ++i) take_piece<T>(p, xn[i], rn[i], w[i], h[i], sum, top);
        fetch(row + step);   // other rows than any output written now
        const int64_t base = row * vecs;
        if (p.total != nullptr && row < p.T) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (in_row + i * row_threads < vecs)
                    static_cast<uint4*>(p.total)[base + in_row + i * row_threads] = pack8<T>(h[i]);
        }
        reduce_row(sum, top, row_threads);
        if (row < p.T) {
            const RowFactors f = row_factors(p, sum, top, row, in_row == 0);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (in_row + i * row_threads < vecs) write_piece<T>(p, f, h[i], w[i], base + in_row + i * row_threads);
        }
        if (row_threads > 32) __syncthreads();   // the sums have been read
    }
}

// Rows too long for registers: read a second time, each piece by the thread that
// writes it, so that outputs may take the place of x or r.  A thread's pieces are added with what
// their roundings leave (`rest`): one after the other in fp32, the squares of 2^27 equal numbers came
// out 0.2 % too small.
template <class T>
__global__ void __launch_bounds__(kNormMaxThreads) norm_long_kernel(const NormParams p) {
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int vecs = p.H / kNormVec;
    const int64_t row = blockIdx.x, base = row * vecs;
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    float sum = 0.0f, rest = 0.0f;
    uint32_t top = 0u;
    for (int v = threadIdx.x; v < vecs; v += kNormMaxThreads) {
        float h[8], piece = 0.0f;
        take_piece<T>(p, load8<T>(p.X, base + v), p.R != nullptr ? load8<T>(p.R, base + v) : none,
                      p.W != nullptr ? load8<T>(p.W, v) : none, h, piece, top);
        const float add = __fadd_rn(piece, rest), next = __fadd_rn(sum, add);
        rest = next <= FLT_MAX ? __fsub_rn(add, __fsub_rn(next, sum)) : 0.0f;   // an infinite sum stays one
        sum = next;
    }
    reduce_row(sum, top, kNormMaxThreads);
    const RowFactors f = row_factors(p, sum, top, row, threadIdx.x == 0);
    for (int v = threadIdx.x; v < vecs; v += kNormMaxThreads) {
        const uint4 wv = p.W != nullptr ? load8<T>(p.W, v) : none;
        float h[8], s = 0.0f;
        uint32_t t = 0u;
        take_piece<T>(p, load8<T>(p.X, base + v), p.R != nullptr ? load8<T>(p.R, base + v) : none, wv, h, s, t);
        if (p.total != nullptr) static_cast<uint4*>(p.total)[base + v] = pack8<T>(h);
        write_piece<T>(p, f, h, wv, base + v);
    }
}

int power_of_two(int n) {
    int p = 1;
    while (p < n) p *= 2;
    return p;
}

template <class T>
gemm_status_t run(NormParams p, const DeviceView& dev, cudaStream_t s) {
    const int vecs = p.H / kNormVec;
    if (vecs > kNormMaxThreads * kNormMaxVecs) {
        p.row_threads = kNormMaxThreads;
        return launch_clusters(norm_long_kernel<T>, dev.dev, static_cast<int>(p.T), kNormMaxThreads, 1, 0, true, s, p);
    }
    // Few rows leave SMs idle whatever the split, so a row gets a thread per piece; with
    // many, four pieces per thread keep enough loads under way.
    const int want = p.T <= 2 * dev.sms ? 1 : kNormMaxVecs;
    const int each = (vecs + want - 1) / want;
    p.row_threads = each > 128 ? std::min(kNormMaxThreads, (each + 31) / 32 * 32) : std::max(want == 1 ? 32 : 4, power_of_two(each));
    if (want > 1 && each > 128 && p.row_threads < kStayThreads)   // as many as cost no CTA
        p.row_threads = kStayThreads / (kStayThreads / p.row_threads) / 32 * 32;
    const int nv = (vecs + p.row_threads - 1) / p.row_threads;
    const int rows = want == 1 ? 1 : std::max(1, 256 / p.row_threads);
    const int grid = static_cast<int>((p.T + rows - 1) / rows), threads = rows * p.row_threads;
    // CTAs stay where each has several turns (4096 x 8192 bf16 to E4M3 48 -> 39 us)
    const int stay = dev.sms * (kStayThreads / std::min(threads, kStayThreads));
    if (threads <= kStayThreads && grid >= 2 * stay) {
        if (nv <= 1) return launch_clusters(norm_stay_kernel<T, 1>, dev.dev, stay, threads, 1, 0, true, s, p);
        if (nv <= 2) return launch_clusters(norm_stay_kernel<T, 2>, dev.dev, stay, threads, 1, 0, true, s, p);
        if (nv <= 3) return launch_clusters(norm_stay_kernel<T, 3>, dev.dev, stay, threads, 1, 0, true, s, p);
        return launch_clusters(norm_stay_kernel<T, 4>, dev.dev, stay, threads, 1, 0, true, s, p);
    }
    if (nv <= 1) return launch_clusters(norm_kernel<T, 1, 1024>, dev.dev, grid, threads, 1, 0, true, s, p);
    if (nv <= 2) return launch_clusters(norm_kernel<T, 2, 1024>, dev.dev, grid, threads, 1, 0, true, s, p);
    // 512 threads have registers enough for four pieces, 1024 (rows of more than 16384) spill 72 bytes
    if (threads <= 512) return launch_clusters(norm_kernel<T, 4, 512>, dev.dev, grid, threads, 1, 0, true, s, p);
    return launch_clusters(norm_kernel<T, 4, 1024>, dev.dev, grid, threads, 1, 0, true, s, p);
}

}  // namespace

gemm_status_t run_rmsnorm(bool bf16, const NormArgs& a, const DeviceView& dev, cudaStream_t s) {
    NormParams p{};
    p.X = a.X;
    p.R = a.residual;
    p.W = a.weight;
    p.Y = a.Y;
    p.Y8 = static_cast<uint8_t*>(a.Y8);
    p.scales = a.scales;
    p.total = a.total;
    p.T = a.T;
    p.H = static_cast<int32_t>(a.H);
    p.eps = a.eps;
    p.scale = a.scale;
    p.top = a.e5m2 ? 57344.0f : 448.0f;
    p.e5m2 = a.e5m2;
    return bf16 ? run<__nv_bfloat16>(p, dev, s) : run<__half>(p, dev, s);
}

}  // namespace gemm_gb300
