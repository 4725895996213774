// w4_codes.cu -- 16-bit weights to 4-bit codes with group scales, and back.
//
// A CTA takes 16 rows by 512 k; a warp two of the rows, each thread 8 consecutive
// k of a row at a time (16 bytes of W, 4 bytes of codes), four such pieces loaded
// before the first is used.  The 4, 8 or 16 threads of a group share its
// extremes by shuffles.  Scales lie [K/group][N]: they pass through shared
// memory so that 16 rows' worth is written (or read) side by side.
//
// Both directions are bound by memory: 2 bytes of W and half a byte of codes per
// weight.  The quantiser is close to the fp32 pipes' limit too, so w / s is not
// divided out: with t = w * (1 / s), off by less than 2^-20, rint(t) is rint(w / s)
// unless w / s is exactly half-way.  (w and s have at most 11 significant bits, so
// a quotient that is not half-way is at least 2^-14 away from it.)  Half-way means
// |w - s r| = s / 2, which fma computes exactly, and r then becomes the even
// neighbour.
#include "llm/llm.h"
#include "llm/w4.cuh"

namespace gemm_gb300 {
namespace {

constexpr int kCodesThreads = 256;
constexpr int kCodesRows = 16, kCodesK = 512;
constexpr int kCodesGroups = kCodesK / 32;   // most groups of a row in a tile
constexpr float kRound = 12582912.0f;        // 1.5 * 2^23: adding it rounds to whole numbers, ties to even
constexpr float kWhole = 8388608.0f;         // 2^23

// Rows are numbered through the whole stack: row r is row r % N of matrix r / N,
// and its scales are at [(r / N) * (K / group) + k / group][r % N].
struct CodesTile {
    int64_t row0, k0;
    __device__ __forceinline__ CodesTile(int64_t k_tiles) {
        row0 = static_cast<int64_t>(blockIdx.x) / k_tiles * kCodesRows;
        k0 = static_cast<int64_t>(blockIdx.x) % k_tiles * kCodesK;
    }
};

// Element (row, group) of the tile's scales that this thread moves; -1: none.
__device__ __forceinline__ int64_t side_at(const CodesTile& t, int64_t rows, int64_t N, int64_t K, int group, int& row,
                                           int& grp) {
    row = threadIdx.x % kCodesRows;
    grp = threadIdx.x / kCodesRows;
    const int64_t r = t.row0 + row, g = t.k0 / group + grp, b = r / N;
    if (r >= rows || grp >= kCodesK / group || g >= K / group) return -1;
    return (b * (K / group) + g) * N + (r - b * N);
}

template <class T, bool ASYM>
__global__ void __launch_bounds__(kCodesThreads)
w4_quantize_kernel(const T* __restrict__ W, int64_t rows, int64_t N, int64_t K, int64_t k_tiles, int group,
                   uint8_t* __restrict__ codes, T* __restrict__ scales, T* __restrict__ zeros) {
    __shared__ T s_scale[kCodesGroups][kCodesRows], s_zero[kCodesGroups][kCodesRows];
    const CodesTile tile(k_tiles);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int width = group / 8;   // threads per group: 4, 8 or 16
    uint4 raw[4];
    bool in[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = tile.row0 + warp + 8 * (i >> 1), k = tile.k0 + 256 * (i & 1) + lane * 8;
        in[i] = r < rows && k < K;   // K is a multiple of the group: a group's threads are all in or all out
        raw[i] = in[i] ? __ldcs(reinterpret_cast<const uint4*>(W + r * K + k)) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = warp + 8 * (i >> 1), k = 256 * (i & 1) + lane * 8;
        float w[8];
        unpack8<T>(raw[i], w);
        float lo = 0.0f, hi = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            lo = fminf(lo, w[j]);
            hi = fmaxf(hi, w[j]);
        }
        for (int d = 1; d < width; d *= 2) {
            lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, d));
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, d));
        }
        const T st = Elem<T>::from_float(ASYM ? __fdiv_rn(hi - lo, 15.0f) : __fdiv_rn(fmaxf(hi, -lo), 7.0f));
        const float s = Elem<T>::to_float(st);
        float z = 8.0f;
        if constexpr (ASYM) z = s == 0.0f ? 0.0f : fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.0f), 15.0f);
        const float inv = s == 0.0f ? 0.0f : __frcp_rn(s), half = 0.5f * s;
        float q[8];
        bool tie = false;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            q[j] = __fadd_rn(__fmaf_rn(w[j], inv, kRound), -kRound);
            tie = tie || fabsf(__fmaf_rn(-s, q[j], w[j])) == half;
        }
        if (tie && s != 0.0f) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float e = __fmaf_rn(-s, q[j], w[j]);
                if (fabsf(e) == half && (static_cast<int>(q[j]) & 1)) q[j] += e > 0.0f ? 1.0f : -1.0f;
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) q[j] = fminf(fmaxf(q[j] + z, 0.0f), 15.0f);
        // four codes as one whole number below 2^16, exact in fp32
        const float a = q[0] + 16.0f * (q[1] + 16.0f * (q[2] + 16.0f * q[3]));
        const float b = q[4] + 16.0f * (q[5] + 16.0f * (q[6] + 16.0f * q[7]));
        if (in[i]) {
            reinterpret_cast<uint32_t*>(codes)[((tile.row0 + row) * K + tile.k0 + k) / 8] =
                __byte_perm(__float_as_uint(a + kWhole), __float_as_uint(b + kWhole), 0x5410);
            if ((lane & (width - 1)) == 0) {
                s_scale[k / group][row] = st;
                if constexpr (ASYM) s_zero[k / group][row] = Elem<T>::from_float(z);
            }
        }
    }
    __syncthreads();
    int row, grp;
    const int64_t at = side_at(tile, rows, N, K, group, row, grp);
    if (at >= 0) {
        scales[at] = s_scale[grp][row];
        if constexpr (ASYM) zeros[at] = s_zero[grp][row];
    }
}

template <class T>
__global__ void __launch_bounds__(kCodesThreads)
w4_dequantize_kernel(const uint8_t* __restrict__ codes, const T* __restrict__ scales, const T* __restrict__ zeros,
                     int64_t rows, int64_t N, int64_t K, int64_t k_tiles, int group, T* __restrict__ W) {
    __shared__ float s_scale[kCodesGroups][kCodesRows], s_zero[kCodesGroups][kCodesRows];
    const CodesTile tile(k_tiles);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t c[4];
    bool in[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = tile.row0 + warp + 8 * (i >> 1), k = tile.k0 + 256 * (i & 1) + lane * 8;
        in[i] = r < rows && k < K;
        c[i] = in[i] ? __ldcs(reinterpret_cast<const uint32_t*>(codes) + (r * K + k) / 8) : 0u;
    }
    int row, grp;
    const int64_t at = side_at(tile, rows, N, K, group, row, grp);
    if (at >= 0) {
        s_scale[grp][row] = Elem<T>::to_float(scales[at]);
        s_zero[grp][row] = zeros != nullptr ? Elem<T>::to_float(zeros[at]) : 8.0f;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (!in[i]) continue;
        const int r = warp + 8 * (i >> 1), k = 256 * (i & 1) + lane * 8;
        const float s = s_scale[k / group][r], z = s_zero[k / group][r];
        float w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float q = __uint_as_float(((c[i] >> (4 * j)) & 15u) | 0x4B000000u) - kWhole;
            w[j] = s * (q - z);
        }
        __stcs(reinterpret_cast<uint4*>(W + (tile.row0 + r) * K + tile.k0 + k), pack8<T>(w));
    }
}

// CTAs over row tiles and k tiles; -1 where a grid cannot hold them
int64_t grid_of(int64_t rows, int64_t K, int64_t* k_tiles) {
    *k_tiles = (K + kCodesK - 1) / kCodesK;
    const int64_t n = (rows + kCodesRows - 1) / kCodesRows * *k_tiles;
    return n <= 0x7FFFFFFFll ? n : -1;
}

template <class T>
void quantize(unsigned grid, const void* W, int64_t rows, int64_t N, int64_t K, int64_t k_tiles, int group, void* codes,
              void* scales, void* zeros, cudaStream_t s) {
    const T* w = static_cast<const T*>(W);
    uint8_t* c = static_cast<uint8_t*>(codes);
    if (zeros != nullptr)
        w4_quantize_kernel<T, true><<<grid, kCodesThreads, 0, s>>>(w, rows, N, K, k_tiles, group, c, static_cast<T*>(scales), static_cast<T*>(zeros));
    else
        w4_quantize_kernel<T, false><<<grid, kCodesThreads, 0, s>>>(w, rows, N, K, k_tiles, group, c, static_cast<T*>(scales), nullptr);
}

}  // namespace

cudaError_t launch_w4_quantize(bool bf16, const void* W, int64_t batch, int64_t N, int64_t K, int group, void* codes,
                               void* scales, void* zeros, cudaStream_t s) {
    const int64_t rows = batch * N;
    int64_t k_tiles;
    const int64_t n = grid_of(rows, K, &k_tiles);
    if (n < 0) return cudaErrorInvalidConfiguration;
    if (bf16) quantize<__nv_bfloat16>(static_cast<unsigned>(n), W, rows, N, K, k_tiles, group, codes, scales, zeros, s);
    else quantize<__half>(static_cast<unsigned>(n), W, rows, N, K, k_tiles, group, codes, scales, zeros, s);
    return cudaGetLastError();
}

cudaError_t launch_w4_dequantize(bool bf16, const Weights& w, int64_t batch, int64_t N, int64_t K, void* W,
                                 cudaStream_t s) {
    const int64_t rows = batch * N;
    int64_t k_tiles;
    const int64_t n = grid_of(rows, K, &k_tiles);
    if (n < 0) return cudaErrorInvalidConfiguration;
    const unsigned grid = static_cast<unsigned>(n);
    const uint8_t* c = static_cast<const uint8_t*>(w.data);
    if (bf16)
        w4_dequantize_kernel<__nv_bfloat16><<<grid, kCodesThreads, 0, s>>>(
            c, static_cast<const __nv_bfloat16*>(w.scales), static_cast<const __nv_bfloat16*>(w.zeros), rows, N, K,
            k_tiles, w.group, static_cast<__nv_bfloat16*>(W));
    else
        w4_dequantize_kernel<__half><<<grid, kCodesThreads, 0, s>>>(c, static_cast<const __half*>(w.scales),
                                                                    static_cast<const __half*>(w.zeros), rows, N, K,
                                                                    k_tiles, w.group, static_cast<__half*>(W));
    return cudaGetLastError();
}

}  // namespace gemm_gb300
