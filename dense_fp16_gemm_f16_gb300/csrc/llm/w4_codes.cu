// w4_codes.cu -- 16-bit weights to 4-bit codes with group scales, and back.
//
// One thread takes 8 consecutive k of one row (16 bytes of W, 4 bytes of
// codes); the 4, 8 or 16 threads of a group share its extremes by shuffles.
// Both directions are bound by memory: 2 bytes of W and half a byte of codes
// per weight.
#include "llm/llm.h"
#include "llm/w4.cuh"

namespace gemm_gb300 {
namespace {

constexpr int kCodesThreads = 256;

// Rows are numbered through the whole stack: row r is row r % N of matrix r / N,
// and its scales are at [(r / N) * (K / group) + k / group][r % N].
template <class T>
__global__ void __launch_bounds__(kCodesThreads)
w4_quantize_kernel(const T* __restrict__ W, int64_t rows, int64_t N, int64_t K, int group, uint8_t* __restrict__ codes,
                   T* __restrict__ scales, T* __restrict__ zeros) {
    const int64_t units = rows * (K / 8);
    const int width = group / 8;   // threads per group: 4, 8 or 16
    // K is a multiple of the group, so a group's threads are all in or all out
    for (int64_t u0 = static_cast<int64_t>(blockIdx.x) * kCodesThreads; u0 < units;
         u0 += static_cast<int64_t>(gridDim.x) * kCodesThreads) {
        const int64_t u = u0 + threadIdx.x;
        const bool in = u < units;
        float w[8] = {};
        if (in) unpack8<T>(reinterpret_cast<const uint4*>(W)[u], w);
        float lo = 0.0f, hi = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo = fminf(lo, w[i]);
            hi = fmaxf(hi, w[i]);
        }
        for (int d = 1; d < width; d *= 2) {
            lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, d));
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, d));
        }
        const T st = Elem<T>::from_float(zeros != nullptr ? __fdiv_rn(hi - lo, 15.0f) : __fdiv_rn(fmaxf(hi, -lo), 7.0f));
        const float s = Elem<T>::to_float(st);
        float z = 8.0f;
        if (zeros != nullptr) z = s == 0.0f ? 0.0f : fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.0f), 15.0f);
        if (!in) continue;
        uint32_t packed = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q = fminf(fmaxf((s == 0.0f ? 0.0f : rintf(__fdiv_rn(w[i], s))) + z, 0.0f), 15.0f);
            packed |= static_cast<uint32_t>(q) << (4 * i);
        }
        reinterpret_cast<uint32_t*>(codes)[u] = packed;
        if ((threadIdx.x & (width - 1)) == 0) {
            const int64_t r = u / (K / 8), g = (u - r * (K / 8)) / width, b = r / N;
            const int64_t at = (b * (K / group) + g) * N + (r - b * N);
            scales[at] = st;
            if (zeros != nullptr) zeros[at] = Elem<T>::from_float(z);
        }
    }
}

template <class T>
__global__ void __launch_bounds__(kCodesThreads)
w4_dequantize_kernel(const uint8_t* __restrict__ codes, const T* __restrict__ scales, const T* __restrict__ zeros,
                     int64_t rows, int64_t N, int64_t K, int group, T* __restrict__ W) {
    const int64_t units = rows * (K / 8);
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * kCodesThreads + threadIdx.x; u < units;
         u += static_cast<int64_t>(gridDim.x) * kCodesThreads) {
        const uint32_t c = reinterpret_cast<const uint32_t*>(codes)[u];
        const int64_t r = u / (K / 8), g = (u - r * (K / 8)) / (group / 8), b = r / N;
        const int64_t at = (b * (K / group) + g) * N + (r - b * N);
        const float s = Elem<T>::to_float(scales[at]);
        const float z = zeros != nullptr ? Elem<T>::to_float(zeros[at]) : 8.0f;
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = s * (static_cast<float>((c >> (4 * i)) & 15u) - z);
        reinterpret_cast<uint4*>(W)[u] = pack8<T>(w);
    }
}

unsigned blocks_for(int64_t units) {
    const int64_t b = (units + kCodesThreads - 1) / kCodesThreads;
    return static_cast<unsigned>(b < (1 << 20) ? b : (1 << 20));
}

}  // namespace

cudaError_t launch_w4_quantize(bool bf16, const void* W, int64_t batch, int64_t N, int64_t K, int group, void* codes,
                               void* scales, void* zeros, cudaStream_t s) {
    const int64_t rows = batch * N;
    const unsigned blocks = blocks_for(rows * (K / 8));
    uint8_t* c = static_cast<uint8_t*>(codes);
    if (bf16)
        w4_quantize_kernel<__nv_bfloat16><<<blocks, kCodesThreads, 0, s>>>(
            static_cast<const __nv_bfloat16*>(W), rows, N, K, group, c, static_cast<__nv_bfloat16*>(scales),
            static_cast<__nv_bfloat16*>(zeros));
    else
        w4_quantize_kernel<__half><<<blocks, kCodesThreads, 0, s>>>(static_cast<const __half*>(W), rows, N, K, group, c,
                                                                    static_cast<__half*>(scales),
                                                                    static_cast<__half*>(zeros));
    return cudaGetLastError();
}

cudaError_t launch_w4_dequantize(bool bf16, const Weights& w, int64_t batch, int64_t N, int64_t K, void* W,
                                 cudaStream_t s) {
    const int64_t rows = batch * N;
    const unsigned blocks = blocks_for(rows * (K / 8));
    const uint8_t* c = static_cast<const uint8_t*>(w.data);
    if (bf16)
        w4_dequantize_kernel<__nv_bfloat16><<<blocks, kCodesThreads, 0, s>>>(
            c, static_cast<const __nv_bfloat16*>(w.scales), static_cast<const __nv_bfloat16*>(w.zeros), rows, N, K,
            w.group, static_cast<__nv_bfloat16*>(W));
    else
        w4_dequantize_kernel<__half><<<blocks, kCodesThreads, 0, s>>>(c, static_cast<const __half*>(w.scales),
                                                                      static_cast<const __half*>(w.zeros), rows, N, K,
                                                                      w.group, static_cast<__half*>(W));
    return cudaGetLastError();
}

}  // namespace gemm_gb300
