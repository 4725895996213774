// w4_gemm.cu -- D = A·Bᵀ with the weights B in 4 bits.
//
// Simple form: one warp per output column n and 8 rows of A; the lanes share
// K, each taking 8 consecutive k (4 bytes of codes) at a time.
#include "llm/llm.h"
#include "llm/w4.cuh"

namespace gemm_gb300 {
namespace {

constexpr int kRowsPerWarp = 8;

template <class T>
__global__ void __launch_bounds__(256)
w4_gemm_kernel(const T* __restrict__ A, const uint8_t* __restrict__ codes, const T* __restrict__ scales,
               const T* __restrict__ zeros, T* D, int64_t M, int64_t N, int64_t K, int group, EpiParams epi) {
    const int lane = threadIdx.x & 31;
    const int64_t n = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (n >= N) return;
    for (int64_t m0 = static_cast<int64_t>(blockIdx.y) * kRowsPerWarp; m0 < M;
         m0 += static_cast<int64_t>(gridDim.y) * kRowsPerWarp) {
        float acc[kRowsPerWarp] = {};
        for (int64_t k = lane * 8; k < K; k += 256) {
            const uint32_t c = *reinterpret_cast<const uint32_t*>(codes + n * (K / 2) + k / 2);
            const int64_t at = (k / group) * N + n;
            const float s = Elem<T>::to_float(scales[at]);
            const float z = zeros != nullptr ? Elem<T>::to_float(zeros[at]) : 8.0f;
#pragma unroll
            for (int r = 0; r < kRowsPerWarp; ++r) {
                if (m0 + r >= M) break;
                float x[8], sum = 0.0f;
                unpack8<T>(*reinterpret_cast<const uint4*>(A + (m0 + r) * K + k), x);
#pragma unroll
                for (int i = 0; i < 8; ++i) sum += x[i] * (static_cast<float>((c >> (4 * i)) & 15u) - z);
                acc[r] += s * sum;
            }
        }
#pragma unroll
        for (int r = 0; r < kRowsPerWarp; ++r) {
            for (int d = 16; d > 0; d >>= 1) acc[r] += __shfl_xor_sync(0xffffffffu, acc[r], d);
            if (lane == 0 && m0 + r < M) {
                const float v = epi.on ? epi_apply1<T>(epi, acc[r], m0 + r, n, N) : acc[r];
                D[(m0 + r) * N + n] = Elem<T>::from_float(v);
            }
        }
    }
}

template <class T>
cudaError_t launch(const void* A, const Weights& w, void* D, int64_t M, int64_t N, int64_t K, const EpiParams& epi,
                   cudaStream_t s) {
    const int64_t my = (M + kRowsPerWarp - 1) / kRowsPerWarp;
    const dim3 grid(static_cast<unsigned>((N + 7) / 8), static_cast<unsigned>(my < 65535 ? my : 65535), 1);
    w4_gemm_kernel<T><<<grid, 256, 0, s>>>(static_cast<const T*>(A), static_cast<const uint8_t*>(w.data),
                                           static_cast<const T*>(w.scales), static_cast<const T*>(w.zeros),
                                           static_cast<T*>(D), M, N, K, w.group, epi);
    return cudaGetLastError();
}

}  // namespace

gemm_status_t run_w4_gemm(bool bf16, const void* A, const Weights& w, void* D, int64_t M, int64_t N, int64_t K,
                          const EpiParams& epi, const DeviceView&, gemm_stream_t stream) {
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = bf16 ? launch<__nv_bfloat16>(A, w, D, M, N, K, epi, s) : launch<__half>(A, w, D, M, N, K, epi, s);
    return e == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

}  // namespace gemm_gb300
