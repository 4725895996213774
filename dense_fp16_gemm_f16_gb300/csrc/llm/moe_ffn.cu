// moe_ffn.cu -- the experts' gated products for a few tokens.
//
// Simple form: one warp per (token's choice, row of the expert's first
// product), fp32 h in scratch, then one warp per (token, output).
#include "llm/llm.h"
#include "llm/w4.cuh"

namespace gemm_gb300 {
namespace {

__device__ __forceinline__ float silu(float v) { return v / (1.0f + expf(-v)); }

// One row of one matrix times a vector x of K elements (type TX), by a warp.
template <class T, class TX>
__device__ float row_dot(const Weights& w, int64_t matrix, int64_t rows, int64_t row, int64_t K, const TX* x, int lane) {
    const int64_t r = matrix * rows + row;
    float acc = 0.0f;
    for (int64_t k = lane * 8; k < K; k += 256) {
        float b[8];
        if (w.scales == nullptr) {
            unpack8<T>(*reinterpret_cast<const uint4*>(static_cast<const T*>(w.data) + r * K + k), b);
        } else {
            const uint32_t c = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(w.data) + r * (K / 2) + k / 2);
            const int64_t at = (matrix * (K / w.group) + k / w.group) * rows + row;
            const float s = Elem<T>::to_float(static_cast<const T*>(w.scales)[at]);
            const float z = w.zeros != nullptr ? Elem<T>::to_float(static_cast<const T*>(w.zeros)[at]) : 8.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) b[i] = s * (static_cast<float>((c >> (4 * i)) & 15u) - z);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (sizeof(TX) == 4) acc += x[k + i] * b[i];
            else acc += Elem<T>::to_float(x[k + i]) * b[i];
        }
    }
    for (int d = 16; d > 0; d >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, d);
    return acc;
}

template <class T>
__global__ void __launch_bounds__(256) moe_up_kernel(const FfnParams p, float* h) {
    const int lane = threadIdx.x & 31;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int slot = blockIdx.y;
    const int e = p.ids[slot];
    if (i >= p.I || e < 0 || e >= p.E) return;
    const T* x = static_cast<const T*>(p.X) + static_cast<int64_t>(slot / p.k) * p.H;
    const float gate = row_dot<T, T>(p.w13, e, 2 * static_cast<int64_t>(p.I), i, p.H, x, lane);
    const float up = row_dot<T, T>(p.w13, e, 2 * static_cast<int64_t>(p.I), p.I + i, p.H, x, lane);
    if (lane == 0) h[static_cast<int64_t>(slot) * p.I + i] = silu(gate) * up;
}

template <class T>
__global__ void __launch_bounds__(256) moe_down_kernel(const FfnParams p, const float* h) {
    const int lane = threadIdx.x & 31;
    const int64_t r = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int t = blockIdx.y;
    if (r >= p.H) return;
    float y = 0.0f;
    for (int j = 0; j < p.k; ++j) {
        const int e = p.ids[t * p.k + j];
        if (e < 0 || e >= p.E) continue;
        y += p.weights[t * p.k + j] * row_dot<T, float>(p.w2, e, p.H, r, p.I, h + static_cast<int64_t>(t * p.k + j) * p.I, lane);
    }
    if (lane == 0) static_cast<T*>(p.Y)[static_cast<int64_t>(t) * p.H + r] = Elem<T>::from_float(y);
}

template <class T>
cudaError_t launch(const FfnParams& p, float* h, cudaStream_t s) {
    moe_up_kernel<T><<<dim3(static_cast<unsigned>((p.I + 7) / 8), static_cast<unsigned>(p.T * p.k), 1), 256, 0, s>>>(p, h);
    moe_down_kernel<T><<<dim3(static_cast<unsigned>((p.H + 7) / 8), static_cast<unsigned>(p.T), 1), 256, 0, s>>>(p, h);
    return cudaGetLastError();
}

}  // namespace

size_t ffn_scratch_bytes(int64_t T, int64_t I, int k) { return static_cast<size_t>(T) * k * I * 4; }

gemm_status_t run_ffn(bool bf16, const FfnParams& p, uint8_t* data, const DeviceView&, gemm_stream_t stream) {
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    float* h = reinterpret_cast<float*>(data);
    const cudaError_t e = bf16 ? launch<__nv_bfloat16>(p, h, s) : launch<__half>(p, h, s);
    return e == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

}  // namespace gemm_gb300
