// llm.h -- launch entry points of the 4-bit-weight, mixture-of-experts,
// normalisation and adapter kernels.  Arguments are checked by llm_api.cu before these are called.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "epilogue.cuh"
#include "gemm_llm.h"
#include "internal.h"

namespace gemm_gb300 {

// A stack of weight matrices on the device (gemm_weights_t, checked).
struct Weights {
    const void* data;
    const void* scales;   // nullptr: 16-bit data
    const void* zeros;    // nullptr: zero point 8
    int32_t group;
};

constexpr int kMoeMaxTokens = 64;
constexpr int kMoeMaxChoices = 16;
constexpr int kMoeMaxExperts = 1024;

struct RouteParams {
    const void* X;        // [T][H]
    const void* Wr;       // [E][H]
    const float* bias;    // [E] or nullptr
    int64_t T;
    int32_t H, E, k;
    int32_t scoring;      // gemm_moe_scoring_t
    int32_t renormalize;
    int32_t* ids;         // [T][k]
    float* weights;       // [T][k]
};

struct FfnParams {
    const void* X;        // [T][H]
    const int32_t* ids;   // [T][k]
    const float* weights; // [T][k]
    Weights w13, w2;
    void* Y;              // [T][H]
    int32_t T, H, I, E, k;
};

cudaError_t launch_w4_quantize(bool bf16, const void* W, int64_t batch, int64_t N, int64_t K, int group, void* codes,
                               void* scales, void* zeros, int sms, cudaStream_t s);
cudaError_t launch_w4_dequantize(bool bf16, const Weights& w, int64_t batch, int64_t N, int64_t K, void* W,
                                 int sms, cudaStream_t s);

// The product on tcgen05, for more than a few rows of A, and its estimated clocks.
double w4_tiles_clocks(int64_t M, int64_t N, int64_t K, const DeviceView& dev);
gemm_status_t run_w4_tiles(bool bf16, const void* A, const Weights& w, void* D, int64_t M, int64_t N, int64_t K,
                           const EpiParams& epi, const DeviceView& dev, cudaStream_t s);

gemm_status_t run_w4_gemm(bool bf16, const void* A, const Weights& w, void* D, int64_t M, int64_t N, int64_t K,
                          const EpiParams& epi, const DeviceView& dev, gemm_stream_t stream);

struct NormArgs {
    const void *X, *residual, *weight;
    void *Y, *Y8;
    float* scales;        // nullptr: `scale` for every row
    void* total;
    int64_t T, H;
    float eps, scale;
    bool e5m2;
};
gemm_status_t run_rmsnorm(bool bf16, const NormArgs& a, const DeviceView& dev, cudaStream_t s);

// U = beta C + the adapters' part of the rows: c_a (X A_aT) B_aT, a = ids[m]
struct LoraArgs {
    const void *X, *A, *B;
    const float* factors;  // nullptr: ones
    const int32_t* ids;
    const void* C;         // nullptr: none
    float beta;
    void* U;               // may be C
    float* V;              // [M][R], M <= kLoraEpiRows: c_a X A_aT is all that is wanted; else nullptr
    uint32_t* ready;       // with V: set as soon as all before has ended (LoraEpi)
    int64_t M, N, K, R, count;
};
constexpr int kLoraMaxRank = 256;
// bytes of scratch that run_lora needs at `data` (M: rows)
size_t lora_scratch_bytes(int64_t M);
gemm_status_t run_lora(bool bf16, const LoraArgs& a, uint8_t* data, const DeviceView& dev, cudaStream_t s);

// bytes of scratch that run_route needs at `data`; counters: one zero, left at zero
size_t route_scratch_bytes(int64_t T, int64_t E);
gemm_status_t run_route(bool bf16, const RouteParams& p, uint8_t* data, uint32_t* counters, const DeviceView& dev,
                        gemm_stream_t stream);

// bytes of scratch that run_ffn needs at `data`
size_t ffn_scratch_bytes(int64_t T, int64_t I, int k);
gemm_status_t run_ffn(bool bf16, const FfnParams& p, uint8_t* data, const DeviceView& dev, gemm_stream_t stream);

}  // namespace gemm_gb300
