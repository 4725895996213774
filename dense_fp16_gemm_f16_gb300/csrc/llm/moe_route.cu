// moe_route.cu -- the k experts of each token and their weights.
//
// Simple form: one block per token; each warp sums the logits of its experts,
// then one warp picks the k largest keys, one at a time.
#include <math_constants.h>

#include "llm/llm.h"
#include "llm/w4.cuh"

namespace gemm_gb300 {
namespace {

template <class T>
__global__ void __launch_bounds__(256)
moe_route_kernel(const RouteParams p) {
    __shared__ float logit[kMoeMaxExperts];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const T* Wr = static_cast<const T*>(p.Wr);
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        const T* x = static_cast<const T*>(p.X) + t * p.H;
        for (int e = warp; e < p.E; e += 8) {
            float acc = 0.0f;
            for (int h = lane * 8; h < p.H; h += 256) {
                float a[8], b[8];
                unpack8<T>(*reinterpret_cast<const uint4*>(x + h), a);
                unpack8<T>(*reinterpret_cast<const uint4*>(Wr + static_cast<int64_t>(e) * p.H + h), b);
#pragma unroll
                for (int i = 0; i < 8; ++i) acc += a[i] * b[i];
            }
            for (int d = 16; d > 0; d >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, d);
            if (lane == 0) logit[e] = acc;
        }
        __syncthreads();
        if (warp == 0) {
            // softmax: the largest logit and the sum of exponentials
            float top = -CUDART_INF_F, sum = 0.0f;
            if (p.scoring == GEMM_MOE_SOFTMAX) {
                for (int e = lane; e < p.E; e += 32) top = fmaxf(top, logit[e]);
                for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                for (int e = lane; e < p.E; e += 32) sum += expf(logit[e] - top);
                for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            }
            auto score = [&](int e) {
                return p.scoring == GEMM_MOE_SOFTMAX ? expf(logit[e] - top) / sum : 1.0f / (1.0f + expf(-logit[e]));
            };
            uint32_t taken[kMoeMaxExperts / 1024] = {};   // bit i: expert lane + 32 i
            float total = 0.0f, mine = 0.0f;
            for (int j = 0; j < p.k; ++j) {
                float best = -CUDART_INF_F;
                int at = -1;
                for (int e = lane, i = 0; e < p.E; e += 32, ++i) {
                    if (taken[0] >> i & 1u) continue;
                    const float key = p.bias != nullptr ? score(e) + p.bias[e] : logit[e];
                    if (key > best) {   // false for NaN; the lower expert stays where keys are equal
                        best = key;
                        at = e;
                    }
                }
                for (int d = 16; d > 0; d >>= 1) {
                    const float ob = __shfl_xor_sync(0xffffffffu, best, d);
                    const int oa = __shfl_xor_sync(0xffffffffu, at, d);
                    if (oa >= 0 && (at < 0 || ob > best || (ob == best && oa < at))) {
                        best = ob;
                        at = oa;
                    }
                }
                float w = 0.0f;
                if (at >= 0) {
                    w = score(at);
                    if ((at & 31) == lane) taken[0] |= 1u << (at >> 5);
                }
                total += w;
                if (lane == j) mine = w;
                if (lane == 0) p.ids[t * p.k + j] = at;
            }
            if (p.renormalize && total != 0.0f) mine /= total;
            if (lane < p.k) p.weights[t * p.k + lane] = mine;
        }
        __syncthreads();
    }
}

}  // namespace

gemm_status_t run_route(bool bf16, const RouteParams& p, const DeviceView&, gemm_stream_t stream) {
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const unsigned blocks = static_cast<unsigned>(p.T < 65536 ? p.T : 65536);
    if (bf16) moe_route_kernel<__nv_bfloat16><<<blocks, 256, 0, s>>>(p);
    else moe_route_kernel<__half><<<blocks, 256, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

}  // namespace gemm_gb300
