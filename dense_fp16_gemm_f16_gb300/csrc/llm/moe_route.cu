// moe_route.cu -- the k experts of each token and their weights.
//
// Logits.  X·Wrᵀ for up to 64 tokens and 16 experts per cluster of up to 8
// CTAs, which split K between them and their 8 warps; mma.sync m16n8k16 with the
// experts as rows.  A thread loads 16 bytes of each operand row straight from
// global memory (the k order within an MMA is free, so 8 consecutive k are the
// thread's slots of two steps); there is nothing to stage, each byte is used
// once per CTA.  The partial sums of warps and CTAs are added in a fixed order
// in (distributed) shared memory.  Chains of MMAs stay short, so a logit is
// as exact as an fp32 sum in pieces.
// Choice.  One warp per token holds E / 32 keys per lane as integers that
// order like the floats; k times, a warp-wide maximum (redux) and the lowest
// expert that has it.  Up to 8 tokens the last CTA to finish its logits makes
// the choice, above that a second kernel with a warp for every token.
//
// Bound by latency: 64 tokens x 256 experts x 8192 read 5 MB (0.8 us of HBM) and
// take 11 us, one token x 64 experts x 2048 takes 4 us (on one warp per logit from
// plain loads they took 126 and 14).
#include <math_constants.h>

#include <algorithm>

#include "llm/llm.h"
#include "llm/stream.cuh"

namespace gemm_gb300 {
namespace {

constexpr int kRouteThreads = 256;
constexpr int kRouteWarps = kRouteThreads / 32;
constexpr int kRouteTile = 16;         // experts per cluster
constexpr int kRouteTokens = 64;       // tokens per cluster
constexpr int kRouteFewTokens = 8;     // up to here the last CTA chooses

struct LogitsParams {
    const void* X;
    const void* Wr;
    float* logits;         // [T][E]
    uint32_t* counter;     // CTAs done, zero before and after (few tokens only)
    int32_t T, H, E, split;
};

struct ChoiceParams {
    const float* logits;
    const float* bias;
    int32_t T, E, k, scoring, renormalize;
    int32_t* ids;
    float* weights;
};

// floats in the order of unsigned integers, 0 for minus infinity and NaN
__device__ __forceinline__ uint32_t key_of(float v) {
    if (!(v > -CUDART_INF_F)) return 0u;
    const uint32_t u = __float_as_uint(v + 0.0f);   // -0 becomes +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// One token's choice by a warp; EPL experts per lane, expert i * 32 + lane.
template <int EPL>
__device__ void choose(const ChoiceParams& p, int64_t t, int lane) {
    const float* row = p.logits + t * p.E;
    float prob[EPL];
    uint32_t key[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = i * 32 + lane;
        prob[i] = e < p.E ? row[e] : -CUDART_INF_F;
        key[i] = e < p.E ? key_of(prob[i]) : 0u;
    }
    if (p.scoring == GEMM_MOE_SOFTMAX) {
        float top = -CUDART_INF_F, sum = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) top = fmaxf(top, prob[i]);
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            prob[i] = i * 32 + lane < p.E ? expf(prob[i] - top) : 0.0f;
            sum += prob[i];
        }
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
#pragma unroll
        for (int i = 0; i < EPL; ++i) prob[i] = prob[i] / sum;
    } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) prob[i] = 1.0f / (1.0f + expf(-prob[i]));
    }
    if (p.bias != nullptr) {
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (i * 32 + lane < p.E) key[i] = key_of(prob[i] + p.bias[i * 32 + lane]);
    }
    float total = 0.0f, mine = 0.0f;
    int my_id = -1;
    for (int j = 0; j < p.k; ++j) {
        uint32_t best = 0u;
        int at = 0;
        float w = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            if (key[i] > best) {   // the lane's lowest expert where keys are equal
                best = key[i];
                at = i * 32 + lane;
                w = prob[i];
            }
        }
        const uint32_t top = __reduce_max_sync(0xffffffffu, best);
        int id = -1;
        if (top != 0u) {
            id = static_cast<int>(__reduce_min_sync(0xffffffffu, best == top ? static_cast<uint32_t>(at) : 0xffffffffu));
            w = __shfl_sync(0xffffffffu, w, id & 31);
            if (lane == (id & 31)) {
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (i == id >> 5) key[i] = 0u;
            }
        } else {
            w = 0.0f;
        }
        total += w;
        if (lane == j) {
            mine = w;
            my_id = id;
        }
    }
    if (lane < p.k) {
        if (p.renormalize && total != 0.0f) mine /= total;
        p.ids[t * p.k + lane] = my_id;
        p.weights[t * p.k + lane] = mine;
    }
}

__device__ __forceinline__ void choose_any(const ChoiceParams& p, int64_t t, int lane) {
    if (p.E <= 64) choose<2>(p, t, lane);
    else if (p.E <= 256) choose<8>(p, t, lane);
    else choose<32>(p, t, lane);
}

// NT groups of 8 tokens
template <class T, int NT>
__global__ void __launch_bounds__(kRouteThreads)
moe_logits_kernel(const LogitsParams p, const ChoiceParams c) {
    __shared__ float part[kRouteWarps][NT * 8][kRouteTile + 1];
    __shared__ float recv[8][NT * 8 * kRouteTile];   // [CTA of the cluster][outputs of this CTA's share]
    __shared__ uint32_t last;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int P = p.split;
    const int j = static_cast<int>(blockIdx.x % P);
    const int e0 = static_cast<int>(blockIdx.x / P) * kRouteTile;
    const int64_t t0 = static_cast<int64_t>(blockIdx.y) * kRouteTokens;
    const int tokens = static_cast<int>(min(static_cast<int64_t>(NT * 8), p.T - t0));
    if (P > 1) ptx::cluster_sync();   // every CTA of the cluster runs before any writes to another's memory
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    // rows past the end are read from the last one; their sums are not used
    const T* w0 = static_cast<const T*>(p.Wr) + static_cast<int64_t>(min(e0 + g, p.E - 1)) * p.H + t * 8;
    const T* w1 = static_cast<const T*>(p.Wr) + static_cast<int64_t>(min(e0 + g + 8, p.E - 1)) * p.H + t * 8;
    const T* x[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) x[n] = static_cast<const T*>(p.X) + (t0 + min(n * 8 + g, tokens - 1)) * p.H + t * 8;
    float acc[NT][4] = {};
    // steps of 32 k, dealt in turn to the cluster's warps
    constexpr int kUnroll = NT <= 2 ? 4 : 2;
    const uint32_t stride = P * kRouteWarps, H = p.H;   // unsigned: an element past the end may pass 2^31
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    for (uint32_t s = j * kRouteWarps + warp; s * 32u < H; s += kUnroll * stride) {
        uint4 a[kUnroll][2], b[kUnroll][NT];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint32_t k = (s + u * stride) * 32u;
            const bool in = k + t * 8u < H;   // H is a multiple of 8
            a[u][0] = in ? *reinterpret_cast<const uint4*>(w0 + k) : zero;
            a[u][1] = in ? *reinterpret_cast<const uint4*>(w1 + k) : zero;
#pragma unroll
            for (int n = 0; n < NT; ++n) b[u][n] = in ? *reinterpret_cast<const uint4*>(x[n] + k) : zero;
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint32_t lo[4] = {a[u][0].x, a[u][1].x, a[u][0].y, a[u][1].y};
            const uint32_t hi[4] = {a[u][0].z, a[u][1].z, a[u][0].w, a[u][1].w};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                ptx::mma16816<T>(acc[n], lo, b[u][n].x, b[u][n].y);
                ptx::mma16816<T>(acc[n], hi, b[u][n].z, b[u][n].w);
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        part[warp][n * 8 + 2 * t][g] = acc[n][0];
        part[warp][n * 8 + 2 * t + 1][g] = acc[n][1];
        part[warp][n * 8 + 2 * t][g + 8] = acc[n][2];
        part[warp][n * 8 + 2 * t + 1][g + 8] = acc[n][3];
    }
    __syncthreads();
    const int outs = tokens * kRouteTile, per = (outs + P - 1) / P;
    auto store = [&](int o, float v) {
        const int e = e0 + o % kRouteTile;
        if (e < p.E) p.logits[(t0 + o / kRouteTile) * p.E + e] = v;
    };
    for (int o = threadIdx.x; o < outs; o += kRouteThreads) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kRouteWarps; ++w) v += part[w][o / kRouteTile][o % kRouteTile];
        if (P == 1) {
            store(o, v);
        } else {
            const int d = o / per;
            ptx::st_cluster_f32(ptx::mapa(ptx::smem_u32(&recv[j][o - d * per]), static_cast<uint32_t>(d)), v);
        }
    }
    if (P > 1) {
        ptx::cluster_sync();
        for (int i = threadIdx.x; i < per && j * per + i < outs; i += kRouteThreads) {
            float v = 0.0f;
            for (int q = 0; q < P; ++q) v += recv[q][i];
            store(j * per + i, v);
        }
    }
    if (p.T > kRouteFewTokens) return;
    // the last CTA to get here sees every logit
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        last = ptx::atom_add_acq_rel_gpu(p.counter, 1u) == gridDim.x - 1 ? 1u : 0u;
        if (last) *p.counter = 0u;
    }
    __syncthreads();
    if (last && warp < p.T) choose_any(c, warp, lane);
}

__global__ void __launch_bounds__(kRouteThreads) moe_choose_kernel(const ChoiceParams c) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5);
    if (t < c.T) choose_any(c, t, threadIdx.x & 31);
}

template <class T, int NT>
cudaError_t launch_logits(const LogitsParams& p, const ChoiceParams& c, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((p.E + kRouteTile - 1) / kRouteTile * p.split),
                       static_cast<unsigned>((p.T + kRouteTokens - 1) / kRouteTokens), 1);
    cfg.blockDim = dim3(kRouteThreads, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 1;
    if (p.split > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = static_cast<unsigned>(p.split);
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    cfg.attrs = attr;
    return cudaLaunchKernelEx(&cfg, moe_logits_kernel<T, NT>, p, c);
}

template <class T>
cudaError_t run(const LogitsParams& p, const ChoiceParams& c, cudaStream_t s) {
    cudaError_t e;
    if (p.T <= 8) e = launch_logits<T, 1>(p, c, s);
    else if (p.T <= 16) e = launch_logits<T, 2>(p, c, s);
    else if (p.T <= 32) e = launch_logits<T, 4>(p, c, s);
    else e = launch_logits<T, 8>(p, c, s);
    if (e != cudaSuccess || p.T <= kRouteFewTokens) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((p.T + kRouteWarps - 1) / kRouteWarps), 1, 1);
    cfg.blockDim = dim3(kRouteThreads, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, moe_choose_kernel, c);
}

// tokens whose logits are in scratch at one time
constexpr int64_t kRouteBlock = 8192;

}  // namespace

size_t route_scratch_bytes(int64_t T, int64_t E) {
    return static_cast<size_t>((std::min(T, kRouteBlock) * E * 4 + 255) / 256 * 256);
}

gemm_status_t run_route(bool bf16, const RouteParams& r, uint8_t* data, uint32_t* counters, const DeviceView&,
                        gemm_stream_t stream) {
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    for (int64_t t0 = 0; t0 < r.T; t0 += kRouteBlock) {
        const int T = static_cast<int>(std::min(kRouteBlock, r.T - t0));
        LogitsParams p;
        p.X = static_cast<const uint16_t*>(r.X) + t0 * r.H;
        p.Wr = r.Wr;
        p.logits = reinterpret_cast<float*>(data);
        p.counter = counters;
        p.T = T;
        p.H = r.H;
        p.E = r.E;
        // as many CTAs per cluster as leave every warp about two steps of 32 k
        p.split = 1;
        while (p.split < 8 && p.split * kRouteWarps * 2 * 32 < r.H) p.split *= 2;
        const ChoiceParams c{p.logits, r.bias, T, r.E, r.k, r.scoring, r.renormalize, r.ids + t0 * r.k, r.weights + t0 * r.k};
        const cudaError_t e = bf16 ? run<__nv_bfloat16>(p, c, s) : run<__half>(p, c, s);
        if (e != cudaSuccess) {
            cudaGetLastError();
            return GEMM_ERR_LAUNCH;
        }
    }
    return GEMM_OK;
}

}  // namespace gemm_gb300
