// llm_api.cu -- the C ABI declared in include/gemm_llm.h: argument checks,
// per-stream scratch and the calls into the kernels' launchers.  Nothing here
// computes on the CPU.
#include <algorithm>
#include <climits>
#include <map>
#include <mutex>
#include <vector>

#include "llm/llm.h"

using namespace gemm_gb300;

namespace gemm_gb300 {

namespace {
struct StreamScratch {
    std::mutex mu;   // held by the call whose launches use the buffer
    uint8_t* data = nullptr;
    size_t bytes = 0;
    uint32_t* counters = nullptr;
};
std::mutex g_scratch_mu;
std::map<StreamKey, StreamScratch> g_scratch;
}  // namespace

// A buffer that has become too small is not freed: work queued on the stream,
// or a captured graph, may still use it.  Buffers at least double, so the ones
// left behind hold less than the one in use.
gemm_status_t get_scratch(int dev, gemm_stream_t stream, size_t bytes, Scratch* out) {
    StreamKey key;
    const gemm_status_t st = stream_key(dev, stream, &key);
    if (st != GEMM_OK) return st;
    StreamScratch* found = nullptr;
    {
        std::lock_guard<std::mutex> lock(g_scratch_mu);
        found = &g_scratch[key];   // stays where it is
    }
    StreamScratch& w = *found;
    w.mu.lock();
    out->held = &w.mu;
    if (w.counters == nullptr) {
        uint32_t* c = nullptr;
        if (cudaMalloc(&c, kScratchCounters * sizeof(uint32_t)) != cudaSuccess) {
            cudaGetLastError();
            return GEMM_ERR_CUDA;
        }
        if (cudaMemset(c, 0, kScratchCounters * sizeof(uint32_t)) != cudaSuccess ||
            cudaDeviceSynchronize() != cudaSuccess) {   // zero before any stream's kernel reads them
            cudaGetLastError();
            cudaFree(c);
            return GEMM_ERR_CUDA;
        }
        w.counters = c;
    }
    if (w.bytes < bytes) {
        const size_t want = std::max(bytes, 2 * w.bytes);
        uint8_t* d = nullptr;
        if (cudaMalloc(&d, want) != cudaSuccess) {
            cudaGetLastError();
            return GEMM_ERR_CUDA;
        }
        w.data = d;
        w.bytes = want;
    }
    out->data = w.data;
    out->counters = w.counters;
    return GEMM_OK;
}

}  // namespace gemm_gb300

namespace {

constexpr int64_t kMaxDim = INT32_MAX;

bool dim_ok(int64_t v) { return v >= 0 && v <= kMaxDim; }
bool type16(int dtype) { return dtype == GEMM_DTYPE_F16 || dtype == GEMM_DTYPE_BF16; }
bool group_ok(int32_t g) { return g == 32 || g == 64 || g == 128; }

// a * b, or -1 where it passes 2^62 (sizes that no array can have)
int64_t mul_sat(int64_t a, int64_t b) {
    if (a < 0 || b < 0) return -1;
    if (a != 0 && b > (int64_t{1} << 62) / a) return -1;
    return a * b;
}

// The checks of one stack of weights: `rows` rows in all of K elements, each
// matrix `rows_each` rows.  Fills the kernel form; *bytes the size of `data`.
gemm_status_t check_weights(const gemm_weights_t* w, int64_t rows, int64_t rows_each, int64_t K, bool need4,
                            Weights* out) {
    if (w == nullptr) return GEMM_ERR_INVALID_VALUE;
    const bool some = rows > 0 && K > 0;
    const bool four = need4 || w->scales != nullptr;   // an empty array may have no address
    if (four && some && w->scales == nullptr) return GEMM_ERR_INVALID_VALUE;
    if (!four && (w->zeros != nullptr || w->group != 0)) return GEMM_ERR_INVALID_VALUE;
    if (four && !group_ok(w->group)) return GEMM_ERR_INVALID_VALUE;
    if (rows > kMaxDim || mul_sat(rows, K) < 0) return GEMM_ERR_INVALID_VALUE;
    if (some && w->data == nullptr) return GEMM_ERR_INVALID_VALUE;
    if (four && (K % w->group != 0 || rows_each % 8 != 0)) return GEMM_ERR_MISALIGNED;
    if (!four && K % 8 != 0) return GEMM_ERR_MISALIGNED;
    if (!aligned16(w->data) || !aligned16(w->scales) || !aligned16(w->zeros)) return GEMM_ERR_MISALIGNED;
    *out = Weights{w->data, w->scales, w->zeros, w->group};
    return GEMM_OK;
}

bool overlaps_weights(const void* p, int64_t bytes, const Weights& w, int64_t rows, int64_t K) {
    if (w.scales == nullptr) return ranges_overlap(p, bytes, w.data, rows * K * 2);
    const int64_t side = rows * (K / w.group) * 2;
    return ranges_overlap(p, bytes, w.data, rows * K / 2) || ranges_overlap(p, bytes, w.scales, side) ||
           (w.zeros != nullptr && ranges_overlap(p, bytes, w.zeros, side));
}

gemm_status_t from_launch(cudaError_t e) {
    if (e == cudaSuccess) return GEMM_OK;
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
}

// No exception leaves a C entry (the maps behind device state and scratch allocate).
template <class F>
gemm_status_t guarded(F&& f) {
    try {
        return f();
    } catch (...) {
        return GEMM_ERR_CUDA;
    }
}

gemm_status_t quantize(int dtype, const void* W, int64_t batch, int64_t N, int64_t K, int32_t group, void* codes,
                       void* scales, void* zeros, gemm_stream_t stream) {
    if (!type16(dtype) || !dim_ok(batch) || !dim_ok(N) || !dim_ok(K) || !group_ok(group)) return GEMM_ERR_INVALID_VALUE;
    const int64_t rows = mul_sat(batch, N);
    if (rows < 0 || rows > kMaxDim || mul_sat(rows, K) < 0) return GEMM_ERR_INVALID_VALUE;
    if (rows == 0 || K == 0) return GEMM_OK;
    if (W == nullptr || codes == nullptr || scales == nullptr) return GEMM_ERR_INVALID_VALUE;
    if (K % group != 0 || N % 8 != 0) return GEMM_ERR_MISALIGNED;
    if (!aligned16(W) || !aligned16(codes) || !aligned16(scales) || !aligned16(zeros)) return GEMM_ERR_MISALIGNED;
    const int64_t side = rows * (K / group) * 2, in = rows * K * 2, out = rows * K / 2;
    const int64_t zside = zeros != nullptr ? side : 0;
    if (ranges_overlap(codes, out, W, in) || ranges_overlap(scales, side, W, in) || ranges_overlap(zeros, zside, W, in) ||
        ranges_overlap(codes, out, scales, side) || ranges_overlap(codes, out, zeros, zside) ||
        ranges_overlap(scales, side, zeros, zside))
        return GEMM_ERR_INVALID_VALUE;
    DeviceView dev;
    const gemm_status_t st = device_view(&dev);
    if (st != GEMM_OK) return st;
    return from_launch(launch_w4_quantize(dtype == GEMM_DTYPE_BF16, W, batch, N, K, group, codes, scales, zeros,
                                          dev.sms, reinterpret_cast<cudaStream_t>(stream)));
}

gemm_status_t dequantize(int dtype, const gemm_weights_t* weights, int64_t batch, int64_t N, int64_t K, void* W,
                         gemm_stream_t stream) {
    if (!type16(dtype) || !dim_ok(batch) || !dim_ok(N) || !dim_ok(K)) return GEMM_ERR_INVALID_VALUE;
    const int64_t rows = mul_sat(batch, N);
    if (rows < 0) return GEMM_ERR_INVALID_VALUE;
    Weights w;
    gemm_status_t st = check_weights(weights, rows, N, K, true, &w);
    if (st != GEMM_OK) return st;
    if (rows == 0 || K == 0) return GEMM_OK;
    if (W == nullptr) return GEMM_ERR_INVALID_VALUE;
    if (!aligned16(W)) return GEMM_ERR_MISALIGNED;
    if (overlaps_weights(W, rows * K * 2, w, rows, K)) return GEMM_ERR_INVALID_VALUE;
    DeviceView dev;
    st = device_view(&dev);
    if (st != GEMM_OK) return st;
    return from_launch(launch_w4_dequantize(dtype == GEMM_DTYPE_BF16, w, batch, N, K, W,
                                            dev.sms, reinterpret_cast<cudaStream_t>(stream)));
}

gemm_status_t w4_nt(int dtype, const void* A, const gemm_weights_t* B, void* D, int64_t M, int64_t N, int64_t K,
                    const gemm_epilogue_t* epilogue, gemm_stream_t stream) {
    if (!type16(dtype) || !dim_ok(M) || !dim_ok(N) || !dim_ok(K)) return GEMM_ERR_INVALID_VALUE;
    Weights w;
    gemm_status_t st = check_weights(B, N, N, K, true, &w);
    if (st != GEMM_OK) return st;
    st = check_epilogue(epilogue, D, M, N);
    if (st != GEMM_OK) return st;
    const EpiParams epi = epi_params(epilogue);
    if (M == 0 || N == 0) return GEMM_OK;
    if (D == nullptr || (K > 0 && A == nullptr)) return GEMM_ERR_INVALID_VALUE;
    const int64_t d_bytes = M * N * 2;
    if (ranges_overlap(D, d_bytes, A, M * K * 2) || (K > 0 && overlaps_weights(D, d_bytes, w, N, K)))
        return GEMM_ERR_INVALID_VALUE;
    if (!aligned16(D) || !aligned16(A)) return GEMM_ERR_MISALIGNED;
    DeviceView dev;
    st = device_view(&dev);
    if (st != GEMM_OK) return st;
    if (K == 0) return run_empty_sum(D, M, N, epi, dtype, dev.sms, reinterpret_cast<cudaStream_t>(stream));
    return run_w4_gemm(dtype == GEMM_DTYPE_BF16, A, w, D, M, N, K, epi, dev, stream);
}

gemm_status_t check_route(int dtype, const void* X, const void* Wr, const float* bias, int64_t T, int64_t H, int64_t E,
                          int32_t k, int scoring) {
    if (!type16(dtype) || !dim_ok(T) || !dim_ok(H) || E < 1 || E > kMoeMaxExperts || k < 1 || k > kMoeMaxChoices || k > E)
        return GEMM_ERR_INVALID_VALUE;
    if (scoring != GEMM_MOE_SOFTMAX && scoring != GEMM_MOE_SIGMOID) return GEMM_ERR_INVALID_VALUE;
    if (T > 0 && H > 0 && (X == nullptr || Wr == nullptr)) return GEMM_ERR_INVALID_VALUE;
    if (H % 8 != 0) return GEMM_ERR_MISALIGNED;
    if (!aligned16(X) || !aligned16(Wr) || !aligned16(bias)) return GEMM_ERR_MISALIGNED;
    return GEMM_OK;
}

gemm_status_t route(int dtype, const void* X, const void* Wr, const float* bias, int64_t T, int64_t H, int64_t E,
                    int32_t k, int scoring, int32_t renormalize, int32_t* ids, float* weights, gemm_stream_t stream) {
    gemm_status_t st = check_route(dtype, X, Wr, bias, T, H, E, k, scoring);
    if (st != GEMM_OK) return st;
    if (T == 0) return GEMM_OK;
    if (ids == nullptr || weights == nullptr) return GEMM_ERR_INVALID_VALUE;
    if (!aligned16(ids) || !aligned16(weights)) return GEMM_ERR_MISALIGNED;
    const int64_t out = T * k * 4;
    for (const void* o : {static_cast<const void*>(ids), static_cast<const void*>(weights)})
        if (ranges_overlap(o, out, X, T * H * 2) || ranges_overlap(o, out, Wr, E * H * 2) ||
            (bias != nullptr && ranges_overlap(o, out, bias, E * 4)))
            return GEMM_ERR_INVALID_VALUE;
    if (ranges_overlap(ids, out, weights, out)) return GEMM_ERR_INVALID_VALUE;
    DeviceView dev;
    st = device_view(&dev);
    if (st != GEMM_OK) return st;
    const RouteParams p{X, Wr, bias, T, static_cast<int32_t>(H), static_cast<int32_t>(E), k, scoring, renormalize, ids,
                        weights};
    Scratch ws;
    st = get_scratch(dev.dev, stream, route_scratch_bytes(T, E), &ws);
    if (st != GEMM_OK) return st;
    return run_route(dtype == GEMM_DTYPE_BF16, p, ws.data, ws.counters, dev, stream);
}

// The checks that gemm_moe_ffn and gemm_moe_layer share; fills all of `p` but ids and weights.
gemm_status_t check_ffn(int dtype, const void* X, const gemm_weights_t* w13, const gemm_weights_t* w2, void* Y,
                        int64_t T, int64_t H, int64_t I, int64_t E, int32_t k, FfnParams* p) {
    if (!type16(dtype) || T < 0 || T > kMoeMaxTokens || !dim_ok(H) || !dim_ok(I) || E < 1 || E > kMoeMaxExperts ||
        k < 1 || k > kMoeMaxChoices || H < 1 || I < 1)
        return GEMM_ERR_INVALID_VALUE;
    gemm_status_t st = check_weights(w13, E * 2 * I, 2 * I, H, false, &p->w13);
    if (st != GEMM_OK) return st;
    st = check_weights(w2, E * H, H, I, false, &p->w2);
    if (st != GEMM_OK) return st;
    if (H % 8 != 0 || I % 8 != 0) return GEMM_ERR_MISALIGNED;
    if (T > 0 && (X == nullptr || Y == nullptr)) return GEMM_ERR_INVALID_VALUE;
    if (!aligned16(X) || !aligned16(Y)) return GEMM_ERR_MISALIGNED;
    const int64_t bytes = T * H * 2;
    if (ranges_overlap(Y, bytes, X, bytes) || overlaps_weights(Y, bytes, p->w13, E * 2 * I, H) ||
        overlaps_weights(Y, bytes, p->w2, E * H, I))
        return GEMM_ERR_INVALID_VALUE;
    p->X = X;
    p->Y = Y;
    p->T = static_cast<int32_t>(T);
    p->H = static_cast<int32_t>(H);
    p->I = static_cast<int32_t>(I);
    p->E = static_cast<int32_t>(E);
    p->k = k;
    return GEMM_OK;
}

gemm_status_t ffn(int dtype, const void* X, const int32_t* ids, const float* weights, const gemm_weights_t* w13,
                  const gemm_weights_t* w2, void* Y, int64_t T, int64_t H, int64_t I, int64_t E, int32_t k,
                  gemm_stream_t stream) {
    FfnParams p;
    gemm_status_t st = check_ffn(dtype, X, w13, w2, Y, T, H, I, E, k, &p);
    if (st != GEMM_OK) return st;
    if (T == 0) return GEMM_OK;
    if (ids == nullptr || weights == nullptr) return GEMM_ERR_INVALID_VALUE;
    if (!aligned16(ids) || !aligned16(weights)) return GEMM_ERR_MISALIGNED;
    if (ranges_overlap(Y, T * H * 2, ids, T * k * 4) || ranges_overlap(Y, T * H * 2, weights, T * k * 4))
        return GEMM_ERR_INVALID_VALUE;
    p.ids = ids;
    p.weights = weights;
    DeviceView dev;
    st = device_view(&dev);
    if (st != GEMM_OK) return st;
    Scratch ws;
    st = get_scratch(dev.dev, stream, ffn_scratch_bytes(T, I, k), &ws);
    if (st != GEMM_OK) return st;
    return run_ffn(dtype == GEMM_DTYPE_BF16, p, ws.data, dev, stream);
}

gemm_status_t layer(int dtype, const void* X, const void* Wr, const float* bias, const gemm_weights_t* w13,
                    const gemm_weights_t* w2, void* Y, int64_t T, int64_t H, int64_t I, int64_t E, int32_t k,
                    int scoring, int32_t renormalize, gemm_stream_t stream) {
    gemm_status_t st = check_route(dtype, X, Wr, bias, T, H, E, k, scoring);
    if (st != GEMM_OK) return st;
    FfnParams p;
    st = check_ffn(dtype, X, w13, w2, Y, T, H, I, E, k, &p);
    if (st != GEMM_OK) return st;
    if (T == 0) return GEMM_OK;
    if (ranges_overlap(Y, T * H * 2, Wr, E * H * 2) || (bias != nullptr && ranges_overlap(Y, T * H * 2, bias, E * 4)))
        return GEMM_ERR_INVALID_VALUE;
    DeviceView dev;
    st = device_view(&dev);
    if (st != GEMM_OK) return st;
    // scratch: run_route's, ids and weights (256-byte padded each), run_ffn's
    const size_t logits = route_scratch_bytes(T, E), side = (static_cast<size_t>(T) * k * 4 + 255) / 256 * 256;
    Scratch ws;
    st = get_scratch(dev.dev, stream, logits + 2 * side + ffn_scratch_bytes(T, I, k), &ws);
    if (st != GEMM_OK) return st;
    int32_t* ids = reinterpret_cast<int32_t*>(ws.data + logits);
    float* weights = reinterpret_cast<float*>(ws.data + logits + side);
    const RouteParams r{X, Wr, bias, T, static_cast<int32_t>(H), static_cast<int32_t>(E), k, scoring, renormalize, ids,
                        weights};
    const bool bf16 = dtype == GEMM_DTYPE_BF16;
    st = run_route(bf16, r, ws.data, ws.counters, dev, stream);
    if (st != GEMM_OK) return st;
    p.ids = ids;
    p.weights = weights;
    return run_ffn(bf16, p, ws.data + logits + 2 * side, dev, stream);
}

}  // namespace

extern "C" {

GEMM_API gemm_status_t gemm_w4_quantize(gemm_dtype_t dtype, const void* W, int64_t batch, int64_t N, int64_t K,
                                        int32_t group, void* codes, void* scales, void* zeros, gemm_stream_t stream) {
    return guarded([&] { return quantize(dtype, W, batch, N, K, group, codes, scales, zeros, stream); });
}

GEMM_API gemm_status_t gemm_w4_dequantize(gemm_dtype_t dtype, const gemm_weights_t* weights, int64_t batch, int64_t N,
                                          int64_t K, void* W, gemm_stream_t stream) {
    return guarded([&] { return dequantize(dtype, weights, batch, N, K, W, stream); });
}

GEMM_API gemm_status_t gemm_w4_nt(gemm_dtype_t dtype, const void* A, const gemm_weights_t* B, void* D, int64_t M,
                                  int64_t N, int64_t K, const gemm_epilogue_t* epilogue, gemm_stream_t stream) {
    return guarded([&] { return w4_nt(dtype, A, B, D, M, N, K, epilogue, stream); });
}

GEMM_API gemm_status_t gemm_moe_route(gemm_dtype_t dtype, const void* X, const void* Wr, const float* bias, int64_t T,
                                      int64_t H, int64_t E, int32_t k, gemm_moe_scoring_t scoring,
                                      int32_t renormalize, int32_t* ids, float* weights, gemm_stream_t stream) {
    return guarded([&] { return route(dtype, X, Wr, bias, T, H, E, k, scoring, renormalize, ids, weights, stream); });
}

GEMM_API gemm_status_t gemm_moe_ffn(gemm_dtype_t dtype, const void* X, const int32_t* ids, const float* weights,
                                    const gemm_weights_t* w13, const gemm_weights_t* w2, void* Y, int64_t T,
                                    int64_t H, int64_t I, int64_t E, int32_t k, gemm_stream_t stream) {
    return guarded([&] { return ffn(dtype, X, ids, weights, w13, w2, Y, T, H, I, E, k, stream); });
}

GEMM_API gemm_status_t gemm_moe_layer(gemm_dtype_t dtype, const void* X, const void* Wr, const float* bias,
                                      const gemm_weights_t* w13, const gemm_weights_t* w2, void* Y, int64_t T,
                                      int64_t H, int64_t I, int64_t E, int32_t k, gemm_moe_scoring_t scoring,
                                      int32_t renormalize, gemm_stream_t stream) {
    return guarded(
        [&] { return layer(dtype, X, Wr, bias, w13, w2, Y, T, H, I, E, k, scoring, renormalize, stream); });
}

}  // extern "C"
