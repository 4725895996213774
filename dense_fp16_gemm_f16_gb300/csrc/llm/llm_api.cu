// llm_api.cu -- the C ABI declared in include/gemm_llm.h: argument checks,
// per-stream scratch and the calls into the kernels' launchers.  Nothing here
// computes on the CPU.
#include <algorithm>
#include <cfloat>
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

gemm_status_t rmsnorm(int dtype, const void* X, const void* residual, const void* weight, float eps, int64_t T, int64_t H,
                      const gemm_norm_out_t* out, gemm_stream_t stream) {
    if (!type16(dtype) || !dim_ok(T) || !dim_ok(H) || out == nullptr) return GEMM_ERR_INVALID_VALUE;
    if (!(eps >= 0.0f) || eps > FLT_MAX) return GEMM_ERR_INVALID_VALUE;
    if (out->Y == nullptr && out->Y8 == nullptr && T > 0 && H > 0) return GEMM_ERR_INVALID_VALUE;
    const bool eight = out->Y8 != nullptr;
    if (eight && out->dtype8 != GEMM_DTYPE_E4M3 && out->dtype8 != GEMM_DTYPE_E5M2) return GEMM_ERR_INVALID_VALUE;
    // one scale for all rows, or a place for one per row, and neither without an 8-bit output
    const bool fixed = out->scale != 0.0f;
    if (fixed && (!(out->scale > 0.0f) || out->scale > FLT_MAX)) return GEMM_ERR_INVALID_VALUE;
    if (eight ? fixed == (out->scales != nullptr) : fixed || out->scales != nullptr) return GEMM_ERR_INVALID_VALUE;
    if (T == 0 || H == 0) return GEMM_OK;
    if (X == nullptr) return GEMM_ERR_INVALID_VALUE;
    if (H % 8 != 0) return GEMM_ERR_MISALIGNED;
    if (!aligned16(X) || !aligned16(residual) || !aligned16(weight) || !aligned16(out->Y) || !aligned16(out->Y8) ||
        !aligned4(out->scales) || !aligned16(out->total))
        return GEMM_ERR_MISALIGNED;
    if (mul_sat(T, H) < 0) return GEMM_ERR_INVALID_VALUE;
    // Y and total may be X or the residual themselves (a row is read before it is
    // written); no output may overlap anything else
    const struct { const void* p; int64_t bytes; } outs[4] = {{out->Y, T * H * 2}, {out->total, T * H * 2},
                                                              {out->Y8, T * H}, {out->scales, T * 4}};
    for (int i = 0; i < 4; ++i) {
        if (outs[i].p == nullptr) continue;
        for (const void* in : {X, residual})
            if (in != nullptr && ranges_overlap(outs[i].p, outs[i].bytes, in, T * H * 2) && (i > 1 || outs[i].p != in))
                return GEMM_ERR_INVALID_VALUE;
        if (weight != nullptr && ranges_overlap(outs[i].p, outs[i].bytes, weight, H * 2)) return GEMM_ERR_INVALID_VALUE;
        for (int j = 0; j < i; ++j)
            if (outs[j].p != nullptr && ranges_overlap(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes))
                return GEMM_ERR_INVALID_VALUE;
    }
    DeviceView dev;
    const gemm_status_t st = device_view(&dev);
    if (st != GEMM_OK) return st;
    const NormArgs a{X, residual, weight, out->Y, out->Y8, out->scales, out->total, T, H, eps, out->scale,
                     out->dtype8 == GEMM_DTYPE_E5M2};
    return run_rmsnorm(dtype == GEMM_DTYPE_BF16, a, dev, reinterpret_cast<cudaStream_t>(stream));
}

// The checks of adapters beside X [M][K] and an output U [M][N]; fills all of `a` but C, beta and U.
gemm_status_t check_lora(int dtype, const void* X, const gemm_lora_t* l, const int32_t* ids, const void* U, int64_t M,
                         int64_t N, int64_t K, LoraArgs* a) {
    if (!type16(dtype) || !dim_ok(M) || !dim_ok(N) || !dim_ok(K) || l == nullptr) return GEMM_ERR_INVALID_VALUE;
    if (l->count < 0 || l->R < 1 || l->R > kLoraMaxRank) return GEMM_ERR_INVALID_VALUE;
    const int64_t count = l->count, R = l->R, a_size = mul_sat(mul_sat(count, R), K), b_size = mul_sat(mul_sat(count, R), N);
    if (a_size < 0 || b_size < 0) return GEMM_ERR_INVALID_VALUE;
    if (M > 0 && N > 0) {
        if (U == nullptr || (K > 0 && X == nullptr)) return GEMM_ERR_INVALID_VALUE;
        if (count > 0 && K > 0 && (l->A == nullptr || l->B == nullptr || ids == nullptr)) return GEMM_ERR_INVALID_VALUE;
    }
    if (K % 8 != 0 || N % 8 != 0 || R % 8 != 0) return GEMM_ERR_MISALIGNED;
    if (!aligned16(X) || !aligned16(U) || !aligned4(ids) || !aligned16(l->A) || !aligned16(l->B) || !aligned4(l->factors))
        return GEMM_ERR_MISALIGNED;
    const int64_t out = mul_sat(M, N) < 0 ? -1 : M * N * 2;
    if (out < 0 || mul_sat(M, K) < 0) return GEMM_ERR_INVALID_VALUE;
    if (ranges_overlap(U, out, X, M * K * 2) || (l->A != nullptr && ranges_overlap(U, out, l->A, a_size * 2)) ||
        (l->B != nullptr && ranges_overlap(U, out, l->B, b_size * 2)) ||
        (l->factors != nullptr && ranges_overlap(U, out, l->factors, count * 4)) ||
        (ids != nullptr && ranges_overlap(U, out, ids, M * 4)))
        return GEMM_ERR_INVALID_VALUE;
    *a = LoraArgs{X, l->A, l->B, l->factors, ids, nullptr, 0.0f, nullptr, nullptr, nullptr, M, N, K, R, count};
    return GEMM_OK;
}

gemm_status_t lora_delta(int dtype, const void* X, const gemm_lora_t* l, const int32_t* ids, float beta, const void* C, void* U,
                         int64_t M, int64_t N, int64_t K, gemm_stream_t stream) {
    LoraArgs a;
    gemm_status_t st = check_lora(dtype, X, l, ids, U, M, N, K, &a);
    if (st != GEMM_OK) return st;
    const gemm_epilogue_t epilogue{1.0f, beta, C, nullptr, GEMM_ACT_NONE, 0, nullptr};
    st = check_epilogue(&epilogue, U, M, N);
    if (st != GEMM_OK) return st;
    if (M == 0 || N == 0) return GEMM_OK;
    a.C = beta != 0.0f ? C : nullptr;
    a.beta = beta;
    a.U = U;
    DeviceView dev;
    st = device_view(&dev);
    if (st != GEMM_OK) return st;
    Scratch ws;
    const size_t bytes = lora_scratch_bytes(M);
    if (bytes > 0) st = get_scratch(dev.dev, stream, bytes, &ws);
    if (st != GEMM_OK) return st;
    return run_lora(dtype == GEMM_DTYPE_BF16, a, ws.data, dev, reinterpret_cast<cudaStream_t>(stream));
}

gemm_status_t lora_nt(int dtype, const void* X, const gemm_weights_t* weights, const gemm_lora_t* l, const int32_t* ids,
                      void* D, int64_t M, int64_t N, int64_t K, const gemm_epilogue_t* epilogue, gemm_stream_t stream) {
    LoraArgs a;
    gemm_status_t st = check_lora(dtype, X, l, ids, D, M, N, K, &a);
    if (st != GEMM_OK) return st;
    Weights w;
    st = check_weights(weights, N, N, K, false, &w);
    if (st != GEMM_OK) return st;
    st = check_epilogue(epilogue, D, M, N);
    if (st != GEMM_OK) return st;
    if (M == 0 || N == 0) return GEMM_OK;
    if (K > 0 && overlaps_weights(D, M * N * 2, w, N, K)) return GEMM_ERR_INVALID_VALUE;
    DeviceView dev;
    st = device_view(&dev);
    if (st != GEMM_OK) return st;
    // beta C and the adapters' part go to D, and the projection's epilogue adds them
    gemm_epilogue_t epi{1.0f, 0.0f, nullptr, nullptr, GEMM_ACT_NONE, 0, nullptr};
    if (epilogue != nullptr) epi = *epilogue;
    if (K == 0 || a.count == 0) {
        const EpiParams plain = epi_params(epilogue);
        if (K == 0) return run_empty_sum(D, M, N, plain, dtype, dev.sms, reinterpret_cast<cudaStream_t>(stream));
        return w.scales != nullptr ? run_w4_gemm(dtype == GEMM_DTYPE_BF16, X, w, D, M, N, K, plain, dev, stream)
                                   : run_dense(dtype, X, w.data, D, M, N, K, epilogue, nullptr, stream);
    }
    if (w.scales == nullptr && M <= kLoraEpiRows && M * a.R <= kLoraEpiFloats) {
        // few rows: X Aᵀ by itself, its product with B on the idle warps of the projection's kernel
        Scratch ws;
        st = get_scratch(dev.dev, stream, static_cast<size_t>(M * a.R * 4), &ws);
        if (st != GEMM_OK) return st;
        a.V = reinterpret_cast<float*>(ws.data);
        a.ready = ws.counters + kCounterLora;
        st = run_lora(dtype == GEMM_DTYPE_BF16, a, nullptr, dev, reinterpret_cast<cudaStream_t>(stream));
        if (st != GEMM_OK) return st;
        const LoraEpi part{a.V, l->B, ids, a.ready, static_cast<int32_t>(a.R), static_cast<int32_t>(a.count)};
        st = run_dense(dtype, X, w.data, D, M, N, K, epilogue, &part, stream);
        if (st != GEMM_OK) cudaMemsetAsync(a.ready, 0, sizeof(uint32_t), reinterpret_cast<cudaStream_t>(stream));   // nobody took it back
        return st;
    }
    a.C = epi.beta != 0.0f ? epi.C : nullptr;
    a.beta = epi.beta;
    a.U = D;
    epi.beta = 1.0f;
    epi.C = D;
    Scratch ws;
    const size_t bytes = lora_scratch_bytes(M);
    if (bytes > 0) st = get_scratch(dev.dev, stream, bytes, &ws);
    if (st != GEMM_OK) return st;
    st = run_lora(dtype == GEMM_DTYPE_BF16, a, ws.data, dev, reinterpret_cast<cudaStream_t>(stream));
    if (st != GEMM_OK) return st;
    return w.scales != nullptr ? run_w4_gemm(dtype == GEMM_DTYPE_BF16, X, w, D, M, N, K, epi_params(&epi), dev, stream)
                               : run_dense(dtype, X, w.data, D, M, N, K, &epi, nullptr, stream);
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

GEMM_API gemm_status_t gemm_rmsnorm(gemm_dtype_t dtype, const void* X, const void* residual, const void* weight, float eps,
                                    int64_t T, int64_t H, const gemm_norm_out_t* out, gemm_stream_t stream) {
    return guarded([&] { return rmsnorm(dtype, X, residual, weight, eps, T, H, out, stream); });
}

GEMM_API gemm_status_t gemm_moe_route(gemm_dtype_t dtype, const void* X, const void* Wr, const float* bias, int64_t T,
                                      int64_t H, int64_t E, int32_t k, gemm_moe_scoring_t scoring,
                                      int32_t renormalize, int32_t* ids, float* weights, gemm_stream_t stream) {
    return guarded([&] { return route(dtype, X, Wr, bias, T, H, E, k, scoring, renormalize, ids, weights, stream); });
}

GEMM_API gemm_status_t gemm_lora_delta(gemm_dtype_t dtype, const void* X, const gemm_lora_t* lora, const int32_t* ids,
                                       float beta, const void* C, void* U, int64_t M, int64_t N, int64_t K,
                                       gemm_stream_t stream) {
    return guarded([&] { return lora_delta(dtype, X, lora, ids, beta, C, U, M, N, K, stream); });
}

GEMM_API gemm_status_t gemm_lora_nt(gemm_dtype_t dtype, const void* X, const gemm_weights_t* W, const gemm_lora_t* lora,
                                    const int32_t* ids, void* D, int64_t M, int64_t N, int64_t K,
                                    const gemm_epilogue_t* epilogue, gemm_stream_t stream) {
    return guarded([&] { return lora_nt(dtype, X, W, lora, ids, D, M, N, K, epilogue, stream); });
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
