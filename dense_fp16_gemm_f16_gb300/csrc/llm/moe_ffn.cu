// moe_ffn.cu -- launches of the experts' two products (moe_up.cuh, rows.cuh).
#include <algorithm>
#include <mutex>

#include "llm/moe_up.cuh"
#include "llm/rows.cuh"
#include "llm/rows_host.cuh"

namespace gemm_gb300 {
namespace {

// Shared memory of each of the two kernels: at most half of an SM's, so the
// second product's CTA finds room beside the first's and has its first ring of
// weights in flight when the first product ends.
constexpr int kFfnSmem = 200 * 1024;

template <class T, bool W4, int NT>
gemm_status_t launch_up(const FfnParams& f, void* h, const DeviceView& dev, cudaStream_t s) {
    UpParams p{};
    p.H = f.H;
    p.I = f.I;
    p.k_stages = (f.H + kStageElems<W4> - 1) / kStageElems<W4>;
    const SideGroups sg(f.w13, f.H);
    p.groups_k = sg.groups_k;
    p.stage_groups = sg.stage_groups;
    p.chunks_per_group = sg.chunks_per_group;
    p.has_zeros = f.w13.zeros != nullptr;
    const int64_t rows = 2ll * f.I * f.E;
    p.stream_w = stream_weights(W4, rows, f.H);
    p.X = f.X;
    p.h = h;
    p.ids = f.ids;
    p.weights = f.weights;
    p.T = f.T;
    p.k = f.k;
    p.E = f.E;
    p.status = dev.status;
    p.timeout_ns = kStreamTimeoutNs;
    const int lists = list_offsets(f.T * f.k, f.E).end;
    const int cols = std::min(8 * NT, f.T);
    int smem = 0;
    for (p.mw = kUpGranules / kTilesPerWarp<NT>; p.mw <= kUpGranules; p.mw *= 2) {
        // as few warps per stage as the registers allow, more where the sums or
        // a ring of KW stages would leave too little in flight
        const int kw = kConsumers / p.mw;
        const int sums = 2 * kw * 8 * NT * kUpPitch * 4;
        p.ring = ring_layout(W4, kUpRows, 2 * kUpGranules * 8, sg.stage_groups, cols, kFfnSmem - 1024 - lists - sums, kw);
        p.list_off = p.ring.end;
        p.sums_off = p.list_off + lists;
        smem = p.sums_off + sums + 1024;
        if (smem <= kFfnSmem && p.ring.stages >= 4) break;
    }
    if (p.mw > kUpGranules) {
        p.mw = kUpGranules;
        if (smem > kMaxDynamicSmem) return GEMM_ERR_CUDA;
    }
    CUtensorMap w, sc, zr;
    if (!encode_weights(f.w13, rows, static_cast<int64_t>(f.E) * sg.groups_k, 2 * f.I, f.H, 8, kUpGranules * 8, sg.stage_groups, &w, &sc, &zr))
        return GEMM_ERR_INVALID_VALUE;
    return launch_stream(moe_up_kernel<T, W4, NT>, dev.dev, dev.sms, 1, smem, s, w, sc, zr, p);
}

template <class T, bool W4, int NT>
gemm_status_t launch_down(const FfnParams& f, const void* h, const DeviceView& dev, cudaStream_t s) {
    RowsParams p{};
    const SideGroups sg(f.w2, f.I);
    const int lists = list_offsets(f.T * f.k, f.E).end;
    p.N = f.H;
    p.K = f.I;
    p.k_stages = (f.I + kStageElems<W4> - 1) / kStageElems<W4>;
    const int smem = plan_rows<T, W4, NT, true>(&p, f.T, std::min(8 * NT, 2 * f.T), sg.stage_groups, lists, kFfnSmem, dev);
    if (smem <= 0) return GEMM_ERR_CUDA;
    p.groups_k = sg.groups_k;
    p.stage_groups = sg.stage_groups;
    p.chunks_per_group = sg.chunks_per_group;
    p.has_zeros = f.w2.zeros != nullptr;
    const int64_t rows = static_cast<int64_t>(f.H) * f.E;
    p.stream_w = stream_weights(W4, rows, f.I);
    p.cols = f.T;
    p.X = h;
    p.D = f.Y;
    p.ids = f.ids;
    p.weights = f.weights;
    p.k = f.k;
    p.E = f.E;
    p.status = dev.status;
    p.timeout_ns = kStreamTimeoutNs;
    CUtensorMap w, sc, zr;
    if (!encode_weights(f.w2, rows, static_cast<int64_t>(f.E) * sg.groups_k, f.H, f.I, p.width, p.width, sg.stage_groups, &w, &sc, &zr))
        return GEMM_ERR_INVALID_VALUE;
    return launch_stream(weight_rows_kernel<T, W4, NT, true>, dev.dev, p.ranges * p.pieces, p.pieces, smem, s, w, sc, zr, p);
}

// Columns a segment may have: as many as one expert can get, up to 64 for
// 16-bit weights and 32 for 4-bit ones, whose group sums take registers too.
template <class T>
gemm_status_t up(const FfnParams& f, void* h, const DeviceView& dev, cudaStream_t s) {
    if (f.w13.scales != nullptr) {
        if (f.T <= 8) return launch_up<T, true, 1>(f, h, dev, s);
        if (f.T <= 16) return launch_up<T, true, 2>(f, h, dev, s);
        return launch_up<T, true, 4>(f, h, dev, s);
    }
    if (f.T <= 8) return launch_up<T, false, 1>(f, h, dev, s);
    if (f.T <= 16) return launch_up<T, false, 2>(f, h, dev, s);
    if (f.T <= 32) return launch_up<T, false, 4>(f, h, dev, s);
    return launch_up<T, false, 8>(f, h, dev, s);
}

template <class T>
gemm_status_t down(const FfnParams& f, const void* h, const DeviceView& dev, cudaStream_t s) {
    if (f.w2.scales != nullptr) {
        if (f.T <= 4) return launch_down<T, true, 1>(f, h, dev, s);
        if (f.T <= 8) return launch_down<T, true, 2>(f, h, dev, s);
        return launch_down<T, true, 4>(f, h, dev, s);
    }
    if (f.T <= 4) return launch_down<T, false, 1>(f, h, dev, s);
    if (f.T <= 8) return launch_down<T, false, 2>(f, h, dev, s);
    if (f.T <= 16) return launch_down<T, false, 4>(f, h, dev, s);
    return launch_down<T, false, 8>(f, h, dev, s);
}

}  // namespace

size_t ffn_scratch_bytes(int64_t T, int64_t I, int k) { return static_cast<size_t>(T) * k * 2 * I * 2; }

gemm_status_t run_ffn(bool bf16, const FfnParams& p, uint8_t* data, const DeviceView& dev, gemm_stream_t stream) {
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const gemm_status_t st = bf16 ? up<__nv_bfloat16>(p, data, dev, s) : up<__half>(p, data, dev, s);
    if (st != GEMM_OK) return st;
    return bf16 ? down<__nv_bfloat16>(p, data, dev, s) : down<__half>(p, data, dev, s);
}

}  // namespace gemm_gb300
