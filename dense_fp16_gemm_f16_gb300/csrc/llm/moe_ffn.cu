// moe_ffn.cu -- launches of the experts' two products (moe_up.cuh, rows.cuh).
#include <algorithm>
#include <mutex>

#include "llm/moe_up.cuh"
#include "llm/rows.cuh"
#include "llm/rows_host.cuh"

namespace gemm_gb300 {
namespace {

// Slots of an expert when the choices are even, for the experts that get any.
int typical_slots(const FfnParams& f) { return std::max(1, (f.T * f.k + f.E - 1) / f.E); }

template <class T, int CPG, int NT>
gemm_status_t launch_up(const FfnParams& f, void* h, const DeviceView& dev, cudaStream_t s) {
    constexpr bool W4 = CPG != 0;
    UpParams p{};
    p.H = f.H;
    p.I = f.I;
    const SideGroups sg(f.w13, f.H);
    p.groups_k = sg.groups_k;
    p.atom_groups = sg.atom_groups;
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
    constexpr int kBudget = kSmemBudget<W4, NT, true>;
    int smem = 0;
    for (int mw = kUpGranules / kTilesPerWarp<W4, NT, true>; mw <= kUpGranules; mw *= 2) {
        // as few warps per stage as the registers allow, more where the sums
        // would leave too little in flight
        const int kw = kConsumers / mw;
        const int sums = kw * 8 * NT * kUpPitch * 4;
        p.mw = mw;
        // 4-bit weights: a segment's columns stay in shared memory over all its
        // pieces if they take at most half of it; a stage of columns would be as
        // large as the weights beside it
        const int fixed = 1024 + lists + sums;
        // in 64 bits: eight columns of 2^27 elements pass 2^31 bytes
        const int64_t x_pitch = (2ll * f.H + 127) / 128 * 128 + 64;
        const int64_t all_columns = W4 ? (up_to(cols, 8) * x_pitch + 127) / 128 * 128 : 0;
        p.x_resident = W4 && all_columns <= kBudget / 2 && fixed + all_columns + kw * 12 * 1024 <= kBudget;
        p.x_pitch = p.x_resident ? static_cast<int32_t>(x_pitch) : 0;
        const int resident = p.x_resident ? static_cast<int>(all_columns) : 0;
        p.ring = ring_layout(W4, 1, kUpRows, 2 * kUpGranules * 8, sg.atom_groups, p.x_resident ? 0 : cols,
                             kBudget - fixed - resident, kw);
        p.x_off = p.ring.end;
        p.list_off = p.x_off + resident;
        p.sums_off = p.list_off + lists;
        smem = p.sums_off + sums + 1024;
        if (smem <= kBudget && p.ring.slots >= 8) break;
    }
    if (smem > kMaxDynamicSmem) return GEMM_ERR_CUDA;
    p.k_stages = count_of(f.H, kAtomElems<W4>);
    CUtensorMap w, sc, zr;
    if (!encode_weights(f.w13, rows, static_cast<int64_t>(f.E) * sg.groups_k, 2 * f.I, f.H, 8, kUpGranules * 8,
                        sg.atom_groups, &w, &sc, &zr) ||
        !encode_weights_box(f.w13, rows, f.H, 8 * kUpGranules, &p.tm_piece))
        return GEMM_ERR_INVALID_VALUE;
    return launch_stream(moe_up_kernel<T, CPG, NT>, dev.dev, kCtasPerSm<W4, NT, true> * dev.sms, 1, smem, true, s, w, sc,
                         zr, p);
}

template <class T, int CPG, int NT>
gemm_status_t launch_down(const FfnParams& f, const void* h, const DeviceView& dev, cudaStream_t s) {
    constexpr bool W4 = CPG != 0;
    RowsParams p{};
    const SideGroups sg(f.w2, f.I);
    const int lists = list_offsets(f.T * f.k, f.E).end;
    p.N = f.H;
    p.K = f.I;
    const int cols = std::min(8 * NT, 2 * f.T), typical_cols = std::min(8 * NT, 2 * typical_slots(f));
    const int smem = plan_rows<W4, NT, true>(reinterpret_cast<const void*>(weight_rows_kernel<T, CPG, NT, true>), &p, f.T,
                                             cols, typical_cols, std::min(f.E, f.T * f.k), sg.atom_groups, lists, dev);
    if (smem <= 0) return GEMM_ERR_CUDA;
    p.groups_k = sg.groups_k;
    p.atom_groups = sg.atom_groups;
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
    if (!encode_weights(f.w2, rows, static_cast<int64_t>(f.E) * sg.groups_k, f.H, f.I, p.width, p.width,
                        p.ring.atoms * sg.atom_groups, &w, &sc, &zr))
        return GEMM_ERR_INVALID_VALUE;
    // Clusters of 8 that start while the CTAs of the first product end here and there
    // are placed so that some are left for a second round: 64 tokens, 2 of 64
    // experts of 2048 x 1408 in 4 bits 184 us, 134 if they wait for its end.  The
    // smaller clusters gain 1 to 3 us by starting early.
    return launch_stream(weight_rows_kernel<T, CPG, NT, true>, dev.dev, p.ranges * p.pieces, p.pieces, smem, p.pieces < 8,
                         s, w, sc, zr, p);
}

// How many columns a kernel is built for (8 NT).  An expert with more slots than
// that has its weights read again for the rest; few columns leave registers for
// more tiles per warp or for two CTAs per SM, and shared memory for weights in
// flight.  Matrices of up to kResident bytes are still in L2 when they are read again,
// so for them the narrow kernels win well past the slots that an expert
// usually gets.  Measured, E experts of H x I, T tokens with k choices, us of the whole
// layer for each width of the product named:
//   first product, 16 bits: 64 of 2048 x 1024, T = 64, k = 6: 8 columns 184, 16
//     columns 202; k = 8: 226, 222.  8 of 4096 x 8200, k = 2, T = 16: 265, 275;
//     T = 32: 390, 338; T = 64: 16 columns 550, 32 columns 564.
//   first product, 4 bits: 64 of 2048 x 1408, k = 8, T = 4: 8 columns 56, 16 columns
//     65; T = 8: 107, 85; T = 16: 147, 117; T = 64: 16 columns 206, 32 columns 397.
//     16 of them, T = 64, k = 4: 128, 98, 32 columns 164.
//   second product (two columns per slot), 16 bits: 64 of 2048 x 1024, T = 64, k = 6: 8
//     columns 198, 16 columns 184, 32 columns 218; 8 of them, k = 4: 110, 98, 103, 64
//     columns 126.  8 of 4096 x 8200, k = 2, T = 16: 290, 265; T = 64: 16 columns
//     608, 32 columns 575, 64 columns 551.
//   second product, 4 bits: 64 of 2048 x 1408, k = 8, T = 32: 8 columns 147, 16
//     columns 165, 32 columns 171; T = 64: 246, 240, 206.
constexpr int64_t kResident = 24ll << 20;

bool resident(const Weights& w, int64_t rows, int64_t K) {
    return (w.scales != nullptr ? rows * K / 2 : rows * K * 2) <= kResident;
}

int up_columns(const FfnParams& f) {
    const int usual = typical_slots(f);
    if (f.w13.scales != nullptr) return f.T <= 4 || f.T * f.k <= 16 ? 8 : 16;
    return std::min(f.T, resident(f.w13, 2ll * f.I, f.H) ? (usual <= 6 ? 8 : 16) : usual <= 4 ? 8 : usual <= 16 ? 16 : 32);
}

int down_columns(const FfnParams& f) {
    const int usual = typical_slots(f);
    const bool small = resident(f.w2, f.H, f.I);
    if (f.w2.scales != nullptr) return std::min(2 * f.T, usual <= (small ? 4 : 2) ? 8 : 32);
    return std::min(2 * f.T, small ? (usual <= 2 ? 8 : 16) : 4 * usual);
}

template <class T, int CPG>
gemm_status_t up(const FfnParams& f, void* h, const DeviceView& dev, cudaStream_t s) {
    const int cols = up_columns(f);
    if (cols <= 8) return launch_up<T, CPG, 1>(f, h, dev, s);
    if constexpr (CPG == 0) {
        if (cols > 16) return launch_up<T, CPG, 4>(f, h, dev, s);
    }
    return launch_up<T, CPG, 2>(f, h, dev, s);
}

template <class T, int CPG>
gemm_status_t down(const FfnParams& f, const void* h, const DeviceView& dev, cudaStream_t s) {
    const int cols = down_columns(f);
    if (cols <= 8) return launch_down<T, CPG, 1>(f, h, dev, s);
    if constexpr (CPG == 0) {
        if (cols <= 16) return launch_down<T, CPG, 2>(f, h, dev, s);
        if (cols > 32) return launch_down<T, CPG, 8>(f, h, dev, s);
    }
    return launch_down<T, CPG, 4>(f, h, dev, s);
}

template <class T>
gemm_status_t both(const FfnParams& f, void* h, const DeviceView& dev, cudaStream_t s) {
    gemm_status_t st;
    switch (f.w13.group) {
        case 32: st = up<T, 1>(f, h, dev, s); break;
        case 64: st = up<T, 2>(f, h, dev, s); break;
        case 128: st = up<T, 4>(f, h, dev, s); break;
        default: st = up<T, 0>(f, h, dev, s);
    }
    if (st != GEMM_OK) return st;
    switch (f.w2.group) {
        case 32: return down<T, 1>(f, h, dev, s);
        case 64: return down<T, 2>(f, h, dev, s);
        case 128: return down<T, 4>(f, h, dev, s);
        default: return down<T, 0>(f, h, dev, s);
    }
}

}  // namespace

size_t ffn_scratch_bytes(int64_t T, int64_t I, int k) { return static_cast<size_t>(T) * k * 2 * I * 2; }

gemm_status_t run_ffn(bool bf16, const FfnParams& p, uint8_t* data, const DeviceView& dev, gemm_stream_t stream) {
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return bf16 ? both<__nv_bfloat16>(p, data, dev, s) : both<__half>(p, data, dev, s);
}

}  // namespace gemm_gb300
