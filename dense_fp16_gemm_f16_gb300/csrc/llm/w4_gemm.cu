// w4_gemm.cu -- D = A·Bᵀ with the weights B in 4 bits: few rows of A stream the
// weights (rows.cuh), more go to the tensor cores (w4_tiles.cuh).
#include <algorithm>

#include "llm/rows.cuh"
#include "llm/rows_host.cuh"

namespace gemm_gb300 {
namespace {

template <class T, int CPG, int NT>
gemm_status_t launch(const void* A, const Weights& w, void* D, int64_t row0, int M, int64_t N, int64_t K,
                     const EpiParams& epi, const DeviceView& dev, cudaStream_t s) {
    RowsParams p{};
    const SideGroups sg(w, K);
    p.N = static_cast<int32_t>(N);
    p.K = static_cast<int32_t>(K);
    const int smem = plan_rows<true, NT, false>(reinterpret_cast<const void*>(weight_rows_kernel<T, CPG, NT, false>), &p,
                                                M, M, M, 1, sg.atom_groups, 0, dev);
    if (smem <= 0) return GEMM_ERR_CUDA;
    p.groups_k = sg.groups_k;
    p.atom_groups = sg.atom_groups;
    p.has_zeros = w.zeros != nullptr;
    p.stream_w = stream_weights(true, N, K);
    p.cols = M;
    p.X = static_cast<const T*>(A) + row0 * K;
    p.D = D;
    p.epi = epi;
    p.row0 = row0;
    p.status = dev.status;
    p.timeout_ns = kStreamTimeoutNs;
    CUtensorMap tw, ts, tz;
    if (!encode_weights(w, N, sg.groups_k, N, K, p.width, p.width, p.ring.atoms * sg.atom_groups, &tw, &ts, &tz))
        return GEMM_ERR_INVALID_VALUE;
    return launch_stream(weight_rows_kernel<T, CPG, NT, false>, dev.dev, p.ranges * p.pieces, p.pieces, smem, true, s, tw,
                         ts, tz, p);
}

template <class T, int CPG>
gemm_status_t run(const void* A, const Weights& w, void* D, int64_t M, int64_t N, int64_t K, const EpiParams& epi,
                  const DeviceView& dev, cudaStream_t s) {
    for (int64_t m0 = 0; m0 < M; m0 += 32) {
        const int m = static_cast<int>(std::min<int64_t>(32, M - m0));
        gemm_status_t st;
        if (m <= 8) st = launch<T, CPG, 1>(A, w, D, m0, m, N, K, epi, dev, s);
        else if (m <= 16) st = launch<T, CPG, 2>(A, w, D, m0, m, N, K, epi, dev, s);
        else st = launch<T, CPG, 4>(A, w, D, m0, m, N, K, epi, dev, s);
        if (st != GEMM_OK) return st;
    }
    return GEMM_OK;
}

template <class T>
gemm_status_t by_group(const void* A, const Weights& w, void* D, int64_t M, int64_t N, int64_t K, const EpiParams& epi,
                       const DeviceView& dev, cudaStream_t s) {
    if (w.group == 32) return run<T, 1>(A, w, D, M, N, K, epi, dev, s);
    if (w.group == 64) return run<T, 2>(A, w, D, M, N, K, epi, dev, s);
    return run<T, 4>(A, w, D, M, N, K, epi, dev, s);
}

// Clocks of the streaming kernel for 17 to 64 rows of A, in passes of up to 32,
// fitted to measured times.  Against the tiles of w4_tiles.cuh (us): 8192 x 8192,
// 17 rows 29.5 / 22.5, 48 rows 69 / 24; 2048 x 8192, 17 rows 10.9 / 13.2, 48 rows
// 24.6 / 13.6; 1024 x 4096, 17 rows 7.0 / 7.3, 32 rows 8.3 / 7.3.
double rows_clocks(int64_t M, int64_t N, int64_t K) {
    const double passes = static_cast<double>((M + 31) / 32), weights = static_cast<double>(N) * static_cast<double>(K);
    return passes * 10500.0 + weights * (4.4e-4 * passes + 1.5e-5 * static_cast<double>(M));
}

}  // namespace

gemm_status_t run_w4_gemm(bool bf16, const void* A, const Weights& w, void* D, int64_t M, int64_t N, int64_t K,
                          const EpiParams& epi, const DeviceView& dev, gemm_stream_t stream) {
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (M > 64 || (M > 16 && w4_tiles_clocks(M, N, K, dev) < rows_clocks(M, N, K)))
        return run_w4_tiles(bf16, A, w, D, M, N, K, epi, dev, s);
    return bf16 ? by_group<__nv_bfloat16>(A, w, D, M, N, K, epi, dev, s) : by_group<__half>(A, w, D, M, N, K, epi, dev, s);
}

}  // namespace gemm_gb300
