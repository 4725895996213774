// w4_tiles.cu -- launches of the 4-bit product on tcgen05 (w4_tiles.cuh).
#include <algorithm>

#include "config.h"
#include "llm/rows_host.cuh"
#include "llm/w4_tiles.cuh"

namespace gemm_gb300 {
namespace {

// The split of one product over tiles and clusters, and its time in clocks.
struct TileShape {
    int rows_a, m_tiles, n_tiles, split;
    double clocks;
};

// Clocks of a K block of 64, fitted to measured times: what decoding and handing
// it over takes (with and without remainders), or its MMAs; then a CTA's start and
// end, and an exchange between split parts.
constexpr double kPairClocks = 520.0, kDecodeClocks = 400.0, kMmaClocksPerRow = 2.1;
constexpr double kTileFixedClocks = 8000.0, kTileExchangeClocks = 2000.0;

template <class T, bool PAIRS>
TileShape tile_shape(int64_t M, int64_t N, int64_t K, const DeviceView& dev) {
    TileShape t{};
    t.m_tiles = static_cast<int>((M + 255) / 256);
    t.rows_a = up_to(static_cast<int>((M + t.m_tiles - 1) / t.m_tiles), 16);
    t.n_tiles = static_cast<int>((N + kTileRows - 1) / kTileRows);
    const int64_t atoms = (K + 255) / 256, tiles = static_cast<int64_t>(t.m_tiles) * t.n_tiles;
    const double block = std::max(kMmaClocksPerRow * t.rows_a, PAIRS ? kPairClocks : kDecodeClocks);
    for (int s = 1; s <= 8 && s <= atoms; s *= 2) {
        const int at_once = active_clusters(reinterpret_cast<const void*>(w4_tiles_kernel<T, PAIRS, 1>), dev, kTileThreads,
                                            kMaxDynamicSmem, s);
        if (at_once < 1) continue;
        const double rounds = static_cast<double>((tiles + at_once - 1) / at_once);
        const double c = rounds * (4.0 * static_cast<double>((atoms + s - 1) / s) * block + kTileFixedClocks) +
                         (s > 1 ? kTileExchangeClocks : 0.0);
        if (t.split == 0 || c < t.clocks) {
            t.split = s;
            t.clocks = c;
        }
    }
    return t;
}

template <class T, bool PAIRS, int KB>
gemm_status_t launch(const void* A, const Weights& w, void* D, int64_t M, int64_t N, int64_t K, const EpiParams& epi,
                     const TileShape& t, const DeviceView& dev, cudaStream_t s) {
    const SideGroups sg(w, K);
    TileParams p{};
    p.M = static_cast<int32_t>(M);
    p.N = static_cast<int32_t>(N);
    p.K = static_cast<int32_t>(K);
    p.rows_a = t.rows_a;
    p.m_tiles = t.m_tiles;
    p.split = t.split;
    p.atoms = static_cast<int32_t>((K + 255) / 256);
    p.atom_groups = sg.atom_groups;
    p.group = w.group;
    p.has_zeros = w.zeros != nullptr;
    p.stream_w = stream_weights(true, N, K);
    p.side_bytes = kTileRows * sg.atom_groups * 2;
    p.codes_off = kTileStages * KB * t.rows_a * 128;
    const int code_slot = kTileRows * 128 + 2 * p.side_bytes;
    p.codes = std::min(kTileCodes, (kMaxDynamicSmem - 1024 - p.codes_off) / code_slot) / 2 * 2;
    if (p.codes < 2) return GEMM_ERR_CUDA;
    p.side_off = p.codes_off + p.codes * kTileRows * 128;
    p.end = p.side_off + p.codes * 2 * p.side_bytes;
    // the output's exchange lies over the operands
    const int per = (t.rows_a / 16 + t.split - 1) / t.split * 16;
    if (t.split > 1) p.end = std::max(p.end, t.split * per * 512);
    // more than half an SM's: a CTA takes all of an SM's TMEM, so it shares none
    const int smem = std::max(p.end + 1024, 116 * 1024);
    if (smem > kMaxDynamicSmem) return GEMM_ERR_CUDA;
    p.ab_format = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
    p.D = D;
    p.epi = epi;
    p.status = dev.status;
    p.timeout_ns = kStreamTimeoutNs;
    CUtensorMap tw, ts, tz, ta;
    if (!encode_weights(w, N, sg.groups_k, N, K, kTileRows, kTileRows, sg.atom_groups, &tw, &ts, &tz) ||
        !encode_map(&ta, A, 2, K, M, 64, static_cast<uint32_t>(t.rows_a), true))
        return GEMM_ERR_INVALID_VALUE;
    const int64_t ctas = static_cast<int64_t>(t.m_tiles) * t.n_tiles * t.split;
    if (ctas > INT32_MAX) return GEMM_ERR_INVALID_VALUE;
    return launch_clusters(w4_tiles_kernel<T, PAIRS, KB>, dev.dev, static_cast<int>(ctas), kTileThreads, t.split, smem,
                           true, s, tw, ts, tz, ta, p);
}

template <class T>
gemm_status_t run(const void* A, const Weights& w, void* D, int64_t M, int64_t N, int64_t K, const EpiParams& epi,
                  const DeviceView& dev, cudaStream_t s) {
    const TileShape t = M <= 64 ? tile_shape<T, true>(M, N, K, dev) : tile_shape<T, false>(M, N, K, dev);
    if (t.split == 0) return GEMM_ERR_CUDA;
    if (M <= 64) return launch<T, true, 1>(A, w, D, M, N, K, epi, t, dev, s);
    return t.rows_a <= 128 ? launch<T, false, 2>(A, w, D, M, N, K, epi, t, dev, s)
                           : launch<T, false, 1>(A, w, D, M, N, K, epi, t, dev, s);
}

}  // namespace

double w4_tiles_clocks(int64_t M, int64_t N, int64_t K, const DeviceView& dev) {
    return M <= 64 ? tile_shape<__half, true>(M, N, K, dev).clocks : tile_shape<__half, false>(M, N, K, dev).clocks;
}

gemm_status_t run_w4_tiles(bool bf16, const void* A, const Weights& w, void* D, int64_t M, int64_t N, int64_t K,
                           const EpiParams& epi, const DeviceView& dev, cudaStream_t s) {
    return bf16 ? run<__nv_bfloat16>(A, w, D, M, N, K, epi, dev, s) : run<__half>(A, w, D, M, N, K, epi, dev, s);
}

}  // namespace gemm_gb300
