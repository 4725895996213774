// w4_tiles.cu -- launches of the 4-bit product on tcgen05 (w4_tiles.cuh).
#include <algorithm>

#include "config.h"
#include "llm/rows_host.cuh"
#include "llm/w4_tiles.cuh"

namespace gemm_gb300 {
namespace {

// The split of one product over tiles and clusters, and its time in clocks.
struct TileShape {
    int rows_a, rows_b, m_tiles, n_tiles, split;
    double clocks;
};

// A K block of 64 takes the MMA 2 clocks per row of A (128 weight rows), and
// decoding it about kDecodeClocks; a CTA's start and end, and an exchange
// between split parts, are added.
constexpr double kDecodeClocks = 230.0, kTileFixedClocks = 7000.0, kTileExchangeClocks = 2500.0;

TileShape tile_shape(int64_t M, int64_t N, int64_t K, int sms) {
    TileShape t{};
    t.rows_b = M <= 64 ? 64 : 128;
    t.m_tiles = static_cast<int>((M + 255) / 256);
    t.rows_a = up_to(static_cast<int>((M + t.m_tiles - 1) / t.m_tiles), 16);
    t.n_tiles = static_cast<int>((N + t.rows_b - 1) / t.rows_b);
    const int64_t atoms = (K + 255) / 256, tiles = static_cast<int64_t>(t.m_tiles) * t.n_tiles;
    const double block = std::max(2.0 * t.rows_a, kDecodeClocks);
    for (int s = 1; s <= 8 && s <= atoms; s *= 2) {
        const double rounds = static_cast<double>((tiles * s + sms - 1) / sms);
        const double c = rounds * (4.0 * static_cast<double>((atoms + s - 1) / s) * block + kTileFixedClocks) + (s > 1 ? kTileExchangeClocks : 0.0);
        if (t.split == 0 || c < t.clocks) {
            t.split = s;
            t.clocks = c;
        }
    }
    return t;
}

template <class T, bool PAIRS>
gemm_status_t launch(const void* A, const Weights& w, void* D, int64_t M, int64_t N, int64_t K, const EpiParams& epi,
                     const TileShape& t, const DeviceView& dev, cudaStream_t s) {
    const SideGroups sg(w, K);
    TileParams p{};
    p.M = static_cast<int32_t>(M);
    p.N = static_cast<int32_t>(N);
    p.K = static_cast<int32_t>(K);
    p.rows_a = t.rows_a;
    p.rows_b = t.rows_b;
    p.m_tiles = t.m_tiles;
    p.split = t.split;
    p.atoms = static_cast<int32_t>((K + 255) / 256);
    p.atom_groups = sg.atom_groups;
    p.group = w.group;
    p.has_zeros = w.zeros != nullptr;
    p.stream_w = stream_weights(true, N, K);
    p.side_bytes = up_to(t.rows_b * sg.atom_groups * 2, 128);
    p.stages = t.rows_a <= 128 ? kTileStages : kTileStages / 2;   // 32 KB of A each at 256 rows
    p.codes_off = p.stages * t.rows_a * 128;
    const int code_slot = t.rows_b * 128 + 2 * p.side_bytes;
    p.codes = std::min(kTileCodes, (kMaxDynamicSmem - 1024 - p.codes_off) / code_slot);
    p.side_off = p.codes_off + p.codes * t.rows_b * 128;
    p.end = p.side_off + p.codes * 2 * p.side_bytes;
    // the output's exchange lies over the operands
    const int per = (t.rows_a / 16 + t.split - 1) / t.split * 16;
    if (PAIRS || t.split > 1) p.end = std::max(p.end, t.split * per * 512);
    // more than half an SM's: a CTA takes all of an SM's TMEM, so it shares none
    const int smem = std::max(p.end + 1024, 116 * 1024);
    if (smem > kMaxDynamicSmem) return GEMM_ERR_CUDA;
    p.ab_format = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
    p.D = D;
    p.epi = epi;
    p.status = dev.status;
    p.timeout_ns = kStreamTimeoutNs;
    CUtensorMap tw, ts, tz, ta;
    if (!encode_weights(w, N, sg.groups_k, N, K, t.rows_b, t.rows_b, sg.atom_groups, &tw, &ts, &tz) ||
        !encode_map(&ta, A, 2, K, M, 64, static_cast<uint32_t>(t.rows_a), true))
        return GEMM_ERR_INVALID_VALUE;
    const int64_t ctas = static_cast<int64_t>(t.m_tiles) * t.n_tiles * t.split;
    if (ctas > INT32_MAX) return GEMM_ERR_INVALID_VALUE;
    return launch_clusters(w4_tiles_kernel<T, PAIRS>, dev.dev, static_cast<int>(ctas), kTileThreads, t.split, smem, s, tw, ts, tz, ta, p);
}

template <class T>
gemm_status_t run(const void* A, const Weights& w, void* D, int64_t M, int64_t N, int64_t K, const EpiParams& epi,
                  const DeviceView& dev, cudaStream_t s) {
    const TileShape t = tile_shape(M, N, K, dev.sms);
    return M <= 64 ? launch<T, true>(A, w, D, M, N, K, epi, t, dev, s) : launch<T, false>(A, w, D, M, N, K, epi, t, dev, s);
}

}  // namespace

double w4_tiles_clocks(int64_t M, int64_t N, int64_t K, int sms) { return tile_shape(M, N, K, sms).clocks; }

gemm_status_t run_w4_tiles(bool bf16, const void* A, const Weights& w, void* D, int64_t M, int64_t N, int64_t K,
                           const EpiParams& epi, const DeviceView& dev, cudaStream_t s) {
    return bf16 ? run<__nv_bfloat16>(A, w, D, M, N, K, epi, dev, s) : run<__half>(A, w, D, M, N, K, epi, dev, s);
}

}  // namespace gemm_gb300
