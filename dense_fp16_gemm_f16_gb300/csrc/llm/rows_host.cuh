// rows_host.cuh -- host side of the weight-streaming kernels: tensor maps,
// the split of rows over clusters, launches.
#pragma once

#include <algorithm>
#include <cmath>
#include <functional>
#include <map>
#include <mutex>

#include "llm/rows.cuh"

namespace gemm_gb300 {

constexpr uint64_t kStreamTimeoutNs = 4000000000ull;
constexpr int kMaxDynamicSmem = 226 * 1024;   // 227 KB less the barriers
// dynamic shared memory of a launch, so that kCtasPerSm CTAs fit (1 KB of an SM's goes to each)
template <bool W4, int NT, bool MOE>
constexpr int kSmemBudget = kCtasPerSm<W4, NT, MOE> == 2 ? kSmemPerSm / 2 - 2048 : 210 * 1024;

struct SideGroups {
    int groups_k = 0, atom_groups = 0;
    SideGroups(const Weights& w, int64_t K) {
        if (w.scales == nullptr) return;
        groups_k = static_cast<int>(K / w.group);
        atom_groups = 256 / w.group;
    }
};

// Parts of up to `part` that n falls into.  n may be all but 2^31, so nothing is added to it.
inline int count_of(int n, int part) { return n / part + (n % part != 0); }

// Weights that cannot stay in L2 (129 MB) from one call to the next anyway
// are read with evict-first, so they do not push out what can.
inline int32_t stream_weights(bool w4, int64_t rows, int64_t K) {
    return (w4 ? rows * K / 2 : rows * K * 2) > (48ll << 20);
}

// Tensor maps of a stack: rows x K codes or 16-bit numbers in boxes of
// box_rows x 128 bytes; scales and zero points [side_rows][N] in boxes of
// side_groups x side_box.
inline bool encode_weights(const Weights& w, int64_t rows, int64_t side_rows, int64_t N, int64_t K, int box_rows,
                           int side_box, int side_groups, CUtensorMap* tw, CUtensorMap* ts, CUtensorMap* tz) {
    if (w.scales == nullptr) {
        if (!encode_map(tw, w.data, 2, K, rows, 64, static_cast<uint32_t>(box_rows), true)) return false;
        *ts = *tz = *tw;   // not used
        return true;
    }
    if (!encode_map(tw, w.data, 1, K / 2, rows, 128, static_cast<uint32_t>(box_rows), true)) return false;
    const uint32_t box_n = static_cast<uint32_t>(side_box), box_groups = static_cast<uint32_t>(side_groups);
    if (!encode_map(ts, w.scales, 2, N, side_rows, box_n, box_groups, false)) return false;
    if (w.zeros == nullptr) {
        *tz = *ts;
        return true;
    }
    return encode_map(tz, w.zeros, 2, N, side_rows, box_n, box_groups, false);
}

// The same rows in boxes of another height.
inline bool encode_weights_box(const Weights& w, int64_t rows, int64_t K, int box_rows, CUtensorMap* t) {
    return w.scales == nullptr ? encode_map(t, w.data, 2, K, rows, 64, static_cast<uint32_t>(box_rows), true)
                               : encode_map(t, w.data, 1, K / 2, rows, 128, static_cast<uint32_t>(box_rows), true);
}

// What the facts about a kernel's launches are known by.  A type of this
// namespace also keeps the maps' symbols out of the library's exports.
struct LaunchKey {
    const void* kernel;
    int dev, smem, cluster;
    bool operator<(const LaunchKey& o) const {
        if (kernel != o.kernel) return std::less<const void*>()(kernel, o.kernel);
        if (dev != o.dev) return dev < o.dev;
        if (smem != o.smem) return smem < o.smem;
        return cluster < o.cluster;
    }
};

// Lifts a kernel's shared-memory limit, once per kernel and device.
inline cudaError_t allow_smem(const void* kernel, int dev) {
    static std::mutex mu;
    static std::map<LaunchKey, bool> done;
    std::lock_guard<std::mutex> lock(mu);
    bool& ready = done[LaunchKey{kernel, dev, 0, 0}];
    if (ready) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxDynamicSmem);
    ready = e == cudaSuccess;
    return e;
}

// Clusters of `cluster` CTAs that run at one time (0: none), looked up once.
inline int active_clusters(const void* kernel, const DeviceView& dev, int threads, int smem, int cluster) {
    static std::mutex mu;
    static std::map<LaunchKey, int> known;
    std::lock_guard<std::mutex> lock(mu);
    const LaunchKey key{kernel, dev.dev, smem, cluster};
    const auto it = known.find(key);
    if (it != known.end()) return it->second;
    int n = 0;
    if (allow_smem(kernel, dev.dev) == cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(cluster), 1, 1);
        cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
        cfg.dynamicSmemBytes = static_cast<size_t>(smem);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
            cudaGetLastError();
            n = 0;
        }
    }
    known[key] = n;
    return n;
}

// Programmatic stream serialisation (where `early`), and clusters of `cluster` CTAs.
template <class Kernel, class... Args>
gemm_status_t launch_clusters(Kernel kernel, int dev, int grid, int threads, int cluster, int smem, bool early,
                              cudaStream_t s, const Args&... args) {
    if (allow_smem(reinterpret_cast<const void*>(kernel), dev) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_CUDA;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = early ? 1 : 0;
    cfg.numAttrs = 1;
    if (cluster > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    cfg.attrs = attr;
    if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_LAUNCH;
    }
    return GEMM_OK;
}

template <class Kernel, class Params>
gemm_status_t launch_stream(Kernel kernel, int dev, int grid, int cluster, int smem, bool early, cudaStream_t s,
                            const CUtensorMap& w, const CUtensorMap& sc, const CUtensorMap& zr, const Params& p) {
    return launch_clusters(kernel, dev, grid, kStreamThreads, cluster, smem, early, s, w, sc, zr, p);
}

// What plan_rows decides from, and the decision.  A thread keeps its last few: a
// model's calls repeat a handful of shapes, and deciding takes microseconds.
struct RowsPlan {
    const void* kernel = nullptr;
    int dev = 0, N = 0, K = 0, tokens = 0, cols = 0, typical_cols = 0, segments = 0, atom_groups = 0, lists = 0;
    RowsParams p;
    int smem = 0;
    bool same(const RowsPlan& o) const {
        return kernel == o.kernel && dev == o.dev && N == o.N && K == o.K && tokens == o.tokens && cols == o.cols &&
               typical_cols == o.typical_cols && segments == o.segments && atom_groups == o.atom_groups && lists == o.lists;
    }
};

template <bool W4, int NT, bool MOE>
int plan_rows_anew(const void* kernel, RowsParams* p, int tokens, int cols, int typical_cols, int segments,
                   int atom_groups, int lists, const DeviceView& dev);

template <bool W4, int NT, bool MOE>
int plan_rows(const void* kernel, RowsParams* p, int tokens, int cols, int typical_cols, int segments, int atom_groups,
              int lists, const DeviceView& dev) {
    thread_local RowsPlan known[8];
    thread_local int next = 0;
    RowsPlan want;
    want.kernel = kernel;
    want.dev = dev.dev;
    want.N = p->N;
    want.K = p->K;
    want.tokens = tokens;
    want.cols = cols;
    want.typical_cols = typical_cols;
    want.segments = segments;
    want.atom_groups = atom_groups;
    want.lists = lists;
    for (const RowsPlan& k : known)
        if (k.same(want)) {
            *p = k.p;
            return k.smem;
        }
    want.smem = plan_rows_anew<W4, NT, MOE>(kernel, p, tokens, cols, typical_cols, segments, atom_groups, lists, dev);
    want.p = *p;
    if (want.smem > 0) {
        known[next] = want;
        next = (next + 1) % 8;
    }
    return want.smem;
}

// Fills the split and the shared-memory layout of `p` (N and K set): `tokens`
// outputs per row, at most `cols` columns per stage, mostly typical_cols, about `segments`
// matrices.  Returns the dynamic shared memory
// of the launch, 0 when nothing fits.
template <bool W4, int NT, bool MOE>
int plan_rows_anew(const void* kernel, RowsParams* p, int tokens, int cols, int typical_cols, int segments,
                   int atom_groups, int lists, const DeviceView& dev) {
    constexpr int budget = kSmemBudget<W4, NT, MOE>;
    constexpr int MT = kTilesPerWarp<W4, NT, MOE>;
    const int table_cols = MOE ? tokens : 8 * NT;
    const int k_atoms = count_of(p->K, kAtomElems<W4>);
    const int nt = std::min(NT, (typical_cols + 7) / 8);
    int best = 0;
    bool best_fits = false;
    double best_t = 0.0;
    RowsParams got = *p;
    for (int P = 1; P <= 8; P *= 2) {
        const int clusters = active_clusters(kernel, dev, kStreamThreads, budget, P);
        if (clusters < 1) continue;
        // as few rounds of clusters as keep a range within a TMA box (256 rows)
        // and the consumers' registers
        const int most = std::min(256, kConsumers * MT * 16);
        const int rounds = count_of(p->N, clusters * most);
        const int width = up_to(count_of(p->N, clusters * rounds), 8);
        const int tiles = (width + 15) / 16;
        for (int mw = 1; mw <= kConsumers; mw *= 2) {
            if (mw * MT < tiles) continue;
            const int kw = kConsumers / mw;
            for (int atoms = 1; atoms <= kMaxAtoms; atoms *= 2) {
                if (atoms > 1 && atoms * width * 128 > 16384) break;
                RowsParams c = *p;
                c.width = width;
                c.ranges = count_of(p->N, width);
                c.pieces = P;
                c.mw = mw;
                c.k_stages = (k_atoms + atoms - 1) / atoms;
                c.table_pitch = up_to(tiles * 16, 32) + 8;
                const int tables = kw * table_cols * c.table_pitch * 4;
                const int recv = P > 1 ? up_to((tokens * width + P - 1) / P * P * 4, 128) : 0;
                const int fixed = lists + tables + recv + 1024;
                c.ring = ring_layout(W4, atoms, width, width, atom_groups, cols, budget - fixed, kw);
                // more than the budget (fewer CTAs per SM than planned) only where nothing fits it
                const bool fits = c.ring.end + fixed <= budget;
                if (c.ring.end + fixed > kMaxDynamicSmem || (best != 0 && best_fits && !fits)) continue;
                // Clocks per atom.  Arithmetic: a warp's instructions for its
                // columns and tiles, about one per clock and SM.  Copies: the
                // CTA's share of HBM for the weights and of L2 for the columns,
                // slowed when less is in flight than their latency needs.
                // Latency: what a group takes for a stage however small, with
                // kw groups side by side; warps that share a stage wait for one
                // another.
                const int per_warp = (tiles + mw - 1) / mw;
                const double work = W4 ? 8.0 * (10.0 * nt + per_warp * (22.0 + 6.0 * nt))
                                       : 4.0 * (6.0 * nt + per_warp * (5.0 + 3.0 * nt));
                const double arith = kCtasPerSm<W4, NT, MOE> * (work + 200.0 / atoms) * mw * (0.9 + 0.1 * mw) / 2.0;
                const double flight = std::min(1.0, c.ring.slots * atoms * width * 128 / (65536.0 / kCtasPerSm<W4, NT, MOE>));
                const double copies =
                    kCtasPerSm<W4, NT, MOE> * (width * 128 / 23.5 + typical_cols * (W4 ? 512 : 128) / 50.0) / flight;
                const double latency = (1500.0 + 1500.0 * (mw - 1)) / (kw * atoms) + 2.0 * work / kw;
                const double n_atoms = std::ceil(std::ceil(static_cast<double>(segments) * c.k_stages / P) / kw) * kw * atoms;
                const double t = rounds * n_atoms * std::max(std::max(arith, copies), latency) + (P > 1 ? 800.0 : 0.0) +
                                 tables / 100.0;
                if (best == 0 || t < best_t || (fits && !best_fits)) {
                    best_t = t;
                    best_fits = fits;
                    c.list_off = c.ring.end;
                    c.table_off = c.list_off + lists;
                    c.recv_off = c.table_off + tables;
                    best = c.recv_off + recv + 1024;
                    got = c;
                }
            }
        }
    }
    if (best) *p = got;
    return best;
}

}  // namespace gemm_gb300
