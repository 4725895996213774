// w4_codes.cu -- 16-bit weights to 4-bit codes with group scales, and back.
//
// A tile is 16 rows by 512 k; a warp takes two of the rows, each thread 8 consecutive
// k of a row at a time (16 bytes of W, 4 bytes of codes), four such pieces per tile,
// the next tile's loaded before this one's are worked on.  A CTA walks a run of
// tiles.  The 4, 8 or 16 threads of a group find its extremes by shuffles, two
// numbers to a register, and share out the divisions: lane i (mod 4) does piece i's.
// Scales lie [K/group][N]: they pass through shared memory so that 16 rows' worth
// is written (or read) side by side.
//
// The least that either direction moves is 2.5 bytes per weight.  Unpacking runs at
// 85 % of that; packing is bound by instructions (190 per 256 weights, 2.9 of 4
// issued per clock), so w / s is not divided out: with t = w * (1 / s), off by less
// than 2^-20, rint(t) is rint(w / s) unless w / s is exactly half-way.  (w and s have
// at most 11 significant bits, so a quotient that is not half-way is at least 2^-14
// away from it.)  Half-way means |w - s r| = s / 2, which fma computes exactly, and r
// then becomes the even neighbour; only threads with a quotient within 0.0001 of
// half-way look.
// Measured, 8 matrices of 11000 x 4096, bf16, zero points, groups of 128: packing
// 306 us (3.0 TB/s), unpacking 156 us (5.9 TB/s); one of 1024 x 2048, both in 6.6 us.
#include <algorithm>
#include <type_traits>

#include "llm/llm.h"
#include "llm/w4.cuh"

namespace gemm_gb300 {
namespace {

constexpr int kCodesThreads = 256;
constexpr int kPackPerSm = 3, kUnpackPerSm = 4;   // CTAs, each with the next tile's loads in flight; the quantiser's registers spill with 4
constexpr int kCodesRows = 16, kCodesK = 512;
constexpr int kCodesGroups = kCodesK / 32;   // most groups of a row in a tile: one scale per thread
constexpr float kRound = 12582912.0f;        // 1.5 * 2^23: adding it rounds to whole numbers, ties to even
constexpr float kWhole = 8388608.0f;         // 2^23

// Rows are numbered through the whole stack: row r is row r % N of matrix r / N,
// and its scales are at [(r / N) * (K / group) + k / group][r % N].
//
// A CTA walks a run of tiles, along k and then to the next 16 rows, by additions
// alone: a 64-bit division costs about 100 instructions, as much as eight weights.
// A thread's pieces of a tile are 2 * half + j: row warp + 8 half, k 256 j + 8 lane.
struct Walk {
    int64_t row0, k0;        // the tile
    int64_t off[2];          // this thread's first weight in it, of each half
    int64_t N, K, k_end, rows;
    int row_end, k_left;     // what this thread has: halves below row_end, pieces below k_left
    __device__ __forceinline__ Walk(int64_t tile, int64_t k_tiles, int64_t rows_, int64_t N_, int64_t K_) {
        const int64_t strip = tile / k_tiles;
        row0 = strip * kCodesRows;
        k0 = (tile - strip * k_tiles) * kCodesK;
        rows = rows_, N = N_, K = K_, k_end = k_tiles * kCodesK;
        off[0] = (row0 + (threadIdx.x >> 5)) * K + k0 + (threadIdx.x & 31) * 8;
        off[1] = off[0] + 8 * K;
        ends();
    }
    __device__ __forceinline__ void ends() {
        row_end = static_cast<int>(min(rows - row0, static_cast<int64_t>(kCodesRows))) - static_cast<int>(threadIdx.x >> 5);
        k_left = static_cast<int>(min(K - k0, static_cast<int64_t>(kCodesK))) - static_cast<int>(threadIdx.x & 31) * 8;
    }
    __device__ __forceinline__ void next() {
        k0 += kCodesK;
        int64_t step = kCodesK;
        if (k0 == k_end) {
            k0 = 0;
            row0 += kCodesRows;
            step += kCodesRows * K - k_end;
        }
        off[0] += step;
        off[1] += step;
        ends();
    }
    __device__ __forceinline__ bool has(int i) const { return 8 * (i >> 1) < row_end && 256 * (i & 1) < k_left; }
    template <class P>
    __device__ __forceinline__ P* wide(P* base, int i) const { return base + off[i >> 1] + 256 * (i & 1); }
    template <class P>
    __device__ __forceinline__ P* word(P* codes, int i) const { return codes + (off[i >> 1] >> 1) + 128 * (i & 1); }
};

// Where the scale lies that this thread moves: row threadIdx % 16 of the tile,
// group threadIdx / 16.  The row's matrix is followed along with the walk.
struct Side {
    int64_t row0, n, base;   // base: the row's first scale
    __device__ __forceinline__ Side(const Walk& t, int shift) {
        const int64_t r = t.row0 + threadIdx.x % kCodesRows, b = r / t.N;
        row0 = t.row0;
        n = r - b * t.N;
        base = b * (t.K >> shift) * t.N + n;
    }
    __device__ __forceinline__ int64_t at(const Walk& t, int shift) {
        const int grp = threadIdx.x / kCodesRows;
        if (grp >= (kCodesK >> shift)) return -1;   // whole warps leave here but for the smallest groups
        if (t.row0 != row0) {
            row0 = t.row0;
            n += kCodesRows;
            base += kCodesRows;
            for (; n >= t.N; n -= t.N) base += ((t.K >> shift) - 1) * t.N;
        }
        const int64_t g = (t.k0 >> shift) + grp;
        if (row0 + threadIdx.x % kCodesRows >= t.rows || g >= (t.K >> shift)) return -1;
        return base + g * t.N;
    }
};

// The smallest normal number of T with room to spare: from here on a scale is
// within 2^-8 of the quotient it was rounded from.
template <class T>
constexpr float kSmall = std::is_same<T, __half>::value ? 1.220703125e-4f : 2.4e-38f;

template <class T>
using Pair = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;

template <class T>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    const Pair<T> m = __hmax2(*reinterpret_cast<const Pair<T>*>(&a), *reinterpret_cast<const Pair<T>*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
}

// max(0, -w) in the low half and max(0, w) in the high half over 8 numbers; with
// one zero point for all, max |w| in both.
template <class T, bool ASYM>
__device__ __forceinline__ uint32_t extremes(const uint4& v) {
    constexpr uint32_t kAbs = 0x7FFF7FFFu, kSign = 0x80008000u;
    if constexpr (ASYM) {
        const uint32_t up = max2<T>(max2<T>(v.x, v.y), max2<T>(v.z, v.w));
        const uint32_t down = max2<T>(max2<T>(v.x ^ kSign, v.y ^ kSign), max2<T>(v.z ^ kSign, v.w ^ kSign));
        return max2<T>(0u, max2<T>(__byte_perm(down, up, 0x5410), __byte_perm(down, up, 0x7632)));
    } else {
        const uint32_t m = max2<T>(max2<T>(v.x & kAbs, v.y & kAbs), max2<T>(v.z & kAbs, v.w & kAbs));
        return max2<T>(m, __byte_perm(m, m, 0x1032));
    }
}

// This thread's pieces of a tile (Walk's halves and ends) whose scale has no finite
// reciprocal: bf16 scales of at most 2^-128.  They divide.  Apart from the kernel, whose
// registers are full (as a branch of it, it cost every tile 2 %).
template <bool ASYM>
__device__ __noinline__ void quantize_smallest(const __nv_bfloat16* W, uint8_t* codes, int64_t off0, int64_t off1,
                                               int row_end, int k_left, int shift,
                                               const __nv_bfloat16 (*scales)[kCodesRows],
                                               const __nv_bfloat16 (*zeros)[kCodesRows]) {
    using B = Elem<__nv_bfloat16>;
    for (int i = 0; i < 4; ++i) {
        if (8 * (i >> 1) >= row_end || 256 * (i & 1) >= k_left) continue;
        const int row = (threadIdx.x >> 5) + 8 * (i >> 1), grp = (256 * (i & 1) + (threadIdx.x & 31) * 8) >> shift;
        const float s = B::to_float(scales[grp][row]), z = ASYM ? B::to_float(zeros[grp][row]) : 8.0f;
        if (s == 0.0f || !isinf(__frcp_rn(s))) continue;
        const int64_t at = (i >> 1 ? off1 : off0) + 256 * (i & 1);
        float w[8];
        unpack8<__nv_bfloat16>(*reinterpret_cast<const uint4*>(W + at), w);
        uint32_t word = 0u;
        for (int j = 0; j < 8; ++j)
            word |= static_cast<uint32_t>(fminf(fmaxf(rintf(__fdiv_rn(w[j], s)) + z, 0.0f), 15.0f)) << (4 * j);
        *reinterpret_cast<uint32_t*>(codes + at / 2) = word;
    }
}

template <class T, bool ASYM>
__global__ void __launch_bounds__(kCodesThreads, kPackPerSm)
w4_quantize_kernel(const T* __restrict__ W, int64_t rows, int64_t N, int64_t K, int64_t k_tiles, int64_t tiles, int shift,
                   uint8_t* __restrict__ codes, T* __restrict__ scales, T* __restrict__ zeros) {
    __shared__ T s_scale[2][kCodesGroups][kCodesRows], s_zero[2][kCodesGroups][kCodesRows];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int width = 1 << (shift - 3);   // threads per group: 4, 8 or 16
    const int64_t first = tiles * blockIdx.x / gridDim.x, last = tiles * (blockIdx.x + 1) / gridDim.x;
    Walk tile(first, k_tiles, rows, N, K), ahead = tile;
    Side side(tile, shift);
    uint4 raw[4], coming[4];
    // zeros outside; K is a multiple of the group, so a group's threads are all in or all out
    auto load = [&] {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            coming[i] = ahead.has(i) ? __ldcs(reinterpret_cast<const uint4*>(ahead.wide(W, i))) : make_uint4(0u, 0u, 0u, 0u);
    };
    load();
    for (int64_t t = first; t < last; ++t, tile.next()) {
        const int buf = static_cast<int>(t - first) & 1;
        uint32_t ext[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            raw[i] = coming[i];
            ext[i] = extremes<T, ASYM>(raw[i]);
        }
        if (t + 1 < last) {   // in flight while this tile is worked on
            ahead.next();
            load();
        }
        for (int d = 1; d < width; d *= 2) {
#pragma unroll
            for (int i = 0; i < 4; ++i) ext[i] = max2<T>(ext[i], __shfl_xor_sync(0xffffffffu, ext[i], d));
        }
        // scale and zero point of piece i in lane i (mod 4) of its group: one set of
        // divisions for the four pieces
        const int mine = lane & 3;
        const uint32_t e = mine == 0 ? ext[0] : mine == 1 ? ext[1] : mine == 2 ? ext[2] : ext[3];
        const float down = Elem<T>::lo(e), up = Elem<T>::hi(e);
        const T st = Elem<T>::from_float(ASYM ? __fdiv_rn(up + down, 15.0f) : __fdiv_rn(up, 7.0f));
        const float s_mine = Elem<T>::to_float(st);
        float z_mine = 8.0f;
        if constexpr (ASYM) z_mine = s_mine == 0.0f ? 0.0f : fminf(fmaxf(rintf(__fdiv_rn(down, s_mine)), 0.0f), 15.0f);
        const float inv_mine = s_mine == 0.0f ? 0.0f : __frcp_rn(s_mine);
        // r + z leaves 0 to 15 only where s is subnormal and far from the quotient it
        // was rounded from, and by one step above 15 with zero points: those groups
        // get their scale's sign set and are clamped below
        bool edge = s_mine < kSmall<T>;
        if constexpr (ASYM) edge = edge || __fmaf_rn(up, inv_mine, z_mine) > 15.4999f;
        const float s_sent = edge ? -s_mine : s_mine;
        if ((lane & (width - 1)) < 4) {
            const int row = warp + 8 * (mine >> 1), grp = (256 * (mine & 1) + 8 * (lane & ~(width - 1))) >> shift;
            s_scale[buf][grp][row] = st;
            if constexpr (ASYM) s_zero[buf][grp][row] = Elem<T>::from_float(z_mine);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int src = (lane & ~(width - 1)) + i;
            const float s_sign = __shfl_sync(0xffffffffu, s_sent, src), inv = __shfl_sync(0xffffffffu, inv_mine, src);
            const float z = ASYM ? __shfl_sync(0xffffffffu, z_mine, src) : 8.0f;
            float w[8], r[8];
            unpack8<T>(raw[i], w);
            float far = 0.0f;   // the farthest that a quotient is from a whole number
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                r[j] = __fadd_rn(__fmaf_rn(w[j], inv, kRound), -kRound);
                far = fmaxf(far, fabsf(__fmaf_rn(w[j], inv, -r[j])));
            }
            if (far > 0.4999f || __float_as_int(s_sign) < 0) {   // perhaps half-way, or past an end
                const float s = fabsf(s_sign), half = 0.5f * s;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float d = __fmaf_rn(-s, r[j], w[j]);
                    if (s != 0.0f && fabsf(d) == half && (static_cast<int>(r[j]) & 1)) r[j] += d > 0.0f ? 1.0f : -1.0f;
                    r[j] = fminf(fmaxf(r[j], -z), 15.0f - z);
                }
            }
            // four codes as one whole number below 2^16, exact in fp32 as are the sums before it
            const float whole = __fmaf_rn(z, 4369.0f, kWhole);
            const float a = r[0] + 16.0f * (r[1] + 16.0f * (r[2] + 16.0f * r[3])) + whole;
            const float b = r[4] + 16.0f * (r[5] + 16.0f * (r[6] + 16.0f * r[7])) + whole;
            if (tile.has(i))
                __stcs(reinterpret_cast<uint32_t*>(tile.word(codes, i)),
                       __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x5410));
        }
        // two buffers: the next tile's writes go to the other one
        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
            if (__syncthreads_or(isinf(inv_mine)))
                quantize_smallest<ASYM>(W, codes, tile.off[0], tile.off[1], tile.row_end, tile.k_left, shift, s_scale[buf],
                                        s_zero[buf]);
        } else {
            __syncthreads();
        }
        const int64_t at = side.at(tile, shift);
        if (at >= 0) {
            scales[at] = s_scale[buf][threadIdx.x / kCodesRows][threadIdx.x % kCodesRows];
            if constexpr (ASYM) zeros[at] = s_zero[buf][threadIdx.x / kCodesRows][threadIdx.x % kCodesRows];
        }
    }
}

template <class T>
__global__ void __launch_bounds__(kCodesThreads, kUnpackPerSm)
w4_dequantize_kernel(const uint8_t* __restrict__ codes, const T* __restrict__ scales, const T* __restrict__ zeros,
                     int64_t rows, int64_t N, int64_t K, int64_t k_tiles, int64_t tiles, int shift, T* __restrict__ W) {
    __shared__ float2 s_side[2][kCodesGroups][kCodesRows];   // scale, zero point
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t first = tiles * blockIdx.x / gridDim.x, last = tiles * (blockIdx.x + 1) / gridDim.x;
    Walk tile(first, k_tiles, rows, N, K), ahead = tile;
    Side side(tile, shift);
    uint32_t c[4], coming[4];
    T sc = Elem<T>::from_float(0.0f), ze = Elem<T>::from_float(8.0f);
    auto load = [&] {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            coming[i] = ahead.has(i) ? __ldcs(reinterpret_cast<const uint32_t*>(ahead.word(codes, i))) : 0u;
        const int64_t at = side.at(ahead, shift);
        if (at >= 0) {
            sc = scales[at];
            if (zeros != nullptr) ze = zeros[at];
        }
    };
    load();
    for (int64_t t = first; t < last; ++t, tile.next()) {
        const int buf = static_cast<int>(t - first) & 1;
        s_side[buf][threadIdx.x / kCodesRows][threadIdx.x % kCodesRows] = make_float2(Elem<T>::to_float(sc), Elem<T>::to_float(ze));
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = coming[i];
        if (t + 1 < last) {   // in flight while this tile is worked on
            ahead.next();
            load();
        }
        __syncthreads();   // two buffers: the next tile's scales go to the other one
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (!tile.has(i)) continue;
            const float2 sz = s_side[buf][(256 * (i & 1) + lane * 8) >> shift][warp + 8 * (i >> 1)];
            float w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                // the code stays where it is in the word, below the exponent of 2^23:
                // 2^23 + 16^m q, brought down to q by one fma
                const int m = j & 3;
                const float down = 1.0f / static_cast<float>(1 << (4 * m));
                const float u = __uint_as_float(((j < 4 ? c[i] : c[i] >> 16) & (15u << (4 * m))) | 0x4B000000u);
                w[j] = sz.x * (__fmaf_rn(u, down, -kWhole * down) - sz.y);
            }
            __stcs(reinterpret_cast<uint4*>(tile.wide(W, i)), pack8<T>(w));
        }
    }
}

int64_t k_tiles_of(int64_t K) { return (K + kCodesK - 1) / kCodesK; }
int64_t tiles_of(int64_t rows, int64_t K) { return (rows + kCodesRows - 1) / kCodesRows * k_tiles_of(K); }
int shift_of(int group) { return group == 32 ? 5 : group == 64 ? 6 : 7; }
unsigned grid_of(int64_t tiles, int ctas) { return static_cast<unsigned>(std::min<int64_t>(tiles, ctas)); }

template <class T>
void quantize(const void* W, int64_t rows, int64_t N, int64_t K, int group, void* codes, void* scales, void* zeros, int sms,
              cudaStream_t s) {
    const int64_t tiles = tiles_of(rows, K);
    const unsigned grid = grid_of(tiles, kPackPerSm * sms);
    const T* w = static_cast<const T*>(W);
    uint8_t* c = static_cast<uint8_t*>(codes);
    if (zeros != nullptr)
        w4_quantize_kernel<T, true><<<grid, kCodesThreads, 0, s>>>(w, rows, N, K, k_tiles_of(K), tiles, shift_of(group), c,
                                                                   static_cast<T*>(scales), static_cast<T*>(zeros));
    else
        w4_quantize_kernel<T, false><<<grid, kCodesThreads, 0, s>>>(w, rows, N, K, k_tiles_of(K), tiles, shift_of(group), c,
                                                                    static_cast<T*>(scales), nullptr);
}

template <class T>
void dequantize(const Weights& w, int64_t rows, int64_t N, int64_t K, void* W, int sms, cudaStream_t s) {
    const int64_t tiles = tiles_of(rows, K);
    w4_dequantize_kernel<T><<<grid_of(tiles, kUnpackPerSm * sms), kCodesThreads, 0, s>>>(
        static_cast<const uint8_t*>(w.data), static_cast<const T*>(w.scales), static_cast<const T*>(w.zeros), rows, N, K,
        k_tiles_of(K), tiles, shift_of(w.group), static_cast<T*>(W));
}

}  // namespace

cudaError_t launch_w4_quantize(bool bf16, const void* W, int64_t batch, int64_t N, int64_t K, int group, void* codes,
                               void* scales, void* zeros, int sms, cudaStream_t s) {
    if (bf16) quantize<__nv_bfloat16>(W, batch * N, N, K, group, codes, scales, zeros, sms, s);
    else quantize<__half>(W, batch * N, N, K, group, codes, scales, zeros, sms, s);
    return cudaGetLastError();
}

cudaError_t launch_w4_dequantize(bool bf16, const Weights& w, int64_t batch, int64_t N, int64_t K, void* W, int sms,
                                 cudaStream_t s) {
    if (bf16) dequantize<__nv_bfloat16>(w, batch * N, N, K, W, sms, s);
    else dequantize<__half>(w, batch * N, N, K, W, sms, s);
    return cudaGetLastError();
}

}  // namespace gemm_gb300
