// internal.h -- what the C-ABI layers share: the current device's state, tensor
// map encoding, the fused epilogue's checks and per-stream scratch.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <mutex>

#include "epilogue.cuh"
#include "gemm_f16.h"

namespace gemm_gb300 {

struct DeviceView {
    int dev;            // CUDA device ordinal
    int sms;
    uint32_t* status;   // device status word (wait.cuh)
};

// The current device, set up on first use (api.cu).
gemm_status_t device_view(DeviceView* out);

// The epilogue's argument checks and its kernel form (api.cu).
gemm_status_t check_epilogue(const gemm_epilogue_t* e, const void* D, int64_t M, int64_t N);
EpiParams epi_params(const gemm_epilogue_t* e);

// gemm_nt_ex of 16-bit operands with AUTO, and with the second half of a few rows'
// adapters in its epilogue (nullptr: none) (api.cu).
gemm_status_t run_dense(int dtype, const void* A, const void* B, void* D, int64_t M, int64_t N, int64_t K,
                        const gemm_epilogue_t* epilogue, const LoraEpi* lora, gemm_stream_t stream);

// D = act(beta * C + bias), the K == 0 result (api.cu).
gemm_status_t run_empty_sum(void* D, int64_t M, int64_t N, const EpiParams& epi, int out_dtype, int sms,
                            cudaStream_t s);

// 2-D tensor map over `outer` rows of `inner` elements of elem_bytes (1 or 2),
// rows `inner` elements apart, zero fill outside (api.cu).
bool encode_map(CUtensorMap* map, const void* base, int elem_bytes, int64_t inner, int64_t outer, uint32_t box_inner,
                uint32_t box_outer, bool swizzle128);

bool ranges_overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes);
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// What scratch memory belongs to: one stream of one device.  A handle does not tell
// streams apart: cudaStreamPerThread is another stream in every thread, and a
// destroyed stream's handle may come back while its work still runs.
struct StreamKey {
    int dev;
    unsigned long long id;   // cudaStreamGetId: never used twice in a process
    bool operator<(const StreamKey& o) const { return dev != o.dev ? dev < o.dev : id < o.id; }
};
gemm_status_t stream_key(int dev, gemm_stream_t stream, StreamKey* out);   // api.cu

// `bytes` of scratch for (device, stream), 256-byte aligned, and its counters:
// kScratchCounters zeros that every kernel using them leaves at zero (llm/llm_api.cu).
// The kernels of one call pass values to one another through it, so a Scratch keeps
// other threads' calls on the pair waiting for as long as it lives: until the call's
// last launch.
constexpr int kScratchCounters = 1024;
constexpr int kCounterLora = 32;   // of the adapters' small calls; the first is the router's
struct Scratch {
    uint8_t* data = nullptr;
    uint32_t* counters = nullptr;
    std::mutex* held = nullptr;
    Scratch() = default;
    Scratch(const Scratch&) = delete;
    Scratch& operator=(const Scratch&) = delete;
    ~Scratch() {
        if (held != nullptr) held->unlock();
    }
};
gemm_status_t get_scratch(int dev, gemm_stream_t stream, size_t bytes, Scratch* out);

}  // namespace gemm_gb300
