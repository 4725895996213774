// w4.cuh -- eight 16-bit weights as fp32 numbers and back.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "epilogue.cuh"

namespace gemm_gb300 {

// 16 bytes of T as 8 floats
template <class T>
__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = Elem<T>::lo(w[i]);
        x[2 * i + 1] = Elem<T>::hi(w[i]);
    }
}

template <class T>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(Elem<T>::pack2(x[0], x[1]), Elem<T>::pack2(x[2], x[3]), Elem<T>::pack2(x[4], x[5]),
                      Elem<T>::pack2(x[6], x[7]));
}

}  // namespace gemm_gb300
