// Device helpers shared by the kernels around an adapted layer (layer norm,
// low-rank adapters, gradient clipping): element types and block sums.
#pragma once

#include "device_common.h"

namespace i8mm {
namespace {

typedef __bf16 v8b __attribute__((ext_vector_type(8)));

template <typename T>
__device__ __forceinline__ float to_float(T v) { return static_cast<float>(v); }

// fp32 -> T, to nearest even (the identity for float)
template <typename T>
__device__ __forceinline__ T from_float(float v) { return static_cast<T>(v); }

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
    return v;
}

// Sum over a block of NW wavefronts, in every thread; the same order on
// every call. red: NW floats of LDS, free for reuse when the call returns
// in every thread.
template <int NW>
__device__ __forceinline__ float block_sum(float v, float* red) {
    v = wave_sum(v);
    if constexpr (NW == 1) return v;
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) t += red[w];
    __syncthreads();
    return t;
}

}  // namespace
}  // namespace i8mm
