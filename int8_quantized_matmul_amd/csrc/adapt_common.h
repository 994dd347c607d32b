// Device helpers shared by the kernels around an adapted layer (layer norm,
// low-rank adapters, gradient clipping): element types, groups of eight
// elements and sums over a wavefront.
#pragma once

#include "device_common.h"

namespace i8mm {
namespace {

typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef float v8f __attribute__((ext_vector_type(8)));
typedef float v2f __attribute__((ext_vector_type(2)));

template <typename T>
__device__ __forceinline__ float to_float(T v) { return static_cast<float>(v); }

// fp32 -> T, to nearest even (the identity for float)
template <typename T>
__device__ __forceinline__ T from_float(float v) { return static_cast<T>(v); }

// Eight neighbouring elements, loaded and stored by one 16-byte access (two
// for fp32) at any element alignment: global memory is accessed at byte
// granularity on this target, an unaligned access only touches one more line.
template <typename T>
struct Eight {
    typedef T vec __attribute__((ext_vector_type(8)));
    vec v;

    // elements [0, n) of p, zeros beyond (n >= 8: all)
    __device__ __forceinline__ void load(const T* p, int n) {
        if (n >= 8) {
            __builtin_memcpy(&v, p, sizeof(v));
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = k < n ? p[k] : static_cast<T>(0.0f);
        }
    }
    __device__ __forceinline__ void store(T* p, int n) const {
        if (n >= 8) {
            __builtin_memcpy(p, &v, sizeof(v));
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < n) p[k] = v[k];
        }
    }
    // The same past the caches, for results that are not read again soon.
    __device__ __forceinline__ void store_through(T* p, int n) const {
        typedef vec loose __attribute__((aligned(sizeof(T))));
        if (n >= 8) __builtin_nontemporal_store(v, reinterpret_cast<loose*>(p));
        else store(p, n);
    }
    __device__ __forceinline__ float at(int k) const { return to_float<T>(v[k]); }
    __device__ __forceinline__ void set(int k, float f) { v[k] = from_float<T>(f); }
};

// -inf in fp64 from a register that the compiler does not look into: as a
// constant of a whole wavefront it would become a scalar move of a 64-bit
// literal, which this target has no encoding for and the compiler drops to 0.
__device__ __forceinline__ double minus_infinity() {
    float f = -INFINITY;
    asm("" : "+v"(f));
    return f;
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __builtin_bit_cast(
        float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}

// Sum over the wavefront, in every lane. Within 16 lanes the partners come by
// lane permutes in the adder's own operand path; the swaps of 16- and 32-lane
// halves are register moves too, so nothing goes through LDS.
__device__ __forceinline__ float wave_sum(float v) {
    v += dpp<0xb1>(v);     // lanes xor 1
    v += dpp<0x4e>(v);     // lanes xor 2
    v += dpp<0x141>(v);    // mirrored within 8
    v += dpp<0x140>(v);    // mirrored within 16
    {
        const auto p = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, v),
                                                        __builtin_bit_cast(unsigned, v), false, false);
        v = __builtin_bit_cast(float, static_cast<unsigned>(p[0])) +
            __builtin_bit_cast(float, static_cast<unsigned>(p[1]));
    }
    const auto p = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, v), __builtin_bit_cast(unsigned, v),
                                                    false, false);
    return __builtin_bit_cast(float, static_cast<unsigned>(p[0])) +
           __builtin_bit_cast(float, static_cast<unsigned>(p[1]));
}

}  // namespace
}  // namespace i8mm
