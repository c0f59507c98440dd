// elements.h -- elements of bf16 or fp32 tensors, one by one and in vectors of
// up to 16 bytes.
#pragma once

#include "common.h"

namespace gdn2 {

template <class T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32<uint16_t>(uint16_t x) { return bf16_to_f32(x); }

// fp32 -> the stored type, to nearest even (bf16: the hardware's conversion,
// two elements an instruction).
template <class T>
__device__ __forceinline__ T from_f32(float x) {
    if constexpr (sizeof(T) == 2) return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
    else return x;
}

template <class T, int VE>
struct alignas(VE * sizeof(T) < 16 ? VE * sizeof(T) : 16) Pack {
    T e[VE];
};

}  // namespace gdn2
