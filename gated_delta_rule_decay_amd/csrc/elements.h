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

template <class T, int VE>
struct alignas(VE * sizeof(T) < 16 ? VE * sizeof(T) : 16) Pack {
    T e[VE];
};

}  // namespace gdn2
