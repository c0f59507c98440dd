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

// Elements of a tensor from a uniform one on: loads behind the last read as
// zero and stores there are dropped, so a lane goes to NOWHERE with what it does
// not need instead of branching by itself.
template <class E>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void *tensor, int64_t first, int elements) {
    const uint64_t at = reinterpret_cast<uint64_t>(static_cast<const E *>(tensor) + first);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(at)), hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(at >> 32));
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void *>(static_cast<uint64_t>(hi) << 32 | lo), 0,
                                             elements * static_cast<int>(sizeof(E)), 0x00027000);
}
// an offset behind the end, also with up to 2^31 - 1 added
constexpr unsigned NOWHERE = 0x80000000u;

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

// Keeps the compiler from working on all elements of a lane at once, for which
// the registers do not suffice: what follows in the program starts after `v` is
// there (an empty instruction that is said to change it).
__device__ __forceinline__ void settle(float &v) { asm volatile("" : "+v"(v)); }

}  // namespace gdn2
