// kmeans_types.h -- element types of the codebook-training kernels (lookup,
// linear, gradient clipping): bf16, fp16 and fp32 in memory, fp32 (or more)
// in every sum.  Not part of the public interface.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kmeans_mi355x.h"

namespace kmeans {

// Each type's conversions between its stored bits and fp32.  Narrowing rounds
// to nearest, ties to even; bf16 NaNs become quiet, values past the largest
// finite one become infinite.
struct Bf16 {
    typedef uint16_t bits;
    typedef __bf16 mfma __attribute__((ext_vector_type(8)));
    static __device__ __forceinline__ float widen(bits b) {
        return __uint_as_float(static_cast<uint32_t>(b) << 16);
    }
    static __device__ __forceinline__ bits narrow(float f) {
        return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));
    }
};

struct Fp16 {
    typedef uint16_t bits;
    typedef _Float16 mfma __attribute__((ext_vector_type(8)));
    static __device__ __forceinline__ float widen(bits b) {
        return static_cast<float>(__builtin_bit_cast(_Float16, b));
    }
    static __device__ __forceinline__ bits narrow(float f) {
        // The empty asm keeps f an fp32 value: a product or sum fused into
        // the conversion would be rounded to fp16 alone, not to fp32 first as
        // the formulas say (and as the other types do it).
#if defined(__HIP_DEVICE_COMPILE__)
        asm("" : "+v"(f));
#endif
        return __builtin_bit_cast(uint16_t, static_cast<_Float16>(f));
    }
};

struct Fp32 {
    typedef float bits;
    static __device__ __forceinline__ float widen(bits b) { return b; }
    static __device__ __forceinline__ bits narrow(float f) { return f; }
};

// n consecutive elements at an address aligned to one element only: one
// vector access where the hardware takes unaligned ones (global memory does).
template <typename B, int n>
struct __attribute__((packed, aligned(sizeof(B)))) Packed {
    B v[n];
};

inline size_t dtype_size(int32_t dtype) { return dtype == KMEANS_FP32 ? 4 : 2; }

}  // namespace kmeans
