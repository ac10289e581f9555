// kmeans_types.h -- element types of the kernels around a codebook (lookup,
// linear, gradient clipping, norm, quantisation, sampling): bf16, fp16 and fp32 in
// memory, fp32 (or more) in every sum.  Not part of the public interface.
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
    // Two values in one conversion (v_cvt_pk_bf16_f32).
    static __device__ __forceinline__ uint32_t narrow2(float a, float b) {
        typedef float f32x2 __attribute__((ext_vector_type(2)));
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
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
    static __device__ __forceinline__ uint32_t narrow2(float a, float b) {
        return narrow(a) | static_cast<uint32_t>(narrow(b)) << 16;
    }
};

struct Fp32 {
    typedef float bits;
    static __device__ __forceinline__ float widen(bits b) { return b; }
    static __device__ __forceinline__ bits narrow(float f) { return f; }
};

// n consecutive elements at an address aligned to one element only.
template <typename B, int n>
struct __attribute__((packed, aligned(sizeof(B)))) Packed {
    B v[n];
};

// Their loads and stores as one vector access each (two for 32 bytes), which
// global memory takes at any alignment.  The vector type matters: an access
// typed as n elements is split and merged with neighbouring ones.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
template <typename B, int n>
__device__ __forceinline__ Packed<B, n> load_packed(const B *p) {
    constexpr size_t bytes = sizeof(B) * n;
    static_assert(n == 1 || bytes == 8 || bytes == 16 || bytes == 32, "vector accesses");
    if constexpr (n == 1) {
        return Packed<B, n>{{*p}};
    } else if constexpr (bytes == 8) {
        return __builtin_bit_cast(Packed<B, n>, *reinterpret_cast<const u32x2_any *>(p));
    } else if constexpr (bytes == 16) {
        return __builtin_bit_cast(Packed<B, n>, *reinterpret_cast<const u32x4_any *>(p));
    } else {
        struct { u32x4_any a, b; } v;
        v.a = reinterpret_cast<const u32x4_any *>(p)[0];
        v.b = reinterpret_cast<const u32x4_any *>(p)[1];
        return __builtin_bit_cast(Packed<B, n>, v);
    }
}
template <typename B, int n>
__device__ __forceinline__ void store_packed(B *p, const Packed<B, n> &q) {
    constexpr size_t bytes = sizeof(B) * n;
    static_assert(n == 1 || bytes == 8 || bytes == 16 || bytes == 32, "vector accesses");
    if constexpr (n == 1) {
        *p = q.v[0];
    } else if constexpr (bytes == 8) {
        *reinterpret_cast<u32x2_any *>(p) = __builtin_bit_cast(u32x2_any, q);
    } else if constexpr (bytes == 16) {
        *reinterpret_cast<u32x4_any *>(p) = __builtin_bit_cast(u32x4_any, q);
    } else {
        struct Halves { u32x4_any a, b; };
        const Halves v = __builtin_bit_cast(Halves, q);
        reinterpret_cast<u32x4_any *>(p)[0] = v.a;
        reinterpret_cast<u32x4_any *>(p)[1] = v.b;
    }
}

// The first m of n elements (all where m >= n).
template <typename B, int n>
__device__ __forceinline__ Packed<B, n> load_run(const B *p, int m) {
    if (m >= n)
        return load_packed<B, n>(p);
    Packed<B, n> q = {};
#pragma unroll
    for (int c = 0; c < n - 1; ++c)
        if (c < m)
            q.v[c] = p[c];
    return q;
}
template <typename B, int n>
__device__ __forceinline__ void store_run(B *p, int m, const Packed<B, n> &q) {
    if (m >= n) {
        store_packed(p, q);
        return;
    }
#pragma unroll
    for (int c = 0; c < n - 1; ++c)
        if (c < m)
            p[c] = q.v[c];
}

// n values rounded to T.
template <typename T, int n>
__device__ __forceinline__ Packed<typename T::bits, n> narrow_run(const float (&v)[n]) {
    if constexpr (sizeof(typename T::bits) == 2 && n % 2 == 0) {
        Packed<uint32_t, n / 2> q;
#pragma unroll
        for (int c = 0; c < n / 2; ++c)
            q.v[c] = T::narrow2(v[2 * c], v[2 * c + 1]);
        return __builtin_bit_cast(Packed<typename T::bits, n>, q);
    } else {
        Packed<typename T::bits, n> q;
#pragma unroll
        for (int c = 0; c < n; ++c)
            q.v[c] = T::narrow(v[c]);
        return q;
    }
}

inline size_t dtype_size(int32_t dtype) { return dtype == KMEANS_FP32 ? 4 : 2; }

}  // namespace kmeans
