// kmeans_fp8.h -- 8-bit floating point (OCP e4m3: 4 exponent and 3 mantissa
// bits, largest value 448, no infinities) with a scale for each block of 128
// columns, as the norm and kmeans_quantize write it and kmeans_linear_fp8 reads
// it.  Not part of the public interface.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kmeans_internal.h"
#include "kmeans_types.h"

namespace kmeans {

constexpr int kFp8Block = 128;
constexpr float kFp8Max = 448.0f;

inline int64_t fp8_blocks(int64_t D) { return (D + kFp8Block - 1) / kFp8Block; }

// A matrix argument: rows of `cols` elements of `element` bytes, `ld` apart.
kmeans_status_t check_matrix(const char *name, const void *p, int64_t cols, int64_t ld,
                             size_t element);
// An array argument that may be null.
kmeans_status_t check_array(const char *name, const void *p, size_t element);

// |v| as an unsigned number of the same order, NaN above all others.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The largest magnitude among aligned groups of LANES lanes.
template <int LANES>
__device__ __forceinline__ uint32_t block_most(uint32_t m) {
#pragma unroll
    for (int x = LANES / 2; x >= 1; x >>= 1)
        m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), x, 64)));
    return m;
}

// The scale of a block by its largest magnitude: 1 where all values are zero,
// and no less than the smallest normal number (its inverse stays finite).  A
// NaN or an infinity in the block is its scale.
__device__ __forceinline__ float fp8_scale(uint32_t most) {
    const float s = __uint_as_float(most) / kFp8Max;
    return most == 0 ? 1.0f : s < 0x1p-126f ? 0x1p-126f : s;
}

// The first n of 8 values, times `inv`, in e4m3 (to nearest, ties to even; the
// scale keeps them at 448 or below but for a rounding).
struct __attribute__((packed, aligned(1))) Fp8Run {
    uint32_t lo, hi;
};
__device__ __forceinline__ void store_fp8_run(uint8_t *p, int n, const float (&v)[8], float inv) {
#if defined(__HIP_DEVICE_COMPILE__)
    Fp8Run q;
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * inv, v[1] * inv, 0, false);
    q.lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * inv, v[3] * inv, w, true);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4] * inv, v[5] * inv, 0, false);
    q.hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6] * inv, v[7] * inv, w, true);
    if (n >= 8) {
        typedef uint32_t u32x2_bytes __attribute__((ext_vector_type(2), aligned(1)));
        *reinterpret_cast<u32x2_bytes *>(p) = __builtin_bit_cast(u32x2_bytes, q);
        return;
    }
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (e < n)
            p[e] = static_cast<uint8_t>((e < 4 ? q.lo : q.hi) >> (8 * (e & 3)));
#endif
}

}  // namespace kmeans
