// kmeans_fp8.h -- 8-bit floating point (OCP e4m3: 4 exponent and 3 mantissa
// bits, largest value 448, no infinities) with a scale for each block of 128
// columns, as the norm and kmeans_quantize write it and kmeans_linear_fp8 reads
// it.  Not part of the public interface.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
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

// The first n of 8 values, divided by their scale and rounded to e4m3 (to nearest,
// ties to even; the scale keeps them at 448 or below but for a rounding).  The
// quotient is the correctly rounded one: quotients of 16-bit values often lie on a
// tie of e4m3, which a product with 1 / scale would leave to either side (one bf16
// value of 2000).  q0 = v inv is off by a unit or two, and its remainder, exact in
// one fused operation, brings it to the nearest (262144 x 128 in rows 22.7 us, 21.4
// with the product alone, 26.2 with a division for each; 16384 x 4096 in the norm
// 88, 88 and 96).  Remainders below 2^-149 are
// kept from vanishing by a power of two on both sides; zeros keep their sign, and an
// infinite scale makes zeros of finite values, as in a division.
struct __attribute__((packed, aligned(1))) Fp8Run {
    uint32_t lo, hi;
};
__device__ __forceinline__ void store_fp8_run(uint8_t *p, int n, float (&v)[8], float scale) {
#if defined(__HIP_DEVICE_COMPILE__)
    if (scale < 0x1p-90f) {
        scale *= 0x1p60f;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] *= 0x1p60f;
    }
    const float inv = 1.0f / scale;
    const float finite = scale == INFINITY ? 0.0f : scale;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float q0 = v[e] * inv;
        v[e] = fmaf(-fmaf(q0, finite, -v[e]), inv, q0);
    }
    Fp8Run q;
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
    q.lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], w, true);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], 0, false);
    q.hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], w, true);
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
