// kmeans_linear_tile.h -- what the linear layer's kernels share: activations and
// the epilogue, the staging of operand tiles in LDS and their fragments, the
// order of tiles over the XCDs, and the joining of a split product.  Device
// code; not part of the public interface.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "kmeans_linear_plan.h"
#include "kmeans_types.h"

namespace kmeans {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

#define KM_LDS __attribute__((address_space(3)))
#define KM_INLINE __attribute__((always_inline))

constexpr uint32_t kOutOfRange = 0x80000000u;

// ---- activations -----------------------------------------------------------

constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

// (erfc(|x|) / 2, exp(-x^2)): exp(x^2) erfc(x) as a quotient of polynomials of
// degree 3 and 4 (least largest relative error over x >= 0, fitted by linear
// programming: 3.9e-7) times the Gaussian.  The error is relative, so that
// z Phi(z) keeps its digits in the negative tail, where it is this value alone:
// 7e-7 with the roundings, and 1e-7 for each unit of x^2 from the exponential.
// Past 16 the Gaussian is zero in fp32.
__device__ __forceinline__ float half_erfc_abs(float x, float &gauss) {
    const float a = fminf(fabsf(x), 16.0f);
    gauss = exp_fast(-a * a);
    float n = 0.5f * 0.09663902589f;
    n = fmaf(n, a, 0.5f * 0.4787308077f);
    n = fmaf(n, a, 0.5f * 1.024552540f);
    n = fmaf(n, a, 0.5f * 0.9999996149f);
    float d = 0.1713078895f;
    d = fmaf(d, a, 0.8479616586f);
    d = fmaf(d, a, 1.908325611f);
    d = fmaf(d, a, 2.152904719f);
    d = fmaf(d, a, 1.0f);
    return n * __builtin_amdgcn_rcpf(d) * gauss;
}

// 1 / (1 + exp(-x)): 0 and 1 at the infinities.
__device__ __forceinline__ float logistic(float x) {
    return __builtin_amdgcn_rcpf(1.0f + exp_fast(-x));
}

constexpr float kTanhC = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kTanhA = 0.044715f;

__device__ __forceinline__ float activate(int act, float z) {
    switch (act) {
    case KMEANS_ACT_RELU:
        return z <= 0.0f ? 0.0f : z;
    case KMEANS_ACT_GELU: {
        float g;
        const float h = half_erfc_abs(z * kSqrtHalf, g);
        return z * (z < 0.0f ? h : 1.0f - h);
    }
    case KMEANS_ACT_GELU_TANH:
        // (1 + tanh(u)) / 2 = logistic(2 u)
        return z * logistic(kTanhC * fmaf(kTanhA * z, z * z, z));
    case KMEANS_ACT_SILU:
        return z * logistic(z);
    default:
        return z;
    }
}

// d * act'(z).  Past 128 every slope but relu's is 1 or 0 to the last bit in
// fp32; z is held there, since its square or cube would overflow, or an
// infinite z (a pre-activation kept in fp16) meet a zero, and make NaN of it.
// A NaN stays.
__device__ __forceinline__ float activate_grad(int act, float z, float d) {
    if (act != KMEANS_ACT_NONE && act != KMEANS_ACT_RELU)
        z = z > 128.0f ? 128.0f : z < -128.0f ? -128.0f : z;
    switch (act) {
    case KMEANS_ACT_RELU:
        return z <= 0.0f ? 0.0f : d;
    case KMEANS_ACT_GELU: {
        float g;
        const float h = half_erfc_abs(z * kSqrtHalf, g);
        const float phi = z < 0.0f ? h : 1.0f - h;
        return d * fmaf(z * 0.3989422804014327f, g, phi);   // 1 / sqrt(2 pi)
    }
    case KMEANS_ACT_GELU_TANH: {
        const float s = logistic(kTanhC * fmaf(kTanhA * z, z * z, z));
        const float du = kTanhC * fmaf(3.0f * kTanhA * z, z, 1.0f);
        return d * fmaf(z * s * (1.0f - s), du, s);
    }
    case KMEANS_ACT_SILU: {
        const float s = logistic(z);
        return d * fmaf(z * s, 1.0f - s, s);
    }
    default:
        return d;
    }
}

// ---- the product -----------------------------------------------------------

template <int ACT, int V>
__device__ __forceinline__ void activate_run(float (&v)[V]) {
#pragma unroll
    for (int c = 0; c < V; ++c)
        v[c] = activate(ACT, v[c]);
}

template <int V>
__device__ __forceinline__ void activate_run(int act, float (&v)[V]) {
    switch (act) {
    case KMEANS_ACT_RELU: activate_run<KMEANS_ACT_RELU>(v); break;
    case KMEANS_ACT_GELU: activate_run<KMEANS_ACT_GELU>(v); break;
    case KMEANS_ACT_GELU_TANH: activate_run<KMEANS_ACT_GELU_TANH>(v); break;
    case KMEANS_ACT_SILU: activate_run<KMEANS_ACT_SILU>(v); break;
    default: break;
    }
}

// V consecutive outputs of row i from column j on (those below J): bias,
// activation, residual, one rounding.
template <typename T, int V>
__device__ __forceinline__ void finish_run(const Epilogue &e, int i, int j, int J, float (&v)[V]) {
    typedef typename T::bits B;
    const int n = J - j;
    if (e.bias != nullptr) {
        const Packed<B, V> q = load_run<B, V>(static_cast<const B *>(e.bias) + j, n);
#pragma unroll
        for (int c = 0; c < V; ++c)
            v[c] += T::widen(q.v[c]);
    }
    if (e.pre != nullptr)
        store_run<B, V>(static_cast<B *>(e.pre) + i * e.ldp + j, n, narrow_run<T, V>(v));
    activate_run(e.act, v);
    if (e.residual != nullptr) {
        const Packed<B, V> q = load_run<B, V>(static_cast<const B *>(e.residual) + i * e.ldr + j, n);
#pragma unroll
        for (int c = 0; c < V; ++c)
            v[c] += T::widen(q.v[c]);
    }
    store_run<B, V>(static_cast<B *>(e.out) + i * e.ldo + j, n, narrow_run<T, V>(v));
}

__device__ __forceinline__ f32x4 mfma(Bf16::mfma a, Bf16::mfma b, f32x4 c) {
#if defined(__HIP_DEVICE_COMPILE__)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
#else
    return c;
#endif
}
__device__ __forceinline__ f32x4 mfma(Fp16::mfma a, Fp16::mfma b, f32x4 c) {
#if defined(__HIP_DEVICE_COMPILE__)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
#else
    return c;
#endif
}

// s_waitcnt vmcnt(N): all but the last N global-to-LDS copies of this wave
// have landed (a workgroup barrier does not imply it).
template <int N>
__device__ __forceinline__ void wait_vmem() {
    static_assert(N < 64, "vmcnt has six bits");
    __builtin_amdgcn_s_waitcnt(0x0f70 | (N & 15) | ((N >> 4) << 14));
}

// Workgroup barrier for LDS traffic alone: this wave's LDS reads and writes are
// done, its copies may still be on their way (__syncthreads would wait for
// every copy).
__device__ __forceinline__ void lds_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xc07f);   // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Copies tiles of one operand from global memory into LDS, THREADS threads
// together; tile t covers k in [t * 64, t * 64 + 64) of the workgroup's range.
// Values past the range of k are zero (so they add nothing); values past the
// own index are anything (their outputs are not stored), but nothing outside
// the operand is read.
//
// DMA (16-byte aligned rows of whole chunks): buffer loads straight into LDS,
// nothing held in registers.  Else: 16-byte buffer loads at the rows' own
// alignment into registers at issue(), written to LDS at commit().  Such a load
// may run past the end of its row, into the rows after it, where those hold it
// (runs_stay_inside).  The last tile, where there may be no next row, loads a
// run that is cut short so that it ends with its row, and commit() shifts it
// down (4133 x 515 x 1001 24.6 us, 26.5 with those values loaded one by one).
// Rows of less than eight values have no such run: their last tile, and the
// one before it where its runs would leave the operand, is loaded value by
// value.
template <typename T, bool OWN, int R, int THREADS, bool DMA>
struct Stager {
    typedef TileMap<OWN, R> Map;
    typedef TilePieces<OWN, R, THREADS, DMA> Pieces;
    typedef typename T::bits B;
    static constexpr int kPieces = Pieces::kCount;

    const B *base;        // element (0, 0) of the current range, own offset included
    int64_t ld;
    int own_lim;          // values of the own index that exist from base on
    int k_len;            // k values of the range
    int back;             // values of a row known to lie before base, 8 at most
    bool narrow;          // rows of less than eight values
    int tid;
    uint32_t off[kPieces];
    u32x4 held[DMA ? 1 : kPieces];
    struct Halves { uint64_t lo, hi; };

    // Piece u of this thread: row r and chunk c (elements 8 c ..) it fetches.
    __device__ __forceinline__ void piece(int u, int &r, int &c) const {
        Pieces::at(tid, u, r, c);
    }
    // Whether a tile with k_left values of k to the end of the range (its own
    // among them) may load whole runs.
    __device__ __forceinline__ bool whole_runs(int k_left) const {
        return runs_stay_inside(OWN, k_left, ld, own_lim);
    }
    // Tiles at the end of the range that may not.
    __device__ __forceinline__ int cut_tiles() const {
        const int last = (k_len - 1) % kTileK + 1;
        return k_len > kTileK && !whole_runs(last + kTileK) ? 2 : 1;
    }
    __device__ __forceinline__ void init(const void *p, int64_t stride, int own0, int own,
                                         int64_t k0, int k_n, int thread) {
        ld = stride;
        tid = thread;
        own_lim = own - own0;
        k_len = k_n;
        back = (OWN ? own0 : k0) > 0 ? 8 : 0;
        narrow = back == 0 && (OWN ? own_lim : k_len) < 8;
        base = static_cast<const B *>(p) + (OWN ? k0 * stride + own0 : own0 * stride + k0);
#pragma unroll
        for (int u = 0; u < kPieces; ++u) {
            int r, c;
            piece(u, r, c);
            if (OWN)
                off[u] = c * 8 < own_lim ? static_cast<uint32_t>(r * ld + c * 8) * 2u
                                         : kOutOfRange;
            else
                off[u] = static_cast<uint32_t>(min(r, own_lim - 1) * ld + c * 8) * 2u;
        }
    }
    // FULL: the tile is known to hold kTileK values of k, and to be none of the
    // last cut_tiles() ones where those count (without DMA).
    template <bool FULL>
    __device__ __forceinline__ void issue(int t, uint8_t *stage) {
#if defined(__HIP_DEVICE_COMPILE__)
        const B *src = base + static_cast<int64_t>(t) * (OWN ? kTileK * ld : kTileK);
        const int k_left = k_len - t * kTileK;
        const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<B *>(src), 0, 0x7fffffff, 0x00020000);
        if constexpr (DMA) {
            uint8_t *dst = stage + __builtin_amdgcn_readfirstlane(tid >> 6) * (kPieces * 1024);
            if (FULL || k_left >= kTileK) {
#pragma unroll
                for (int u = 0; u < kPieces; ++u)
                    __builtin_amdgcn_raw_ptr_buffer_load_lds(
                        rs, (KM_LDS void *)(dst + u * 1024), 16, off[u], 0, 0, 0);
            } else {
#pragma unroll
                for (int u = 0; u < kPieces; ++u) {
                    int r, c;
                    piece(u, r, c);
                    const uint32_t o = (OWN ? r : c * 8) < k_left ? off[u] : kOutOfRange;
                    __builtin_amdgcn_raw_ptr_buffer_load_lds(
                        rs, (KM_LDS void *)(dst + u * 1024), 16, o, 0, 0, 0);
                }
            }
        } else if (FULL || whole_runs(k_left)) {
#pragma unroll
            for (int u = 0; u < kPieces; ++u)
                held[u] = __builtin_bit_cast(
                    u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, off[u], 0, 0));
        } else if (narrow) {
            for (int u = 0; u < kPieces; ++u) {
                int r, c;
                piece(u, r, c);
                const bool row = OWN ? r < k_left : true;
                const int n = row ? (OWN ? own_lim : k_left) - c * 8 : 0;   // that exist
                const uint32_t at = static_cast<uint32_t>((OWN ? r : min(r, own_lim - 1)) * ld +
                                                          c * 8) * 2u;
                uint32_t e[8];
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    e[x] = __builtin_amdgcn_raw_buffer_load_b16(
                        rs, x < n ? at + 2 * x : kOutOfRange, 0, 0);
                const u32x4 v = {e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16,
                                 e[6] | e[7] << 16};
#pragma unroll
                for (int x = 0; x < kPieces; ++x)      // keeps held[] in registers
                    held[x] = x == u ? v : held[x];
            }
        } else {
            // The resource starts `before` values earlier, so that offsets are
            // not negative.
            const int before = OWN || t == 0 ? back : 8;
            const __amdgpu_buffer_rsrc_t tail = __builtin_amdgcn_make_buffer_rsrc(
                const_cast<B *>(src - before), 0, 0x7fffffff, 0x00020000);
#pragma unroll
            for (int u = 0; u < kPieces; ++u) {
                int r, c;
                piece(u, r, c);
                const bool some = OWN ? r < k_left && c * 8 < own_lim : c * 8 < k_left;
                const int at = before + c * 8 - cut(c, k_left);
                held[u] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                    tail, some ? static_cast<uint32_t>((OWN ? r : min(r, own_lim - 1)) * ld + at) *
                                     2u : kOutOfRange, 0, 0));
            }
        }
#endif
    }
    // Values by which the last tile's run c starts early to end with its row.
    __device__ __forceinline__ int cut(int c, int k_left) const {
        return values_cut(c, OWN ? own_lim : k_left);
    }
    // Tile t, issued last, is in LDS once this returned on every wave and
    // they met at a barrier.  FULL: it is not the last one.
    template <bool FULL>
    __device__ __forceinline__ void commit(int t, uint8_t *stage) {
        if constexpr (!DMA) {
            const int k_left = k_len - t * kTileK;
            if (!FULL && k_left <= kTileK && !narrow) {
#pragma unroll
                for (int u = 0; u < kPieces; ++u) {
                    int r, c;
                    piece(u, r, c);
                    const int shift = 16 * cut(c, k_left);
                    Halves h = __builtin_bit_cast(Halves, held[u]);
                    if (shift >= 64) {
                        h.lo = shift >= 128 ? 0 : h.hi >> (shift - 64);
                        h.hi = 0;
                    } else if (shift > 0) {
                        h.lo = h.lo >> shift | h.hi << (64 - shift);
                        h.hi >>= shift;
                    }
                    held[u] = __builtin_bit_cast(u32x4, h);
                }
            }
#pragma unroll
            for (int u = 0; u < kPieces; ++u)
                *reinterpret_cast<u32x4 *>(stage + (u * THREADS + tid) * 16) = held[u];
        }
    }
};

// Fragments of one operand for the 16x16x32 matrix instruction: lane l holds
// own index l % 16 of a 16-wide block, k = 8 (l / 16) .. + 7 of a k-step.
template <typename T, bool OWN, int R, int BLOCKS>
struct Reader {
    typedef TileMap<OWN, R> Map;
    uint32_t off[OWN ? BLOCKS : 2];

    __device__ __forceinline__ void init(int own0, int lane) {
        const int l = lane & 15, g = lane >> 4;
        if constexpr (OWN) {
            const int k = 8 * g + (l >> 2);
#pragma unroll
            for (int b = 0; b < BLOCKS; ++b)
                off[b] = k * Map::kRowBytes + ((own0 / 16 + b) ^ Map::spread(k)) * 32 + (l & 3) * 8;
        } else {
#pragma unroll
            for (int s = 0; s < 2; ++s)
                off[s] = (own0 + l) * Map::kRowBytes + Map::chunk(l, 4 * s + g) * 16;
        }
    }
    __device__ __forceinline__ typename T::mfma read(const uint8_t *stage, int b, int s) const {
        if constexpr (OWN) {
            // Lane l of a group of 16 addresses k row l / 4, values 4 (l % 4)
            // .. + 3; it receives value l of k rows 0 .. 3.  Two such reads
            // make a lane's eight k.
#if defined(__HIP_DEVICE_COMPILE__)
            struct { s16x4 lo, hi; } v;
            const uint8_t *p = stage + off[b] + s * 32 * Map::kRowBytes;
            v.lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((KM_LDS s16x4 *)(p));
            v.hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (KM_LDS s16x4 *)(p + 4 * Map::kRowBytes));
            return __builtin_bit_cast(typename T::mfma, v);
#else
            return typename T::mfma{};
#endif
        } else {
            return __builtin_bit_cast(typename T::mfma,
                                      *reinterpret_cast<const u32x4 *>(
                                          stage + off[s] + b * 16 * Map::kRowBytes));
        }
    }
};

// Split and output tile of workgroup b: XCD x = b % 8 takes a contiguous eighth
// of the (split, tile) pairs (each XCD has its own L2), the tiles of a split in
// bands of 8 tile rows, so that the tiles in flight together share rows of both
// operands.
__device__ __forceinline__ void tile_of(int b, int ni, int nj, int splits, int &split, int &ti,
                                        int &tj) {
    constexpr int kBand = 8;
    const int tiles = ni * nj, n = tiles * splits;
    const int x = b & 7, q = n >> 3, rem = n & 7;
    int t = x * q + min(x, rem) + (b >> 3);
    split = t / tiles;
    t -= split * tiles;
    const int band = t / (kBand * nj);
    const int i0 = band * kBand;
    const int h = min(kBand, ni - i0);
    const int in = t - i0 * nj;
    tj = in / h;
    ti = i0 + in - tj * h;
}

template <int I>
using Index = std::integral_constant<int, I>;

// db[j] = sum of linear_dz_kernel's column partials.  A workgroup takes COLS
// columns, THREADS / COLS threads a column, each a fixed interleaved share of
// the rows (kBiasBatch in flight), joined in LDS.
struct BiasSums {
    const float *col_partial;    // [rows][F]; null: no bias gradient
    int rows, F;
    void *db;
};
constexpr int kBiasThreads = 1024;
constexpr int kBiasCols = 32;
constexpr int kBiasBatch = 8;
template <typename T, int THREADS, int COLS>
__device__ __forceinline__ void sum_bias(const BiasSums &b, int block) {
    constexpr int kShares = THREADS / COLS;
    __shared__ float sums[kShares][COLS + 1];
    const int c = threadIdx.x % COLS, w = threadIdx.x / COLS;
    const int col = block * COLS + c;
    float v = 0.0f;
    if (col < b.F)
        for (int r0 = w; r0 < b.rows; r0 += kBiasBatch * kShares) {
            float x[kBiasBatch];
#pragma unroll
            for (int u = 0; u < kBiasBatch; ++u)
                x[u] = b.col_partial[static_cast<int64_t>(min(r0 + u * kShares, b.rows - 1)) * b.F +
                                     col];
#pragma unroll
            for (int u = 0; u < kBiasBatch; ++u)
                v += r0 + u * kShares < b.rows ? x[u] : 0.0f;
        }
    sums[w][c] = v;
    __syncthreads();
    if (w == 0 && col < b.F) {
        for (int q = 1; q < kShares; ++q)
            v += sums[q][c];
        static_cast<typename T::bits *>(b.db)[col] = T::narrow(v);
    }
}

// Joins the splits of a product: the partial sums of a run of four outputs are
// added by four threads, one of each wave (every fourth split each, kJoinBatch
// loads in flight), whose sums meet in LDS; then the epilogue.  Workgroups from
// join_wgs on sum the bias gradient instead, where there is one: a launch less
// (65536 x 512 x 128 gradients 50.2 us, 52.8 with linear_bias_kernel alone).
constexpr int kJoinThreads = 256;
constexpr int kJoinRuns = 64;          // of one workgroup
constexpr int kJoinBatch = 8;
constexpr int kJoinBiasCols = 8;
template <typename T>
__global__ __launch_bounds__(kJoinThreads)
void linear_join_kernel(const Product g, int join_wgs, const BiasSums bias) {
    if (static_cast<int>(blockIdx.x) >= join_wgs) {
        sum_bias<T, kJoinThreads, kJoinBiasCols>(bias, blockIdx.x - join_wgs);
        return;
    }
    constexpr int kShares = kJoinThreads / kJoinRuns;
    __shared__ f32x4 sums[kShares][kJoinRuns];
    const int share = threadIdx.x / kJoinRuns, lane = threadIdx.x % kJoinRuns;
    const int runs = (g.J + 3) / 4;
    const int64_t total = static_cast<int64_t>(g.I) * runs;
    const int64_t plane = static_cast<int64_t>(g.I) * g.J;
    for (int64_t x0 = static_cast<int64_t>(blockIdx.x) * kJoinRuns; x0 < total;
         x0 += static_cast<int64_t>(join_wgs) * kJoinRuns) {
        const int64_t x = min(x0 + lane, total - 1);
        const int i = static_cast<int>(x / runs), j = static_cast<int>(x % runs) * 4;
        const float *p = g.partial + static_cast<int64_t>(i) * g.J + j;
        f32x4 v = {0, 0, 0, 0};
        for (int s0 = share; s0 < g.splits; s0 += kShares * kJoinBatch) {
            Packed<float, 4> w[kJoinBatch];
#pragma unroll
            for (int u = 0; u < kJoinBatch; ++u)
                w[u] = load_run<float, 4>(p + min(s0 + u * kShares, g.splits - 1) * plane, g.J - j);
#pragma unroll
            for (int u = 0; u < kJoinBatch; ++u)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    v[c] += s0 + u * kShares < g.splits ? w[u].v[c] : 0.0f;
        }
        sums[share][lane] = v;
        __syncthreads();
        if (share == 0 && x0 + lane < total) {
#pragma unroll
            for (int q = 1; q < kShares; ++q)
                v += sums[q][lane];
            float y[4] = {v[0], v[1], v[2], v[3]};
            finish_run<T, 4>(g.epi, i, j, g.J, y);
        }
        __syncthreads();
    }
}

}  // namespace
}  // namespace kmeans
