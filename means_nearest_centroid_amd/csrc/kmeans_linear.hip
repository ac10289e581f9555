// kmeans_linear.hip -- gfx950 kernels of the linear layer around a codebook
// and of its gradients.
//
//     forward   Z = X W^T + b,  Y = act(Z) + R
//     backward  dZ = dY * act'(Z),  dX = dZ W,  dW = dZ^T X,  db = sum_i dZ[i]
//
// All three products are one kernel, out[i][j] = sum_k P[i][k] Q[j][k], on
// operands that lie in memory either with k contiguous or with their own row
// index contiguous:
//
//     Y  (i = row,     j = F, k = D):  P = X  (k contiguous),  Q = W  (k contiguous)
//     dX (i = row,     j = D, k = F):  P = dZ (k contiguous),  Q = W  (j contiguous)
//     dW (i = feature, j = D, k = N):  P = dZ (i contiguous),  Q = X  (j contiguous)
//
// so no operand is ever transposed in memory: an operand whose own index is
// contiguous is staged in LDS as it lies and transposed by the LDS reads
// (ds_read_b64_tr_b16) on its way to the matrix instruction.
#include <stdint.h>

#include <algorithm>
#include <optional>
#include <type_traits>
#include <utility>

#include "kmeans_internal.h"
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

// One workgroup of WI x WJ waves computes a tile of (WI 16 TI) x (WJ 16 TJ)
// outputs over one split of k.  The matrix instruction's A operand is Q and B
// is P, so that a lane's four accumulator values are four consecutive j of
// one row i.
//
// S LDS stages; while tile t is multiplied, tiles t + 1 .. t + S - 1 are on
// their way.  Each k-step is worked in phases of four P blocks: a phase's
// fragments are read one phase ahead (double-buffered registers).  The
// barrier between tiles stands before the last phase of a tile, whose
// fragments are in registers by then: behind it the next tile's first
// fragments are read and the copy of tile t + S starts into the stage just
// freed, both under the last phase's matrix instructions.  The stages are
// distinct arrays and the loop is unrolled by S so that the compiler can tell
// an LDS read of one stage from a copy into another.
//
// Where k is long the matrix pipe is busy 0.66 to 0.69 of the time (8192 x 4096
// x 4096 forward 192 us, 1430 TFLOP/s; a kernel of matrix instructions alone
// reaches 0.87 by the same counters); waves wait at the barriers between tiles
// for the rest, and while the first copies and the epilogue run alone: nothing
// overlaps them with one workgroup per CU.  Where k is short or the epilogue has
// more to move, its bytes bound it: 16384 x 4096 x 4096 with tanh-gelu, residual
// and pre-activations kept is 484 us (busy 0.54), of which about 37 are the
// residual, 24 the pre-activations and 10 to 20 the activation (all residual
// loads ahead of both passes spill: 505).
template <int I>
using Index = std::integral_constant<int, I>;

template <typename T, bool POWN, bool QOWN, int WI, int WJ, int TI, int TJ, int S, bool DMA>
__global__ __launch_bounds__(WI * WJ * 64, DMA ? 2 : 4)
void linear_tile_kernel(const Product g) {
    constexpr int kThreads = WI * WJ * 64;
    constexpr int RI = WI * TI * 16, RJ = WJ * TJ * 16;
    constexpr int HB = TI < 4 ? TI : 4;       // P blocks of one phase
    constexpr int NH = TI / HB;               // phases per k-step
    constexpr int NP = 2 * NH;                // phases per tile
    static_assert(TI % HB == 0 && NP % 2 == 0, "phases alternate fragment buffers");
    static_assert(S == 2 || (S == 4 && DMA), "registers hold one tile on its way");
    typedef typename T::mfma Frag;
    typedef TileMap<POWN, RI> PMap;
    typedef TileMap<QOWN, RJ> QMap;
    __shared__ __attribute__((aligned(16))) uint8_t p0[PMap::kBytes];
    __shared__ __attribute__((aligned(16))) uint8_t q0[QMap::kBytes];
    __shared__ __attribute__((aligned(16))) uint8_t p1[PMap::kBytes];
    __shared__ __attribute__((aligned(16))) uint8_t q1[QMap::kBytes];
    __shared__ __attribute__((aligned(16))) uint8_t p2[S > 2 ? PMap::kBytes : 16];
    __shared__ __attribute__((aligned(16))) uint8_t q2[S > 2 ? QMap::kBytes : 16];
    __shared__ __attribute__((aligned(16))) uint8_t p3[S > 2 ? PMap::kBytes : 16];
    __shared__ __attribute__((aligned(16))) uint8_t q3[S > 2 ? QMap::kBytes : 16];
    auto p_stage = [&](auto i) KM_INLINE -> uint8_t * {
        constexpr int n = decltype(i)::value % S;
        return n == 0 ? p0 : n == 1 ? p1 : n == 2 ? p2 : p3;
    };
    auto q_stage = [&](auto i) KM_INLINE -> uint8_t * {
        constexpr int n = decltype(i)::value % S;
        return n == 0 ? q0 : n == 1 ? q1 : n == 2 ? q2 : q3;
    };

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ni = (g.I + RI - 1) / RI, nj = (g.J + RJ - 1) / RJ;
    int split, ti, tj;
    tile_of(g.first_wg + static_cast<int>(blockIdx.x), ni, nj, g.splits, split, ti, tj);
    const int i0 = ti * RI, j0 = tj * RJ;
    const int wi = (wave % WI) * TI * 16, wj = (wave / WI) * TJ * 16;
    const int64_t k0 = static_cast<int64_t>(split) * g.k_chunk;
    const int k_len = static_cast<int>(min(static_cast<int64_t>(g.k_chunk), g.K - k0));
    const int tiles = (k_len + kTileK - 1) / kTileK;

    Stager<T, POWN, RI, kThreads, DMA> ps;
    Stager<T, QOWN, RJ, kThreads, DMA> qs;
    ps.init(g.P, g.ldp, i0, g.I, k0, k_len, tid);
    qs.init(g.Q, g.ldq, j0, g.J, k0, k_len, tid);
    Reader<T, POWN, RI, TI> pr;
    Reader<T, QOWN, RJ, TJ> qr;
    pr.init(wi, lane);
    qr.init(wj, lane);

    f32x4 acc[TI][TJ];
#pragma unroll
    for (int a = 0; a < TI; ++a)
#pragma unroll
        for (int b = 0; b < TJ; ++b)
            acc[a][b] = f32x4{0, 0, 0, 0};
    Frag pf[2][HB], qf[2][TJ];

    auto read_phase = [&](const uint8_t *pst, const uint8_t *qst, int ph) KM_INLINE {
        const int s = ph / NH, h = ph % NH;
        if (h == 0) {
#pragma unroll
            for (int b = 0; b < TJ; ++b)
                qf[s][b] = qr.read(qst, b, s);
        }
#pragma unroll
        for (int a = 0; a < HB; ++a)
            pf[ph & 1][a] = pr.read(pst, h * HB + a, s);
    };
    auto multiply = [&](int ph) KM_INLINE {
        const int s = ph / NH, h = ph % NH;
#pragma unroll
        for (int a = 0; a < HB; ++a)
#pragma unroll
            for (int b = 0; b < TJ; ++b)
                acc[h * HB + a][b] = mfma(qf[s][b], pf[ph & 1][a], acc[h * HB + a][b]);
    };
    constexpr int kReads = (POWN ? 2 : 1) * HB + (QOWN ? 2 : 1) * TJ;
    constexpr int kCopies = decltype(ps)::kPieces + decltype(qs)::kPieces;
    // Tile t, in stage at % S.  FULL: tiles t + 1 .. t + S exist and t + S is a
    // whole one (without DMA: and none of the last cut_tiles()), so the step has
    // no branches (a branch around the copies would cost the compiler its
    // knowledge of which stage they write, and a wait before the next reads).
    auto step = [&](auto full, auto at, int t) KM_INLINE {
        constexpr bool FULL = decltype(full)::value;
        uint8_t *pc = p_stage(at), *qc = q_stage(at);
        uint8_t *pn = p_stage(Index<decltype(at)::value + 1>{});
        uint8_t *qn = q_stage(Index<decltype(at)::value + 1>{});
#pragma unroll
        for (int ph = 0; ph + 1 < NP; ++ph) {
            read_phase(pc, qc, ph + 1);
            multiply(ph);
            // Fragment reads one by one between the matrix instructions.
            const int reads = (POWN ? 2 : 1) * HB + ((ph + 1) % NH == 0 ? (QOWN ? 2 : 1) * TJ : 0);
#pragma unroll
            for (int r = 0; r < reads; ++r) {
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // one LDS read
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // one MFMA
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if (FULL || t + 1 < tiles) {
            ps.template commit<FULL>(t + 1, pn);
            qs.template commit<FULL>(t + 1, qn);
            if constexpr (DMA)
                wait_vmem<FULL ? (S - 2) * kCopies : 0>();
            lds_barrier();
            read_phase(pn, qn, 0);
            if (FULL || t + S < tiles) {
                ps.template issue<FULL>(t + S, pc);
                qs.template issue<FULL>(t + S, qc);
            }
        }
        multiply(NP - 1);
        if (FULL) {
#pragma unroll
            for (int r = 0; r < kCopies; ++r) {
                __builtin_amdgcn_sched_group_barrier(0x100, kReads / kCopies, 0);
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);   // one copy
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    auto start = [&](auto at) KM_INLINE {
        constexpr int n = decltype(at)::value;
        if (n < tiles) {
            ps.template issue<false>(n, p_stage(at));
            qs.template issue<false>(n, q_stage(at));
        }
    };

    start(Index<0>{});
    ps.template commit<false>(0, p0);
    qs.template commit<false>(0, q0);
    start(Index<1>{});
    if constexpr (S > 2) {
        start(Index<2>{});
        start(Index<3>{});
    }
    if constexpr (DMA) {
        // All stages were started: only the first need have landed.
        if (tiles >= S)
            wait_vmem<(S - 1) * kCopies>();
        else
            wait_vmem<0>();
    }
    lds_barrier();
    read_phase(p0, q0, 0);
    int t = 0;
    const int full = DMA ? k_len / kTileK : tiles - max(ps.cut_tiles(), qs.cut_tiles());
    for (; t + 2 * S - 1 < full; t += S) {
        step(std::true_type{}, Index<0>{}, t);
        step(std::true_type{}, Index<1>{}, t + 1);
        if constexpr (S > 2) {
            step(std::true_type{}, Index<2>{}, t + 2);
            step(std::true_type{}, Index<3>{}, t + 3);
        }
    }
    for (; t < tiles; t += S) {
        step(std::false_type{}, Index<0>{}, t);
        if (t + 1 < tiles)
            step(std::false_type{}, Index<1>{}, t + 1);
        if constexpr (S > 2) {
            if (t + 2 < tiles)
                step(std::false_type{}, Index<2>{}, t + 2);
            if (t + 3 < tiles)
                step(std::false_type{}, Index<3>{}, t + 3);
        }
    }

    const int l = lane & 15, g4 = lane >> 4;
    if (g.splits > 1) {
        float *part = g.partial + static_cast<int64_t>(split) * g.I * g.J;
#pragma unroll
        for (int a = 0; a < TI; ++a) {
            const int i = i0 + wi + a * 16 + l;
            if (i >= g.I)
                continue;
#pragma unroll
            for (int b = 0; b < TJ; ++b) {
                const int j = j0 + wj + b * 16 + g4 * 4;
                store_run<float, 4>(part + static_cast<int64_t>(i) * g.J + j, g.J - j,
                                    __builtin_bit_cast(Packed<float, 4>, acc[a][b]));
            }
        }
        return;
    }
    // The accumulators hold quads scattered over 16 rows.  Each wave passes
    // them, 64 rows at a time, through its own part of the first two stages
    // (rows of 16 TJ floats; chunk c of row r at a place that spreads both
    // sides' accesses over the banks) and takes them back as runs of eight
    // columns: a wave's loads and stores then cover whole rows, and the
    // epilogue's code exists once.
    constexpr int kRowFloats = TJ * 16;
    constexpr int kPass = 64 * kRowFloats * 4;          // bytes of one wave's pass
    constexpr int kPerArray = WI * WJ / 4;              // waves sharing one stage array
    static_assert((TJ == 4 || TJ == 2) && TI % 4 == 0, "64-row passes");
    static_assert(WI * WJ % 4 == 0 && kPerArray * kPass <= sizeof(p0) && sizeof(p0) == sizeof(q0),
                  "the first two stages hold a pass of every wave");
    auto spot = [](int r, int c) KM_INLINE {
        return r * kRowFloats * 4 + (c ^ (TJ == 4 ? r & 15 : (r >> 1) & 7)) * 16;
    };
    uint8_t *mine = wave / kPerArray == 0 ? p0 : wave / kPerArray == 1 ? p1
                  : wave / kPerArray == 2 ? q0 : q1;
    mine += (wave % kPerArray) * kPass;
    __syncthreads();
    constexpr int kRuns = TJ * 2;                       // runs of eight columns per row
    constexpr int kSteps = kRuns;                       // a wave's steps over 64 rows
    typedef typename T::bits B;
    const Epilogue &e = g.epi;
    const int c8 = lane % kRuns;
    const int j = j0 + wj + c8 * 8;
    const int n = g.J - j;                              // columns that exist
    const int i_first = i0 + wi + lane / kRuns;
    // A run that the right edge cuts short is left to one last step, in which
    // each lane finishes it for one row.
    const bool whole = n >= 8;
    const int cut = g.J % 8 == 0 ? -1 : (g.J / 8 * 8 - j0 - wj) / 8;     // run, uniform
    const bool has_cut = g.J % 8 != 0 && g.J / 8 * 8 >= j0 + wj && cut < kRuns;
    float bias[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (!QOWN && e.bias != nullptr && whole) {
        const Packed<B, 8> q = load_packed<B, 8>(static_cast<const B *>(e.bias) + j);
#pragma unroll
        for (int c = 0; c < 8; ++c)
            bias[c] = T::widen(q.v[c]);
    }
    auto take = [&](int r, int run, float (&v)[8]) KM_INLINE {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const f32x4 x = *reinterpret_cast<const f32x4 *>(mine + spot(r, 2 * run + h));
#pragma unroll
            for (int c = 0; c < 4; ++c)
                v[4 * h + c] = x[c];
        }
    };
    auto pass = [&](auto which) KM_INLINE {
        constexpr int half = decltype(which)::value;
        const int i_pass = i_first + half * 64;
        // All residual loads of the pass are in flight while the accumulators
        // go through LDS.
        Packed<B, 8> res[kSteps];
        if (!QOWN && e.residual != nullptr && whole) {
            const B *p = static_cast<const B *>(e.residual) + i_pass * e.ldr + j;
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                res[s] = Packed<B, 8>{};
                if (i_pass + s * (64 / kRuns) < g.I)
                    res[s] = load_packed<B, 8>(p + s * (64 / kRuns) * e.ldr);
            }
        }
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int b = 0; b < TJ; ++b)
                *reinterpret_cast<f32x4 *>(mine + spot(a * 16 + l, b * 4 + g4)) =
                    acc[half * 4 + a][b];
        // One wave writes and reads the region, in program order; the fence
        // keeps the compiler to it.
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        auto finish = [&](auto act, auto stream) KM_INLINE {
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const int i = i_pass + s * (64 / kRuns);
                float v[8];
                take(lane / kRuns + s * (64 / kRuns), c8, v);
                if (i >= g.I || !whole)
                    continue;
                if constexpr (!QOWN) {
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        v[c] += bias[c];
                    if (e.pre != nullptr)
                        store_packed(static_cast<B *>(e.pre) + i * e.ldp + j, narrow_run<T, 8>(v));
                    activate_run<decltype(act)::value>(v);
                    if (e.residual != nullptr) {
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            v[c] += T::widen(res[s].v[c]);
                    }
                }
                B *o = static_cast<B *>(e.out) + i * e.ldo + j;
                const Packed<B, 8> y = narrow_run<T, 8>(v);
                // Gradients of aligned rows go past the caches, which leaves
                // the operands there (65536 x 512 x 128: 56 us for both gradients,
                // 63 with plain stores); unaligned rows do not (100 x 8001 x
                // 8001 113 us, 137 past the caches), nor forward outputs (4096
                // x 4096 x 1000 37 us, 41 so).
                if constexpr (decltype(stream)::value)
                    __builtin_nontemporal_store(__builtin_bit_cast(u32x4_any, y),
                                                reinterpret_cast<u32x4_any *>(o));
                else
                    store_packed(o, y);
            }
        };
        if constexpr (QOWN) {
            if (DMA && e.ldo % 8 == 0)
                finish(Index<KMEANS_ACT_NONE>{}, std::bool_constant<DMA>{});
            else
                finish(Index<KMEANS_ACT_NONE>{}, std::false_type{});
        } else {
            switch (e.act) {
            case KMEANS_ACT_RELU: finish(Index<KMEANS_ACT_RELU>{}, std::false_type{}); break;
            case KMEANS_ACT_GELU: finish(Index<KMEANS_ACT_GELU>{}, std::false_type{}); break;
            case KMEANS_ACT_GELU_TANH: finish(Index<KMEANS_ACT_GELU_TANH>{}, std::false_type{}); break;
            case KMEANS_ACT_SILU: finish(Index<KMEANS_ACT_SILU>{}, std::false_type{}); break;
            default: finish(Index<KMEANS_ACT_NONE>{}, std::false_type{}); break;
            }
        }
        if (has_cut) {
            const int i = i0 + wi + half * 64 + lane;
            float v[8];
            take(lane, cut, v);
            if (i < g.I)
                finish_run<T, 8>(e, i, g.J / 8 * 8, g.J, v);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    };
    pass(Index<0>{});
    if constexpr (TI > 4)
        pass(Index<1>{});
    static_assert(TI <= 8, "two passes");
}

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

template <typename T>
__global__ __launch_bounds__(kBiasThreads)
void linear_bias_kernel(const BiasSums b) {
    sum_bias<T, kBiasThreads, kBiasCols>(b, blockIdx.x);
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

// Few rows: the weights are read once, straight into fragments, and that is
// the whole cost.  One workgroup takes 16 features and all (at most 16) rows;
// its WAVES waves split D between them in runs of kRowsStep values (each wave
// every WAVES-th run, so that together they read along the rows of W) and add
// their sums in LDS in wave order.  kRowsUnroll matrix instructions' operands
// are in flight per wave.  Loads are 16 bytes per lane at the rows' own
// alignment; the last values of a row that is no multiple of 8 are loaded one
// by one.  1 x 4096 x 4096: 7.9 us (33.6 MB, 4.2 TB/s: 256 workgroups of 16
// waves start and end together, which a stream this short feels).  Against the
// tile kernels, per call without an epilogue: 8.5 us instead of 11.5, 16 rows
// 9.3 instead of 11.6, but 32 rows (two row blocks) 12.9 instead of 12.7, so it
// stops at 16.
constexpr int kRowsUnroll = 4;
constexpr int kRowsStep = 32 * kRowsUnroll;
template <typename T, int WAVES>
__global__ __launch_bounds__(WAVES * 64)
void linear_rows_kernel(const Product g) {
    typedef typename T::bits B;
    typedef typename T::mfma Frag;
    __shared__ f32x4 sums[WAVES][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l = lane & 15, q = lane >> 4;
    const int j0 = blockIdx.x * 16;
    const B *w = static_cast<const B *>(g.Q) + min(j0 + l, g.J - 1) * g.ldq + q * 8;
    const B *x = static_cast<const B *>(g.P) + min(l, g.I - 1) * g.ldp + q * 8;
    f32x4 acc = {0, 0, 0, 0};
    int k = wave * kRowsStep;
    for (; k + kRowsStep <= g.K; k += WAVES * kRowsStep) {
        Packed<B, 8> wf[kRowsUnroll], xf[kRowsUnroll];
#pragma unroll
        for (int u = 0; u < kRowsUnroll; ++u)
            wf[u] = load_packed<B, 8>(w + k + u * 32);
#pragma unroll
        for (int u = 0; u < kRowsUnroll; ++u)
            xf[u] = load_packed<B, 8>(x + k + u * 32);
#pragma unroll
        for (int u = 0; u < kRowsUnroll; ++u)
            acc = mfma(__builtin_bit_cast(Frag, wf[u]), __builtin_bit_cast(Frag, xf[u]), acc);
    }
    // The one run that D cuts short, if it is this wave's.
    for (int e = min(g.K, k + kRowsStep); k < e; k += 32) {
        const int n = e - k - q * 8;
        acc = mfma(__builtin_bit_cast(Frag, load_run<B, 8>(w + k, n)),
                   __builtin_bit_cast(Frag, load_run<B, 8>(x + k, n)), acc);
    }
    sums[wave][lane] = acc;
    __syncthreads();
    // Four features of one row per lane: element c of lane (l, q) is feature
    // 4 q + c of row l.
    const int j = j0 + q * 4;
    if (tid >= 64 || l >= g.I || j >= g.J)
        return;
    f32x4 s = sums[0][lane];
#pragma unroll
    for (int v = 1; v < WAVES; ++v)
        s += sums[v][lane];
    float v[4] = {s[0], s[1], s[2], s[3]};
    finish_run<T, 4>(g.epi, l, j, g.J, v);
}

// ---- dZ and the bias gradient ----------------------------------------------

// dZ = dY * act'(Z), rounded once, rows ldz apart (a multiple of 8 elements,
// 16-byte aligned), and the column sums of the unrounded dZ over this
// workgroup's rows.  A lane owns eight columns; the workgroup's 256 lanes
// cover `lanes` groups of eight columns (a power of two) and 256 / lanes rows
// at a time, kDzRows of them in flight per lane.  The sums of the row groups
// meet in LDS in a fixed order.  dZ == null: the sums alone.  Without an
// activation and sums it lays rows out anew (Operand).  Bound by memory: 8192 x
// 4096 with silu 35 us (201 MB, 5.8 TB/s); the activation is chosen at compile
// time (20000 x 1111 with gelu: 12 us less for the call than by a branch per
// value).
template <typename T, int ACT>
__global__ __launch_bounds__(kDzThreads)
void linear_dz_kernel(const void *dY, int64_t ldy, const void *pre, int64_t ldp, int N, int F,
                      int lanes_log2, int rows_per_wg, void *dZ, int64_t ldz,
                      float *col_partial) {
    typedef typename T::bits B;
    __shared__ float sums[kDzThreads][9];
    const int tid = threadIdx.x;
    const int lanes = 1 << lanes_log2;
    const int groups = kDzThreads >> lanes_log2;
    const int c0 = (blockIdx.y * lanes + (tid & (lanes - 1))) * 8;
    const int r_first = blockIdx.x * rows_per_wg;
    const int r_end = min(N, r_first + rows_per_wg);
    const int n = F - c0;     // columns that exist (may be <= 0)
    float s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    // A lane whose columns the row's end cuts short loads the row's last eight
    // values and shifts out the first `back` (20000 x 77 x 1111 gradients 77 us,
    // 85 with its values loaded one by one).
    const int back = F >= 8 ? min(max(8 - n, 0), 8) : 0;
    auto shifted = [&](const Packed<B, 8> &q) KM_INLINE {
        typedef unsigned __int128 u128;
        return __builtin_bit_cast(Packed<B, 8>, __builtin_bit_cast(u128, q) >> (16 * back));
    };
    auto put = [&](int64_t r, Packed<B, 8> d, Packed<B, 8> z) KM_INLINE {
        if (back > 0) {
            d = shifted(d);
            if (ACT != KMEANS_ACT_NONE)
                z = shifted(z);
        }
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[e] = activate_grad(ACT, T::widen(z.v[e]), T::widen(d.v[e]));
            s[e] += v[e];
        }
        if (dZ != nullptr)    // the row's padding may be written
            *reinterpret_cast<u32x4 *>(static_cast<B *>(dZ) + r * ldz + c0) =
                __builtin_bit_cast(u32x4, narrow_run<T, 8>(v));
    };
    const B *y = static_cast<const B *>(dY) + c0 - back;
    const B *z = static_cast<const B *>(pre) + c0 - back;
    int r = r_first + (tid >> lanes_log2);
    if (n > 0 && F >= 8) {
        for (; r + (kDzRows - 1) * groups < r_end; r += kDzRows * groups) {
            Packed<B, 8> d[kDzRows], p[kDzRows];
#pragma unroll
            for (int u = 0; u < kDzRows; ++u) {
                d[u] = load_packed<B, 8>(y + (r + u * groups) * ldy);
                p[u] = Packed<B, 8>{};
            }
            if (ACT != KMEANS_ACT_NONE) {
#pragma unroll
                for (int u = 0; u < kDzRows; ++u)
                    p[u] = load_packed<B, 8>(z + (r + u * groups) * ldp);
            }
#pragma unroll
            for (int u = 0; u < kDzRows; ++u)
                put(r + u * groups, d[u], p[u]);
        }
    }
    if (n > 0)
        for (; r < r_end; r += groups) {
            Packed<B, 8> p = {};
            if (ACT != KMEANS_ACT_NONE)
                p = load_run<B, 8>(z + r * ldp, F);
            put(r, load_run<B, 8>(y + r * ldy, F), p);
        }
    if (col_partial == nullptr)
        return;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        sums[tid][e] = s[e];
    __syncthreads();
    for (int x = tid; x < lanes * 8; x += kDzThreads) {
        const int lane = x >> 3, e = x & 7;
        float v = 0.0f;
        for (int q = 0; q < groups; ++q)
            v += sums[q * lanes + lane][e];
        const int col = (blockIdx.y * lanes + lane) * 8 + e;
        if (col < F)
            col_partial[static_cast<int64_t>(blockIdx.x) * F + col] = v;
    }
}

// Zeroes rows of 16-bit values (dW and db of an empty batch, dX of no features).
__global__ __launch_bounds__(256)
void linear_zero_kernel(uint16_t *p, int64_t rows, int cols, int64_t ld) {
    const int64_t total = rows * cols;
    for (int64_t x = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; x < total;
         x += static_cast<int64_t>(gridDim.x) * 256)
        p[x / cols * ld + x % cols] = 0;
}

// ---- launch ----------------------------------------------------------------

template <typename T, int ACT>
hipError_t launch_dz(const RowPlan &r, const void *dY, int64_t ldy, const void *pre, int64_t ldp,
                     int N, int F, void *dZ, float *col_partial, hipStream_t stream) {
    hipLaunchKernelGGL((linear_dz_kernel<T, ACT>), dim3(r.row_wgs, r.col_wgs), dim3(kDzThreads), 0,
                       stream, dY, ldy, pre, ldp, N, F, r.lanes_log2, r.rows_per_wg, dZ, r.ld,
                       col_partial);
    return hipGetLastError();
}

// Lays the operand out anew if it was planned so, and points (p, ld) to it.
template <typename T>
hipError_t move_operand(const Operand &o, int compute_units, char *ws, const void *&p, int64_t &ld,
                        hipStream_t stream) {
    if (!o.moved)
        return hipSuccess;
    const RowPlan r(o.rows, o.cols, compute_units);
    p = ws + o.at;
    ld = r.ld;
    return launch_dz<T, KMEANS_ACT_NONE>(r, o.p, o.ld, nullptr, 0, static_cast<int>(o.rows),
                                         static_cast<int>(o.cols), ws + o.at, nullptr, stream);
}

template <typename T, bool POWN, bool QOWN>
hipError_t launch_product_modes(const Product &product, const BiasSums &bias, hipStream_t stream) {
    // A launch has less than 2^32 threads: products of more tiles take several.
    constexpr int64_t kMaxGrid = int64_t(1) << 22;
    Product g = product;
    const int64_t tiles = tiles_of(g, g.shape == kWide ? 256 : 128) * g.splits;
    hipError_t e = hipSuccess;
    for (int64_t first = 0; first < tiles && e == hipSuccess; first += kMaxGrid) {
        g.first_wg = static_cast<int>(first);
        const dim3 grid(static_cast<unsigned>(std::min(tiles - first, kMaxGrid)));
        switch (g.shape) {
        case kWide:
            hipLaunchKernelGGL((linear_tile_kernel<T, POWN, QOWN, 2, 4, 8, 4, 2, true>), grid,
                               dim3(512), 0, stream, g);
            break;
        case kDeep:
            hipLaunchKernelGGL((linear_tile_kernel<T, POWN, QOWN, 2, 4, 4, 2, 4, true>), grid,
                               dim3(512), 0, stream, g);
            break;
        case kPaired:
            hipLaunchKernelGGL((linear_tile_kernel<T, POWN, QOWN, 2, 2, 4, 4, 2, true>), grid,
                               dim3(256), 0, stream, g);
            break;
        default:
            hipLaunchKernelGGL((linear_tile_kernel<T, POWN, QOWN, 2, 4, 4, 2, 2, false>), grid,
                               dim3(512), 0, stream, g);
            break;
        }
        e = hipGetLastError();
    }
    if (e == hipSuccess && g.splits > 1) {
        const int64_t runs = static_cast<int64_t>(g.I) * ((g.J + 3) / 4);
        const int wgs = static_cast<int>(
            std::min<int64_t>((runs + kJoinRuns - 1) / kJoinRuns, 4096));
        const int bias_wgs =
            bias.col_partial != nullptr ? (bias.F + kJoinBiasCols - 1) / kJoinBiasCols : 0;
        hipLaunchKernelGGL((linear_join_kernel<T>), dim3(wgs + bias_wgs), dim3(kJoinThreads), 0,
                           stream, g, wgs, bias);
        e = hipGetLastError();
    }
    return e;
}

enum Modes { kForward, kInputGrad, kWeightGrad };

// `bias` is for the joining launch of a split product.
template <typename T>
hipError_t launch_product(const Product &g, Modes m, const BiasSums &bias, hipStream_t stream) {
    switch (m) {
    case kForward:
        return launch_product_modes<T, false, false>(g, bias, stream);
    case kInputGrad:
        return launch_product_modes<T, false, true>(g, bias, stream);
    default:
        return launch_product_modes<T, true, true>(g, bias, stream);
    }
}

kmeans_status_t check_linear(int64_t N, int64_t D, int64_t F, int32_t dtype, int32_t activation) {
    if (N < 0 || D < 1 || F < 1)
        return fail(KMEANS_ERR_INVALID_ARG, "N=%lld must be >= 0, D=%lld and F=%lld >= 1",
                    static_cast<long long>(N), static_cast<long long>(D),
                    static_cast<long long>(F));
    if (activation < KMEANS_ACT_NONE || activation > KMEANS_ACT_SILU)
        return fail(KMEANS_ERR_INVALID_ARG, "activation=%d is not a kmeans_activation_t",
                    activation);
    if (dtype != KMEANS_BF16 && dtype != KMEANS_FP16)
        return dtype == KMEANS_FP32
                   ? fail(KMEANS_ERR_UNSUPPORTED, "fp32 is not supported: bf16 or fp16")
                   : fail(KMEANS_ERR_INVALID_ARG, "dtype=%d is not a kmeans_dtype_t", dtype);
    if (N > kMaxRows || D > kMaxWidth || F > kMaxWidth)
        return fail(KMEANS_ERR_UNSUPPORTED, "N=%lld, D=%lld or F=%lld too large (max %lld, "
                    "%lld, %lld)", static_cast<long long>(N), static_cast<long long>(D),
                    static_cast<long long>(F), static_cast<long long>(kMaxRows),
                    static_cast<long long>(kMaxWidth), static_cast<long long>(kMaxWidth));
    return KMEANS_OK;
}

// A matrix argument of 16-bit values: rows of `cols`, `ld` apart.
kmeans_status_t check_rows(const char *name, const void *p, int64_t cols, int64_t ld) {
    if (p == nullptr)
        return fail(KMEANS_ERR_INVALID_ARG, "null pointer argument (%s)", name);
    if (!aligned(p, 2))
        return fail(KMEANS_ERR_ALIGNMENT, "%s must be 2-byte aligned", name);
    if (ld < cols)
        return fail(KMEANS_ERR_INVALID_ARG, "%s: row stride %lld below the row length %lld", name,
                    static_cast<long long>(ld), static_cast<long long>(cols));
    if (ld > kMaxWidth)
        return fail(KMEANS_ERR_UNSUPPORTED, "%s: row stride %lld too large (max %lld)", name,
                    static_cast<long long>(ld), static_cast<long long>(kMaxWidth));
    return KMEANS_OK;
}

kmeans_status_t check_vector(const char *name, const void *p) {
    if (!aligned(p, 2))
        return fail(KMEANS_ERR_ALIGNMENT, "%s must be 2-byte aligned", name);
    return KMEANS_OK;
}

template <typename T>
hipError_t run_forward(Product g, const Operand &x, const Operand &w, int compute_units, char *ws,
                       hipStream_t stream) {
    if (g.shape != kRows) {
        hipError_t e = move_operand<T>(x, compute_units, ws, g.P, g.ldp, stream);
        if (e == hipSuccess)
            e = move_operand<T>(w, compute_units, ws, g.Q, g.ldq, stream);
        return e == hipSuccess ? launch_product<T>(g, kForward, BiasSums{}, stream) : e;
    }
    // As many waves as D gives work to, while the CUs hold them (32 each).
    const dim3 grid((g.J + 15) / 16);
    int64_t waves = 4;
    while (waves < 16 && waves * kRowsStep < g.K && grid.x * waves * 2 <= 16 * compute_units)
        waves *= 2;
    if (waves == 16)
        hipLaunchKernelGGL((linear_rows_kernel<T, 16>), grid, dim3(1024), 0, stream, g);
    else if (waves == 8)
        hipLaunchKernelGGL((linear_rows_kernel<T, 8>), grid, dim3(512), 0, stream, g);
    else
        hipLaunchKernelGGL((linear_rows_kernel<T, 4>), grid, dim3(256), 0, stream, g);
    return hipGetLastError();
}

// The launches of kmeans_linear_grad on workspace `ws`.
struct GradPlan {
    bool dz;                    // whether dZ is written (else dY stands for it)
    RowPlan rows;
    size_t dz_at, col_at, part_at, bytes;
    Operand x, w;
    Product dx, dw;
};

template <typename T>
hipError_t run_grad(GradPlan &p, int compute_units, const void *dY, int64_t dy_stride, const void *pre,
                    int64_t pre_stride, int N, int F, int act, bool want_dx, bool want_dw,
                    void *dbias, char *ws, hipStream_t stream) {
    hipError_t e = hipSuccess;
    if (p.dz || dbias != nullptr) {
        auto launch = [&](auto kind) {
            return launch_dz<T, decltype(kind)::value>(
                p.rows, dY, dy_stride, pre, pre_stride, N, F, p.dz ? ws + p.dz_at : nullptr,
                dbias != nullptr ? reinterpret_cast<float *>(ws + p.col_at) : nullptr, stream);
        };
        switch (act) {
        case KMEANS_ACT_RELU: e = launch(Index<KMEANS_ACT_RELU>{}); break;
        case KMEANS_ACT_GELU: e = launch(Index<KMEANS_ACT_GELU>{}); break;
        case KMEANS_ACT_GELU_TANH: e = launch(Index<KMEANS_ACT_GELU_TANH>{}); break;
        case KMEANS_ACT_SILU: e = launch(Index<KMEANS_ACT_SILU>{}); break;
        default: e = launch(Index<KMEANS_ACT_NONE>{}); break;
        }
    }
    // The bias sums go with a product's join if there is one.
    BiasSums bias{}, with_dx{}, with_dw{};
    if (dbias != nullptr)
        bias = {reinterpret_cast<const float *>(ws + p.col_at), p.rows.row_wgs, F, dbias};
    if (want_dw && p.dw.splits > 1) {
        std::swap(bias, with_dw);
    } else if (want_dx && p.dx.splits > 1) {
        std::swap(bias, with_dx);
    }
    if (e == hipSuccess && bias.col_partial != nullptr) {
        hipLaunchKernelGGL((linear_bias_kernel<T>), dim3((F + kBiasCols - 1) / kBiasCols),
                           dim3(kBiasThreads), 0, stream, bias);
        e = hipGetLastError();
    }
    if (e == hipSuccess)
        e = move_operand<T>(p.w, compute_units, ws, p.dx.Q, p.dx.ldq, stream);
    if (e == hipSuccess)
        e = move_operand<T>(p.x, compute_units, ws, p.dw.Q, p.dw.ldq, stream);
    if (e == hipSuccess && want_dx)
        e = launch_product<T>(p.dx, kInputGrad, with_dx, stream);
    if (e == hipSuccess && want_dw)
        e = launch_product<T>(p.dw, kWeightGrad, with_dw, stream);
    return e;
}

hipError_t zero_rows(void *p, int64_t rows, int64_t cols, int64_t ld, hipStream_t stream) {
    if (p == nullptr)
        return hipSuccess;
    const unsigned wgs = static_cast<unsigned>(std::min<int64_t>((rows * cols + 255) / 256, 8192));
    hipLaunchKernelGGL(linear_zero_kernel, dim3(wgs), dim3(256), 0, stream,
                       static_cast<uint16_t *>(p), rows, static_cast<int>(cols), ld);
    return hipGetLastError();
}

}  // namespace
}  // namespace kmeans

// ---- C entry points --------------------------------------------------------

extern "C" kmeans_status_t kmeans_linear(const void *X, int64_t x_stride, const void *W,
                                         int64_t w_stride, const void *bias, const void *residual,
                                         int64_t residual_stride, int64_t N, int64_t D, int64_t F,
                                         int32_t dtype, int32_t activation, void *Y,
                                         int64_t y_stride, void *pre, int64_t pre_stride,
                                         hipStream_t stream) {
    using namespace kmeans;
    kmeans_status_t st = check_linear(N, D, F, dtype, activation);
    if (st != KMEANS_OK)
        return st;
    if (N == 0)
        return ok();
    if ((st = check_rows("X", X, D, x_stride)) != KMEANS_OK ||
        (st = check_rows("W", W, D, w_stride)) != KMEANS_OK ||
        (st = check_rows("Y", Y, F, y_stride)) != KMEANS_OK ||
        (st = check_vector("bias", bias)) != KMEANS_OK ||
        (residual && (st = check_rows("residual", residual, F, residual_stride)) != KMEANS_OK) ||
        (pre && (st = check_rows("pre", pre, F, pre_stride)) != KMEANS_OK))
        return st;

    const int cus = device_compute_units();
    Operand x{X, x_stride, N, D, false, 0}, w{W, w_stride, F, D, false, 0};
    size_t bytes = 0;
    Product g = forward_product(x, w, cus, bytes);
    g.epi = {bias, residual, residual_stride, Y, y_stride, pre, pre_stride, activation};
    if (tiles_of(g, 128) > kMaxRows / kMaxKSplits)
        return fail(KMEANS_ERR_UNSUPPORTED, "N=%lld x F=%lld: too many outputs",
                    static_cast<long long>(N), static_cast<long long>(F));
    const size_t part_at = bytes;
    bytes += partial_bytes(g);
    std::optional<WorkspaceLease> lease;
    char *ws = nullptr;
    if (bytes > 0) {
        lease.emplace(stream, bytes);
        if (lease->error() != hipSuccess)
            return fail(KMEANS_ERR_NO_MEMORY, "workspace of %zu bytes: %s", bytes,
                        hipGetErrorString(lease->error()));
        ws = static_cast<char *>(lease->ptr());
        g.partial = reinterpret_cast<float *>(ws + part_at);
    }
    const hipError_t e = dtype == KMEANS_BF16 ? run_forward<Bf16>(g, x, w, cus, ws, stream)
                                              : run_forward<Fp16>(g, x, w, cus, ws, stream);
    if (e != hipSuccess)
        return fail(KMEANS_ERR_HIP, "linear launch failed: %s", hipGetErrorString(e));
    return ok();
}

extern "C" kmeans_status_t kmeans_linear_grad(const void *dY, int64_t dy_stride, const void *X,
                                              int64_t x_stride, const void *W, int64_t w_stride,
                                              const void *pre, int64_t pre_stride, int64_t N,
                                              int64_t D, int64_t F, int32_t dtype,
                                              int32_t activation, void *dX, int64_t dx_stride,
                                              void *dW, int64_t dw_stride, void *dbias,
                                              hipStream_t stream) {
    using namespace kmeans;
    kmeans_status_t st = check_linear(N, D, F, dtype, activation);
    if (st != KMEANS_OK)
        return st;
    if ((dW && (st = check_rows("dW", dW, D, dw_stride)) != KMEANS_OK) ||
        (st = check_vector("dbias", dbias)) != KMEANS_OK)
        return st;
    if (N == 0) {
        hipError_t e = zero_rows(dW, F, D, dw_stride, stream);
        if (e == hipSuccess)
            e = zero_rows(dbias, 1, F, F, stream);
        if (e != hipSuccess)
            return fail(KMEANS_ERR_HIP, "linear gradient launch failed: %s", hipGetErrorString(e));
        return ok();
    }
    if ((st = check_rows("dY", dY, F, dy_stride)) != KMEANS_OK ||
        (dW && (st = check_rows("X", X, D, x_stride)) != KMEANS_OK) ||
        (dX && (st = check_rows("W", W, D, w_stride)) != KMEANS_OK) ||
        (dX && (st = check_rows("dX", dX, D, dx_stride)) != KMEANS_OK) ||
        (activation != KMEANS_ACT_NONE && (st = check_rows("pre", pre, F, pre_stride)) != KMEANS_OK))
        return st;
    if (!dX && !dW && !dbias)
        return ok();

    const int cus = device_compute_units();
    GradPlan p{false, RowPlan(N, F, cus), 0, 0, 0, 0, {X, x_stride, N, D, false, 0},
               {W, w_stride, F, D, false, 0}, {}, {}};
    // dZ is dY itself without an activation, where its rows can be staged as
    // they lie; otherwise it is written once with rows of whole chunks.
    p.dz = (dX || dW) &&
           (activation != KMEANS_ACT_NONE || !rows_aligned(dY, dy_stride) || F % 8 != 0);

    const void *z = dY;
    int64_t ldz = dy_stride;
    size_t at = 0;
    if (p.dz) {
        p.dz_at = at;
        at += p.rows.bytes(N);
    }
    if (dbias) {
        p.col_at = at;
        at += align_up(static_cast<size_t>(p.rows.row_wgs) * F * sizeof(float));
    }
    // dZ fits the copies (zeros past F in its last chunk); X and W may not.
    size_t part = 0;
    if (dX) {
        p.dx = input_grad_product(N, p.w, cus, at);
        p.dx.epi = {nullptr, nullptr, 0, dX, dx_stride, nullptr, 0, KMEANS_ACT_NONE};
        part = std::max(part, partial_bytes(p.dx));
    }
    if (dW) {
        p.dw = weight_grad_product(F, p.x, cus, at);
        p.dw.epi = {nullptr, nullptr, 0, dW, dw_stride, nullptr, 0, KMEANS_ACT_NONE};
        part = std::max(part, partial_bytes(p.dw));
    }
    if ((dX && tiles_of(p.dx, 128) > kMaxRows / kMaxKSplits) ||
        (dW && tiles_of(p.dw, 128) > kMaxRows / kMaxKSplits))
        return fail(KMEANS_ERR_UNSUPPORTED, "N=%lld x D=%lld: too many outputs",
                    static_cast<long long>(N), static_cast<long long>(D));
    p.part_at = at;
    p.bytes = at + part;
    std::optional<WorkspaceLease> lease;
    char *ws = nullptr;
    if (p.bytes > 0) {
        lease.emplace(stream, p.bytes);
        if (lease->error() != hipSuccess)
            return fail(KMEANS_ERR_NO_MEMORY, "workspace of %zu bytes: %s", p.bytes,
                        hipGetErrorString(lease->error()));
        ws = static_cast<char *>(lease->ptr());
    }
    if (p.dz) {
        z = ws + p.dz_at;
        ldz = p.rows.ld;
    }
    p.dx.P = p.dw.P = z;
    p.dx.ldp = p.dw.ldp = ldz;
    p.dx.partial = p.dw.partial = reinterpret_cast<float *>(ws + p.part_at);
    const hipError_t e =
        dtype == KMEANS_BF16
            ? run_grad<Bf16>(p, cus, dY, dy_stride, pre, pre_stride, static_cast<int>(N),
                             static_cast<int>(F), activation, dX != nullptr, dW != nullptr, dbias,
                             ws, stream)
            : run_grad<Fp16>(p, cus, dY, dy_stride, pre, pre_stride, static_cast<int>(N),
                             static_cast<int>(F), activation, dX != nullptr, dW != nullptr, dbias,
                             ws, stream);
    if (e != hipSuccess)
        return fail(KMEANS_ERR_HIP, "linear gradient launch failed: %s", hipGetErrorString(e));
    return ok();
}
