// kmeans_linear_fp8.hip -- gfx950 kernels of the linear layer on 8-bit operands
// (e4m3) with a scale for each block of 128 columns (of one row of X, of 128
// rows of W):
//
//     Z[i][j] = sum over blocks b of  sx[i][b] sw[j / 128][b]
//                                     (sum over k in b of X[i][k] W[j][k])
//     Y = act(Z + bias) + residual
//
// One 16x16x128 matrix instruction multiplies one block: its fp32 result is
// scaled and added to the sum in fp32, so that no scale is rounded.  The tile of
// 128 columns by R rows that the 16-bit product stages as 64 columns has the
// same bytes here, so staging, fragments, tile order and epilogue are its own
// (kmeans_linear_tile.h), the operands addressed as 16-bit values, two to one.
// Within a block any order of k will do that is the same on both operands, so a
// lane's two 16-byte fragments of a row need not be neighbours.
#include <stdint.h>

#include <algorithm>
#include <optional>

#include "kmeans_fp8.h"
#include "kmeans_internal.h"
#include "kmeans_linear_plan.h"
#include "kmeans_linear_tile.h"
#include "kmeans_types.h"

namespace kmeans {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4_bytes __attribute__((ext_vector_type(4), aligned(1)));

struct Scales {
    const float *x, *w;      // [I][blocks], [J / 128][blocks]
    int64_t ldx, ldw;
    int blocks_j;            // rows of w
};

struct Halves {
    u32x4 lo, hi;
};

// The products of one block of k, unscaled.  The 8-bit matrix instruction adds
// its products in groups of eight neighbouring columns, each cut (towards zero) to a
// multiple of 2^-13 of the largest power of two in the group's largest, and the
// groups in fp32 (measured: 1.4e-5 of a random block's norm; bf16 rounds the result
// by 1.7e-3, fp16 by 2.1e-4).
__device__ __forceinline__ f32x4 mfma_block(const Halves &a, const Halves &b) {
#if defined(__HIP_DEVICE_COMPILE__)
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
        __builtin_bit_cast(i32x8, a), __builtin_bit_cast(i32x8, b), f32x4{0, 0, 0, 0}, 0, 0, 0, 0, 0,
        0);
#else
    return f32x4{};
#endif
}

// The same with full fp32 sums, at half the rate: e4m3 values are bf16 values,
// whose matrix instruction keeps every bit of a product (4e-8 of the magnitudes
// in sums of 128).  For fp32 outputs, and where memory bounds the product (64 rows x
// 4096 x 65536 75 us, 512 rows 257, 4096 rows 1900, 1160 TFLOP/s).
struct Widened {
    Bf16::mfma v[4];
};
__device__ __forceinline__ Widened widen_block(const Halves &h) {
    Widened out{};
#if defined(__HIP_DEVICE_COMPILE__)
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const i32x8 x = __builtin_bit_cast(i32x8, h);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        struct { bf16x2 p[4]; } w;
        w.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[2 * q], 1.0f, false);
        w.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[2 * q], 1.0f, true);
        w.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[2 * q + 1], 1.0f, false);
        w.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[2 * q + 1], 1.0f, true);
        out.v[q] = __builtin_bit_cast(Bf16::mfma, w);
    }
#endif
    return out;
}
__device__ __forceinline__ f32x4 mfma_block(const Widened &a, const Widened &b) {
    f32x4 c = {0, 0, 0, 0};
#pragma unroll
    for (int q = 0; q < 4; ++q)
        c = mfma(a.v[q], b.v[q], c);
    return c;
}

// One workgroup of WI x WJ waves computes a tile of (WI 16 TI) x (WJ 16 TJ)
// outputs over one split of k, in S stages, as linear_tile_kernel does.  A
// staged tile is one block of k: its scales come with it, one copy of 64 values
// to a wave (first the rows of X in the order in which lanes need them, then the
// columns).  A tile is worked in phases of one P block against all TJ Q blocks; a
// phase's P fragment is read one phase ahead.  A product is scaled and added two
// products after its own, so that no instruction waits for the matrix pipe.
//
// 8192 x 8192 x 8192 467 to 500 us by device (2200 to 2350 TFLOP/s; the library's
// product with one scale each 2660), 16384 x 4096 x 4096 250 to 270 us (2040 to 2200;
// 2430).  What is left there: the first copies of each of four rounds, and the output.
// With tanh-gelu, bias and residual 305 to 327 us: with one workgroup per CU nothing
// hides the residual's 134 MB and the output's (both passes' residual loads ahead of
// the first spill: 352).  128 x 128 tiles in pairs hide them, but read LDS twice as often: 364.
template <typename T, int WI, int WJ, int TI, int TJ, int S>
__global__ __launch_bounds__(WI * WJ * 64, 2)
void linear_fp8_kernel(const Product g, const Scales sc) {
    constexpr bool EXACT = sizeof(typename T::bits) == 4;
    constexpr int kThreads = WI * WJ * 64;
    constexpr int RI = WI * TI * 16, RJ = WJ * TJ * 16;
    static_assert(RI + RJ <= kThreads, "one copy of scales to a wave");
    typedef Bf16 Pair;                        // two 8-bit values
    typedef TileMap<false, RI> PMap;
    typedef TileMap<false, RJ> QMap;
    constexpr int kScaleBytes = kThreads * 4;
    __shared__ __attribute__((aligned(16))) uint8_t p0[PMap::kBytes];
    __shared__ __attribute__((aligned(16))) uint8_t q0[QMap::kBytes];
    __shared__ __attribute__((aligned(16))) uint8_t p1[PMap::kBytes];
    __shared__ __attribute__((aligned(16))) uint8_t q1[QMap::kBytes];
    __shared__ __attribute__((aligned(16))) uint8_t p2[S > 2 ? PMap::kBytes : 16];
    __shared__ __attribute__((aligned(16))) uint8_t q2[S > 2 ? QMap::kBytes : 16];
    __shared__ __attribute__((aligned(16))) uint8_t p3[S > 2 ? PMap::kBytes : 16];
    __shared__ __attribute__((aligned(16))) uint8_t q3[S > 2 ? QMap::kBytes : 16];
    __shared__ __attribute__((aligned(16))) uint8_t s0[kScaleBytes];
    __shared__ __attribute__((aligned(16))) uint8_t s1[kScaleBytes];
    __shared__ __attribute__((aligned(16))) uint8_t s2[S > 2 ? kScaleBytes : 16];
    __shared__ __attribute__((aligned(16))) uint8_t s3[S > 2 ? kScaleBytes : 16];
    // Stages by number: one known at compile time, so that the compiler can tell an
    // LDS read of one stage from a copy into another.
    auto p_stage = [&](int i) KM_INLINE -> uint8_t * {
        const int n = i % S;
        return n == 0 ? p0 : n == 1 ? p1 : n == 2 ? p2 : p3;
    };
    auto q_stage = [&](int i) KM_INLINE -> uint8_t * {
        const int n = i % S;
        return n == 0 ? q0 : n == 1 ? q1 : n == 2 ? q2 : q3;
    };
    auto s_stage = [&](int i) KM_INLINE -> uint8_t * {
        const int n = i % S;
        return n == 0 ? s0 : n == 1 ? s1 : n == 2 ? s2 : s3;
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
    const int l = lane & 15, g4 = lane >> 4;

    Stager<Pair, false, RI, kThreads, true> ps;
    Stager<Pair, false, RJ, kThreads, true> qs;
    ps.init(g.P, g.ldp, i0, g.I, k0, k_len, tid);
    qs.init(g.Q, g.ldq, j0, g.J, k0, k_len, tid);
    Reader<Pair, false, RI, TI> pr;
    Reader<Pair, false, RJ, TJ> qr;
    pr.init(wi, lane);
    qr.init(wj, lane);

    // This thread's scale: place tid < RI is row (tid / (16 TI)) 16 TI + a 16 + l
    // with a = tid % TI, so that a lane's TI scales lie together; the next RJ are
    // the columns'; what is left repeats the last.
    [[maybe_unused]] const float *scale_base;
    [[maybe_unused]] uint32_t scale_off;
    if (wave < RI / 64) {
        const int in = tid % (16 * TI);
        const int r = tid - in + in % TI * 16 + in / TI;
        scale_base = sc.x + i0 * sc.ldx;
        scale_off = static_cast<uint32_t>(min(r, g.I - 1 - i0) * sc.ldx) * 4u;
    } else {
        const int c = min(tid - RI, RJ - 1);
        scale_base = sc.w + (j0 / kFp8Block) * sc.ldw;
        scale_off = static_cast<uint32_t>(
                        min(c / kFp8Block, sc.blocks_j - 1 - j0 / kFp8Block) * sc.ldw) * 4u;
    }
    scale_base += k0 / kTileK;
    auto issue_scales = [&](int t, uint8_t *stage) KM_INLINE {
#if defined(__HIP_DEVICE_COMPILE__)
        const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<float *>(scale_base + t), 0, 0x7fffffff, 0x00020000);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (KM_LDS void *)(stage + wave * 256), 4,
                                                 t < tiles ? scale_off : kOutOfRange, 0, 0, 0);
#endif
    };

    f32x4 acc[TI][TJ];
#pragma unroll
    for (int a = 0; a < TI; ++a)
#pragma unroll
        for (int b = 0; b < TJ; ++b)
            acc[a][b] = f32x4{0, 0, 0, 0};
    Halves pf[2], qf[TJ];
    float scale[TI];

    auto read_p = [&](const uint8_t *pst, int a) KM_INLINE {
        pf[a & 1].lo = __builtin_bit_cast(u32x4, pr.read(pst, a, 0));
        pf[a & 1].hi = __builtin_bit_cast(u32x4, pr.read(pst, a, 1));
    };
    auto read_q = [&](const uint8_t *qst, int b) KM_INLINE {
        qf[b].lo = __builtin_bit_cast(u32x4, qr.read(qst, b, 0));
        qf[b].hi = __builtin_bit_cast(u32x4, qr.read(qst, b, 1));
    };
    auto read_scales = [&](const uint8_t *sst) KM_INLINE {
        const float w = *reinterpret_cast<const float *>(sst + (RI + wj) * 4);
#pragma unroll
        for (int a = 0; a < TI; a += 4) {
            const f32x4 x = *reinterpret_cast<const f32x4 *>(sst + (wi + l * TI + a) * 4);
#pragma unroll
            for (int c = 0; c < 4; ++c)
                scale[a + c] = x[c] * w;
        }
    };
    // Product n of the tile (block n / TJ of P with block n % TJ of Q), and the
    // sum that the one before the last goes to.
    f32x4 made[3];
    auto add = [&](int n) KM_INLINE {
#pragma unroll
        for (int c = 0; c < 4; ++c)
            acc[n / TJ][n % TJ][c] = fmaf(made[n % 3][c], scale[n / TJ], acc[n / TJ][n % TJ][c]);
    };
    auto multiply = [&](int n) KM_INLINE {
        if constexpr (EXACT)
            made[n % 3] = mfma_block(widen_block(qf[n % TJ]), widen_block(pf[n / TJ & 1]));
        else
            made[n % 3] = mfma_block(qf[n % TJ], pf[n / TJ & 1]);
        __builtin_amdgcn_sched_barrier(0);
        if (n >= 2)
            add(n - 2);
    };
    constexpr int kCopies = decltype(ps)::kPieces + decltype(qs)::kPieces + 1;
    // Tile t's copies.  What lies past the range of k is copied as zeros, whole
    // tiles behind the last one too: the loop below needs no other form for its
    // end (which would cost it registers: with one, 16384 x 4096 x 4096 took 408
    // us).
    auto issue_piece = [&](auto &st, int u, int t, uint8_t *stage) KM_INLINE {
#if defined(__HIP_DEVICE_COMPILE__)
        typedef std::remove_reference_t<decltype(st)> Stage;
        const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<typename Pair::bits *>(st.base + static_cast<int64_t>(t) * kTileK), 0,
            0x7fffffff, 0x00020000);
        int r, c;
        st.piece(u, r, c);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rs, (KM_LDS void *)(stage + wave * (Stage::kPieces * 1024) + u * 1024), 16,
            c * 8 < k_len - t * kTileK ? st.off[u] : kOutOfRange, 0, 0, 0);
#endif
    };
    // Copy i of kCopies.
    auto issue_copy = [&](int i, int t, int at) KM_INLINE {
        constexpr int kP = decltype(ps)::kPieces, kQ = decltype(qs)::kPieces;
        if (i < kP)
            issue_piece(ps, i, t, p_stage(at));
        else if (i < kP + kQ)
            issue_piece(qs, i - kP, t, q_stage(at));
        else
            issue_scales(t, s_stage(at));
    };
    // Tile t, in stage at % S.
    auto step = [&](auto at, int t) KM_INLINE {
#pragma unroll
        for (int a = 0; a + 1 < TI; ++a) {
            read_p(p_stage(at), a + 1);
#pragma unroll
            for (int b = 0; b < TJ; ++b)
                multiply(a * TJ + b);
        }
        wait_vmem<(S - 2) * kCopies>();
        lds_barrier();
        // A Q fragment is read again as soon as its last product is on its way,
        // and the copies of tile t + S go between the products too.
#pragma unroll
        for (int b = 0; b < TJ; ++b) {
            multiply((TI - 1) * TJ + b);
            read_q(q_stage(at + 1), b);
            if (b == 0)
                read_p(p_stage(at + 1), 0);
#pragma unroll
            for (int i = b * kCopies / TJ; i < (b + 1) * kCopies / TJ; ++i)
                issue_copy(i, t + S, at);
        }
        add(TI * TJ - 2);
        add(TI * TJ - 1);
        read_scales(s_stage(at + 1));
        __builtin_amdgcn_sched_barrier(0);
    };

#pragma unroll
    for (int t = 0; t < S; ++t)
#pragma unroll
        for (int i = 0; i < kCopies; ++i)
            issue_copy(i, t, t);
    wait_vmem<(S - 1) * kCopies>();       // the first tile has landed
    lds_barrier();
    read_p(p0, 0);
#pragma unroll
    for (int b = 0; b < TJ; ++b)
        read_q(q0, b);
    read_scales(s0);
    int t = 0;
#pragma unroll 1
    for (; t + S <= tiles; t += S) {
        step(Index<0>{}, t);
        step(Index<1>{}, t + 1);
        if constexpr (S > 2) {
            step(Index<2>{}, t + 2);
            step(Index<3>{}, t + 3);
        }
    }
    if (t < tiles)
        step(Index<0>{}, t);
    if constexpr (S > 2) {
        if (t + 1 < tiles)
            step(Index<1>{}, t + 1);
        if (t + 2 < tiles)
            step(Index<2>{}, t + 2);
    }
    wait_vmem<0>();                       // of the zeros, before the stages are used again

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
    // The epilogue as in linear_tile_kernel: the accumulators go through the
    // first two stages, 64 rows at a time, and come back as runs of eight
    // columns of one row.
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
    const bool whole = g.J - j >= 8;
    const int i_first = i0 + wi + lane / kRuns;
    // A run that the right edge cuts short is left to one last step, in which
    // each lane finishes it for one row.
    const int cut = g.J % 8 == 0 ? -1 : (g.J / 8 * 8 - j0 - wj) / 8;     // run, uniform
    const bool has_cut = g.J % 8 != 0 && g.J / 8 * 8 >= j0 + wj && cut < kRuns;
    float bias[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (e.bias != nullptr && whole) {
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
        if (e.residual != nullptr && whole) {
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
        auto finish = [&](auto act) KM_INLINE {
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const int i = i_pass + s * (64 / kRuns);
                float v[8];
                take(lane / kRuns + s * (64 / kRuns), c8, v);
                if (i >= g.I || !whole)
                    continue;
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    v[c] += bias[c];
                activate_run<decltype(act)::value>(v);
                if (e.residual != nullptr) {
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        v[c] += T::widen(res[s].v[c]);
                }
                store_packed(static_cast<B *>(e.out) + i * e.ldo + j, narrow_run<T, 8>(v));
            }
        };
        switch (e.act) {
        case KMEANS_ACT_RELU: finish(Index<KMEANS_ACT_RELU>{}); break;
        case KMEANS_ACT_GELU: finish(Index<KMEANS_ACT_GELU>{}); break;
        case KMEANS_ACT_GELU_TANH: finish(Index<KMEANS_ACT_GELU_TANH>{}); break;
        case KMEANS_ACT_SILU: finish(Index<KMEANS_ACT_SILU>{}); break;
        default: finish(Index<KMEANS_ACT_NONE>{}); break;
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

// ---- few rows --------------------------------------------------------------

// 16 bytes of a row, of which n exist from p on (none where n <= 0).
__device__ __forceinline__ u32x4 load_bytes(const uint8_t *p, int n) {
    if (n >= 16)
        return *reinterpret_cast<const u32x4_bytes *>(p);
    u32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int x = 0; x < 15; ++x)
        if (x < n)
            v[x / 4] |= static_cast<uint32_t>(p[x]) << (8 * (x % 4));
    return v;
}

// At most 16 rows: the weights are read once, straight into fragments, and that
// is the whole cost.  One workgroup takes FB blocks of 16 features and all rows
// (so FB blocks share a row fragment); its WAVES waves take the blocks of k in
// turns and add their sums in LDS in wave order.  Loads are at the rows' own
// alignment; a lane takes bytes 16 q .. and 64 + 16 q .. of a block, so that a load
// of a wave covers 64 bytes of each row.  1 x 4096 x 32768: 28.6 us (134 MB, 4.7
// TB/s), 16 rows 30 to 35; with FB = 1 33 and 42, with two or four blocks of k at
// once 29 to 34.  1 x 8192 x 8192 13.6 us (4.9 TB/s).
template <typename T, int WAVES, int FB>
__global__ __launch_bounds__(WAVES * 64)
void linear_fp8_rows_kernel(const Product g, const Scales sc) {
    __shared__ f32x4 sums[FB][WAVES][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l = lane & 15, q = lane >> 4;
    const int j0 = blockIdx.x * (16 * FB);
    const int row = min(l, g.I - 1);
    const uint8_t *w[FB];
#pragma unroll
    for (int f = 0; f < FB; ++f)
        w[f] = static_cast<const uint8_t *>(g.Q) + min(j0 + 16 * f + l, g.J - 1) * g.ldq + q * 16;
    const uint8_t *x = static_cast<const uint8_t *>(g.P) + row * g.ldp + q * 16;
    const float *sx = sc.x + row * sc.ldx;
    const float *sw = sc.w + j0 / kFp8Block * sc.ldw;
    const int blocks = (g.K + kFp8Block - 1) / kFp8Block;
    f32x4 acc[FB] = {};
    auto block = [&](auto whole, int b) KM_INLINE {
        const int n = decltype(whole)::value ? kFp8Block : g.K - b * kFp8Block - q * 16;
        auto load = [&](const uint8_t *p) KM_INLINE {
            return Halves{load_bytes(p + b * kFp8Block, n), load_bytes(p + b * kFp8Block + 64, n - 64)};
        };
        Halves wf[FB];
#pragma unroll
        for (int f = 0; f < FB; ++f)
            wf[f] = load(w[f]);
        const Halves xf = load(x);
        const float s = sx[b] * sw[b];
        const Widened xw = widen_block(xf);
#pragma unroll
        for (int f = 0; f < FB; ++f) {
            const f32x4 v = mfma_block(widen_block(wf[f]), xw);
#pragma unroll
            for (int c = 0; c < 4; ++c)
                acc[f][c] = fmaf(v[c], s, acc[f][c]);
        }
    };
    const int whole = g.K / kFp8Block;
    for (int b = wave; b < whole; b += WAVES)
        block(std::true_type{}, b);
    if (whole < blocks && whole % WAVES == wave)
        block(std::false_type{}, whole);
#pragma unroll
    for (int f = 0; f < FB; ++f)
        sums[f][wave][lane] = acc[f];
    __syncthreads();
    // Four features of one row per lane: element c of lane (l, q) is feature
    // 4 q + c of row l.  Wave f finishes feature block f.
    const int j = j0 + 16 * wave + q * 4;
    if (wave >= FB || l >= g.I || j >= g.J)
        return;
    f32x4 s = sums[wave][0][lane];
#pragma unroll
    for (int v = 1; v < WAVES; ++v)
        s += sums[wave][v][lane];
    float v[4] = {s[0], s[1], s[2], s[3]};
    finish_run<T, 4>(g.epi, l, j, g.J, v);
}

// ---- rows that the copies do not take --------------------------------------

// Rows of `cols` bytes laid out anew, `ld` apart (a multiple of 16, zeros behind
// the last value), up to two matrices in one launch: kLayoutLanes lanes to a row.
struct Layout {
    const uint8_t *from;
    uint8_t *to;
    int64_t ld_from, ld;
    int rows, cols;          // no rows: nothing to do
    int wgs;
};
constexpr int kLayoutLanes = 32;
constexpr int kLayoutRows = 256 / kLayoutLanes;
__global__ __launch_bounds__(256)
void linear_fp8_layout_kernel(const Layout a, const Layout b) {
    const bool second = static_cast<int>(blockIdx.x) >= a.wgs;
    const Layout &m = second ? b : a;
    const int first = (blockIdx.x - (second ? a.wgs : 0)) * kLayoutRows + threadIdx.x / kLayoutLanes;
    for (int64_t row = first; row < m.rows; row += static_cast<int64_t>(m.wgs) * kLayoutRows)
        for (int c = threadIdx.x % kLayoutLanes * 16; c < m.ld; c += kLayoutLanes * 16)
            *reinterpret_cast<u32x4 *>(m.to + row * m.ld + c) =
                load_bytes(m.from + row * m.ld_from + c, m.cols - c);
}

// ---- launch ----------------------------------------------------------------

template <typename T>
hipError_t launch_tiles(const Product &product, const Scales &sc, hipStream_t stream) {
    constexpr int64_t kMaxGrid = int64_t(1) << 22;      // a launch has less than 2^32 threads
    Product g = product;
    const int64_t tiles = tiles_of(g, g.shape == kWide ? 256 : 128) * g.splits;
    hipError_t e = hipSuccess;
    for (int64_t first = 0; first < tiles && e == hipSuccess; first += kMaxGrid) {
        g.first_wg = static_cast<int>(first);
        const dim3 grid(static_cast<unsigned>(std::min(tiles - first, kMaxGrid)));
        switch (g.shape) {
        case kWide:
            if constexpr (sizeof(typename T::bits) == 2)    // the plan has it for no other
                hipLaunchKernelGGL((linear_fp8_kernel<T, 2, 4, 8, 4, 2>), grid, dim3(512), 0,
                                   stream, g, sc);
            break;
        case kDeep:
            hipLaunchKernelGGL((linear_fp8_kernel<T, 2, 4, 4, 2, 4>), grid, dim3(512), 0, stream, g,
                               sc);
            break;
        default:
            hipLaunchKernelGGL((linear_fp8_kernel<T, 2, 2, 4, 4, 2>), grid, dim3(256), 0, stream, g,
                               sc);
            break;
        }
        e = hipGetLastError();
    }
    if (e == hipSuccess && g.splits > 1) {
        const int64_t runs = static_cast<int64_t>(g.I) * ((g.J + 3) / 4);
        const int wgs =
            static_cast<int>(std::min<int64_t>((runs + kJoinRuns - 1) / kJoinRuns, 4096));
        hipLaunchKernelGGL((linear_join_kernel<T>), dim3(wgs), dim3(kJoinThreads), 0, stream, g,
                           wgs, BiasSums{});
        e = hipGetLastError();
    }
    return e;
}

template <typename T>
hipError_t launch_rows(const Product &g, const Scales &sc, int compute_units, hipStream_t stream) {
    // Four feature blocks where that leaves a workgroup for each CU, else as many
    // waves as D gives work to, while the CUs hold them (32 each).
    if (g.J >= 64 * compute_units) {
        hipLaunchKernelGGL((linear_fp8_rows_kernel<T, 8, 4>), dim3((g.J + 63) / 64), dim3(512), 0,
                           stream, g, sc);
        return hipGetLastError();
    }
    const dim3 grid((g.J + 15) / 16);
    int64_t waves = 4;
    while (waves < 16 && waves * kFp8Block < g.K && grid.x * waves * 2 <= 16 * compute_units)
        waves *= 2;
    if (waves == 16)
        hipLaunchKernelGGL((linear_fp8_rows_kernel<T, 16, 1>), grid, dim3(1024), 0, stream, g, sc);
    else if (waves == 8)
        hipLaunchKernelGGL((linear_fp8_rows_kernel<T, 8, 1>), grid, dim3(512), 0, stream, g, sc);
    else
        hipLaunchKernelGGL((linear_fp8_rows_kernel<T, 4, 1>), grid, dim3(256), 0, stream, g, sc);
    return hipGetLastError();
}

template <typename T>
hipError_t run_product(const Product &g, const Scales &sc, int compute_units, hipStream_t stream) {
    return g.shape == kRows ? launch_rows<T>(g, sc, compute_units, stream)
                            : launch_tiles<T>(g, sc, stream);
}

bool takes_copies(const void *p, int64_t ld, int64_t cols) {
    return aligned(p, 16) && ld % 16 == 0 && cols % 16 == 0;
}

// Plans the new layout of rows [rows][D] at workspace offset `at`, or leaves
// them as they are.
Layout layout_of(const void *p, int64_t ld, int64_t rows, int64_t D, size_t &at) {
    Layout m{static_cast<const uint8_t *>(p), nullptr, ld, ld, 0, static_cast<int>(D), 0};
    if (takes_copies(p, ld, D))
        return m;
    m.ld = (D + 15) / 16 * 16;
    m.rows = static_cast<int>(rows);
    m.wgs = static_cast<int>(std::min<int64_t>((rows + kLayoutRows - 1) / kLayoutRows, 4096));
    m.to = reinterpret_cast<uint8_t *>(at);             // an offset until the lease
    at += align_up(static_cast<size_t>(rows) * m.ld);
    return m;
}

kmeans_status_t check_stride(const char *name, int64_t ld) {
    if (ld > kMaxWidth)
        return fail(KMEANS_ERR_UNSUPPORTED, "%s: row stride %lld too large (max %lld)", name,
                    static_cast<long long>(ld), static_cast<long long>(kMaxWidth));
    return KMEANS_OK;
}

}  // namespace
}  // namespace kmeans

// ---- C entry point ---------------------------------------------------------

extern "C" kmeans_status_t kmeans_linear_fp8(const void *X, int64_t x_stride, const float *x_scales,
                                             int64_t xs_stride, const void *W, int64_t w_stride,
                                             const float *w_scales, int64_t ws_stride,
                                             const void *bias, const void *residual,
                                             int64_t residual_stride, int64_t N, int64_t D,
                                             int64_t F, int32_t dtype, int32_t activation, void *Y,
                                             int64_t y_stride, hipStream_t stream) {
    using namespace kmeans;
    if (N < 0 || D < 1 || F < 1)
        return fail(KMEANS_ERR_INVALID_ARG, "N=%lld must be >= 0, D=%lld and F=%lld >= 1",
                    static_cast<long long>(N), static_cast<long long>(D),
                    static_cast<long long>(F));
    if (activation < KMEANS_ACT_NONE || activation > KMEANS_ACT_SILU)
        return fail(KMEANS_ERR_INVALID_ARG, "activation=%d is not a kmeans_activation_t",
                    activation);
    if (dtype < KMEANS_BF16 || dtype > KMEANS_FP32)
        return fail(KMEANS_ERR_INVALID_ARG, "dtype=%d is not a kmeans_dtype_t", dtype);
    if (N > kMaxRows || D > kMaxWidth || F > kMaxWidth)
        return fail(KMEANS_ERR_UNSUPPORTED, "N=%lld, D=%lld or F=%lld too large (max %lld, "
                    "%lld, %lld)", static_cast<long long>(N), static_cast<long long>(D),
                    static_cast<long long>(F), static_cast<long long>(kMaxRows),
                    static_cast<long long>(kMaxWidth), static_cast<long long>(kMaxWidth));
    if (N == 0)
        return ok();
    const size_t size = dtype_size(dtype);
    const int64_t blocks = fp8_blocks(D);
    kmeans_status_t st;
    if ((st = check_matrix("X", X, D, x_stride, 1)) != KMEANS_OK ||
        (st = check_stride("X", x_stride)) != KMEANS_OK ||
        (st = check_matrix("x_scales", x_scales, blocks, xs_stride, 4)) != KMEANS_OK ||
        (st = check_stride("x_scales", xs_stride)) != KMEANS_OK ||
        (st = check_matrix("W", W, D, w_stride, 1)) != KMEANS_OK ||
        (st = check_stride("W", w_stride)) != KMEANS_OK ||
        (st = check_matrix("w_scales", w_scales, blocks, ws_stride, 4)) != KMEANS_OK ||
        (st = check_stride("w_scales", ws_stride)) != KMEANS_OK ||
        (st = check_array("bias", bias, size)) != KMEANS_OK ||
        (residual && (st = check_matrix("residual", residual, F, residual_stride, size)) != KMEANS_OK) ||
        (residual && (st = check_stride("residual", residual_stride)) != KMEANS_OK) ||
        (st = check_matrix("Y", Y, F, y_stride, size)) != KMEANS_OK ||
        (st = check_stride("Y", y_stride)) != KMEANS_OK)
        return st;

    const int cus = device_compute_units();
    const Scales sc{x_scales, w_scales, xs_stride, ws_stride,
                    static_cast<int>((F + kFp8Block - 1) / kFp8Block)};
    Product g{};
    std::optional<WorkspaceLease> lease;
    if (N <= kMaxFewRows) {
        g.I = static_cast<int>(N);
        g.J = static_cast<int>(F);
        g.shape = kRows;
        g.P = X;
        g.Q = W;
        g.ldp = x_stride;
        g.ldq = w_stride;
        g.K = static_cast<int>(D);
    } else {
        size_t bytes = 0;
        Layout x = layout_of(X, x_stride, N, D, bytes), w = layout_of(W, w_stride, F, D, bytes);
        g = fp8_product(N, D, F, cus, dtype != KMEANS_FP32);
        if (tiles_of(g, 128) > kMaxRows / kMaxKSplits)
            return fail(KMEANS_ERR_UNSUPPORTED, "N=%lld x F=%lld: too many outputs",
                        static_cast<long long>(N), static_cast<long long>(F));
        const size_t part_at = bytes;
        bytes += partial_bytes(g);
        char *ws = nullptr;
        if (bytes > 0) {
            lease.emplace(stream, bytes);
            if (lease->error() != hipSuccess)
                return fail(KMEANS_ERR_NO_MEMORY, "workspace of %zu bytes: %s", bytes,
                            hipGetErrorString(lease->error()));
            ws = static_cast<char *>(lease->ptr());
            g.partial = reinterpret_cast<float *>(ws + part_at);
        }
        for (Layout *m : {&x, &w})
            if (m->rows > 0)
                m->to = reinterpret_cast<uint8_t *>(ws + reinterpret_cast<size_t>(m->to));
        if (x.wgs + w.wgs > 0) {
            hipLaunchKernelGGL(linear_fp8_layout_kernel, dim3(x.wgs + w.wgs), dim3(256), 0, stream,
                               x, w);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess)
                return fail(KMEANS_ERR_HIP, "layout launch failed: %s", hipGetErrorString(e));
        }
        g.P = x.rows > 0 ? x.to : X;
        g.Q = w.rows > 0 ? w.to : W;
        g.ldp = x.ld / 2;
        g.ldq = w.ld / 2;
    }
    g.epi = {bias, residual, residual_stride, Y, y_stride, nullptr, 0, activation};
    const hipError_t e = dtype == KMEANS_BF16   ? run_product<Bf16>(g, sc, cus, stream)
                         : dtype == KMEANS_FP16 ? run_product<Fp16>(g, sc, cus, stream)
                                                : run_product<Fp32>(g, sc, cus, stream);
    if (e != hipSuccess)
        return fail(KMEANS_ERR_HIP, "8-bit linear launch failed: %s", hipGetErrorString(e));
    return ok();
}
