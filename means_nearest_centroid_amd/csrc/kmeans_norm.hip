// kmeans_norm.hip -- gfx950 kernels of the root-mean-square norm with the
// residual's addition (its output in the inputs' type, or in 8 bits with a
// scale for each 128 columns), of its gradient, and of quantisation by blocks.
//
//     h = x + residual,  r = 1 / sqrt(mean(h^2) + eps),  y = h r w
//     gradient, with g = dy w:  dx = r g - h r^3 mean(g h) + dh,
//                               dw = sum over rows of dy h r
//     block of values y:  s = max|y| / 448,  q = e4m3(y / s)
//
// All are bound by memory: each row is read once into registers, its sums are
// joined across the lanes that hold it, and what follows is computed from the
// registers.
#include <stdint.h>

#include <algorithm>
#include <optional>
#include <type_traits>

#include "kmeans_fp8.h"
#include "kmeans_internal.h"
#include "kmeans_types.h"

namespace kmeans {
namespace {

constexpr int64_t kMaxNormWidth = 1 << 20;
constexpr int kNormThreads = 256;
constexpr int kRun = 8;                  // values a lane takes at once
constexpr int kLanesPerBlock = kFp8Block / kRun;
// Widest row that a workgroup holds in registers; wider ones are read twice.
constexpr int64_t kMaxHeld = 1024 * 2 * kRun;

// ---- sums over the G lanes that share a row --------------------------------

// Workgroup for G lanes to a row: one row, or several side by side.
constexpr int threads_for(int G) { return G > kNormThreads ? G : kNormThreads; }

// The group's totals of M values, on each of its lanes.  Groups wider than a
// wave meet in LDS (two places in turn: a call may begin while other waves still
// read the one before it, and a third cannot, since the second's barrier lies
// between).
template <int G, int M>
struct GroupSums {
    static constexpr int kGroups = threads_for(G) / G;
    static constexpr int kWaves = G > 64 ? G / 64 : 1;
    float part[G > 64 ? 2 : 1][kGroups][kWaves][M];

    __device__ __forceinline__ void join(float (&v)[M], int &turn) {
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int x = (G < 64 ? G : 64) / 2; x >= 1; x >>= 1)
                v[m] += __shfl_xor(v[m], x, 64);
        if constexpr (G > 64) {
            const int group = threadIdx.x / G, wave = threadIdx.x % G / 64;
            if ((threadIdx.x & 63) == 0) {
#pragma unroll
                for (int m = 0; m < M; ++m)
                    part[turn][group][wave][m] = v[m];
            }
            __syncthreads();
#pragma unroll
            for (int m = 0; m < M; ++m) {
                v[m] = part[turn][group][0][m];
#pragma unroll
                for (int w = 1; w < kWaves; ++w)
                    v[m] += part[turn][group][w][m];
            }
            turn ^= 1;
        }
    }
};

// ---- forward ---------------------------------------------------------------

struct Norm {
    const void *x;
    const void *residual;    // or null
    const void *weight;      // or null
    void *sum;               // or null
    void *y;                 // or null: quantised
    uint8_t *q;
    float *scales;
    int64_t ldx, ldr, ldh, ldy, ldq, lds;
    int64_t first;           // row of this launch
    int N, D;
    float eps;
};

template <typename T>
__device__ __forceinline__ void widen_run(const Packed<typename T::bits, kRun> &p,
                                          float (&v)[kRun]) {
#pragma unroll
    for (int e = 0; e < kRun; ++e)
        v[e] = T::widen(p.v[e]);
}

// Output of one run from column c on: y = h r w, rounded once to the type or by
// its block of 16 lanes to 8 bits.  Every lane of a block calls it (h = 0 past
// the row's end, where n <= 0).
template <typename T, bool QUANT>
__device__ __forceinline__ void norm_out(const Norm &a, int64_t row, int c, float r,
                                         const float (&h)[kRun],
                                         const Packed<typename T::bits, kRun> &w) {
    typedef typename T::bits B;
    const int n = a.D - c;
    float y[kRun], scale[kRun];
    widen_run<T>(w, scale);
#pragma unroll
    for (int e = 0; e < kRun; ++e) {
        y[e] = h[e] * r;
        if (a.weight != nullptr)
            y[e] *= scale[e];
    }
    if constexpr (QUANT) {
        uint32_t most = 0;
#pragma unroll
        for (int e = 0; e < kRun; ++e)
            most = max(most, e < n ? magnitude(y[e]) : 0u);
        most = block_most<kLanesPerBlock>(most);
        const float s = fp8_scale(most);
        if (n > 0) {
            store_fp8_run(a.q + row * a.ldq + c, n, y, s);
            if (c % kFp8Block == 0)
                a.scales[row * a.lds + c / kFp8Block] = s;
        }
    } else if (n > 0) {
        store_run<B, kRun>(static_cast<B *>(a.y) + row * a.ldy + c, n, narrow_run<T, kRun>(y));
    }
}

// G lanes to a row, R runs to a lane: run i of the row is lane i % G's.  One run to
// a lane as far as workgroups go: more rows are on their way at once than with
// more runs to fewer lanes (16384 x 4096 bf16 with residual to 8 bits 88 to 90 us, 471
// MB at 5.3 TB/s, 93 with 256 lanes where it took 86; 4096 x 8192 44 us, 54 so; 2048 x
// 16384 fp16 48 us, 73 with 8 runs to 256 lanes).
template <typename T, bool QUANT, int G, int R>
__global__ __launch_bounds__(threads_for(G))
void norm_kernel(const Norm a) {
    typedef typename T::bits B;
    __shared__ GroupSums<G, 1> sums;
    constexpr int kRows = threads_for(G) / G;
    const int lane = threadIdx.x % G;
    const int64_t row = a.first + static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / G;
    const bool real = row < a.N;
    Packed<B, kRun> px[R], pr[R], pw[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int c = (i * G + lane) * kRun;
        px[i] = load_run<B, kRun>(static_cast<const B *>(a.x) + row * a.ldx + c,
                                  real ? a.D - c : 0);
    }
    if (a.residual != nullptr) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int c = (i * G + lane) * kRun;
            pr[i] = load_run<B, kRun>(static_cast<const B *>(a.residual) + row * a.ldr + c,
                                      real ? a.D - c : 0);
        }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int c = (i * G + lane) * kRun;
        pw[i] = Packed<B, kRun>{};
        if (a.weight != nullptr)
            pw[i] = load_run<B, kRun>(static_cast<const B *>(a.weight) + c, a.D - c);
    }
    float h[R][kRun], ss[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < R; ++i) {
        widen_run<T>(px[i], h[i]);
        if (a.residual != nullptr) {
            float r[kRun];
            widen_run<T>(pr[i], r);
#pragma unroll
            for (int e = 0; e < kRun; ++e)
                h[i][e] += r[e];
        }
#pragma unroll
        for (int e = 0; e < kRun; ++e)
            ss[0] = fmaf(h[i][e], h[i][e], ss[0]);
        const int c = (i * G + lane) * kRun;
        if (a.sum != nullptr && real && c < a.D)
            store_run<B, kRun>(static_cast<B *>(a.sum) + row * a.ldh + c, a.D - c,
                               narrow_run<T, kRun>(h[i]));
    }
    int turn = 0;
    sums.join(ss, turn);
    const float r = 1.0f / sqrtf(ss[0] / static_cast<float>(a.D) + a.eps);
    if (!real)                   // whole groups of lanes
        return;
#pragma unroll
    for (int i = 0; i < R; ++i)
        norm_out<T, QUANT>(a, row, (i * G + lane) * kRun, r, h[i], pw[i]);
}

// Rows wider than the registers of a workgroup: read twice, the second time
// from the caches.  Nothing is written before the row's sum is known, so that
// the outputs may lie on the inputs.
template <typename T, bool QUANT>
__global__ __launch_bounds__(kNormThreads)
void norm_long_kernel(const Norm a) {
    typedef typename T::bits B;
    __shared__ GroupSums<kNormThreads, 1> sums;
    const int64_t row = a.first + blockIdx.x;
    const int step = kNormThreads * kRun;
    auto load = [&](int c, float (&h)[kRun]) __attribute__((always_inline)) {
        widen_run<T>(load_run<B, kRun>(static_cast<const B *>(a.x) + row * a.ldx + c, a.D - c), h);
        if (a.residual == nullptr)
            return;
        float r[kRun];
        widen_run<T>(
            load_run<B, kRun>(static_cast<const B *>(a.residual) + row * a.ldr + c, a.D - c), r);
#pragma unroll
        for (int e = 0; e < kRun; ++e)
            h[e] += r[e];
    };
    float ss[1] = {0.0f};
    for (int c = threadIdx.x * kRun; c < a.D; c += step) {
        float h[kRun];
        load(c, h);
#pragma unroll
        for (int e = 0; e < kRun; ++e)
            ss[0] = fmaf(h[e], h[e], ss[0]);
    }
    int turn = 0;
    sums.join(ss, turn);
    const float r = 1.0f / sqrtf(ss[0] / static_cast<float>(a.D) + a.eps);
    for (int c0 = 0; c0 < a.D; c0 += step) {       // the same trips on every lane
        const int c = c0 + threadIdx.x * kRun;
        float h[kRun];
        load(c, h);
        Packed<B, kRun> w = {};
        if (a.weight != nullptr)
            w = load_run<B, kRun>(static_cast<const B *>(a.weight) + c, a.D - c);
        if (a.sum != nullptr && c < a.D)
            store_run<B, kRun>(static_cast<B *>(a.sum) + row * a.ldh + c, a.D - c,
                               narrow_run<T, kRun>(h));
        norm_out<T, QUANT>(a, row, c, r, h, w);
    }
}

// ---- gradient --------------------------------------------------------------

struct NormGrad {
    const void *dy, *h;
    const void *weight;      // or null
    const void *dh;          // or null
    void *dx;
    void *dw_partial;        // [rows of workgroups][D], or null: fp64 where DEEP, else fp32
    float *r;                // [N]: 1 / rms of each row, for wide rows' dw
    int64_t ldy, ldh, lddh, ldx;
    int N, D;
    float eps;
};

// Terms of dw that a lane adds one after another in fp32, and at most 15 sums of
// other lanes with them: past that (but for eight partial sums in pairs) the sums go
// on in fp64, so that no error grows with the rows (in fp32 alone a lane adds 8192
// terms of 2^27 rows, up to 2^-11 off).
constexpr int kDepth = 44;

// dw of a workgroup's rows so far, summed over its groups, to its row of partial
// sums; DEEP: added to what lies there where `more`, and dw begins anew.
template <int G, int R, bool DEEP>
__device__ __forceinline__ void leave_sums(const NormGrad &a, float (&dw)[R][kRun], float *across,
                                           bool more) {
    constexpr int kThreads = threads_for(G);
    constexpr int kRows = kThreads / G;
    const int lane = threadIdx.x % G, group = threadIdx.x / G;
    const int64_t out = static_cast<int64_t>(blockIdx.x) * a.D;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int c = (i * G + lane) * kRun;
        if constexpr (kRows > 1) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < kRun; ++e)
                across[e * kThreads + threadIdx.x] = dw[i][e];
            __syncthreads();
            if (group == 0)
#pragma unroll
                for (int e = 0; e < kRun; ++e)
                    for (int q = 1; q < kRows; ++q)
                        dw[i][e] += across[e * kThreads + q * G + lane];
        }
        if (group == 0 && c < a.D) {
            if constexpr (DEEP) {
                double *sum = static_cast<double *>(a.dw_partial) + out + c;
#pragma unroll
                for (int e = 0; e < kRun; ++e)
                    if (c + e < a.D)
                        sum[e] = more ? sum[e] + dw[i][e] : dw[i][e];
            } else {
                Packed<float, kRun> p;
#pragma unroll
                for (int e = 0; e < kRun; ++e)
                    p.v[e] = dw[i][e];
                store_run<float, kRun>(static_cast<float *>(a.dw_partial) + out + c, a.D - c, p);
            }
        }
        if constexpr (DEEP)
#pragma unroll
            for (int e = 0; e < kRun; ++e)
                dw[i][e] = 0.0f;
    }
}

// Rows of a workgroup, one after another (kRows at a time): dx from the row's
// two sums, dw summed in registers over kDepth of a lane's rows in their order,
// then over the workgroup's groups in LDS, and those of more rows in fp64 in its row
// of partial sums.  The next row is on its way while this one is worked, where
// registers hold both (R = 1; two runs to a lane, rows of more than 8192, spill 5 to
// 29 of them: 2048 x 16384 68 us, 4096 x 8192 of the same bytes 57); rows stay in
// their own type for that.  As many workgroups as the CUs hold (16 waves each): 16384 x
// 4096 bf16 with dh 102 us (537 MB, 5.3 TB/s), 119 with twice and 149 with half as
// many, and 171 with 256 lanes to a row.  WHOLE: D is a multiple of 8, and no run is
// cut short (50021 x 321 fp32 40 us, 193 MB; 45 with its last runs loaded whole
// and shifted).  DEEP: a lane has more than kDepth rows.
template <typename T, int G, int R, bool WHOLE, bool DEEP>
__global__ __launch_bounds__(threads_for(G))
void norm_grad_kernel(const NormGrad a) {
    typedef typename T::bits B;
    typedef Packed<B, kRun> Run;
    constexpr int kThreads = threads_for(G);
    constexpr int kRows = kThreads / G;
    __shared__ GroupSums<G, 2> sums;
    __shared__ float across[kRows > 1 ? kThreads * kRun : 1];
    const int lane = threadIdx.x % G, group = threadIdx.x / G;
    auto fetch = [&](const void *p, int64_t at, int c, bool real) __attribute__((always_inline)) {
        const B *q = static_cast<const B *>(p) + at + c;
        if constexpr (WHOLE)
            return real && c < a.D ? load_packed<B, kRun>(q) : Run{};
        else
            return load_run<B, kRun>(q, real ? a.D - c : 0);
    };
    float dw[R][kRun] = {};
    Run w[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (a.weight != nullptr)
            w[i] = fetch(a.weight, 0, (i * G + lane) * kRun, true);
    Run h[R], y[R], d[R];
    auto load = [&](int64_t row) __attribute__((always_inline)) {
        const bool real = row < a.N;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int c = (i * G + lane) * kRun;
            h[i] = fetch(a.h, row * a.ldh, c, real);
            y[i] = fetch(a.dy, row * a.ldy, c, real);
            d[i] = Run{};
            if (a.dh != nullptr)
                d[i] = fetch(a.dh, row * a.lddh, c, real);
        }
    };
    auto gain = [&](int i, int e) __attribute__((always_inline)) {
        return a.weight != nullptr ? T::widen(w[i].v[e]) : 1.0f;
    };
    const float inv_d = 1.0f / static_cast<float>(a.D);
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kRows;
    int turn = 0;
    [[maybe_unused]] int held = 0;
    bool more = false;
    int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + group;
    load(row);
    for (; row - group < a.N; row += stride) {
        Run h0[R], y0[R], d0[R];
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < R; ++i) {
            h0[i] = h[i];
            y0[i] = y[i];
            d0[i] = d[i];
#pragma unroll
            for (int e = 0; e < kRun; ++e) {
                const float x = T::widen(h0[i].v[e]);
                s[0] = fmaf(x, x, s[0]);
                s[1] = fmaf(T::widen(y0[i].v[e]) * gain(i, e), x, s[1]);
            }
        }
        if (R == 1)
            load(row + stride);
        sums.join(s, turn);
        const float r = 1.0f / sqrtf(s[0] / static_cast<float>(a.D) + a.eps);
        const float k = (s[1] * inv_d * r) * r;      // dx = r (g - h k) + dh
        if (row < a.N) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int c = (i * G + lane) * kRun;
                float v[kRun];
#pragma unroll
                for (int e = 0; e < kRun; ++e) {
                    const float x = T::widen(h0[i].v[e]), g = T::widen(y0[i].v[e]);
                    v[e] = r * fmaf(-x, k, g * gain(i, e)) + T::widen(d0[i].v[e]);
                    dw[i][e] = fmaf(g * x, r, dw[i][e]);
                }
                B *o = static_cast<B *>(a.dx) + row * a.ldx + c;
                if constexpr (WHOLE) {
                    if (c < a.D)
                        store_packed<B, kRun>(o, narrow_run<T, kRun>(v));
                } else if (c < a.D) {
                    store_run<B, kRun>(o, a.D - c, narrow_run<T, kRun>(v));
                }
            }
        }
        if (R > 1)
            load(row + stride);
        if constexpr (DEEP)
            if (++held == kDepth) {
                leave_sums<G, R, DEEP>(a, dw, across, more);
                held = 0;
                more = true;
            }
    }
    if (a.dw_partial != nullptr)
        leave_sums<G, R, DEEP>(a, dw, across, more);
}

// Wide rows: dx by two readings of the row (the second from the caches).
template <typename T>
__global__ __launch_bounds__(kNormThreads)
void norm_grad_long_kernel(const NormGrad a, int64_t first) {
    typedef typename T::bits B;
    __shared__ GroupSums<kNormThreads, 2> sums;
    const int64_t row = first + blockIdx.x;
    auto load = [&](const void *p, int64_t ld, int c, float (&v)[kRun])
                    __attribute__((always_inline)) {
        widen_run<T>(load_run<B, kRun>(static_cast<const B *>(p) + row * ld + c, a.D - c), v);
    };
    auto load_g = [&](int c, float (&g)[kRun]) __attribute__((always_inline)) {
        load(a.dy, a.ldy, c, g);
        if (a.weight == nullptr)
            return;
        float w[kRun];
        widen_run<T>(load_run<B, kRun>(static_cast<const B *>(a.weight) + c, a.D - c), w);
#pragma unroll
        for (int e = 0; e < kRun; ++e)
            g[e] *= w[e];
    };
    float s[2] = {0.0f, 0.0f};
    for (int c = threadIdx.x * kRun; c < a.D; c += kNormThreads * kRun) {
        float h[kRun], g[kRun];
        load(a.h, a.ldh, c, h);
        load_g(c, g);
#pragma unroll
        for (int e = 0; e < kRun; ++e) {
            s[0] = fmaf(h[e], h[e], s[0]);
            s[1] = fmaf(g[e], h[e], s[1]);
        }
    }
    int turn = 0;
    sums.join(s, turn);
    const float r = 1.0f / sqrtf(s[0] / static_cast<float>(a.D) + a.eps);
    const float k = (s[1] / static_cast<float>(a.D) * r) * r;
    if (a.r != nullptr && threadIdx.x == 0)
        a.r[row] = r;
    for (int c = threadIdx.x * kRun; c < a.D; c += kNormThreads * kRun) {
        float h[kRun], g[kRun], d[kRun] = {};
        load(a.h, a.ldh, c, h);
        load_g(c, g);
        if (a.dh != nullptr)
            load(a.dh, a.lddh, c, d);
#pragma unroll
        for (int e = 0; e < kRun; ++e)
            g[e] = r * fmaf(-h[e], k, g[e]) + d[e];
        store_run<B, kRun>(static_cast<B *>(a.dx) + row * a.ldx + c, a.D - c,
                           narrow_run<T, kRun>(g));
    }
}

// Wide rows: dw's partial sums over a workgroup's rows, a run of columns to each
// lane, every kDepth rows in fp64.
template <typename T>
__global__ __launch_bounds__(kNormThreads)
void norm_columns_kernel(const NormGrad a, int rows_per_wg) {
    typedef typename T::bits B;
    const int c = (blockIdx.y * kNormThreads + threadIdx.x) * kRun;
    if (c >= a.D)
        return;
    const int64_t end = min(static_cast<int64_t>(a.N),
                            (static_cast<int64_t>(blockIdx.x) + 1) * rows_per_wg);
    double sum[kRun] = {};
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * rows_per_wg; row < end;) {
        float dw[kRun] = {};
        for (const int64_t stop = min(end, row + kDepth); row < stop; ++row) {
            float h[kRun], y[kRun];
            widen_run<T>(load_run<B, kRun>(static_cast<const B *>(a.h) + row * a.ldh + c, a.D - c),
                         h);
            widen_run<T>(load_run<B, kRun>(static_cast<const B *>(a.dy) + row * a.ldy + c, a.D - c),
                         y);
            const float r = a.r[row];
#pragma unroll
            for (int e = 0; e < kRun; ++e)
                dw[e] = fmaf(y[e] * h[e], r, dw[e]);
        }
#pragma unroll
        for (int e = 0; e < kRun; ++e)
            sum[e] += dw[e];
    }
    Packed<float, kRun> p;
#pragma unroll
    for (int e = 0; e < kRun; ++e)
        p.v[e] = static_cast<float>(sum[e]);
    store_run<float, kRun>(static_cast<float *>(a.dw_partial) +
                               static_cast<int64_t>(blockIdx.x) * a.D + c, a.D - c, p);
}

// dw[c] = sum of the partials (of type P) of column c: kJoinCols columns to a
// workgroup, kJoinShares threads to a column, kJoinBatch loads of each in flight (1024
// rows of 321: 3 us, 11 with one load), added in pairs and then in fp64 (all of it
// in fp64 1.4 us more), joined in LDS in their order.
constexpr int kJoinCols = 32;
constexpr int kJoinShares = 32;
constexpr int kJoinBatch = 8;
template <typename T, typename P>
__global__ __launch_bounds__(kJoinCols * kJoinShares)
void norm_join_kernel(const P *partial, int rows, int D, void *dw) {
    __shared__ double sums[kJoinShares][kJoinCols + 1];
    const int c = threadIdx.x % kJoinCols, share = threadIdx.x / kJoinCols;
    const int col = blockIdx.x * kJoinCols + c;
    double v = 0.0;
    if (col < D)
        for (int r0 = share; r0 < rows; r0 += kJoinBatch * kJoinShares) {
            P x[kJoinBatch];
#pragma unroll
            for (int u = 0; u < kJoinBatch; ++u)
                x[u] = partial[static_cast<int64_t>(min(r0 + u * kJoinShares, rows - 1)) * D + col];
#pragma unroll
            for (int u = 0; u < kJoinBatch; ++u)
                x[u] = r0 + u * kJoinShares < rows ? x[u] : P(0);
#pragma unroll
            for (int half = kJoinBatch / 2; half >= 1; half /= 2)
#pragma unroll
                for (int u = 0; u < half; ++u)
                    x[u] += x[u + half];
            v += x[0];
        }
    sums[share][c] = v;
    __syncthreads();
    if (share != 0 || col >= D)
        return;
    for (int q = 1; q < kJoinShares; ++q)
        v += sums[q][c];
    static_cast<typename T::bits *>(dw)[col] = T::narrow(static_cast<float>(v));
}

template <typename T>
__global__ __launch_bounds__(256)
void norm_zero_kernel(typename T::bits *p, int n) {
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i < n)
        p[i] = T::narrow(0.0f);
}

// ---- quantisation by blocks ------------------------------------------------

struct Quantize {
    const void *x;
    uint8_t *q;
    float *scales;
    int64_t ldx, ldq, lds;
    int N, D;
};

// A tile of 128 rows x 128 columns to a workgroup, all of it in registers: 16
// lanes across a row, 16 rows at a time.  ROWS (of a block): 1, each row's 16
// lanes have its scale; 128, the workgroup joins them.  262144 x 128 bf16 in rows
// 22.7 us (102 MB, 4.5 TB/s), 4096 x 4096 in blocks 13.0 us (50 MB, 3.9 TB/s).
template <typename T, int ROWS>
__global__ __launch_bounds__(kNormThreads)
void quantize_kernel(const Quantize a) {
    typedef typename T::bits B;
    constexpr int kAtOnce = kNormThreads / kLanesPerBlock;
    constexpr int kPasses = kFp8Block / kAtOnce;
    __shared__ uint32_t part[2][kNormThreads / 64];
    const int across = (a.D + kFp8Block - 1) / kFp8Block;
    const int64_t tiles = (static_cast<int64_t>(a.N) + kFp8Block - 1) / kFp8Block * across;
    int turn = 0;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int b = static_cast<int>(t % across);
        const int64_t row0 = t / across * kFp8Block + threadIdx.x / kLanesPerBlock;
        const int c = b * kFp8Block + threadIdx.x % kLanesPerBlock * kRun;
        const int n = a.D - c;
        Packed<B, kRun> p[kPasses];
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int64_t row = row0 + i * kAtOnce;
            p[i] = load_run<B, kRun>(static_cast<const B *>(a.x) + row * a.ldx + c,
                                     row < a.N ? n : 0);
        }
        uint32_t most[kPasses];
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            most[i] = 0;
#pragma unroll
            for (int e = 0; e < kRun; ++e)
                most[i] = max(most[i], magnitude(T::widen(p[i].v[e])));
        }
        if constexpr (ROWS == kFp8Block) {
            uint32_t m = most[0];
#pragma unroll
            for (int i = 1; i < kPasses; ++i)
                m = max(m, most[i]);
            m = block_most<64>(m);
            if ((threadIdx.x & 63) == 0)
                part[turn][threadIdx.x >> 6] = m;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kNormThreads / 64; ++w)
                m = max(m, part[turn][w]);
            turn ^= 1;
#pragma unroll
            for (int i = 0; i < kPasses; ++i)
                most[i] = m;
        } else {
#pragma unroll
            for (int i = 0; i < kPasses; ++i)
                most[i] = block_most<kLanesPerBlock>(most[i]);
        }
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int64_t row = row0 + i * kAtOnce;
            if (row >= a.N || n <= 0)
                continue;
            const float s = fp8_scale(most[i]);
            float v[kRun];
            widen_run<T>(p[i], v);
            store_fp8_run(a.q + row * a.ldq + c, n, v, s);
            if (c % kFp8Block == 0 && row % ROWS == 0)
                a.scales[row / ROWS * a.lds + b] = s;
        }
    }
}

// ---- launch ----------------------------------------------------------------

// A launch has less than 2^32 threads.
constexpr int64_t kMaxThreads = int64_t(1) << 31;
constexpr int64_t kMaxGrid = kMaxThreads / kNormThreads;

template <typename T, bool QUANT, int G, int R>
hipError_t launch_norm(Norm a, hipStream_t stream) {
    constexpr int kRows = threads_for(G) / G;
    constexpr int64_t kMaxGrid = kMaxThreads / threads_for(G);
    hipError_t e = hipSuccess;
    for (int64_t first = 0; first < a.N && e == hipSuccess; first += kMaxGrid * kRows) {
        a.first = first;
        const int64_t wgs = std::min<int64_t>(kMaxGrid, (a.N - first + kRows - 1) / kRows);
        hipLaunchKernelGGL((norm_kernel<T, QUANT, G, R>), dim3(static_cast<unsigned>(wgs)),
                           dim3(threads_for(G)), 0, stream, a);
        e = hipGetLastError();
    }
    return e;
}

template <typename T, bool QUANT>
hipError_t run_norm(Norm a, hipStream_t stream) {
    const int64_t runs = (static_cast<int64_t>(a.D) + kRun - 1) / kRun;
    if (runs <= 16)
        return launch_norm<T, QUANT, 16, 1>(a, stream);
    if (runs <= 32)
        return launch_norm<T, QUANT, 32, 1>(a, stream);
    if (runs <= 64)
        return launch_norm<T, QUANT, 64, 1>(a, stream);
    if (runs <= 128)
        return launch_norm<T, QUANT, 64, 2>(a, stream);
    if (runs <= 256)
        return launch_norm<T, QUANT, 256, 1>(a, stream);
    if (runs <= 512)
        return launch_norm<T, QUANT, 512, 1>(a, stream);
    if (runs <= 1024)
        return launch_norm<T, QUANT, 1024, 1>(a, stream);
    if (runs <= kMaxHeld / kRun)
        return launch_norm<T, QUANT, 1024, 2>(a, stream);
    hipError_t e = hipSuccess;
    for (int64_t first = 0; first < a.N && e == hipSuccess; first += kMaxGrid) {
        a.first = first;
        hipLaunchKernelGGL((norm_long_kernel<T, QUANT>),
                           dim3(static_cast<unsigned>(std::min<int64_t>(kMaxGrid, a.N - first))),
                           dim3(kNormThreads), 0, stream, a);
        e = hipGetLastError();
    }
    return e;
}

template <typename T>
hipError_t run_norm(const Norm &a, hipStream_t stream) {
    return a.q != nullptr ? run_norm<T, true>(a, stream) : run_norm<T, false>(a, stream);
}

// How the rows of a gradient are divided: workgroups (each leaves one row of
// dw's partial sums) and, for wide rows, how many rows each takes.
struct NormGradPlan {
    bool wide, deep;
    int rows_at_once;        // of a workgroup
    int wgs, rows_per_wg;
    NormGradPlan(int64_t N, int64_t D, int compute_units) : wide(D > kMaxHeld) {
        const int64_t runs = (D + kRun - 1) / kRun;
        int lanes = 16;                      // of a row: norm_grad_kernel's G
        while (lanes < 1024 && lanes < runs)
            lanes *= 2;
        rows_at_once = wide ? 1 : threads_for(lanes) / lanes;
        const int64_t most = wide ? 64 : 1024 / threads_for(lanes) * compute_units;
        wgs = static_cast<int>(std::min<int64_t>(most, (N + rows_at_once - 1) / rows_at_once));
        rows_per_wg = static_cast<int>((N + wgs - 1) / wgs);
        deep = !wide && rows_per_wg > kDepth * rows_at_once;
        if (wide)
            wgs = static_cast<int>((N + rows_per_wg - 1) / rows_per_wg);
    }
    size_t partial_bytes(int64_t D) const {
        return static_cast<size_t>(wgs) * D * (deep ? sizeof(double) : sizeof(float));
    }
};

template <int N>
using Int = std::integral_constant<int, N>;

template <typename T>
hipError_t run_norm_grad(const NormGrad &a, const NormGradPlan &p, void *dw, hipStream_t stream) {
    const int64_t runs = (static_cast<int64_t>(a.D) + kRun - 1) / kRun;
    const dim3 grid(p.wgs), block(kNormThreads);
    hipError_t e = hipSuccess;
    if (p.wide) {
        for (int64_t first = 0; first < a.N && e == hipSuccess; first += kMaxGrid) {
            const int64_t wgs = std::min<int64_t>(kMaxGrid, a.N - first);
            hipLaunchKernelGGL((norm_grad_long_kernel<T>), dim3(static_cast<unsigned>(wgs)), block,
                               0, stream, a, first);
            e = hipGetLastError();
        }
        if (e == hipSuccess && dw != nullptr) {
            const unsigned across = static_cast<unsigned>((runs + kNormThreads - 1) / kNormThreads);
            hipLaunchKernelGGL((norm_columns_kernel<T>), dim3(p.wgs, across), block, 0, stream, a,
                               p.rows_per_wg);
            e = hipGetLastError();
        }
    } else {
        auto launch = [&](auto lanes, auto held) {
            constexpr int G = decltype(lanes)::value, R = decltype(held)::value;
            const dim3 threads(threads_for(G));
            const bool deep = p.deep && dw != nullptr;
            if (a.D % kRun == 0 && !deep)
                hipLaunchKernelGGL((norm_grad_kernel<T, G, R, true, false>), grid, threads, 0,
                                   stream, a);
            else if (a.D % kRun == 0)
                hipLaunchKernelGGL((norm_grad_kernel<T, G, R, true, true>), grid, threads, 0,
                                   stream, a);
            else if (!deep)
                hipLaunchKernelGGL((norm_grad_kernel<T, G, R, false, false>), grid, threads, 0,
                                   stream, a);
            else
                hipLaunchKernelGGL((norm_grad_kernel<T, G, R, false, true>), grid, threads, 0,
                                   stream, a);
        };
        if (runs <= 16)
            launch(Int<16>{}, Int<1>{});
        else if (runs <= 32)
            launch(Int<32>{}, Int<1>{});
        else if (runs <= 64)
            launch(Int<64>{}, Int<1>{});
        else if (runs <= 128)
            launch(Int<128>{}, Int<1>{});
        else if (runs <= 256)
            launch(Int<256>{}, Int<1>{});
        else if (runs <= 512)
            launch(Int<512>{}, Int<1>{});
        else if (runs <= 1024)
            launch(Int<1024>{}, Int<1>{});
        else
            launch(Int<1024>{}, Int<2>{});
        e = hipGetLastError();
    }
    if (e == hipSuccess && dw != nullptr) {
        const dim3 columns((a.D + kJoinCols - 1) / kJoinCols), threads(kJoinCols * kJoinShares);
        if (p.deep)
            hipLaunchKernelGGL((norm_join_kernel<T, double>), columns, threads, 0, stream,
                               static_cast<const double *>(a.dw_partial), p.wgs, a.D, dw);
        else
            hipLaunchKernelGGL((norm_join_kernel<T, float>), columns, threads, 0, stream,
                               static_cast<const float *>(a.dw_partial), p.wgs, a.D, dw);
        e = hipGetLastError();
    }
    return e;
}

template <typename T>
hipError_t run_zero(void *p, int64_t n, hipStream_t stream) {
    hipLaunchKernelGGL((norm_zero_kernel<T>), dim3(static_cast<unsigned>((n + 255) / 256)),
                       dim3(256), 0, stream, static_cast<typename T::bits *>(p),
                       static_cast<int>(n));
    return hipGetLastError();
}

template <typename T, int ROWS>
hipError_t launch_quantize(const Quantize &a, hipStream_t stream) {
    const int64_t tiles = (static_cast<int64_t>(a.N) + kFp8Block - 1) / kFp8Block *
                          ((a.D + kFp8Block - 1) / kFp8Block);
    hipLaunchKernelGGL((quantize_kernel<T, ROWS>),
                       dim3(static_cast<unsigned>(std::min(tiles, kMaxGrid))), dim3(kNormThreads),
                       0, stream, a);
    return hipGetLastError();
}

template <typename T>
hipError_t run_quantize(const Quantize &a, int rows, hipStream_t stream) {
    return rows == 1 ? launch_quantize<T, 1>(a, stream) : launch_quantize<T, kFp8Block>(a, stream);
}

// ---- checks ----------------------------------------------------------------

kmeans_status_t check_sizes(int64_t N, int64_t D, int32_t dtype) {
    if (N < 0 || D < 1)
        return fail(KMEANS_ERR_INVALID_ARG, "N=%lld must be >= 0 and D=%lld >= 1",
                    static_cast<long long>(N), static_cast<long long>(D));
    if (dtype < KMEANS_BF16 || dtype > KMEANS_FP32)
        return fail(KMEANS_ERR_INVALID_ARG, "dtype=%d is not a kmeans_dtype_t", dtype);
    if (N > kMaxRows || D > kMaxNormWidth)
        return fail(KMEANS_ERR_UNSUPPORTED, "N=%lld or D=%lld too large (max %lld, %lld)",
                    static_cast<long long>(N), static_cast<long long>(D),
                    static_cast<long long>(kMaxRows), static_cast<long long>(kMaxNormWidth));
    return KMEANS_OK;
}

}  // namespace

kmeans_status_t check_matrix(const char *name, const void *p, int64_t cols, int64_t ld,
                             size_t element) {
    if (p == nullptr)
        return fail(KMEANS_ERR_INVALID_ARG, "null pointer argument (%s)", name);
    if (!aligned(p, element))
        return fail(KMEANS_ERR_ALIGNMENT, "%s must be %zu-byte aligned", name, element);
    if (ld < cols)
        return fail(KMEANS_ERR_INVALID_ARG, "%s: row stride %lld below the row length %lld", name,
                    static_cast<long long>(ld), static_cast<long long>(cols));
    if (ld > kMaxRows)
        return fail(KMEANS_ERR_UNSUPPORTED, "%s: row stride %lld too large (max %lld)", name,
                    static_cast<long long>(ld), static_cast<long long>(kMaxRows));
    return KMEANS_OK;
}

kmeans_status_t check_array(const char *name, const void *p, size_t element) {
    if (!aligned(p, element))
        return fail(KMEANS_ERR_ALIGNMENT, "%s must be %zu-byte aligned", name, element);
    return KMEANS_OK;
}

}  // namespace kmeans

// ---- C entry points --------------------------------------------------------

extern "C" kmeans_status_t kmeans_rms_norm(const void *X, int64_t x_stride, const void *residual,
                                           int64_t residual_stride, const void *weight, int64_t N,
                                           int64_t D, int32_t dtype, float eps, void *sum,
                                           int64_t sum_stride, void *Y, int64_t y_stride, void *Q,
                                           int64_t q_stride, float *scales, int64_t scales_stride,
                                           hipStream_t stream) {
    using namespace kmeans;
    kmeans_status_t st = check_sizes(N, D, dtype);
    if (st != KMEANS_OK)
        return st;
    if (!(eps >= 0.0f))
        return fail(KMEANS_ERR_INVALID_ARG, "eps=%g must be >= 0", static_cast<double>(eps));
    if (N == 0)
        return ok();
    const size_t size = dtype_size(dtype);
    if ((Y != nullptr) == (Q != nullptr))
        return fail(KMEANS_ERR_INVALID_ARG, "one of Y=%p and Q=%p must be given", Y, Q);
    if ((st = check_matrix("X", X, D, x_stride, size)) != KMEANS_OK ||
        (residual && (st = check_matrix("residual", residual, D, residual_stride, size)) != KMEANS_OK) ||
        (st = check_array("weight", weight, size)) != KMEANS_OK ||
        (sum && (st = check_matrix("sum", sum, D, sum_stride, size)) != KMEANS_OK) ||
        (Y && (st = check_matrix("Y", Y, D, y_stride, size)) != KMEANS_OK) ||
        (Q && (st = check_matrix("Q", Q, D, q_stride, 1)) != KMEANS_OK) ||
        (Q && (st = check_matrix("scales", scales, fp8_blocks(D), scales_stride, 4)) != KMEANS_OK))
        return st;
    const Norm a{X, residual, weight, sum, Y, static_cast<uint8_t *>(Q), scales, x_stride,
                 residual_stride, sum_stride, y_stride, q_stride, scales_stride, 0,
                 static_cast<int>(N), static_cast<int>(D), eps};
    const hipError_t e = dtype == KMEANS_BF16   ? run_norm<Bf16>(a, stream)
                         : dtype == KMEANS_FP16 ? run_norm<Fp16>(a, stream)
                                                : run_norm<Fp32>(a, stream);
    if (e != hipSuccess)
        return fail(KMEANS_ERR_HIP, "norm launch failed: %s", hipGetErrorString(e));
    return ok();
}

extern "C" kmeans_status_t kmeans_rms_norm_grad(const void *dY, int64_t dy_stride, const void *H,
                                                int64_t h_stride, const void *weight,
                                                const void *dH, int64_t dh_stride, int64_t N,
                                                int64_t D, int32_t dtype, float eps, void *dX,
                                                int64_t dx_stride, void *dweight,
                                                hipStream_t stream) {
    using namespace kmeans;
    kmeans_status_t st = check_sizes(N, D, dtype);
    if (st != KMEANS_OK)
        return st;
    if (!(eps >= 0.0f))
        return fail(KMEANS_ERR_INVALID_ARG, "eps=%g must be >= 0", static_cast<double>(eps));
    const size_t size = dtype_size(dtype);
    if ((st = check_array("dweight", dweight, size)) != KMEANS_OK)
        return st;
    if (N == 0) {
        if (dweight == nullptr)
            return ok();
        const hipError_t e = dtype == KMEANS_FP32 ? run_zero<Fp32>(dweight, D, stream)
                                                  : run_zero<Bf16>(dweight, D, stream);
        if (e != hipSuccess)
            return fail(KMEANS_ERR_HIP, "norm gradient launch failed: %s", hipGetErrorString(e));
        return ok();
    }
    if ((st = check_matrix("dY", dY, D, dy_stride, size)) != KMEANS_OK ||
        (st = check_matrix("H", H, D, h_stride, size)) != KMEANS_OK ||
        (st = check_array("weight", weight, size)) != KMEANS_OK ||
        (dH && (st = check_matrix("dH", dH, D, dh_stride, size)) != KMEANS_OK) ||
        (st = check_matrix("dX", dX, D, dx_stride, size)) != KMEANS_OK)
        return st;
    const NormGradPlan p(N, D, device_compute_units());
    const size_t r_bytes = p.wide ? (static_cast<size_t>(N) * sizeof(float) + 255) / 256 * 256 : 0;
    NormGrad a{dY, H, weight, dH, dX, nullptr, nullptr, dy_stride, h_stride, dh_stride, dx_stride,
               static_cast<int>(N), static_cast<int>(D), eps};
    std::optional<WorkspaceLease> lease;
    if (dweight != nullptr) {
        const size_t bytes = r_bytes + p.partial_bytes(D);
        lease.emplace(stream, bytes);
        if (lease->error() != hipSuccess)
            return fail(KMEANS_ERR_NO_MEMORY, "workspace of %zu bytes: %s", bytes,
                        hipGetErrorString(lease->error()));
        char *ws = static_cast<char *>(lease->ptr());
        a.r = p.wide ? reinterpret_cast<float *>(ws) : nullptr;
        a.dw_partial = ws + r_bytes;
    }
    const hipError_t e = dtype == KMEANS_BF16   ? run_norm_grad<Bf16>(a, p, dweight, stream)
                         : dtype == KMEANS_FP16 ? run_norm_grad<Fp16>(a, p, dweight, stream)
                                                : run_norm_grad<Fp32>(a, p, dweight, stream);
    if (e != hipSuccess)
        return fail(KMEANS_ERR_HIP, "norm gradient launch failed: %s", hipGetErrorString(e));
    return ok();
}

extern "C" kmeans_status_t kmeans_quantize(const void *X, int64_t x_stride, int64_t N, int64_t D,
                                           int32_t dtype, int32_t block_rows, void *Q,
                                           int64_t q_stride, float *scales, int64_t scales_stride,
                                           hipStream_t stream) {
    using namespace kmeans;
    kmeans_status_t st = check_sizes(N, D, dtype);
    if (st != KMEANS_OK)
        return st;
    if (block_rows != 1 && block_rows != kFp8Block)
        return fail(KMEANS_ERR_INVALID_ARG, "block_rows=%d must be 1 or %d", block_rows, kFp8Block);
    if (N == 0)
        return ok();
    if ((st = check_matrix("X", X, D, x_stride, dtype_size(dtype))) != KMEANS_OK ||
        (st = check_matrix("Q", Q, D, q_stride, 1)) != KMEANS_OK ||
        (st = check_matrix("scales", scales, fp8_blocks(D), scales_stride, 4)) != KMEANS_OK)
        return st;
    const Quantize a{X, static_cast<uint8_t *>(Q), scales, x_stride, q_stride, scales_stride,
                     static_cast<int>(N), static_cast<int>(D)};
    const hipError_t e = dtype == KMEANS_BF16   ? run_quantize<Bf16>(a, block_rows, stream)
                         : dtype == KMEANS_FP16 ? run_quantize<Fp16>(a, block_rows, stream)
                                                : run_quantize<Fp32>(a, block_rows, stream);
    if (e != hipSuccess)
        return fail(KMEANS_ERR_HIP, "quantize launch failed: %s", hipGetErrorString(e));
    return ok();
}
