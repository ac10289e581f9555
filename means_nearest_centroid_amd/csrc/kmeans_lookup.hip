// kmeans_lookup.hip -- gfx950 kernels of the table lookup and of its gradient.
//
//     lookup     Y[i]  = scale * C[labels[i]]        (zero for a stray label)
//     gradient   dC[k] = scale * sum of dY[i] over labels[i] == k
//
// Both move rows and compute next to nothing: the bound is the bytes of the
// rows, read once and written once.
//
// Gradient.  The positions are sorted by label (the stable radix sort of the
// centroid update), so that a label's rows are one run of sorted positions.
//  1. lookup_sum_kernel walks fixed chunks of sorted positions; a group of
//     lanes that together hold one row's columns owns one chunk and sums each
//     run in position order.  A run inside the chunk is finished there (one
//     rounding); a run cut by a chunk edge leaves its partial sum.  Work per
//     group is bounded whatever the label frequencies are.  Further
//     workgroups of the same launch zero the rows that no label names.
//  2. lookup_join_kernel adds the partial sums of the runs that were cut, in
//     an order fixed by the chunks.
// No atomics: the order of every sum follows from the labels alone.
#include <stdint.h>

#include <algorithm>
#include <memory>

#include "kmeans_types.h"
#include "kmeans_update_internal.h"

namespace kmeans {
namespace {

constexpr int kRowThreads = 256;

// The label as a row of the table, -1 for a stray one.
template <typename L>
__device__ __forceinline__ int table_row(L label, int K) {
    return label < 0 || label >= K ? -1 : static_cast<int>(label);
}

// ---- lookup ----------------------------------------------------------------

// Pieces of V elements (16 bytes), `pieces` per row; the last piece of a row
// of D >= V elements starts at D - V, so it may write elements of the piece
// before it a second time (the same values) and no row needs a scalar tail.
// Rows shorter than V move by elements.  Each thread moves kUnroll pieces
// whose loads are in flight together.
constexpr int kUnroll = 4;
template <typename T, int V, typename L>
__global__ __launch_bounds__(kRowThreads)
void lookup_kernel(const typename T::bits *__restrict__ C, int64_t ldc, const L *__restrict__ labels,
                   int64_t N, int D, int K, float scale, int pieces, uint32_t inv,
                   typename T::bits *__restrict__ Y, int64_t ldy) {
    typedef typename T::bits B;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * (kUnroll * kRowThreads);
    const int64_t row0 = first / pieces;
    const uint32_t rem0 = static_cast<uint32_t>(first - row0 * pieces);
    int64_t row[kUnroll];
    int col[kUnroll], from[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const uint32_t x = rem0 + u * kRowThreads + threadIdx.x;
        // x / pieces for x < pieces + 1024: inv = ceil(2^32 / pieces), one
        // too high at most.
        uint32_t q = inv != 0 ? __umulhi(x, inv) : x;
        q -= q * pieces > x ? 1 : 0;
        row[u] = row0 + q;
        col[u] = min(static_cast<int>(x - q * pieces) * V, max(D - V, 0));
        from[u] = row[u] < N ? table_row(labels[row[u]], K) : -1;
    }
    if (D >= V) {
        Packed<B, V> v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            v[u] = from[u] >= 0 ? load_packed<B, V>(C + from[u] * ldc + col[u]) : Packed<B, V>{};
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            float x[V];
#pragma unroll
            for (int e = 0; e < V; ++e)
                x[e] = from[u] >= 0 ? scale * T::widen(v[u].v[e]) : 0.0f;
            if (row[u] < N)
                store_packed<B, V>(Y + row[u] * ldy + col[u], narrow_run<T, V>(x));
        }
    } else {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (row[u] < N)
                for (int e = 0; e < D; ++e)
                    Y[row[u] * ldy + e] =
                        from[u] >= 0 ? T::narrow(scale * T::widen(C[from[u] * ldc + e])) : B(0);
    }
}

// ---- gradient --------------------------------------------------------------

constexpr int kBatch = 8;          // rows of one group whose loads are in flight together
constexpr int kFillRows = 64;      // table rows per zero-filling workgroup
constexpr int kJoinChunks = 16;    // chunks examined by one join workgroup
constexpr int kLongRun = 64;       // partial sums from which a whole workgroup joins a run

struct GradArgs {
    const void *dY;
    int64_t ldy;
    const int32_t *keys, *vals;   // sorted labels (K: stray) and positions
    int N, D, K;
    float scale;
    int accumulate;
    void *dC;
    int64_t ldc;
    float *partial;               // [chunks][2][D]
    int chunk, chunks;            // positions per chunk
    int lanes_log2;               // lanes of a group
    int slabs;                    // column slabs of (lanes V) columns
};

// Columns c0 .. c0 + n - 1 of row k from the sums: scaled, added to the row
// where asked, rounded once.
template <typename O, int V>
__device__ __forceinline__ void finish_row(const GradArgs &g, int k, int c0, int n,
                                           const float (&sum)[V]) {
    typedef typename O::bits B;
    B *o = static_cast<B *>(g.dC) + k * g.ldc + c0;
    float v[V];
    if (g.accumulate) {
        const Packed<B, V> old = load_run<B, V>(o, n);
#pragma unroll
        for (int e = 0; e < V; ++e)
            v[e] = fmaf(g.scale, sum[e], O::widen(old.v[e]));
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
            v[e] = g.scale * sum[e];
    }
    store_run<B, V>(o, n, narrow_run<O, V>(v));
}

template <int V>
__device__ __forceinline__ void store_partial(float *p, int n, const float (&sum)[V]) {
    store_run<float, V>(p, n, narrow_run<Fp32, V>(sum));
}

// First position whose key is at least `key` (lower) or greater (upper).
__device__ __forceinline__ int bound_of(const int32_t *keys, int lo, int hi, int key, bool upper) {
    while (lo < hi) {
        const int mid = lo + ((hi - lo) >> 1);
        if (keys[mid] < key || (upper && keys[mid] == key))
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo;
}

// Workgroups [0, sum_wgs): chunks; [sum_wgs, ...): rows to be zeroed.
template <typename T, typename O, int V>
__global__ __launch_bounds__(kRowThreads)
void lookup_sum_kernel(const GradArgs g, int sum_wgs) {
    typedef typename T::bits B;
    const int tid = threadIdx.x;
    const int lanes = 1 << g.lanes_log2;
    const int l = tid & (lanes - 1);
    if (static_cast<int>(blockIdx.x) >= sum_wgs) {
        // Zero the rows that no label names: kFillRows of them, this slab.
        __shared__ uint8_t named[kFillRows];
        const int r0 = (blockIdx.x - sum_wgs) * kFillRows;
        if (tid < kFillRows) {
            const int k = r0 + tid;
            const int p = bound_of(g.keys, 0, g.N, k, false);
            named[tid] = p < g.N && g.keys[p] == k;
        }
        __syncthreads();
        const float zero[V] = {};
        const int c0 = (blockIdx.y * lanes + l) * V;
        const int n = g.D - c0;
        if (n <= 0)
            return;
        for (int r = tid >> g.lanes_log2; r < kFillRows; r += kRowThreads >> g.lanes_log2)
            if (r0 + r < g.K && !named[r])
                finish_row<O, V>(g, r0 + r, c0, n, zero);
        return;
    }
    const int c = blockIdx.x * (kRowThreads >> g.lanes_log2) + (tid >> g.lanes_log2);
    const int c0 = (blockIdx.y * lanes + l) * V;
    const int n = g.D - c0;
    if (c >= g.chunks || n <= 0)
        return;
    const int beg = c * g.chunk;
    const int end = static_cast<int>(min(static_cast<int64_t>(g.N),
                                         static_cast<int64_t>(beg) + g.chunk));
    const B *src = static_cast<const B *>(g.dY) + c0;
    float *part = g.partial + static_cast<int64_t>(c) * 2 * g.D + c0;
    int cur = g.keys[beg];
    bool open_left = beg > 0 && g.keys[beg - 1] == cur;
    float sum[V] = {};
    for (int p0 = beg; p0 < end && cur < g.K; p0 += kBatch) {
        int key[kBatch];
        Packed<B, V> row[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int p = min(p0 + u, end - 1);
            key[u] = p0 + u < end ? g.keys[p] : -1;
            row[u] = load_run<B, V>(src + g.vals[p] * g.ldy, n);
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (key[u] < 0)
                continue;
            if (key[u] != cur) {
                if (cur < g.K) {
                    if (open_left)
                        store_partial<V>(part, n, sum);
                    else
                        finish_row<O, V>(g, cur, c0, n, sum);
                }
                open_left = false;
                cur = key[u];
#pragma unroll
                for (int e = 0; e < V; ++e)
                    sum[e] = 0.0f;
            }
#pragma unroll
            for (int e = 0; e < V; ++e)
                sum[e] += T::widen(row[u].v[e]);
        }
    }
    if (cur >= g.K)
        return;
    const bool open_right = end < g.N && g.keys[end] == cur;
    if (open_left)
        store_partial<V>(part, n, sum);
    else if (open_right)
        store_partial<V>(part + g.D, n, sum);
    else
        finish_row<O, V>(g, cur, c0, n, sum);
}

// A run that was cut began in some chunk c (slot 1 of c) and went on through
// chunks c + 1 .. c + m (slot 0 of each).  Each workgroup looks for such
// beginnings in kJoinChunks chunks.  A group of lanes adds a short run's
// partial sums in order; a run of kLongRun or more is shared by the
// workgroup's groups (group q takes the partial sums q, q + groups, ...),
// whose sums are then added in group order.
template <typename O, int V>
__global__ __launch_bounds__(kRowThreads)
void lookup_join_kernel(const GradArgs g) {
    __shared__ int key_of[kJoinChunks], more[kJoinChunks];
    __shared__ float sums[kRowThreads][V + 1];
    const int tid = threadIdx.x;
    const int lanes = 1 << g.lanes_log2, groups = kRowThreads >> g.lanes_log2;
    const int l = tid & (lanes - 1), q = tid >> g.lanes_log2;
    const int first = blockIdx.x * kJoinChunks;
    if (tid < kJoinChunks) {
        const int c = first + tid;
        int m = 0, k = g.K;
        if (c < g.chunks - 1) {           // the last chunk has no next one
            const int beg = c * g.chunk, end = beg + g.chunk;
            k = g.keys[end - 1];
            const bool began_here = g.keys[beg] != k || beg == 0 || g.keys[beg - 1] != k;
            if (k < g.K && began_here && g.keys[end] == k) {
                // Chunks after c that the run reaches: nearly always one.
                int stop = end + 1;
                if (g.chunk <= g.N - end && g.keys[end + g.chunk - 1] == k)
                    stop = bound_of(g.keys, end + g.chunk, g.N, k, true);
                m = (stop - 1) / g.chunk - c;
            }
        }
        key_of[tid] = k;
        more[tid] = m;
    }
    __syncthreads();
    const int c0 = (blockIdx.y * lanes + l) * V;
    const int n = g.D - c0;
    for (int x = q; x < kJoinChunks; x += groups) {
        const int m = more[x];
        if (m == 0 || m >= kLongRun || n <= 0)
            continue;
        const float *p = g.partial + static_cast<int64_t>(first + x) * 2 * g.D + c0;
        const Packed<float, V> head = load_run<float, V>(p + g.D, n);
        float sum[V];
#pragma unroll
        for (int e = 0; e < V; ++e)
            sum[e] = head.v[e];
        for (int s = 1; s <= m; ++s) {
            const Packed<float, V> w =
                load_run<float, V>(p + static_cast<int64_t>(s) * 2 * g.D, n);
#pragma unroll
            for (int e = 0; e < V; ++e)
                sum[e] += w.v[e];
        }
        finish_row<O, V>(g, key_of[x], c0, n, sum);
    }
    for (int x = 0; x < kJoinChunks; ++x) {
        const int m = more[x];
        if (m < kLongRun)
            continue;
        const float *p = g.partial + static_cast<int64_t>(first + x) * 2 * g.D + c0;
        float sum[V] = {};
        if (n > 0)
            for (int s = q; s <= m; s += groups) {
                const Packed<float, V> w = load_run<float, V>(
                    s == 0 ? p + g.D : p + static_cast<int64_t>(s) * 2 * g.D, n);
#pragma unroll
                for (int e = 0; e < V; ++e)
                    sum[e] += w.v[e];
            }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < V; ++e)
            sums[tid][e] = sum[e];
        __syncthreads();
        if (q == 0 && n > 0) {
            for (int r = 1; r < groups; ++r)
#pragma unroll
                for (int e = 0; e < V; ++e)
                    sum[e] += sums[r * lanes + l][e];
            finish_row<O, V>(g, key_of[x], c0, n, sum);
        }
    }
}

// ---- launch ----------------------------------------------------------------

struct GradPlan {
    LabelSort sort;
    int chunk, chunks, lanes_log2, slabs;
    size_t partial, bytes;
};

GradPlan make_grad_plan(int64_t N, int64_t D, int64_t K, int V, int compute_units) {
    GradPlan p{};
    while (p.lanes_log2 < 6 && (int64_t(V) << p.lanes_log2) < D)
        ++p.lanes_log2;
    p.slabs = static_cast<int>((D + (int64_t(V) << p.lanes_log2) - 1) / (int64_t(V) << p.lanes_log2));
    if (N == 0)
        return p;
    // Chunks of at least 8 positions, more when that leaves eight waves or
    // more per CU.
    const int64_t waves_at_1 = ((N << p.lanes_log2) + 63) / 64 * p.slabs;
    int64_t chunk = 8;
    while (chunk < 4096 && waves_at_1 / (2 * chunk) >= 8 * compute_units)
        chunk *= 2;
    p.chunk = static_cast<int>(chunk);
    p.chunks = static_cast<int>((N + chunk - 1) / chunk);
    p.sort = make_label_sort(N, K);
    p.partial = (p.sort.bytes + 255) & ~size_t(255);
    p.bytes = p.partial + static_cast<size_t>(p.chunks) * 2 * D * sizeof(float);
    return p;
}

template <typename T, typename O, int V>
hipError_t launch_grad(const GradPlan &p, const GradArgs &g, hipStream_t stream) {
    const int per_wg = kRowThreads >> p.lanes_log2;
    const int sum_wgs = (p.chunks + per_wg - 1) / per_wg;
    const int fill_wgs = g.accumulate ? 0 : (g.K + kFillRows - 1) / kFillRows;
    if (sum_wgs + fill_wgs > 0) {
        hipLaunchKernelGGL((lookup_sum_kernel<T, O, V>), dim3(sum_wgs + fill_wgs, p.slabs),
                           dim3(kRowThreads), 0, stream, g, sum_wgs);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    if (p.chunks > 1)
        hipLaunchKernelGGL((lookup_join_kernel<O, V>),
                           dim3((p.chunks + kJoinChunks - 1) / kJoinChunks, p.slabs),
                           dim3(kRowThreads), 0, stream, g);
    return hipGetLastError();
}

template <typename T, typename L>
hipError_t launch_lookup(const void *C, int64_t ldc, const void *labels, int64_t N, int64_t D,
                         int64_t K, float scale, void *Y, int64_t ldy, hipStream_t stream) {
    typedef typename T::bits B;
    constexpr int V = 16 / sizeof(B);
    const int64_t pieces = (D + V - 1) / V;
    const uint32_t inv = pieces == 1 ? 0
                                     : static_cast<uint32_t>(((uint64_t(1) << 32) + pieces - 1) / pieces);
    const int64_t wgs = (N * pieces + kUnroll * kRowThreads - 1) / (kUnroll * kRowThreads);
    hipLaunchKernelGGL((lookup_kernel<T, V, L>), dim3(static_cast<unsigned>(wgs)), dim3(kRowThreads),
                       0, stream, static_cast<const B *>(C), ldc, static_cast<const L *>(labels),
                       N, static_cast<int>(D), static_cast<int>(K), scale,
                       static_cast<int>(pieces), inv, static_cast<B *>(Y), ldy);
    return hipGetLastError();
}

kmeans_status_t check_table(int64_t N, int64_t D, int64_t K, int32_t dtype, int32_t label_type,
                            const void *labels) {
    if (N < 0 || D < 1 || K < 1)
        return fail(KMEANS_ERR_INVALID_ARG, "N=%lld must be >= 0, D=%lld and K=%lld >= 1",
                    static_cast<long long>(N), static_cast<long long>(D),
                    static_cast<long long>(K));
    if (N > kMaxRows || D > kMaxRows || K > kMaxRows)
        return fail(KMEANS_ERR_UNSUPPORTED, "N=%lld, D=%lld or K=%lld too large (max %lld)",
                    static_cast<long long>(N), static_cast<long long>(D),
                    static_cast<long long>(K), static_cast<long long>(kMaxRows));
    if (dtype < KMEANS_BF16 || dtype > KMEANS_FP32)
        return fail(KMEANS_ERR_INVALID_ARG, "dtype=%d is not a kmeans_dtype_t", dtype);
    if (label_type != KMEANS_INT32 && label_type != KMEANS_INT64)
        return fail(KMEANS_ERR_INVALID_ARG, "label_type=%d is not a kmeans_label_t", label_type);
    if (N > 0 && labels == nullptr)
        return fail(KMEANS_ERR_INVALID_ARG, "null pointer argument (labels)");
    if (N > 0 && !aligned(labels, label_type == KMEANS_INT64 ? 8 : 4))
        return fail(KMEANS_ERR_ALIGNMENT, "labels must be aligned to their size");
    return KMEANS_OK;
}

kmeans_status_t check_rows(const char *name, const void *p, int64_t D, int64_t ld,
                           int32_t dtype) {
    if (p == nullptr)
        return fail(KMEANS_ERR_INVALID_ARG, "null pointer argument (%s)", name);
    if (ld < D)
        return fail(KMEANS_ERR_INVALID_ARG, "%s: row stride %lld below D=%lld", name,
                    static_cast<long long>(ld), static_cast<long long>(D));
    if (!aligned(p, dtype_size(dtype)))
        return fail(KMEANS_ERR_ALIGNMENT, "%s must be aligned to its element size", name);
    return KMEANS_OK;
}

}  // namespace
}  // namespace kmeans

// ---- C entry points --------------------------------------------------------

extern "C" kmeans_status_t kmeans_lookup(const void *C, int64_t c_stride, const void *labels,
                                         int32_t label_type, int64_t N, int64_t D, int64_t K,
                                         int32_t dtype, float scale, void *Y, int64_t y_stride,
                                         hipStream_t stream) {
    using namespace kmeans;
    kmeans_status_t st = check_table(N, D, K, dtype, label_type, labels);
    if (st != KMEANS_OK)
        return st;
    if (N == 0)
        return ok();
    if ((st = check_rows("C", C, D, c_stride, dtype)) != KMEANS_OK ||
        (st = check_rows("Y", Y, D, y_stride, dtype)) != KMEANS_OK)
        return st;
    const int64_t per_wg = kUnroll * kRowThreads;
    const int64_t v = 16 / static_cast<int64_t>(dtype_size(dtype));
    if ((N * ((D + v - 1) / v) + per_wg - 1) / per_wg > kMaxRows)
        return fail(KMEANS_ERR_UNSUPPORTED, "N=%lld rows of D=%lld: too many elements",
                    static_cast<long long>(N), static_cast<long long>(D));
    hipError_t e;
    const bool wide = label_type == KMEANS_INT64;
    switch (dtype) {
    case KMEANS_BF16:
        e = wide ? launch_lookup<Bf16, int64_t>(C, c_stride, labels, N, D, K, scale, Y, y_stride, stream)
                 : launch_lookup<Bf16, int32_t>(C, c_stride, labels, N, D, K, scale, Y, y_stride, stream);
        break;
    case KMEANS_FP16:
        e = wide ? launch_lookup<Fp16, int64_t>(C, c_stride, labels, N, D, K, scale, Y, y_stride, stream)
                 : launch_lookup<Fp16, int32_t>(C, c_stride, labels, N, D, K, scale, Y, y_stride, stream);
        break;
    default:
        e = wide ? launch_lookup<Fp32, int64_t>(C, c_stride, labels, N, D, K, scale, Y, y_stride, stream)
                 : launch_lookup<Fp32, int32_t>(C, c_stride, labels, N, D, K, scale, Y, y_stride, stream);
        break;
    }
    if (e != hipSuccess)
        return fail(KMEANS_ERR_HIP, "lookup launch failed: %s", hipGetErrorString(e));
    return ok();
}

extern "C" kmeans_status_t kmeans_lookup_grad(const void *dY, int64_t dy_stride,
                                              const void *labels, int32_t label_type, int64_t N,
                                              int64_t D, int64_t K, int32_t dtype, float scale,
                                              int32_t accumulate, void *dC, int32_t out_dtype,
                                              int64_t dc_stride, hipStream_t stream) {
    using namespace kmeans;
    kmeans_status_t st = check_table(N, D, K, dtype, label_type, labels);
    if (st != KMEANS_OK)
        return st;
    if (out_dtype != dtype && out_dtype != KMEANS_FP32)
        return fail(KMEANS_ERR_INVALID_ARG, "out_dtype=%d must be dtype=%d or KMEANS_FP32",
                    out_dtype, dtype);
    if ((st = check_rows("dC", dC, D, dc_stride, out_dtype)) != KMEANS_OK ||
        (N > 0 && (st = check_rows("dY", dY, D, dy_stride, dtype)) != KMEANS_OK))
        return st;
    if (N == 0 && accumulate)
        return ok();
    const int V = 16 / static_cast<int>(dtype_size(dtype));
    const GradPlan p = make_grad_plan(N, D, K, V, device_compute_units());
    if (p.slabs > 65535)
        return fail(KMEANS_ERR_UNSUPPORTED, "D=%lld too large", static_cast<long long>(D));
    GradArgs g{};
    g.dY = dY;
    g.ldy = dy_stride;
    g.N = static_cast<int>(N);
    g.D = static_cast<int>(D);
    g.K = static_cast<int>(K);
    g.scale = scale;
    g.accumulate = accumulate != 0;
    g.dC = dC;
    g.ldc = dc_stride;
    g.chunk = p.chunk;
    g.chunks = p.chunks;
    g.lanes_log2 = p.lanes_log2;
    g.slabs = p.slabs;
    std::unique_ptr<WorkspaceLease> lease;
    hipError_t e = hipSuccess;
    if (N > 0) {
        lease = std::make_unique<WorkspaceLease>(stream, p.bytes);
        if (lease->error() != hipSuccess)
            return fail(KMEANS_ERR_NO_MEMORY, "workspace of %zu bytes: %s", p.bytes,
                        hipGetErrorString(lease->error()));
        auto *ws = static_cast<char *>(lease->ptr());
        g.partial = reinterpret_cast<float *>(ws + p.partial);
        e = launch_label_sort(p.sort, labels, label_type, g.N, g.K, ws, &g.keys, &g.vals, stream);
    }
    if (e == hipSuccess) {
        if (dtype == KMEANS_BF16)
            e = out_dtype == dtype ? launch_grad<Bf16, Bf16, 8>(p, g, stream)
                                   : launch_grad<Bf16, Fp32, 8>(p, g, stream);
        else if (dtype == KMEANS_FP16)
            e = out_dtype == dtype ? launch_grad<Fp16, Fp16, 8>(p, g, stream)
                                   : launch_grad<Fp16, Fp32, 8>(p, g, stream);
        else
            e = launch_grad<Fp32, Fp32, 4>(p, g, stream);
    }
    if (e != hipSuccess)
        return fail(KMEANS_ERR_HIP, "lookup gradient launch failed: %s", hipGetErrorString(e));
    return ok();
}
