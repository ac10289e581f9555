// kmeans_clip.hip -- gfx950 kernels of the global gradient norm over a list of
// tensors and of clipping by it.
//
//     n = sqrt(sum of all squares),   dst = src * min(1, max_norm / (n + 1e-6))
//
// Bound by memory: every element is read once for the norm and, since n is
// needed before the first product, read again and written once.  The list
// travels in the kernel arguments (no device table, nothing to upload), in
// batches of kBatch tensors.  Pass 1: a fixed set of workgroups walks fixed
// chunks of the batch's tensors, each leaving one fp64 partial sum.  Pass 2:
// every workgroup adds all partial sums in one fixed order, so all of them
// derive the same factor without a third launch, and scales its chunks.  A
// list of at most kSmallBytes is one launch of one workgroup, its waves taking
// the chunks, which costs less there than a second launch (one launch, two: 60
// KB 7.8 us, 10.5; 200 KB 9.5, 10.2; 400 KB 15.0, 10.1; 12 tensors of 200 KB,
// bound by the host, 13.0, 16.0).
// 2^28 bf16 values out of place: 278 us (1.61 GB moved, 5.8 TB/s; the norm
// alone 93 us); 322 with the second pass in the first one's order and plain
// stores; 2048 or 4096 workgroups instead of 1024 within 2%.
// Squares are summed in fp64: no fp32 value over- or underflows there, and
// the conversions and additions stay far below the memory time.
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "kmeans_internal.h"
#include "kmeans_types.h"

namespace kmeans {
namespace {

constexpr int kClipThreads = 256;
constexpr int kBatch = 96;                 // tensors per launch: 2.8 KiB of arguments
constexpr int kLoads = 8;                  // 16-byte loads of a thread in flight
// Bytes of a source that `threads` threads take as one chunk.
constexpr int chunk_bytes(int threads) { return kLoads * 16 * threads; }
constexpr int kSmallThreads = 1024;        // waves of the one-workgroup kernel: 16
constexpr int64_t kSmallBytes = 320 << 10;
constexpr int64_t kMaxPartials = 1024;
constexpr int64_t kMaxElements = int64_t(1) << 40;

struct Batch {
    const void *src[kBatch];
    void *dst[kBatch];
    int64_t numel[kBatch];
    int first[kBatch + 1];   // first chunk of each tensor
    uint8_t dtype[kBatch];
    int count;
    int first_partial;       // of this batch's workgroups
};

// Tensor that chunk c belongs to (wave-uniform).
__device__ __forceinline__ int tensor_of(const Batch &b, int c) {
    int lo = 0, hi = b.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (b.first[mid] <= c)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1)
        v += __shfl_xor(v, m, 64);
    return v;
}

// The workgroup's total, on every thread.
template <int THREADS>
__device__ __forceinline__ double group_sum(double v) {
    __shared__ double total[THREADS / 64];
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        total[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w)
        s += total[w];
    return s;
}

// Chunk `c` of a tensor: elements [c E, min(numel, (c + 1) E)), E = elements
// of chunk_bytes(THREADS); `tid` of THREADS threads takes kLoads runs of V
// elements.  A whole chunk has all of them in flight together; one that the
// tensor's end cuts short has kPartLoads, and its last elements (fewer than V)
// go one to a thread.
constexpr int kPartLoads = 4;

template <typename T, int THREADS, typename Run, typename One>
__device__ __forceinline__ void for_chunk(const void *src, int64_t numel, int c, int tid,
                                          const Run &run, const One &one) {
    typedef typename T::bits B;
    constexpr int V = 16 / sizeof(B);
    constexpr int E = chunk_bytes(THREADS) / sizeof(B);
    const int64_t beg = static_cast<int64_t>(c) * E;
    const int left = static_cast<int>(min(static_cast<int64_t>(E), numel - beg));
    const B *p = static_cast<const B *>(src) + beg;
    if (left == E) {
        Packed<B, V> v[kLoads];
#pragma unroll
        for (int u = 0; u < kLoads; ++u)
            v[u] = load_packed<B, V>(p + (u * THREADS + tid) * V);
#pragma unroll
        for (int u = 0; u < kLoads; ++u)
            run(beg + (u * THREADS + tid) * V, v[u]);
        return;
    }
    const int whole = left / V * V;
#pragma unroll 1
    for (int at = tid * V; at < whole; at += kPartLoads * THREADS * V) {
        Packed<B, V> v[kPartLoads];
#pragma unroll
        for (int u = 0; u < kPartLoads; ++u)
            v[u] = load_packed<B, V>(p + min(at + u * THREADS * V, whole - V));
#pragma unroll
        for (int u = 0; u < kPartLoads; ++u)
            if (at + u * THREADS * V < whole)
                run(beg + at + u * THREADS * V, v[u]);
    }
    if (whole + tid < left)
        one(beg + whole + tid, p[whole + tid]);
}

template <typename T, int THREADS>
__device__ __forceinline__ void sum_chunk(const void *src, int64_t numel, int c, int tid,
                                          double (&s)[4]) {
    typedef typename T::bits B;
    constexpr int V = 16 / sizeof(B);
    for_chunk<T, THREADS>(
        src, numel, c, tid,
        [&](int64_t, const Packed<B, V> &v) __attribute__((always_inline)) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const double x = static_cast<double>(T::widen(v.v[e]));
                s[e & 3] = fma(x, x, s[e & 3]);
            }
        },
        [&](int64_t, B b) __attribute__((always_inline)) {
            const double x = static_cast<double>(T::widen(b));
            s[0] = fma(x, x, s[0]);
        });
}

template <typename T, int THREADS>
__device__ __forceinline__ void scale_chunk(const void *src, void *dst, int64_t numel, int c,
                                            int tid, float factor) {
    typedef typename T::bits B;
    constexpr int V = 16 / sizeof(B);
    auto *o = static_cast<B *>(dst);
    for_chunk<T, THREADS>(
        src, numel, c, tid,
        [&](int64_t at, const Packed<B, V> &v) __attribute__((always_inline)) {
            float x[V];
#pragma unroll
            for (int e = 0; e < V; ++e)
                x[e] = T::widen(v.v[e]) * factor;
            // Past the caches, which leaves the rest of the sources there.
            __builtin_nontemporal_store(__builtin_bit_cast(u32x4_any, narrow_run<T, V>(x)),
                                        reinterpret_cast<u32x4_any *>(o + at));
        },
        [&](int64_t at, B b) __attribute__((always_inline)) {
            o[at] = T::narrow(T::widen(b) * factor);
        });
}

// Chunk c of the batch, by its tensor's type.
template <int THREADS>
__device__ __forceinline__ void sum_any(const Batch &b, int c, int tid, double (&s)[4]) {
    const int t = tensor_of(b, c);
    const int in = c - b.first[t];
    if (b.dtype[t] == KMEANS_BF16)
        sum_chunk<Bf16, THREADS>(b.src[t], b.numel[t], in, tid, s);
    else if (b.dtype[t] == KMEANS_FP16)
        sum_chunk<Fp16, THREADS>(b.src[t], b.numel[t], in, tid, s);
    else
        sum_chunk<Fp32, THREADS>(b.src[t], b.numel[t], in, tid, s);
}
template <int THREADS>
__device__ __forceinline__ void scale_any(const Batch &b, int c, int tid, float factor) {
    const int t = tensor_of(b, c);
    const int in = c - b.first[t];
    if (factor == 1.0f && b.src[t] == b.dst[t])
        return;                                          // nothing changes
    if (b.dtype[t] == KMEANS_BF16)
        scale_chunk<Bf16, THREADS>(b.src[t], b.dst[t], b.numel[t], in, tid, factor);
    else if (b.dtype[t] == KMEANS_FP16)
        scale_chunk<Fp16, THREADS>(b.src[t], b.dst[t], b.numel[t], in, tid, factor);
    else
        scale_chunk<Fp32, THREADS>(b.src[t], b.dst[t], b.numel[t], in, tid, factor);
}

__device__ __forceinline__ float clip_factor(float n, float max_norm) {
    const float ratio = max_norm / (n + 1e-6f);
    return ratio > 1.0f ? 1.0f : ratio;                  // a NaN stays
}

__global__ __launch_bounds__(kClipThreads)
void clip_norm_kernel(const Batch b, double *__restrict__ partial) {
    double s[4] = {0.0, 0.0, 0.0, 0.0};
    for (int c = blockIdx.x; c < b.first[b.count]; c += gridDim.x)
        sum_any<kClipThreads>(b, c, threadIdx.x, s);
    const double total = group_sum<kClipThreads>((s[0] + s[1]) + (s[2] + s[3]));
    if (threadIdx.x == 0)
        partial[b.first_partial + blockIdx.x] = total;
}

// The norm from all partial sums, the same on every workgroup.
__device__ __forceinline__ float total_norm(const double *partial, int partials) {
    double v = 0.0;
    for (int i = threadIdx.x; i < partials; i += kClipThreads)
        v += partial[i];
    return static_cast<float>(sqrt(group_sum<kClipThreads>(v)));
}

__global__ __launch_bounds__(kClipThreads)
void clip_scale_kernel(const Batch b, const double *__restrict__ partial, int partials,
                       float max_norm, float *__restrict__ norm) {
    const float n = total_norm(partial, partials);
    if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0)
        *norm = n;
    const float factor = clip_factor(n, max_norm);
    // From the end: what the first pass read last is still in the caches.
    for (int c = b.first[b.count] - 1 - static_cast<int>(blockIdx.x); c >= 0; c -= gridDim.x)
        scale_any<kClipThreads>(b, c, threadIdx.x, factor);
}

__global__ __launch_bounds__(kClipThreads)
void clip_finish_kernel(const double *__restrict__ partial, int partials,
                        float *__restrict__ norm) {
    const float n = total_norm(partial, partials);
    if (threadIdx.x == 0)
        *norm = n;
}

// A small list at once: each wave takes every 16th chunk, in both passes.
__global__ __launch_bounds__(kSmallThreads)
void clip_small_kernel(const Batch b, int clip, float max_norm, float *__restrict__ norm) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    constexpr int kWaves = kSmallThreads / 64;
    double s[4] = {0.0, 0.0, 0.0, 0.0};
    for (int c = wave; c < b.first[b.count]; c += kWaves)
        sum_any<64>(b, c, lane, s);
    const float n = static_cast<float>(
        sqrt(group_sum<kSmallThreads>((s[0] + s[1]) + (s[2] + s[3]))));
    if (threadIdx.x == 0)
        *norm = n;
    if (clip == 0)
        return;
    const float factor = clip_factor(n, max_norm);
    for (int c = wave; c < b.first[b.count]; c += kWaves)
        scale_any<64>(b, c, lane, factor);
}

int64_t chunks_of(const kmeans_gradient_t &t, int threads) {
    const int64_t per = chunk_bytes(threads) / static_cast<int64_t>(dtype_size(t.dtype));
    return (t.numel + per - 1) / per;
}

// The next batch of the list from entry i on (empty tensors left out), chunks
// as `threads` threads take them.
int64_t fill_batch(Batch &b, const kmeans_gradient_t *list, int64_t count, int64_t &i,
                   int threads) {
    int64_t chunks = 0;
    b.count = 0;
    for (; i < count && b.count < kBatch; ++i) {
        const kmeans_gradient_t &t = list[i];
        if (t.numel == 0)
            continue;
        b.src[b.count] = t.src;
        b.dst[b.count] = t.dst;
        b.numel[b.count] = t.numel;
        b.dtype[b.count] = static_cast<uint8_t>(t.dtype);
        b.first[b.count++] = static_cast<int>(chunks);
        chunks += chunks_of(t, threads);
    }
    b.first[b.count] = static_cast<int>(chunks);
    return chunks;
}

kmeans_status_t check_list(const kmeans_gradient_t *list, int64_t count, bool clip,
                           const float *norm) {
    if (count < 0)
        return fail(KMEANS_ERR_INVALID_ARG, "count=%lld must be >= 0",
                    static_cast<long long>(count));
    if (count > kMaxRows)
        return fail(KMEANS_ERR_UNSUPPORTED, "count=%lld too large", static_cast<long long>(count));
    if (!norm || (count > 0 && !list))
        return fail(KMEANS_ERR_INVALID_ARG, "null pointer argument (list=%p norm=%p)",
                    static_cast<const void *>(list), static_cast<const void *>(norm));
    if (!aligned(norm, 4))
        return fail(KMEANS_ERR_ALIGNMENT, "norm must be 4-byte aligned");
    int64_t total = 0;
    for (int64_t i = 0; i < count; ++i) {
        const kmeans_gradient_t &t = list[i];
        const auto at = static_cast<long long>(i);
        if (t.numel < 0)
            return fail(KMEANS_ERR_INVALID_ARG, "gradient %lld: numel=%lld must be >= 0", at,
                        static_cast<long long>(t.numel));
        if (t.dtype < KMEANS_BF16 || t.dtype > KMEANS_FP32)
            return fail(KMEANS_ERR_INVALID_ARG, "gradient %lld: dtype=%d is not a kmeans_dtype_t",
                        at, t.dtype);
        if (t.reserved != 0)
            return fail(KMEANS_ERR_INVALID_ARG, "gradient %lld: reserved must be 0", at);
        if (t.numel == 0)
            continue;
        if (!t.src || (clip && !t.dst))
            return fail(KMEANS_ERR_INVALID_ARG, "gradient %lld: null pointer (src=%p dst=%p)", at,
                        t.src, t.dst);
        if (!aligned(t.src, dtype_size(t.dtype)) || (clip && !aligned(t.dst, dtype_size(t.dtype))))
            return fail(KMEANS_ERR_ALIGNMENT, "gradient %lld must be aligned to its element size",
                        at);
        if (t.numel > kMaxElements || (total += t.numel) > kMaxElements)
            return fail(KMEANS_ERR_UNSUPPORTED, "gradients of more than 2^40 elements");
    }
    return KMEANS_OK;
}

kmeans_status_t run_clip(const kmeans_gradient_t *list, int64_t count, bool clip, float max_norm,
                         float *norm, hipStream_t stream) {
    kmeans_status_t st = check_list(list, count, clip, norm);
    if (st != KMEANS_OK)
        return st;
    int64_t total = 0, tensors = 0, bytes = 0;
    for (int64_t i = 0; i < count; ++i) {
        total += chunks_of(list[i], kClipThreads);
        tensors += list[i].numel > 0;
        bytes += list[i].numel * static_cast<int64_t>(dtype_size(list[i].dtype));
    }
    if (bytes <= kSmallBytes && tensors <= kBatch) {
        Batch b;
        int64_t i = 0;
        fill_batch(b, list, count, i, 64);
        hipLaunchKernelGGL(clip_small_kernel, dim3(1), dim3(kSmallThreads), 0, stream, b,
                           static_cast<int>(clip), max_norm, norm);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return fail(KMEANS_ERR_HIP, "clip launch failed: %s", hipGetErrorString(e));
        return ok();
    }
    const int64_t batches = (tensors + kBatch - 1) / kBatch;
    // Each batch gets its share of the workgroups, by chunks, and one at least.
    const WorkspaceLease lease(stream, static_cast<size_t>(kMaxPartials + batches) * sizeof(double));
    if (lease.error() != hipSuccess)
        return fail(KMEANS_ERR_NO_MEMORY, "workspace of %lld partial sums: %s",
                    static_cast<long long>(kMaxPartials + batches),
                    hipGetErrorString(lease.error()));
    auto *partial = static_cast<double *>(lease.ptr());
    int partials = 0;
    for (int pass = 0; pass < (clip ? 2 : 1); ++pass) {
        int64_t i = 0;
        int used = 0;
        while (i < count) {
            Batch b;
            b.first_partial = used;
            const int64_t chunks = fill_batch(b, list, count, i, kClipThreads);
            if (b.count == 0)
                break;
            const int64_t share =
                total <= kMaxPartials ? chunks : std::max<int64_t>(1, chunks * kMaxPartials / total);
            if (pass == 0)
                hipLaunchKernelGGL(clip_norm_kernel, dim3(static_cast<unsigned>(share)),
                                   dim3(kClipThreads), 0, stream, b, partial);
            else
                hipLaunchKernelGGL(clip_scale_kernel, dim3(static_cast<unsigned>(share)),
                                   dim3(kClipThreads), 0, stream, b, partial, partials, max_norm,
                                   used == 0 ? norm : nullptr);
            used += static_cast<int>(share);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess)
                return fail(KMEANS_ERR_HIP, "clip launch failed: %s", hipGetErrorString(e));
        }
        partials = used;
    }
    if (!clip) {
        hipLaunchKernelGGL(clip_finish_kernel, dim3(1), dim3(kClipThreads), 0, stream, partial,
                           partials, norm);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return fail(KMEANS_ERR_HIP, "norm launch failed: %s", hipGetErrorString(e));
    }
    return ok();
}

}  // namespace
}  // namespace kmeans

// ---- C entry points --------------------------------------------------------

extern "C" kmeans_status_t kmeans_gradient_norm(const kmeans_gradient_t *list, int64_t count,
                                                float *norm, hipStream_t stream) {
    return kmeans::run_clip(list, count, false, 0.0f, norm, stream);
}

extern "C" kmeans_status_t kmeans_clip_gradients(const kmeans_gradient_t *list, int64_t count,
                                                 float max_norm, float *norm,
                                                 hipStream_t stream) {
    if (!(max_norm >= 0.0f))
        return kmeans::fail(KMEANS_ERR_INVALID_ARG, "max_norm=%g must be >= 0",
                            static_cast<double>(max_norm));
    return kmeans::run_clip(list, count, true, max_norm, norm, stream);
}
