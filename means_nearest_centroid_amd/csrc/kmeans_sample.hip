// kmeans_sample.hip -- gfx950 kernel that draws a label from each row of logits
// by temperature, top-k, top-p and min-p, from given random numbers.
//
//     order: logit descending, index ascending;  w_i = exp((z_i - max) / t)
//     kept:  a prefix of that order, the shortest of: the first k; the shortest
//            with p of the first k's weight; those with w_i >= min_p
//     label: first in that order whose running weight exceeds u times the
//            weight of all kept
//
// Weights are whole multiples of 2^-43 in 64-bit integers (K < 2^20 of them
// stay below 2^63), so that every sum is exact and the same in any order, from
// atomics too: the label depends on the row alone, not on the launch.  A weight
// is rounded by 2^-44 of the largest one at most.
//
// All borders (the k-th value, the nucleus's end, the draw) are then one thing:
// the element at which a running amount (of elements or of weight) reaches a
// target.  A histogram over 32 temperatures below the largest logit finds the
// bin where it does, the few elements of the bin are compared with one another
// (or, where they are many, divided further by the bits of their values and
// indexes).  No sorting, and a row is read three or four times, from the caches
// after the first.
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "kmeans_fp8.h"
#include "kmeans_internal.h"
#include "kmeans_types.h"

namespace kmeans {
namespace {

constexpr int64_t kMaxLabels = 1 << 20;
constexpr int kWeightBits = 43;
constexpr float kSpan = 32.0f;       // temperatures below the largest logit: past
                                     // 30.5 of them a weight is zero
constexpr int kSmall = 256;          // elements compared with one another
constexpr int kTable = 128;          // 2^(-i / 128)

struct Sample {
    const void *logits;
    int64_t ld;
    int K;
    const float *u;
    float temperature, top_p, min_p;
    int top_k;
    const float *temperatures, *top_ps, *min_ps;     // of each row, or null
    const int *top_ks;
    void *labels;
    int wide;                                        // 64-bit labels
    int64_t first;                                   // row of this launch
};

// An element as one number that orders as the definition does: value, then the
// lower index.
__device__ __forceinline__ uint32_t key_of(float z) {
    const uint32_t b = __float_as_uint(z);
    return b ^ (static_cast<int32_t>(b) < 0 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key ^ (static_cast<int32_t>(key) < 0 ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint64_t element_of(uint32_t key, int i) {
    return static_cast<uint64_t>(key) << 32 | (0xffffffffu - static_cast<uint32_t>(i));
}
__device__ __forceinline__ int index_of(uint64_t e) {
    return static_cast<int>(0xffffffffu - static_cast<uint32_t>(e));
}

// A logit as the definition takes it: NaN is below all others, zero has no sign.
__device__ __forceinline__ float logit(float z) {
    return z != z ? -INFINITY : z + 0.0f;
}

template <typename T, int THREADS, int BINS, int LIST>
struct Draw {
    typedef typename T::bits B;
    static constexpr int kWaves = THREADS / 64;
    static constexpr int V = 16 / sizeof(B);         // values of a load
    static constexpr int U = 4;                      // loads in flight

    struct Shared {
        uint64_t mass[BINS];         // weight by distance to the largest logit
        uint64_t other[BINS];        // counts, and the finer divisions
        uint64_t list[LIST];         // the first k and the rest of their last bin
        uint64_t small[kSmall], amount[kSmall], before[kSmall];
        double table[kTable];
        uint64_t sums[2][kWaves];
        float most[kWaves];
        uint64_t found_before, found_amount, found_element;
        int found, count;
        uint32_t lo, hi;
    };

    Shared &s;
    const B *row;
    int K, tid;
    float m, scale;                  // largest logit; bins per unit of logit
    double rate;                     // 128 log2(e) / temperature
    uint64_t limit;                  // elements below it are not among the first k
    int listed;                      // elements in list, or -1: the row itself

    // f(z, i) for every element of the row.
    template <typename F>
    __device__ __forceinline__ void for_row(const F &f) const {
        for (int c0 = tid * V; c0 < K; c0 += THREADS * V * U) {
            Packed<B, V> v[U];
#pragma unroll
            for (int x = 0; x < U; ++x) {
                const int c = c0 + x * THREADS * V;
                v[x] = load_run<B, V>(row + c, K - c);
            }
#pragma unroll
            for (int x = 0; x < U; ++x) {
                const int c = c0 + x * THREADS * V;
#pragma unroll
                for (int e = 0; e < V; ++e)
                    if (c + e < K)
                        f(logit(T::widen(v[x].v[e])), c + e);
            }
        }
    }
    // f(z, i, bin) for every element that may still be drawn.
    template <typename F>
    __device__ __forceinline__ void for_kept(const F &f) const {
        if (listed >= 0) {
            for (int x = tid; x < listed; x += THREADS) {
                const uint64_t e = s.list[x];
                const float z = value_of(static_cast<uint32_t>(e >> 32));
                if (e >= limit)
                    f(z, index_of(e), bin_of(z));
            }
            return;
        }
        for_row([&](float z, int i) __attribute__((always_inline)) {
            const int b = bin_of(z);
            if (b < BINS && element_of(key_of(z), i) >= limit)
                f(z, i, b);
        });
    }

    // Bin of a logit, not decreasing with its distance to the largest one; BINS:
    // its weight is zero.
    __device__ __forceinline__ int bin_of(float z) const {
        const float x = z == m ? 0.0f : (m - z) * scale;
        return x < static_cast<float>(BINS) ? static_cast<int>(x) : BINS;
    }
    // exp((z - m) / t) in units of 2^-43, of a logit in a bin.  2^(-y / 128),
    // y = n + f: a table for n's low bits, its high ones an exponent, and a
    // polynomial for f (|f| <= 1/2; the term left out is 1e-15 at most).
    __device__ __forceinline__ uint64_t weight(float z) const {
        constexpr double kMagic = 6755399441055744.0;                // 1.5 2^52
        const double y = z == m ? 0.0 : (static_cast<double>(m) - static_cast<double>(z)) * rate;
        const double magic = y + kMagic;
        const int n = static_cast<int>(__double_as_longlong(magic));
        constexpr double c = 0.69314718055994530942 / kTable;
        const double f = (magic - kMagic) - y;
        double p = c * c * c * c / 24;
        p = fma(p, f, c * c * c / 6);
        p = fma(p, f, c * c / 2);
        p = fma(p, f, c);
        p = fma(p, f, 1.0);
        const double w = ldexp(p * s.table[n & (kTable - 1)], kWeightBits - (n >> 7));
        return __double_as_longlong(w + 4503599627370496.0) & 0xfffffffffffffull;   // 2^52
    }

    __device__ __forceinline__ uint64_t group_sum(uint64_t v) {
#pragma unroll
        for (int x = 32; x >= 1; x >>= 1)
            v += __shfl_xor(v, x, 64);
        __syncthreads();
        if ((tid & 63) == 0)
            s.sums[0][tid >> 6] = v;
        __syncthreads();
        uint64_t total = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            total += s.sums[0][w];
        return total;
    }

    // Where the running sum of hist reaches `target` (1 to the total): the bin in
    // found, the sum before it and its own in found_before and found_amount.
    // Returns the total; a target past it finds nothing (found is BINS).
    __device__ __forceinline__ uint64_t locate(const uint64_t *hist, uint64_t target) {
        constexpr int kEach = BINS / THREADS;
        __syncthreads();
        uint64_t own[kEach], v = 0;
#pragma unroll
        for (int x = 0; x < kEach; ++x) {
            own[x] = hist[tid * kEach + x];
            v += own[x];
        }
        uint64_t run = v;
#pragma unroll
        for (int x = 1; x < 64; x <<= 1) {
            const uint64_t up = __shfl_up(run, x, 64);
            run += (tid & 63) >= x ? up : 0;
        }
        if ((tid & 63) == 63)
            s.sums[1][tid >> 6] = run;
        if (tid == 0)
            s.found = BINS;
        __syncthreads();
        uint64_t total = 0, base = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            base += w < tid >> 6 ? s.sums[1][w] : 0;
            total += s.sums[1][w];
        }
        uint64_t at = base + run - v;
        if (at < target && target <= at + v) {
#pragma unroll
            for (int x = 0; x < kEach; ++x) {
                if (at < target && target <= at + own[x]) {
                    s.found = tid * kEach + x;
                    s.found_before = at;
                    s.found_amount = own[x];
                }
                at += own[x];
            }
        }
        __syncthreads();
        return total;
    }

    __device__ __forceinline__ void clear(uint64_t *hist) {
        for (int x = tid; x < BINS; x += THREADS)
            hist[x] = 0;
    }
    static __device__ __forceinline__ void add(uint64_t *p, uint64_t v) {
        atomicAdd(reinterpret_cast<unsigned long long *>(p), static_cast<unsigned long long>(v));
    }

    // The element of bin b at which the running amount within the bin (of
    // elements where COUNT, else of weight) reaches `target`; `upto` is that
    // running amount, its own included.
    template <bool COUNT>
    __device__ __forceinline__ uint64_t resolve(int b, uint64_t target, uint64_t &upto) {
        auto amount_of = [&](float z) __attribute__((always_inline)) {
            return COUNT ? uint64_t(1) : weight(z);
        };
        __syncthreads();
        if (tid == 0) {
            s.count = 0;
            s.lo = 0xffffffffu;
            s.hi = 0;
        }
        if (tid < kSmall)
            s.before[tid] = 0;
        __syncthreads();
        for_kept([&](float z, int i, int bin) __attribute__((always_inline)) {
            if (bin != b)
                return;
            const uint32_t key = key_of(z);
            const int x = atomicAdd(&s.count, 1);
            if (x < kSmall)
                s.small[x] = element_of(key, i);
            atomicMin(&s.lo, key);
            atomicMax(&s.hi, key);
        });
        __syncthreads();
        const int n = s.count;
        if (n <= kSmall) {
            if (tid < n)
                s.amount[tid] = amount_of(value_of(static_cast<uint32_t>(s.small[tid] >> 32)));
            __syncthreads();
            // Thread (part, x) adds up what of its part comes before element x.
            constexpr int kParts = THREADS / kSmall;
            const int x = tid % kSmall, part = tid / kSmall;
            if (x < n) {
                const uint64_t mine = s.small[x];
                const int beg = n * part / kParts, end = n * (part + 1) / kParts;
                uint64_t sum = 0;
                for (int y = beg; y < end; ++y)
                    sum += s.small[y] > mine ? s.amount[y] : 0;
                add(&s.before[x], sum);
            }
            __syncthreads();
            if (tid < n) {
                const uint64_t at = s.before[tid], own = s.amount[tid];
                if (at < target && target <= at + own) {
                    s.found_element = s.small[tid];
                    s.found_amount = at + own;
                }
            }
            __syncthreads();
            upto = s.found_amount;
            return s.found_element;
        }
        // Many: by the bits of their values, then, among equal ones, of their
        // indexes.
        uint32_t lo = s.lo, hi = s.hi;
        uint64_t sum = 0;
        while (lo < hi) {
            const int shift = max(0, 32 - __builtin_clz(hi - lo) - __builtin_ctz(BINS));
            clear(s.other);
            __syncthreads();
            for_kept([&](float z, int, int bin) __attribute__((always_inline)) {
                const uint32_t key = key_of(z);
                if (bin == b && key >= lo && key <= hi)
                    add(&s.other[(hi - key) >> shift], amount_of(z));
            });
            locate(s.other, target - sum);
            if (s.found >= BINS)                        // only if the row changed meanwhile
                break;
            sum += s.found_before;
            hi -= static_cast<uint32_t>(s.found) << shift;
            const uint32_t rest = (1u << shift) - 1;
            lo = hi - lo > rest ? hi - rest : lo;
        }
        const uint32_t key = lo;
        const uint64_t each = amount_of(value_of(key));
        uint64_t nth = (target - sum + each - 1) / each;              // of the equal ones
        upto = sum + nth * each;
        int first = 0, last = K - 1;
        while (first < last) {
            const int shift = max(0, 32 - __builtin_clz(last - first) - __builtin_ctz(BINS));
            clear(s.other);
            __syncthreads();
            for_kept([&](float z, int i, int) __attribute__((always_inline)) {
                if (key_of(z) == key && i >= first && i <= last)
                    add(&s.other[(i - first) >> shift], 1);
            });
            locate(s.other, nth);
            if (s.found >= BINS)
                break;
            nth -= s.found_before;
            first += s.found << shift;
            last = min(last, first + (1 << shift) - 1);
        }
        return element_of(key, first);
    }

    // The row's label, the same on every thread.
    __device__ __forceinline__ int run(float t, int k, float p, float min_p, float u) {
        for (int x = tid; x < kTable; x += THREADS)
            s.table[x] = exp2(-x / static_cast<double>(kTable));
        clear(s.mass);
        clear(s.other);
        float most = -INFINITY;
        for_row([&](float z, int) __attribute__((always_inline)) { most = fmaxf(most, z); });
#pragma unroll
        for (int x = 32; x >= 1; x >>= 1)
            most = fmaxf(most, __shfl_xor(most, x, 64));
        if ((tid & 63) == 0)
            s.most[tid >> 6] = most;
        if (tid == 0)
            s.count = K;
        __syncthreads();
        m = s.most[0];
#pragma unroll
        for (int w = 1; w < kWaves; ++w)
            m = fmaxf(m, s.most[w]);
        if (m == -INFINITY)
            return -1;                                  // nothing to draw
        if (!(t > 0.0f)) {
            int first = K;
            for_row([&](float z, int i) __attribute__((always_inline)) {
                first = z == m ? min(first, i) : first;
            });
            if (first < K)
                atomicMin(&s.count, first);
            __syncthreads();
            return s.count;
        }
        scale = BINS / kSpan / t;
        rate = kTable * 1.44269504088896340736 / static_cast<double>(t);
        limit = 0;
        listed = -1;

        if (k > 0 && k < K) {
            for_row([&](float z, int) __attribute__((always_inline)) {
                const int b = bin_of(z);
                if (b < BINS)
                    add(&s.other[b], 1);
            });
            locate(s.other, k);
            const int b = s.found;
            if (b < BINS) {                             // there are more than k, or k
                const uint64_t target = k - s.found_before;
                const uint64_t upto = s.found_before + s.found_amount;
                if (upto <= LIST) {
                    __syncthreads();
                    if (tid == 0)
                        s.count = 0;
                    __syncthreads();
                    for_row([&](float z, int i) __attribute__((always_inline)) {
                        if (bin_of(z) > b)
                            return;
                        const int x = atomicAdd(&s.count, 1);
                        if (x < LIST)
                            s.list[x] = element_of(key_of(z), i);
                    });
                    listed = static_cast<int>(upto);
                }
                uint64_t sum;
                limit = resolve<true>(b, target, sum);
            }
        }

        const double least = fmin(static_cast<double>(min_p), 1.0) * (1ull << kWeightBits);
        uint64_t likely = 0;                            // weight of those with w >= min_p
        for_kept([&](float z, int, int b) __attribute__((always_inline)) {
            const uint64_t w = weight(z);
            add(&s.mass[b], w);
            likely += static_cast<double>(w) >= least ? w : 0;
        });
        uint64_t total = locate(s.mass, 1);
        if (min_p > 0.0f)
            likely = group_sum(likely);
        if (p < 1.0f) {
            const double want = ceil(static_cast<double>(p) * static_cast<double>(total));
            const uint64_t target =
                want >= 1.0 ? min(static_cast<uint64_t>(want), total) : uint64_t(1);
            locate(s.mass, target);
            const uint64_t before = s.found_before;
            uint64_t upto;
            resolve<false>(s.found, target - before, upto);
            total = before + upto;
        }
        if (min_p > 0.0f)
            total = min(total, likely);
        const double at = static_cast<double>(u) * static_cast<double>(total);
        const uint64_t target =
            at > 0.0 ? (at < static_cast<double>(total) ? min(static_cast<uint64_t>(at), total - 1)
                                                        : total - 1) + 1
                     : uint64_t(1);
        locate(s.mass, target);
        uint64_t upto;
        return index_of(resolve<false>(s.found, target - s.found_before, upto));
    }
};

template <typename T, int THREADS, int BINS, int LIST>
__global__ __launch_bounds__(THREADS, THREADS == 1024 ? 8 : 4)
void sample_kernel(const Sample a) {
    typedef Draw<T, THREADS, BINS, LIST> D;
    __shared__ typename D::Shared s;
    const int64_t row = a.first + blockIdx.x;
    D d{s, static_cast<const typename T::bits *>(a.logits) + row * a.ld, a.K,
        static_cast<int>(threadIdx.x)};
    const int label = d.run(a.temperatures != nullptr ? a.temperatures[row] : a.temperature,
                            a.top_ks != nullptr ? a.top_ks[row] : a.top_k,
                            a.top_ps != nullptr ? a.top_ps[row] : a.top_p,
                            a.min_ps != nullptr ? a.min_ps[row] : a.min_p, a.u[row]);
    if (threadIdx.x != 0)
        return;
    if (a.wide)
        static_cast<int64_t *>(a.labels)[row] = label;
    else
        static_cast<int32_t *>(a.labels)[row] = label;
}

template <typename T>
hipError_t run_sample(Sample a, int64_t N, hipStream_t stream) {
    constexpr int64_t kMaxGrid = int64_t(1) << 21;      // a launch has less than 2^32 threads
    hipError_t e = hipSuccess;
    for (int64_t first = 0; first < N && e == hipSuccess; first += kMaxGrid) {
        a.first = first;
        const dim3 grid(static_cast<unsigned>(std::min(kMaxGrid, N - first)));
        if (a.K <= 4096)
            hipLaunchKernelGGL((sample_kernel<T, 256, 512, 1024>), grid, dim3(256), 0, stream, a);
        else
            hipLaunchKernelGGL((sample_kernel<T, 1024, 2048, 4096>), grid, dim3(1024), 0, stream,
                               a);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace
}  // namespace kmeans

// ---- C entry point ---------------------------------------------------------

extern "C" kmeans_status_t kmeans_sample(const void *logits, int64_t logits_stride, int64_t N,
                                         int64_t K, int32_t dtype, const float *uniforms,
                                         const kmeans_sampling_t *settings, void *labels,
                                         int32_t label_type, hipStream_t stream) {
    using namespace kmeans;
    if (N < 0 || K < 1)
        return fail(KMEANS_ERR_INVALID_ARG, "N=%lld must be >= 0 and K=%lld >= 1",
                    static_cast<long long>(N), static_cast<long long>(K));
    if (dtype < KMEANS_BF16 || dtype > KMEANS_FP32)
        return fail(KMEANS_ERR_INVALID_ARG, "dtype=%d is not a kmeans_dtype_t", dtype);
    if (label_type != KMEANS_INT32 && label_type != KMEANS_INT64)
        return fail(KMEANS_ERR_INVALID_ARG, "label_type=%d is not a kmeans_label_t", label_type);
    if (N > kMaxRows || K > kMaxLabels)
        return fail(KMEANS_ERR_UNSUPPORTED, "N=%lld or K=%lld too large (max %lld, %lld)",
                    static_cast<long long>(N), static_cast<long long>(K),
                    static_cast<long long>(kMaxRows), static_cast<long long>(kMaxLabels));
    if (settings == nullptr)
        return fail(KMEANS_ERR_INVALID_ARG, "null pointer argument (settings)");
    const kmeans_sampling_t &o = *settings;
    if (!o.temperatures && !(o.temperature >= 0.0f))
        return fail(KMEANS_ERR_INVALID_ARG, "temperature=%g must be >= 0",
                    static_cast<double>(o.temperature));
    if (!o.top_ks && o.top_k < 0)
        return fail(KMEANS_ERR_INVALID_ARG, "top_k=%d must be >= 0", o.top_k);
    if (!o.top_ps && !(o.top_p >= 0.0f && o.top_p <= 1.0f))
        return fail(KMEANS_ERR_INVALID_ARG, "top_p=%g must be in [0, 1]",
                    static_cast<double>(o.top_p));
    if (!o.min_ps && !(o.min_p >= 0.0f && o.min_p <= 1.0f))
        return fail(KMEANS_ERR_INVALID_ARG, "min_p=%g must be in [0, 1]",
                    static_cast<double>(o.min_p));
    if (N == 0)
        return ok();
    kmeans_status_t st;
    if ((st = check_matrix("logits", logits, K, logits_stride, dtype_size(dtype))) != KMEANS_OK ||
        (st = check_matrix("uniforms", uniforms, 1, 1, 4)) != KMEANS_OK ||
        (st = check_matrix("labels", labels, 1, 1, label_type == KMEANS_INT64 ? 8 : 4)) != KMEANS_OK ||
        (st = check_array("temperatures", o.temperatures, 4)) != KMEANS_OK ||
        (st = check_array("top_ks", o.top_ks, 4)) != KMEANS_OK ||
        (st = check_array("top_ps", o.top_ps, 4)) != KMEANS_OK ||
        (st = check_array("min_ps", o.min_ps, 4)) != KMEANS_OK)
        return st;
    const Sample a{logits, logits_stride, static_cast<int>(K), uniforms, o.temperature, o.top_p,
                   o.min_p, o.top_k, o.temperatures, o.top_ps, o.min_ps, o.top_ks, labels,
                   label_type == KMEANS_INT64, 0};
    const hipError_t e = dtype == KMEANS_BF16   ? run_sample<Bf16>(a, N, stream)
                         : dtype == KMEANS_FP16 ? run_sample<Fp16>(a, N, stream)
                                                : run_sample<Fp32>(a, N, stream);
    if (e != hipSuccess)
        return fail(KMEANS_ERR_HIP, "sample launch failed: %s", hipGetErrorString(e));
    return ok();
}
