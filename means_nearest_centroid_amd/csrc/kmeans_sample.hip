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
// target.  Where few elements can be drawn (the first k, those above min_p) they
// are gathered and compared with one another.  Otherwise a histogram over 32
// temperatures below the largest logit finds the bins of the nucleus's end and
// of the draw, whose elements are gathered and compared.  Where even those are
// many, they are divided further by the bits of their values and indexes.  No
// sorting; a row is read two or three times, from the caches after the first.
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
constexpr int kTable = 128;          // 2^(-i / 128), from its two factors
constexpr double kEighths[8] = {
    0x1.0000000000000p+0, 0x1.d5818dcfba487p-1, 0x1.ae89f995ad3adp-1, 0x1.8ace5422aa0dbp-1,
    0x1.6a09e667f3bcdp-1, 0x1.4bfdad5362a27p-1, 0x1.306fe0a31b715p-1, 0x1.172b83c7d517bp-1};
constexpr double k128ths[16] = {
    0x1.0000000000000p+0, 0x1.fd3c22b8f71f1p-1, 0x1.fa7c1819e90d8p-1, 0x1.f7bfdad9cbe14p-1,
    0x1.f50765b6e4540p-1, 0x1.f252b376bba97p-1, 0x1.efa1bee615a27p-1, 0x1.ecf482d8e67f1p-1,
    0x1.ea4afa2a490dap-1, 0x1.e7a51fbc74c83p-1, 0x1.e502ee78b3ff6p-1, 0x1.e264614f5a129p-1,
    0x1.dfc97337b9b5fp-1, 0x1.dd321f301b460p-1, 0x1.da9e603db3285p-1, 0x1.d80e316c98398p-1};

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
    const uint32_t b = __float_as_uint(z + 0.0f);        // zero has no sign
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

template <typename T, int THREADS, int BINS, int LIST>
struct Draw {
    typedef typename T::bits B;
    static constexpr int kWaves = THREADS / 64;
    static constexpr int V = 16 / sizeof(B);         // values of a load
    static constexpr int kEach = BINS / THREADS;

    // Few elements and what comes before each of them.
    struct Few {
        uint64_t element[kSmall], amount[kSmall], before[kSmall];
        int rank[kSmall];
        int count;
    };
    struct Shared {
        uint64_t mass[BINS];         // weight by distance to the largest logit
        uint64_t other[BINS];        // counts, and the finer divisions
        uint64_t list[LIST];         // all that may belong to the first k
        Few end, draw;               // around the nucleus's end, around the draw
        double table[kTable];
        uint64_t sums[2][kWaves];
        float most[kWaves];
        uint64_t found_before[2], found_amount[2], found_element;
        int found[2], count, runs;
        uint32_t lo, hi;
    };
    // A histogram's running sum: this thread's bins and what lies before them.
    struct Running {
        uint64_t own[kEach], before, total;
    };

    Shared &s;
    const B *row;
    int K, tid;
    float m, scale;                  // largest logit; bins per unit of logit
    double rate;                     // 128 log2(e) / temperature
    uint64_t limit;                  // elements below it are not among the first k
    int listed;                      // elements in list, or -1: the row itself

    // f(z, i) for every run of the row: V values from index i on, -infinity past
    // its end; VALUES of a thread in flight.
    template <int VALUES, typename F>
    __device__ __forceinline__ void for_runs(const F &f) const {
        constexpr int U = VALUES / V;
        constexpr int kStep = THREADS * VALUES;
        auto give = [&](const Packed<B, V> &p, int c) __attribute__((always_inline)) {
            float z[V];
#pragma unroll
            for (int e = 0; e < V; ++e)
                z[e] = c + e < K ? T::widen(p.v[e]) : -INFINITY;
            f(z, c);
        };
#pragma unroll 1
        for (int base = 0; base < K; base += kStep) {
            const int c0 = base + tid * V;
            if (base + kStep <= K) {
                Packed<B, V> v[U];
#pragma unroll
                for (int x = 0; x < U; ++x)
                    v[x] = load_packed<B, V>(row + c0 + x * THREADS * V);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int x = 0; x < U; ++x) {
                    float z[V];
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        z[e] = T::widen(v[x].v[e]);
                    f(z, c0 + x * THREADS * V);
                }
            } else {
#pragma unroll 1
                for (int c = c0; c < K; c += THREADS * V)
                    give(load_run<B, V>(row + c, K - c), c);
            }
        }
    }
    // f(z, i) for every element with test(z).  Few are expected: a run without
    // any costs no more than the tests.
    template <typename P, typename F>
    __device__ __forceinline__ void for_some(const P &test, const F &f) const {
        for_runs<32>([&](const float (&z)[V], int i) __attribute__((always_inline)) {
            bool any = false;
#pragma unroll
            for (int e = 0; e < V; ++e)
                any |= test(z[e]);
            if (!any)
                return;
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (test(z[e]))
                    f(z[e], i + e);
        });
    }
    // The same of those that may still be drawn.
    template <typename P, typename F>
    __device__ __forceinline__ void for_kept(const P &test, const F &f) const {
        if (listed >= 0) {
            for (int y = tid; y < listed; y += THREADS) {
                const uint64_t e = s.list[y];
                const float z = value_of(static_cast<uint32_t>(e >> 32));
                if (e >= limit && test(z))
                    f(z, index_of(e));
            }
            return;
        }
        for_some(test, [&](float z, int i) __attribute__((always_inline)) {
            if (limit == 0 || element_of(key_of(z), i) >= limit)
                f(z, i);
        });
    }
    __device__ __forceinline__ bool in_span(float z) const {
        return place(z) < static_cast<float>(BINS);
    }
    // Counts by bin of all that may still be drawn.
    __device__ __forceinline__ void count_bins() {
        __syncthreads();
        clear(s.other);
        __syncthreads();
        for_kept([&](float z) __attribute__((always_inline)) { return in_span(z); },
                 [&](float z, int) __attribute__((always_inline)) {
                     add(&s.other[static_cast<int>(place(z))], 1);
                 });
    }

    // Distance to the largest logit (a finite one) in bins, not decreasing with
    // it; from BINS on a weight is zero.  NaN of a NaN.
    __device__ __forceinline__ float place(float z) const { return (m - z) * scale; }

    // exp((z - m) / t) in units of 2^-43, of a logit in a bin.  2^(-y / 128),
    // y = n + f: a table for n's low bits, its high ones an exponent, and a
    // polynomial for f (|f| <= 1/2; the term left out is 1e-15 at most).
    __device__ __forceinline__ uint64_t weight(float z) const {
        constexpr double kMagic = 6755399441055744.0;                // 1.5 2^52
        const double y = (static_cast<double>(m) - static_cast<double>(z)) * rate;
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
    template <bool COUNT>
    __device__ __forceinline__ uint64_t amount_of(uint64_t e) const {
        return COUNT ? uint64_t(1) : weight(value_of(static_cast<uint32_t>(e >> 32)));
    }

    static __device__ __forceinline__ uint64_t wave_sum(uint64_t v) {
#pragma unroll
        for (int x = 32; x >= 1; x >>= 1)
            v += __shfl_xor(v, x, 64);
        return v;
    }
    __device__ __forceinline__ uint64_t group_sum(uint64_t v) {
        v = wave_sum(v);
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

    // Begins with a barrier: the histogram is whole.
    __device__ __forceinline__ Running running(const uint64_t *hist) {
        Running r;
        __syncthreads();
        uint64_t v = 0;
#pragma unroll
        for (int x = 0; x < kEach; ++x) {
            r.own[x] = hist[tid * kEach + x];
            v += r.own[x];
        }
        uint64_t run = v;
#pragma unroll
        for (int x = 1; x < 64; x <<= 1) {
            const uint64_t up = __shfl_up(run, x, 64);
            run += (tid & 63) >= x ? up : 0;
        }
        if ((tid & 63) == 63)
            s.sums[1][tid >> 6] = run;
        __syncthreads();
        uint64_t total = 0, base = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const uint64_t sum = s.sums[1][w];
            base += w < tid >> 6 ? sum : 0;
            total += sum;
        }
        r.before = base + run - v;
        r.total = total;
        return r;
    }
    // The bins where the running sum reaches two targets (1 to the total), and
    // the sums before them and their own.
    __device__ __forceinline__ void find(const Running &r, uint64_t target, uint64_t second) {
        __syncthreads();
        uint64_t at = r.before;
#pragma unroll
        for (int x = 0; x < kEach; ++x) {
#pragma unroll
            for (int which = 0; which < 2; ++which) {
                const uint64_t want = which == 0 ? target : second;
                if (at < want && want <= at + r.own[x]) {
                    s.found[which] = tid * kEach + x;
                    s.found_before[which] = at;
                    s.found_amount[which] = r.own[x];
                }
            }
            at += r.own[x];
        }
        __syncthreads();
    }
    // The same for one target in a histogram; false where the total is less.
    __device__ __forceinline__ bool locate(const uint64_t *hist, uint64_t target) {
        const Running r = running(hist);
        if (target == 0 || target > r.total)
            return false;
        find(r, target, target);
        return true;
    }

    __device__ __forceinline__ void clear(uint64_t *hist) {
        for (int x = tid; x < BINS; x += THREADS)
            hist[x] = 0;
    }
    static __device__ __forceinline__ void add(uint64_t *p, uint64_t v) {
        atomicAdd(reinterpret_cast<unsigned long long *>(p), static_cast<unsigned long long>(v));
    }
    static __device__ __forceinline__ void put(Few &few, uint64_t e) {
        const int x = atomicAdd(&few.count, 1);
        if (x < kSmall)
            few.element[x] = e;
    }
    // Calls f(z, i) for the elements of the row with test(z), a few hundred of
    // them, in two steps: the runs that hold one are listed, one count for those
    // of a wave; then each thread takes some of them.  So the loop over the row
    // has no more than the tests (a wave's 256 or 512 elements hold a hit more
    // often than not).  Where there are more runs than `runs` holds, one step.
    template <typename P, typename F>
    __device__ __forceinline__ void for_listed(const P &test, const F &f) {
        auto *runs = reinterpret_cast<int *>(s.other);
        constexpr int kRoom = 2 * BINS;
        __syncthreads();
        if (tid == 0)
            s.runs = 0;
        __syncthreads();
        for_runs<32>([&](const float (&z)[V], int i) __attribute__((always_inline)) {
            bool any = false;
#pragma unroll
            for (int e = 0; e < V; ++e)
                any |= test(z[e]);
            const uint64_t mask = __ballot(any);
            if (mask == 0)
                return;
            int at = 0;
            const int before = __builtin_amdgcn_mbcnt_hi(
                static_cast<uint32_t>(mask >> 32),
                __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(mask), 0));
            if (any && before == 0)
                at = atomicAdd(&s.runs, __popcll(mask));
            at = __builtin_amdgcn_readlane(at, __builtin_ctzll(mask)) + before;
            if (any && at < kRoom)
                runs[at] = i;
        });
        __syncthreads();
        const int n = s.runs;
        if (n > kRoom) {
            for_some(test, f);
            return;
        }
        for (int y = tid; y < n; y += THREADS) {
            const int i = runs[y];
            const Packed<B, V> v = load_run<B, V>(row + i, K - i);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float z = i + e < K ? T::widen(v.v[e]) : -INFINITY;
                if (test(z))
                    f(z, i + e);
            }
        }
    }
    // For each of few elements, how many come before it in the order, and their
    // weight.  Thread (part, x) adds up its part's share for element x.
    __device__ __forceinline__ void rank_all(Few &few) {
        constexpr int kParts = THREADS / kSmall;
        const int n = few.count;
        if (tid < n) {
            few.amount[tid] = amount_of<false>(few.element[tid]);
            few.before[tid] = 0;
            few.rank[tid] = 0;
        }
        __syncthreads();
        const int x = tid % kSmall, part = tid / kSmall;
        if (x < n) {
            const uint64_t mine = few.element[x];
            const int beg = n * part / kParts, end = n * (part + 1) / kParts;
            uint64_t sum = 0;
            int rank = 0;
#pragma unroll 4
            for (int y = beg; y < end; ++y) {
                const bool first = few.element[y] > mine;
                sum += first ? few.amount[y] : 0;
                rank += first;
            }
            add(&few.before[x], sum);
            atomicAdd(&few.rank[x], rank);
        }
        __syncthreads();
    }
    // Of few ranked elements the one at which the weight reaches `target`; `upto`
    // is the weight with it.  Ends with a barrier.
    __device__ __forceinline__ uint64_t find_few(const Few &few, uint64_t target, uint64_t &upto) {
        if (tid < few.count) {
            const uint64_t at = few.before[tid], own = few.amount[tid];
            if (at < target && target <= at + own) {
                s.found_element = few.element[tid];
                s.found_amount[0] = at + own;
            }
        }
        __syncthreads();
        upto = s.found_amount[0];
        const uint64_t e = s.found_element;
        __syncthreads();
        return e;
    }

    // The element of bin b at which the running amount within the bin (of
    // elements where COUNT, else of weight) reaches `target`, by the bits of their
    // values, then, among equal ones, of their indexes; `upto` is that running
    // amount, its own included.  For bins of many elements.
    template <bool COUNT>
    __device__ __forceinline__ uint64_t divide(int b, uint64_t target, uint64_t &upto) {
        const float beg = static_cast<float>(b), end = static_cast<float>(b + 1);
        __syncthreads();
        if (tid == 0) {
            s.lo = 0xffffffffu;
            s.hi = 0;
        }
        __syncthreads();
        auto inside = [&](float z) __attribute__((always_inline)) {
            const float x = place(z);
            return x >= beg && x < end;
        };
        for_kept(inside, [&](float z, int) __attribute__((always_inline)) {
            atomicMin(&s.lo, key_of(z));
            atomicMax(&s.hi, key_of(z));
        });
        __syncthreads();
        uint32_t lo = s.lo, hi = s.hi;
        uint64_t sum = 0;
        while (lo < hi) {
            const int shift = max(0, 32 - __builtin_clz(hi - lo) - __builtin_ctz(BINS));
            clear(s.other);
            __syncthreads();
            for_kept(inside, [&](float z, int i) __attribute__((always_inline)) {
                const uint32_t key = key_of(z);
                if (key >= lo && key <= hi)
                    add(&s.other[(hi - key) >> shift], amount_of<COUNT>(element_of(key, i)));
            });
            if (!locate(s.other, target - sum))         // only if the row changed meanwhile
                break;
            sum += s.found_before[0];
            hi -= static_cast<uint32_t>(s.found[0]) << shift;
            const uint32_t rest = (1u << shift) - 1;
            lo = hi - lo > rest ? hi - rest : lo;
        }
        const uint32_t key = lo;
        const uint64_t each = max(amount_of<COUNT>(element_of(key, 0)), uint64_t(1));
        uint64_t nth = (target - sum + each - 1) / each;              // of the equal ones
        upto = sum + nth * each;
        return element_of(key, nth_of(key, nth));
    }
    // Index of the nth (from 1) element of this value.
    __device__ __forceinline__ int nth_of(uint32_t key, uint64_t nth) {
        int first = 0, last = K - 1;
        while (first < last) {
            const int shift = max(0, 32 - __builtin_clz(last - first) - __builtin_ctz(BINS));
            __syncthreads();
            clear(s.other);
            __syncthreads();
            for_some([&](float z) __attribute__((always_inline)) { return key_of(z) == key; },
                     [&](float, int i) __attribute__((always_inline)) {
                         if (i >= first && i <= last)
                             add(&s.other[(i - first) >> shift], 1);
                     });
            if (!locate(s.other, nth))
                break;
            nth -= s.found_before[0];
            first += s.found[0] << shift;
            last = min(last, first + (1 << shift) - 1);
        }
        return first;
    }

    // The running weight that a draw of u from `total` has to reach.
    static __device__ __forceinline__ uint64_t drawn(float u, uint64_t total) {
        const double at = static_cast<double>(u) * static_cast<double>(total);
        if (!(at > 0.0))
            return 1;
        return at < static_cast<double>(total) ? min(static_cast<uint64_t>(at), total - 1) + 1
                                               : total;
    }
    // The least running weight that has p of `total`.
    static __device__ __forceinline__ uint64_t share(float p, uint64_t total) {
        const double want = ceil(static_cast<double>(p) * static_cast<double>(total));
        return want >= 1.0 ? min(static_cast<uint64_t>(want), total) : uint64_t(1);
    }

    static __device__ __forceinline__ uint64_t least_weight(float min_p) {
        return min_p > 0.0f ? static_cast<uint64_t>(ceil(fmin(static_cast<double>(min_p), 1.0) *
                                                         (1ull << kWeightBits)))
                            : 0;
    }

    // Gathers every element up to bin b into the list; false where they are more
    // than it holds.
    __device__ __forceinline__ bool gather(int b) {
        const float end = static_cast<float>(b + 1);
        __syncthreads();
        if (tid == 0)
            s.count = 0;
        __syncthreads();
        for_listed([&](float z) __attribute__((always_inline)) { return place(z) < end; },
                   [&](float z, int i) __attribute__((always_inline)) {
                       const int x = atomicAdd(&s.count, 1);
                       if (x < LIST)
                           s.list[x] = element_of(key_of(z), i);
                   });
        __syncthreads();
        const bool whole = s.count <= LIST;
        listed = whole ? s.count : -1;
        return whole;
    }

    // All that can be drawn is in the list and few: every border from their
    // order.
    __device__ __forceinline__ int from_few(int k, float p, float min_p, float u) {
        Few &few = s.draw;
        __syncthreads();
        if (tid < listed)
            few.element[tid] = s.list[tid];
        if (tid == 0)
            few.count = listed;
        __syncthreads();
        rank_all(few);
        const uint64_t least = least_weight(min_p);
        // Weight of the first k, and of those with w >= min_p.
        uint64_t first = 0, likely = 0;
        if (tid < listed) {
            const uint64_t own = few.amount[tid];
            first = few.rank[tid] < k ? own : 0;
            likely = own >= least ? own : 0;
        }
        uint64_t total = group_sum(first);
        if (min_p > 0.0f)
            likely = group_sum(likely);
        if (p < 1.0f) {
            uint64_t upto;
            find_few(few, share(p, total), upto);
            total = upto;
        }
        if (min_p > 0.0f)
            total = min(total, likely);
        uint64_t upto;
        return index_of(find_few(few, drawn(u, total), upto));
    }

    // Logits of +infinity share the row: weights of one each.
    __device__ __forceinline__ int from_infinities(float t, int k, float p, float u) {
        uint64_t n = 0;
        for_runs<32>([&](const float (&z)[V], int) __attribute__((always_inline)) {
#pragma unroll
            for (int e = 0; e < V; ++e)
                n += z[e] == INFINITY;
        });
        n = group_sum(n);
        if (k > 0)
            n = min(n, static_cast<uint64_t>(k));
        if (p < 1.0f)
            n = (share(p, n << kWeightBits) + (1ull << kWeightBits) - 1) >> kWeightBits;
        const uint64_t target = t > 0.0f ? drawn(u, n << kWeightBits) : 1;
        return nth_of(key_of(INFINITY), (target + (1ull << kWeightBits) - 1) >> kWeightBits);
    }

    // The row's label, the same on every thread.
    __device__ __forceinline__ int run(float t, int k, float p, float min_p, float u) {
        if (tid < kTable)
            s.table[tid] = kEighths[tid >> 4] * k128ths[tid & 15];
        clear(s.mass);
        clear(s.other);
        float mine = -INFINITY;
        for_runs<32>([&](const float (&z)[V], int) __attribute__((always_inline)) {
#pragma unroll
            for (int e = 0; e < V; ++e)
                mine = fmaxf(mine, z[e]);
        });
        float most = mine;
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
        if (m == INFINITY)
            return from_infinities(t, k, p, u);
        if (!(t > 0.0f)) {
            int first = K;
            for_some([&](float z) __attribute__((always_inline)) { return z == m; },
                     [&](float, int i) __attribute__((always_inline)) { first = min(first, i); });
            if (first < K)
                atomicMin(&s.count, first);
            __syncthreads();
            return s.count;
        }
        t = fmaxf(t, 0x1p-120f);                        // scale stays finite
        scale = BINS / kSpan / t;
        rate = kTable * 1.44269504088896340736 / static_cast<double>(t);
        limit = 0;
        listed = -1;
        if (k <= 0 || k > K)
            k = K;

        if (k < K) {
            // The k-th largest of the threads' own largest is no larger than the
            // row's k-th: all from its bin up are gathered, a few more than k.
            // With more than THREADS to keep, or too many gathered, the row's own
            // counts say where the k-th is.
            const float x = place(mine);
            if (x < static_cast<float>(BINS))
                add(&s.other[static_cast<int>(x)], 1);
            bool more = locate(s.other, k);             // than k in the span, or k
            if (!more || !gather(s.found[0])) {
                count_bins();
                more = locate(s.other, k);
                if (more && s.found_before[0] + s.found_amount[0] <= LIST)
                    gather(s.found[0]);
            }
            if (listed >= 0 && listed <= kSmall)
                return from_few(k, p, min_p, u);
            if (more) {
                if (listed >= 0) {
                    count_bins();
                    locate(s.other, k);
                }
                uint64_t upto;
                const int at = s.found[0];
                limit = divide<true>(at, k - s.found_before[0], upto);
            }
        } else if (min_p > 0.0f && !(p < 1.0f)) {
            // Those with w >= min_p, and a bin more for roundings.
            const float x = -logf(fminf(min_p, 1.0f)) * (BINS / kSpan);
            if (x < static_cast<float>(BINS - 2) && gather(static_cast<int>(x) + 1) &&
                listed <= kSmall)
                return from_few(k, p, min_p, u);
            listed = -1;
        }

        const uint64_t least = least_weight(min_p);
        uint64_t likely = 0;                            // weight of those with w >= min_p
        auto weigh = [&](float x, uint64_t w) __attribute__((always_inline)) {
            add(&s.mass[static_cast<int>(x)], w);
            if (min_p > 0.0f)
                likely += w >= least ? w : 0;
        };
        if (listed >= 0 || limit != 0) {
            for_kept(
                [&](float z) __attribute__((always_inline)) { return in_span(z); },
                [&](float z, int) __attribute__((always_inline)) { weigh(place(z), weight(z)); });
        } else {
            // The weights of a run together, without a branch between them (past
            // the span they are anything).
            for_runs<16>([&](const float (&z)[V], int) __attribute__((always_inline)) {
                uint64_t w[V];
#pragma unroll
                for (int e = 0; e < V; ++e)
                    w[e] = weight(z[e]);
#pragma unroll
                for (int e = 0; e < V; ++e)
                    if (in_span(z[e]))
                        weigh(place(z[e]), w[e]);
            });
        }
        if (tid == 0)
            s.end.count = s.draw.count = 0;
        likely = min_p > 0.0f ? group_sum(likely) : ~0ull;
        const Running r = running(s.mass);
        // The weight of all kept lies between lo and hi: the nucleus ends within
        // a bin.
        uint64_t lo = r.total, hi = r.total, before_end = 0, in_end = 0;
        int end = -1;
        if (p < 1.0f) {
            const uint64_t target = share(p, r.total);
            find(r, target, target);
            end = s.found[0];
            before_end = s.found_before[0];
            in_end = target - before_end;
            lo = before_end + 1;
            hi = before_end + s.found_amount[0];
        }
        lo = min(lo, likely);
        hi = min(hi, likely);
        find(r, drawn(u, lo), drawn(u, hi));
        const int from = s.found[0], to = s.found[1];
        const uint64_t before_from = s.found_before[0];
        auto bin = [&](float z) __attribute__((always_inline)) {       // of any value
            return static_cast<int>(fminf(place(z), static_cast<float>(BINS + 1)));
        };
        auto test = [&](float z) __attribute__((always_inline)) {
            const int b = bin(z);
            return b == end || static_cast<uint32_t>(b - from) <= static_cast<uint32_t>(to - from);
        };
        auto sort = [&](float z, int i) __attribute__((always_inline)) {
            const int b = bin(z);
            if (b == end)
                put(s.end, element_of(key_of(z), i));
            if (b >= from && b <= to)
                put(s.draw, element_of(key_of(z), i));
        };
        if (listed >= 0 || limit != 0)
            for_kept(test, sort);
        else
            for_listed(test, sort);
        __syncthreads();
        uint64_t total = hi, upto;
        if (end >= 0) {
            if (s.end.count <= kSmall) {
                rank_all(s.end);
                find_few(s.end, in_end, upto);
            } else {
                divide<false>(end, in_end, upto);
            }
            total = min(before_end + upto, likely);
        }
        const uint64_t target = drawn(u, total);
        if (s.draw.count <= kSmall) {
            rank_all(s.draw);
            return index_of(find_few(s.draw, target - before_from, upto));
        }
        find(r, target, target);
        const int b = s.found[0];
        return index_of(divide<false>(b, target - s.found_before[0], upto));
    }
};

template <typename T, int THREADS, int BINS, int LIST>
__global__ __launch_bounds__(THREADS, 4)
void sample_kernel(const Sample a) {
    typedef Draw<T, THREADS, BINS, LIST> D;
    __shared__ typename D::Shared s;
    const int64_t row = a.first + blockIdx.x;
    D d{s, static_cast<const typename T::bits *>(a.logits) + row * a.ld, a.K,
        static_cast<int>(threadIdx.x)};
    // One value for the workgroup: kept in scalar registers.
    auto uniform = [](float v) __attribute__((always_inline)) {
        return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(v)));
    };
    const int k = __builtin_amdgcn_readfirstlane(a.top_ks != nullptr ? a.top_ks[row] : a.top_k);
    const int label =
        d.run(uniform(a.temperatures != nullptr ? a.temperatures[row] : a.temperature), k,
              uniform(a.top_ps != nullptr ? a.top_ps[row] : a.top_p),
              uniform(a.min_ps != nullptr ? a.min_ps[row] : a.min_p), uniform(a.u[row]));
    if (threadIdx.x != 0)
        return;
    if (a.wide)
        static_cast<int64_t *>(a.labels)[row] = label;
    else
        static_cast<int32_t *>(a.labels)[row] = label;
}

template <typename T>
hipError_t run_sample(Sample a, int64_t N, int compute_units, hipStream_t stream) {
    constexpr int64_t kMaxGrid = int64_t(1) << 21;      // a launch has less than 2^32 threads
    hipError_t e = hipSuccess;
    for (int64_t first = 0; first < N && e == hipSuccess; first += kMaxGrid) {
        a.first = first;
        const dim3 grid(static_cast<unsigned>(std::min(kMaxGrid, N - first)));
        if (a.K <= 4096)
            hipLaunchKernelGGL((sample_kernel<T, 256, 512, 1024>), grid, dim3(256), 0, stream, a);
        else if (N <= compute_units)
            hipLaunchKernelGGL((sample_kernel<T, 1024, 2048, 4096>), grid, dim3(1024), 0, stream,
                               a);
        else
            hipLaunchKernelGGL((sample_kernel<T, 512, 2048, 4096>), grid, dim3(512), 0, stream, a);
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
    const int cus = device_compute_units();
    const hipError_t e = dtype == KMEANS_BF16   ? run_sample<Bf16>(a, N, cus, stream)
                         : dtype == KMEANS_FP16 ? run_sample<Fp16>(a, N, cus, stream)
                                                : run_sample<Fp32>(a, N, cus, stream);
    if (e != hipSuccess)
        return fail(KMEANS_ERR_HIP, "sample launch failed: %s", hipGetErrorString(e));
    return ok();
}
