// kmeans_sample.hip -- gfx950 kernel that draws a label from each row of logits
// by temperature, top-k, top-p and min-p, from given random numbers.
//
//     order: logit descending, index ascending;  w_i = exp((z_i - max) / t)
//     kept:  a prefix of that order, the shortest of: the first k; the shortest
//            with p of the first k's weight; those with w_i >= min_p
//     label: first in that order whose running weight exceeds u times the
//            weight of all kept
//
// Weights are summed in 64-bit integers, so that every sum is exact and the same
// in any order, from atomics too: the label depends on the row and its settings
// alone, not on the launch (which way below a row takes goes by its length, its
// settings and its values).  A weight is a multiple of 2^-43 of its bin's centre
// (below); a bin's sum is brought to the scale of the largest weight with one
// rounding, to 2^-43 of that.  32-bit sums would shift the borders by 1e-7 of the whole and draw other
// labels in one row of some thousands.
//
// All borders (the k-th value, the nucleus's end, the draw) are one thing: the
// element at which a running amount (of elements or of weight) reaches a target.
// Where few elements can be drawn (the first k, those above min_p) they are
// gathered and compared with one another.  Otherwise a histogram by the distance
// to a large logit finds the bins of the nucleus's end and of the draw, whose
// elements are gathered and compared.  Where even those are many, they are
// divided further by the bits of their values and indexes.  No sorting.
//
// The histogram needs no maximum first: its bins lie around the largest of the
// row's first values, BINS on either side, and the weights within a bin are
// relative to the bin.  So a row is read from memory once for it (the weights
// under the loads), and once more, from the memory-side cache, to gather.
//
// 512 x 65536 fp32, top-p: 58 us (134 MB; 25 us to read them once).  Each workgroup
// first waits for memory, then for its weights (22 VALU instructions an element,
// 14 of them fp64), then for the second reading (10 us), and all run in step.
// The adds of a row's many likely labels to a few bins cost LDS conflicts too (0.63 of
// the LDS's active cycles).  Three readings (maximum, weights, borders) took 81 us,
// five 125.  16 x 32768 with top-k 50: 10 us of which 1.5 read the row, the rest 20
// barriers; top-p and the draw 21, the histogram and the second reading more.
#include <float.h>
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
constexpr float kSpan = 32.0f;       // temperatures that BINS bins span; labels that
                                     // far below the largest are never drawn
constexpr int kFirst = 4096;         // values whose largest the bins lie around

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

// A value that is the same on every lane, into scalar registers.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ float uniform(float v) {
    return __uint_as_float(uniform(__float_as_uint(v)));
}
__device__ __forceinline__ uint64_t uniform(uint64_t v) {
    return static_cast<uint64_t>(uniform(static_cast<uint32_t>(v >> 32))) << 32 |
           uniform(static_cast<uint32_t>(v));
}
__device__ __forceinline__ double uniform(double v) {
    return __longlong_as_double(uniform(static_cast<uint64_t>(__double_as_longlong(v))));
}

template <typename T, int THREADS, int BINS, int SMALL>
struct Draw {
    typedef typename T::bits B;
    static constexpr int kWaves = THREADS / 64;
    static constexpr int V = 16 / sizeof(B);         // values of a load
    // Most elements compared with one another (a bin of 1/64 temperature of 131072 normal
    // logits, deviation 3, holds up to 272: 256 rows of those 114 us with 256).
    static constexpr int kSmall = SMALL;
    static_assert(THREADS % SMALL == 0, "a thread for each, and whole parts of a row");
    static constexpr float kBins = BINS;

    struct Few {
        uint64_t element[kSmall];
        int count;
    };
    struct Shared {
        uint64_t wide[2 * BINS];     // units by bin, then the running weight with
                                     // each; or all that may belong to the first k
        union {                      // (LDS past 64 KB costs registers)
            uint64_t other[BINS];    // counts, the finer divisions, listed runs
            struct {                 // of few elements
                uint64_t amount[kSmall], before[kSmall];
                int rank[kSmall];
            };
        };
        Few end, draw, likely;       // around the k-th or the nucleus's end, around
                                     // the draw, around min_p
        double coarse[2 * BINS / 64], fine[64], lift;   // see factor()
        uint64_t sums[2][kWaves];
        float most[kWaves];
        uint64_t found_element, found_upto, total;
        uint64_t kept;               // by the first k, of few elements
        int count, runs;
        uint32_t lo, hi;
    };

    Shared &s;
    const B *row;
    int K, tid;
    float m, scale;                  // largest logit; bins per unit of logit
    float ref;                       // the bins lie around it, BINS on either side
    double rate;                     // bins per unit of logit
    uint64_t limit;                  // elements below it are not among the first k

    // Loads U runs of V values, THREADS V values from one to the next, the first
    // from c0 on (of the workgroup's block from base on); -infinity past n.
    template <int U>
    __device__ __forceinline__ void load_block(Packed<B, V> (&v)[U], int base, int c0, int n) const {
        if (base + THREADS * V * U <= n) {
#pragma unroll
            for (int x = 0; x < U; ++x)
                v[x] = load_packed<B, V>(row + c0 + x * THREADS * V);
        } else {
#pragma unroll
            for (int x = 0; x < U; ++x) {
                const int c = c0 + x * THREADS * V;
#pragma unroll
                for (int e = 0; e < V; ++e)
                    v[x].v[e] = T::narrow(-INFINITY);
                if (c + V <= n)
                    v[x] = load_packed<B, V>(row + c);
                else
                    for (int e = 0; c + e < n; ++e)
#pragma unroll
                        for (int y = 0; y < V; ++y)
                            if (y == e)
                                v[x].v[y] = row[c + e];
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    // f(z, i) for every run of the row's first n values: V of them from index i on,
    // -infinity past the end; VALUES of a thread in flight.
    template <int VALUES, typename F>
    __device__ __forceinline__ void for_runs(int n, const F &f) const {
        constexpr int U = VALUES / V;
#pragma unroll 1
        for (int base = 0; base < n; base += THREADS * VALUES) {
            const int c0 = base + tid * V;
            Packed<B, V> v[U];
            load_block(v, base, c0, n);
#pragma unroll
            for (int x = 0; x < U; ++x) {
                float z[V];
#pragma unroll
                for (int e = 0; e < V; ++e)
                    z[e] = T::widen(v[x].v[e]);
                f(z, c0 + x * THREADS * V);
            }
        }
    }
    template <int VALUES, typename F>
    __device__ __forceinline__ void for_runs(const F &f) const {
        for_runs<VALUES>(K, f);
    }
    // f(z, i) for every element with test(z).  Few are expected: a run without
    // any costs no more than the tests.
    template <typename P, typename F>
    __device__ __forceinline__ void for_some(const P &test, const F &f) const {
        for_runs<2 * V>([&](const float (&z)[V], int i) __attribute__((always_inline)) {
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
    // The same of those among the first k.
    template <typename P, typename F>
    __device__ __forceinline__ void for_kept(const P &test, const F &f) const {
        for_some(test, [&](float z, int i) __attribute__((always_inline)) {
            if (limit == 0 || element_of(key_of(z), i) >= limit)
                f(z, i);
        });
    }

    // Distance to ref in bins, not decreasing as logits do, and a half: a bin's
    // centre lies at a whole distance, so that logits as good as equal to ref get
    // the weight one exactly.  NaN of a NaN.
    __device__ __forceinline__ float place(float z) const { return (ref - z) * scale + 0.5f; }
    // Whether a logit has a bin, and which.
    __device__ __forceinline__ bool in_span(float z) const { return fabsf(place(z)) < kBins; }
    __device__ __forceinline__ int bin_of(float z) const {
        return static_cast<int>(floorf(place(z))) + BINS;
    }

    // exp(-d h) in units of 2^-43, d the distance of a logit to its bin's centre in
    // bins (of h temperatures): the powers of d up to one whose successor is 4e-16
    // at most.  The last sum puts the integer into the low bits.
    __device__ __forceinline__ uint64_t unit(float z, int b) const {
        constexpr double h = kSpan / BINS;
        constexpr int kTerms = BINS >= 2048 ? 6 : 8;
        static_assert(BINS >= 512, "terms by the width of a bin");
        constexpr double one = 8796093022208.0;                      // 2^43
        constexpr double kMagic = 4503599627370496.0;                // 2^52
        const double d = fma(static_cast<double>(ref) - static_cast<double>(z), rate,
                             -static_cast<double>(b - BINS));
        double c[kTerms];
        c[0] = one;
#pragma unroll
        for (int n = 1; n < kTerms; ++n)
            c[n] = c[n - 1] * -h / n;
        double p = c[kTerms - 1];
#pragma unroll
        for (int n = kTerms - 2; n >= 1; --n)
            p = fma(p, d, c[n]);
        p = fma(p, d, c[0] + kMagic);
        return __double_as_longlong(p) & 0xfffffffffffffull;
    }
    // Weight of a bin's centre against the largest logit: exp(h (distance of the
    // largest - that of the centre)), from exp(-h i) in two factors and `lift`,
    // exp(h distance of the largest).
    __device__ __forceinline__ double factor(int b) const {
        return s.coarse[b / 64] * s.fine[b % 64] * s.lift;
    }
    __device__ __forceinline__ void make_table() {
        constexpr int kCoarse = 2 * BINS / 64;
        static_assert(kCoarse + 64 <= THREADS, "one entry to a thread");
        if (tid < kCoarse + 64) {
            const int i = tid < kCoarse ? 64 * tid - BINS : tid - kCoarse;
            (tid < kCoarse ? s.coarse[tid] : s.fine[i]) = exp(-static_cast<double>(kSpan / BINS) * i);
        }
    }
    static __device__ __forceinline__ uint64_t whole(double v) {
        return static_cast<uint64_t>(v + 0.5);
    }
    // exp((z - m) / t) in units of 2^-43, of one of few.
    __device__ __forceinline__ uint64_t weight(float z) const {
        const double x = (static_cast<double>(m) - static_cast<double>(z)) * rate * (kSpan / BINS);
        return x < kSpan ? whole(exp(-x) * (1ull << kWeightBits)) : 0;
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
        return uniform(total);
    }
    __device__ __forceinline__ float group_most(float v) {
#pragma unroll
        for (int x = 32; x >= 1; x >>= 1)
            v = fmaxf(v, __shfl_xor(v, x, 64));
        __syncthreads();
        if ((tid & 63) == 0)
            s.most[tid >> 6] = v;
        __syncthreads();
        v = s.most[0];
#pragma unroll
        for (int w = 1; w < kWaves; ++w)
            v = fmaxf(v, s.most[w]);
        return uniform(v);
    }

    // Replaces N bins by the running sums with each of what amount(bin, sum) makes
    // of them; returns the total.  Begins and ends with a barrier.
    template <int N, typename F>
    __device__ __forceinline__ uint64_t run_sums(uint64_t *hist, const F &amount) {
        constexpr int kEach = N / THREADS;
        uint64_t own[kEach], v = 0;
        __syncthreads();
#pragma unroll
        for (int x = 0; x < kEach; ++x) {
            own[x] = hist[tid * kEach + x];
            v |= own[x];
        }
        const bool any = __ballot(v != 0) != 0;         // often not: few bins are in use
        v = 0;
        if (any) {
#pragma unroll
            for (int x = 0; x < kEach; ++x) {
                own[x] = amount(tid * kEach + x, own[x]);
                v += own[x];
            }
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
        uint64_t total = 0, at = run - v;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const uint64_t sum = s.sums[1][w];
            at += w < tid >> 6 ? sum : 0;
            total += sum;
        }
#pragma unroll
        for (int x = 0; x < kEach; ++x) {
            at += own[x];
            hist[tid * kEach + x] = at;
        }
        __syncthreads();
        return uniform(total);
    }
    // The first of N bins whose running sum reaches `target` (N: none does): each
    // lane looks at the last of 64 bins, then at one of those 64.
    template <int N>
    __device__ __forceinline__ int find(const uint64_t *sums, uint64_t target) const {
        const int lane = tid & 63;
        static_assert(N % 64 == 0 && N <= 64 * 64, "two looks");
        const uint64_t last = sums[min(lane, N / 64 - 1) * 64 + 63];
        const int block = __popcll(__ballot(lane < N / 64 && last < target));
        if (block == N / 64)
            return N;
        return block * 64 + __popcll(__ballot(sums[block * 64 + lane] < target));
    }
    static __device__ __forceinline__ uint64_t before(const uint64_t *sums, int b) {
        return uniform(b > 0 ? sums[b - 1] : uint64_t(0));
    }

    template <int N>
    __device__ __forceinline__ void clear(uint64_t *hist) {
        for (int x = tid; x < N; x += THREADS)
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
    // Calls f(z, i) for the elements of the row with miss(z) <= 0 (a number, since
    // masks of lanes are slow to combine), a few hundred of them, in two steps: the
    // runs that hold one are listed, one count for those of a wave; then each thread
    // takes some of them.  So the loop over the row has little more than the tests
    // (a wave's 256 or 512 elements hold a hit more often than not).  Where there are
    // more runs than `runs` holds, one step.
    template <typename P, typename F>
    __device__ __forceinline__ void for_listed(const P &miss, const F &f) {
        auto *runs = reinterpret_cast<int *>(s.other);
        constexpr int kRoom = 2 * BINS;
        constexpr int U = 32 / V;
        __syncthreads();
        if (tid == 0)
            s.runs = 0;
        __syncthreads();
#pragma unroll 1
        for (int base = 0; base < K; base += THREADS * 32) {
            const int c0 = base + tid * V;
            Packed<B, V> v[U];
            load_block(v, base, c0, K);
            uint32_t hits = 0;
#pragma unroll
            for (int x = 0; x < U; ++x) {
                float least = INFINITY;
#pragma unroll
                for (int e = 0; e < V; ++e)
                    least = fminf(least, miss(T::widen(v[x].v[e])));
                hits |= least <= 0.0f ? 1u << x : 0;
            }
            for (;;) {                                  // a run of each lane at a time
                const uint64_t mask = __ballot(hits != 0);
                if (mask == 0)
                    break;
                const int before = __builtin_amdgcn_mbcnt_hi(
                    static_cast<uint32_t>(mask >> 32),
                    __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(mask), 0));
                int at = 0;
                if (hits != 0 && before == 0)
                    at = atomicAdd(&s.runs, __popcll(mask));
                at = __builtin_amdgcn_readlane(at, __builtin_ctzll(mask)) + before;
                if (hits != 0 && at < kRoom)
                    runs[at] = c0 + __builtin_ctz(hits) * THREADS * V;
                hits &= hits - 1;
            }
        }
        __syncthreads();
        const int n = s.runs;
        if (n > kRoom) {
            for_some([&](float z) __attribute__((always_inline)) { return miss(z) <= 0.0f; }, f);
            return;
        }
        for (int y = tid; y < n; y += THREADS) {
            const int i = runs[y];
            const Packed<B, V> v = load_run<B, V>(row + i, K - i);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float z = i + e < K ? T::widen(v.v[e]) : -INFINITY;
                if (miss(z) <= 0.0f)
                    f(z, i + e);
            }
        }
    }

    // For each of few elements, how many come before it in the order, and their
    // amounts (amount(z)).  Thread (part, x) adds up its part's share for element
    // x, in as many parts as there are threads for.
    template <typename F>
    __device__ __forceinline__ void rank_all(const Few &few, const F &amount) {
        const int n = uniform(few.count);
        if (tid < n) {
            s.amount[tid] = amount(value_of(static_cast<uint32_t>(few.element[tid] >> 32)));
            s.before[tid] = 0;
            s.rank[tid] = 0;
        }
        __syncthreads();
        const int shift = n <= 64 ? 6 : n <= 128 ? 7 : n <= 256 ? 8 : 9;
        const int x = tid & ((1 << shift) - 1), part = tid >> shift;
        if (x < n) {
            const uint64_t mine = few.element[x];
            const int parts = THREADS >> shift;
            const int beg = n * part / parts, end = n * (part + 1) / parts;
            uint64_t sum = 0;
            int rank = 0;
#pragma unroll 4
            for (int y = beg; y < end; ++y) {
                const bool first = few.element[y] > mine;
                sum += first ? s.amount[y] : 0;
                rank += first;
            }
            add(&s.before[x], sum);
            atomicAdd(&s.rank[x], rank);
        }
        __syncthreads();
        if (tid < n && s.rank[tid] == n - 1)
            s.total = s.before[tid] + s.amount[tid];
        __syncthreads();
    }
    // Of few ranked elements the one at which the amount reaches `target`, the
    // last one with an amount where none does; `upto` is the amount with it.  Ends
    // with a barrier.
    __device__ __forceinline__ uint64_t find_few(const Few &few, uint64_t target, uint64_t &upto) {
        const bool real = tid < few.count;
        const uint64_t at = real ? s.before[tid] : 0, own = real ? s.amount[tid] : 0;
        target = min(target, uniform(s.total));
        if (real && at < target && target <= at + own) {
            s.found_element = few.element[tid];
            s.found_upto = at + own;
        }
        __syncthreads();
        upto = uniform(s.found_upto);
        const uint64_t e = uniform(s.found_element);
        __syncthreads();
        return e;
    }

    // The value in bin b at which the running amount within the bin (of elements
    // where `count`, else of units) reaches `target`, by the values' bits, and
    // which of the elements of that value; `upto` is that running amount, its own
    // included.  For bins of many elements.
    __device__ __forceinline__ uint32_t divide(bool count, int b, uint64_t target, uint64_t &nth,
                                               uint64_t &upto) {
        auto inside = [&](float z) __attribute__((always_inline)) {
            return in_span(z) && bin_of(z) == b;
        };
        if (tid == 0) {
            s.lo = 0xffffffffu;
            s.hi = 0;
        }
        __syncthreads();
        for_kept(inside, [&](float z, int) __attribute__((always_inline)) {
            atomicMin(&s.lo, key_of(z));
            atomicMax(&s.hi, key_of(z));
        });
        __syncthreads();
        uint32_t lo = uniform(s.lo), hi = uniform(s.hi);
        uint64_t sum = 0;
        while (lo < hi) {
            const int shift = max(0, 32 - __builtin_clz(hi - lo) - __builtin_ctz(BINS));
            clear<BINS>(s.other);
            __syncthreads();
            for_kept(inside, [&](float z, int) __attribute__((always_inline)) {
                const uint32_t key = key_of(z);
                if (key >= lo && key <= hi)
                    add(&s.other[(hi - key) >> shift], count ? uint64_t(1) : unit(z, b));
            });
            const uint64_t total =
                run_sums<BINS>(s.other, [](int, uint64_t v) __attribute__((always_inline)) { return v; });
            target = min(target, sum + total);
            const int at = find<BINS>(s.other, target - sum);
            sum += before(s.other, at);
            __syncthreads();
            if (at >= BINS)                             // only if the row changed meanwhile
                break;
            hi -= static_cast<uint32_t>(at) << shift;
            const uint32_t rest = (1u << shift) - 1;
            lo = hi - lo > rest ? hi - rest : lo;
        }
        const uint64_t each = uniform(count ? 1 : max(unit(value_of(lo), b), uint64_t(1)));
        nth = max((target - sum + each - 1) / each, uint64_t(1));
        upto = sum + nth * each;
        return lo;
    }
    // Index of the nth (from 1) element of this value.
    __device__ __forceinline__ int nth_of(uint32_t key, uint64_t nth) {
        int first = 0, last = K - 1;
        while (first < last) {
            const int shift = max(0, 32 - __builtin_clz(last - first) - __builtin_ctz(BINS));
            clear<BINS>(s.other);
            __syncthreads();
            for_some([&](float z) __attribute__((always_inline)) { return key_of(z) == key; },
                     [&](float, int i) __attribute__((always_inline)) {
                         if (i >= first && i <= last)
                             add(&s.other[(i - first) >> shift], 1);
                     });
            const uint64_t total =
                run_sums<BINS>(s.other, [](int, uint64_t v) __attribute__((always_inline)) { return v; });
            nth = min(nth, total);                      // less only if the row changed
            const int at = find<BINS>(s.other, nth);
            nth -= before(s.other, at);
            __syncthreads();
            if (at >= BINS || nth == 0)
                break;
            first += at << shift;
            last = min(last, first + (1 << shift) - 1);
        }
        return first;
    }

    // The running weight that a draw of u from `total` has to reach.
    static __device__ __forceinline__ uint64_t drawn(float u, uint64_t total) {
        const double at = static_cast<double>(u) * static_cast<double>(total);
        if (!(at > 0.0))
            return 1;
        return uniform(at < static_cast<double>(total)
                           ? min(static_cast<uint64_t>(at), total - 1) + 1
                           : total);
    }
    // The least running weight that has p of `total`.
    static __device__ __forceinline__ uint64_t share(float p, uint64_t total) {
        const double want = ceil(static_cast<double>(p) * static_cast<double>(total));
        return uniform(want >= 1.0 ? min(static_cast<uint64_t>(want), total) : uint64_t(1));
    }

    // Gathers every element with place(z) <= end; their number, -1 where they are
    // more than fit.
    __device__ __forceinline__ int gather(float end) {
        __syncthreads();
        if (tid == 0)
            s.count = 0;
        for_listed([&](float z) __attribute__((always_inline)) { return place(z) - end; },
                   [&](float z, int i) __attribute__((always_inline)) {
                       const int x = atomicAdd(&s.count, 1);
                       if (x < 2 * BINS)
                           s.wide[x] = element_of(key_of(z), i);
                   });
        __syncthreads();
        return s.count <= 2 * BINS ? s.count : -1;
    }

    // All that can be drawn is gathered and few: every border from their order.
    __device__ __forceinline__ int from_few(int n, int k, float p, float min_p, float u) {
        Few &few = s.draw;
        __syncthreads();
        if (tid < n)
            few.element[tid] = s.wide[tid];
        if (tid == 0)
            few.count = n;
        __syncthreads();
        rank_all(few, [&](float z) __attribute__((always_inline)) { return weight(z); });
        // Weight of the first k, and of those with w >= min_p.
        uint64_t total = uniform(s.total), likely = 0;
        if (k < n) {
            if (tid < n && s.rank[tid] == k - 1)
                s.kept = s.before[tid] + s.amount[tid];
            __syncthreads();
            total = uniform(s.kept);
        }
        if (min_p > 0.0f) {
            const double least = fmin(static_cast<double>(min_p), 1.0) * (1ull << kWeightBits);
            likely = group_sum(tid < n && static_cast<double>(s.amount[tid]) >= least ? s.amount[tid]
                                                                                      : 0);
        }
        uint64_t upto;
        if (p < 1.0f) {
            find_few(few, share(p, total), upto);
            total = upto;
        }
        if (min_p > 0.0f)
            total = min(total, likely);
        return index_of(find_few(few, drawn(u, total), upto));
    }

    // The histogram around ref of the whole row; returns the row's largest.
    __device__ __forceinline__ float weigh_row() {
        __syncthreads();
        clear<2 * BINS>(s.wide);
        __syncthreads();
        float most = -INFINITY;
        // The units of a run together, without a branch between them (outside the
        // span they are anything).
        for_runs<16>([&](const float (&z)[V], int) __attribute__((always_inline)) {
            uint64_t w[V];
            float x[V];
            int b[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                most = fmaxf(most, z[e]);
                x[e] = place(z[e]);
                b[e] = static_cast<int>(floorf(x[e])) + BINS;
                w[e] = unit(z[e], b[e]);
            }
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (fabsf(x[e]) < kBins)
                    add(&s.wide[b[e]], w[e]);
        });
        return group_most(most);
    }

    // The row's label, the same on every thread.
    __device__ __forceinline__ int run(float t, int k, float p, float min_p, float u) {
        if (k <= 0 || k > K)
            k = K;
        const bool greedy = !(t > 0.0f);
        t = fminf(fmaxf(t, 0x1p-120f), 0x1p120f);       // scale and its inverse stay finite
        scale = uniform(BINS / kSpan / t);
        rate = uniform((BINS / kSpan) / static_cast<double>(t));
        limit = 0;
        make_table();
        // What the loop below is to find: the border `border` in bin `bin`, where
        // the running units (or elements) reach `target`, or the nth element of
        // the value `key`.
        enum { kValue, kLimit, kEnd, kDraw } border = kValue;
        uint32_t key = 0;
        uint64_t nth = 1, target = 0;
        int bin = 0;
        // Whether all may be drawn: then all are weighed, around the largest of
        // the first ones.
        bool weighed = false;
        if (!greedy && K > kSmall && k == K && (p < 1.0f || !(min_p > 0.0f))) {
            float most = -INFINITY;
            for_runs<V>(min(K, kFirst), [&](const float (&z)[V], int) __attribute__((always_inline)) {
#pragma unroll
                for (int e = 0; e < V; ++e)
                    most = fmaxf(most, z[e]);
            });
            ref = group_most(most);
            if (fabsf(ref) < INFINITY) {
                // Again where the row's largest lies far above the first ones.
                for (int twice = 0; twice < 2 && !weighed; ++twice) {
                    m = weigh_row();
                    weighed = m < INFINITY && place(m) > -kBins;
                    ref = weighed ? ref : m;
                    if (m == INFINITY)
                        break;
                }
            }
        }
        if (!weighed) {
            float mine = -INFINITY;
            clear<BINS>(s.other);
            for_runs<32>([&](const float (&z)[V], int) __attribute__((always_inline)) {
#pragma unroll
                for (int e = 0; e < V; ++e)
                    mine = fmaxf(mine, z[e]);
            });
            m = ref = group_most(mine);
            if (m == -INFINITY)
                return -1;                              // nothing to draw
            if (greedy) {
                int first = K;
                for_some([&](float z) __attribute__((always_inline)) { return z == m; },
                         [&](float, int i) __attribute__((always_inline)) { first = min(first, i); });
                if (tid == 0)
                    s.count = K;
                __syncthreads();
                if (first < K)
                    atomicMin(&s.count, first);
                __syncthreads();
                return s.count;
            } else if (m == INFINITY) {
                // They share the row: weights of one each.
                uint64_t n = 0;
                for_runs<V>([&](const float (&z)[V], int) __attribute__((always_inline)) {
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        n += z[e] == INFINITY;
                });
                n = min(group_sum(n), static_cast<uint64_t>(k));
                auto rounded_up = [](uint64_t v) {
                    return (v + (1ull << kWeightBits) - 1) >> kWeightBits;
                };
                if (p < 1.0f)
                    n = rounded_up(share(p, n << kWeightBits));
                key = key_of(m);
                nth = rounded_up(drawn(u, n << kWeightBits));
            } else {
                // The k-th largest of the largest of kSmall parts of the row is
                // no larger than the row's k-th: all from its bin up are gathered,
                // a few more than k.  Without k, those with w >= min_p and a bin
                // more for roundings.  Of a short row, all.
                float end = kBins;
                if (k < K && K > kSmall) {
                    if constexpr (THREADS > kSmall) {
                        auto *most = reinterpret_cast<float *>(s.wide);
                        most[tid] = mine;
                        __syncthreads();
                        for (int x = tid + kSmall; x < THREADS; x += kSmall)
                            mine = fmaxf(mine, most[x]);
                    }
                    if (tid < kSmall && in_span(mine))
                        add(&s.other[bin_of(mine) - BINS], 1);
                    run_sums<BINS>(s.other, [](int, uint64_t v) __attribute__((always_inline)) { return v; });
                    end = static_cast<float>(find<BINS>(s.other, k) + 1);
                    __syncthreads();
                } else if (!(p < 1.0f) && K > kSmall && min_p > 0.0f) {
                    end = floorf(-logf(fminf(min_p, 1.0f)) * (BINS / kSpan)) + 2.0f;
                }
                if (end < kBins || K <= kSmall) {
                    const int n = gather(end);
                    if (n >= 0 && n <= kSmall)
                        return from_few(n, k, p, min_p, u);
                }
                if (k < K) {
                    // The row's own counts say where the k-th is.
                    __syncthreads();
                    clear<BINS>(s.other);
                    __syncthreads();
                    for_some([&](float z) __attribute__((always_inline)) { return in_span(z); },
                             [&](float z, int) __attribute__((always_inline)) {
                                 add(&s.other[bin_of(z) - BINS], 1);
                             });
                    const uint64_t total = run_sums<BINS>(
                        s.other, [](int, uint64_t v) __attribute__((always_inline)) { return v; });
                    if (total > static_cast<uint64_t>(k)) {
                        const int b = find<BINS>(s.other, k);
                        target = k - before(s.other, b);
                        bin = b + BINS;
                        border = kLimit;
                        __syncthreads();
                    }
                }
            }
        }

        const bool direct = m == INFINITY;
        if (!direct && border != kLimit)
            border = kDraw;
        bool fresh = !direct;                           // the borders' bins are to be gathered
        // The weight of all kept: `top` as far as it is known, between lo and hi.
        uint64_t top = 0, lo = 0, hi = 0, before_end = 0, end_amount = 0, before_likely = 0;
        int from = 0, likely_from = -1, likely_to = -1;
        uint32_t width = 0;                             // bins of the draw, from `from` on
        // Units kept of the nucleus's last bin (a target brought to units may
        // otherwise reach the element behind it).
        int end_bin = -1;
        uint64_t end_units = 0;
#pragma unroll 1
        for (;;) {
            if (fresh && border != kLimit) {
                if (!weighed && limit == 0) {
                    weigh_row();
                } else if (!weighed) {
                    __syncthreads();
                    clear<2 * BINS>(s.wide);
                    __syncthreads();
                    for_kept([&](float z) __attribute__((always_inline)) { return in_span(z); },
                             [&](float z, int) __attribute__((always_inline)) {
                                 add(&s.wide[bin_of(z)], unit(z, bin_of(z)));
                             });
                }
                if (tid < 64)
                    s.lift = exp((static_cast<double>(ref) - static_cast<double>(m)) * rate *
                                 (kSpan / BINS));
                top = run_sums<2 * BINS>(
                    s.wide, [&](int b, uint64_t v) __attribute__((always_inline)) {
                        const double f = v != 0 ? factor(b) : 0.0;
                        return f > 0x1p-46 ? whole(static_cast<double>(v) * f) : uint64_t(0);
                    });
                lo = hi = top;
                if (p < 1.0f) {
                    border = kEnd;
                    const uint64_t want = share(p, top);
                    bin = find<2 * BINS>(s.wide, want);
                    before_end = before(s.wide, bin);
                    end_amount = uniform(s.wide[bin]) - before_end;
                    target = want - before_end;
                    lo = before_end + 1;
                    hi = before_end + end_amount;
                }
                if (min_p > 0.0f) {
                    // The bins that its border may lie in (roundings in 32 bits).
                    const float far = place(m) - logf(fminf(min_p, 1.0f)) * (BINS / kSpan);
                    if (far < kBins - 1.0f) {
                        likely_from = uniform(max(static_cast<int>(floorf(far - 0x1p-6f)) + BINS, 0));
                        likely_to = uniform(max(static_cast<int>(floorf(far + 0x1p-6f)) + BINS, 0));
                        before_likely = before(s.wide, likely_from);
                        lo = min(lo, max(before_likely, uint64_t(1)));
                        hi = min(hi, uniform(s.wide[likely_to]));
                    }
                }
                from = find<2 * BINS>(s.wide, drawn(u, lo));
                width = find<2 * BINS>(s.wide, drawn(u, hi)) - from + 1;
            }
            if (fresh) {
                const int end = border == kDraw ? -1 : bin;
                // The middle and half the width of the logits that the bins may
                // hold, wider by all roundings; a width below zero where there is
                // no bin.  A middle past the type's range is at its end: no
                // logit is further out.
                auto middle = [&](int b, int bins) __attribute__((always_inline)) {
                    const float at = ref - (static_cast<float>(b - BINS) +
                                            0.5f * static_cast<float>(bins - 1)) / scale;
                    return uniform(fminf(fmaxf(at, -FLT_MAX), FLT_MAX));
                };
                auto half = [&](int bins) __attribute__((always_inline)) {
                    return uniform((0.5f * static_cast<float>(bins) + 0.01f + kBins * 0x1p-20f) /
                                       scale + fabsf(ref) * 0x1p-20f);
                };
                const float a = end < 0 ? 0.0f : middle(end, 1);
                const float a_half = end < 0 ? -1.0f : half(1);
                const float b = middle(from, width), b_half = width == 0 ? -1.0f : half(width);
                const int likely = likely_to - likely_from + 1;
                const float c = likely_from < 0 ? 0.0f : middle(likely_from, likely);
                const float c_half = likely_from < 0 ? -1.0f : half(likely);
                __syncthreads();
                if (tid == 0)
                    s.end.count = s.draw.count = s.likely.count = 0;
                for_listed(
                    [&](float z) __attribute__((always_inline)) {
                        return fminf(fminf(fabsf(z - a) - a_half, fabsf(z - b) - b_half),
                                     fabsf(z - c) - c_half);
                    },
                    [&](float z, int i) __attribute__((always_inline)) {
                        const int b = bin_of(z);
                        const uint64_t e = element_of(key_of(z), i);
                        if (!in_span(z) || e < limit)
                            return;
                        if (b == end)
                            put(s.end, e);
                        if (static_cast<uint32_t>(b - from) < width)
                            put(s.draw, e);
                        if (b == likely_from || b == likely_to)
                            put(s.likely, e);
                    });
                __syncthreads();
                fresh = false;
            }
            if (border == kEnd)
                target = uniform(
                    static_cast<uint64_t>(ceil(__ull2double_rz(target) / factor(bin))));
            if (border == kDraw) {
                uint64_t a = 0, b = 0;                  // units of min_p's bins that reach it
                if (likely_from >= 0) {
                    uint64_t sum[2] = {0, 0};
                    const double least =
                        fmin(static_cast<double>(min_p), 1.0) * (1ull << kWeightBits);
                    auto reach = [&](float z, int) __attribute__((always_inline)) {
                        const int b = bin_of(z);
                        const uint64_t own = unit(z, b);
                        if (static_cast<double>(own) * factor(b) >= least * (1.0 - 0x1p-43))
                            sum[b != likely_from] += own;
                    };
                    if (s.likely.count <= kSmall) {
                        if (tid < s.likely.count)
                            reach(value_of(static_cast<uint32_t>(s.likely.element[tid] >> 32)), 0);
                    } else {
                        for_kept([&](float z) __attribute__((always_inline)) {
                                     return in_span(z) &&
                                            (bin_of(z) == likely_from || bin_of(z) == likely_to);
                                 }, reach);
                    }
                    a = group_sum(sum[0]);
                    b = likely_to != likely_from ? group_sum(sum[1]) : 0;
                    top = min(top, uniform(before_likely +
                                           whole(static_cast<double>(a) * factor(likely_from)) +
                                           whole(static_cast<double>(b) * factor(likely_to))));
                }
                const uint64_t want = drawn(u, max(lo, min(hi, top)));
                bin = find<2 * BINS>(s.wide, want);
                // More than what `want` exceeds by one (rounded down: a sum of many
                // equal weights is one that doubles hold).
                target = uniform(1 + static_cast<uint64_t>(
                    __ull2double_rz(want - 1 - before(s.wide, bin)) / factor(bin)));
                if (bin == end_bin)
                    target = min(target, end_units);
                if (bin == likely_from)
                    target = min(target, a);
                else if (bin == likely_to)
                    target = min(target, b);
            }
            Few &few = border == kDraw ? s.draw : s.end;
            uint64_t e, upto = 0;
            if (border != kValue && few.count <= kSmall) {
                rank_all(few, [&](float z) __attribute__((always_inline)) {
                    return border == kLimit ? 1 : bin_of(z) == bin ? unit(z, bin) : 0;
                });
                e = find_few(few, target, upto);
            } else {
                if (border != kValue)
                    key = divide(border == kLimit, bin, target, nth, upto);
                e = element_of(key, nth_of(key, nth));
            }
            if (border == kLimit) {
                limit = e;
                fresh = true;
            } else if (border == kEnd) {
                end_bin = bin;
                end_units = upto;
                // At least what was wanted, at most the bin's amount.
                const uint64_t least = lo > before_end ? lo - before_end : 1;
                top = before_end +
                      uniform(max(least, min(whole(static_cast<double>(upto) * factor(bin)),
                                             end_amount)));
            } else {
                return index_of(e);
            }
            border = kDraw;
        }
    }
};

template <typename T, int THREADS, int BINS, int SMALL>
__global__ __launch_bounds__(THREADS, 4)
void sample_kernel(const Sample a) {
    typedef Draw<T, THREADS, BINS, SMALL> D;
    __shared__ typename D::Shared s;
    const int64_t row = a.first + blockIdx.x;
    D d{s, static_cast<const typename T::bits *>(a.logits) + row * a.ld, a.K,
        static_cast<int>(threadIdx.x)};
    const int k = uniform(a.top_ks != nullptr ? a.top_ks[row] : a.top_k);
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

// The bins, and how many labels are compared with one another, go by the number of
// labels alone: roundings differ with them, and a row's label does not depend on the
// batch.  Few bins are quick to add up, many leave few labels in one.  The threads
// change no result: many rows fill the CUs with small workgroups, of few rows each
// has a large one.  us, plain draw and top-p:
//   bins 1024, threads      256         512
//   2048 x 16384            62, 67      73, 83
//   600 x 16384             28, 31      30, 34
//   512 x 16384             24, 27      21, 24
//   16 x 16384              18, 20      15, 17
//   bins 2048, threads      512         1024
//   512 x 65536             55, 58      74, 82
//   256 x 32768             22, 24      25, 28
//   300 x 131072            95, 99      107, 116
//   256 x 131072            78, 84      71, 75
//   16 x 131072             56, 66      47, 54
// (1024 threads spill 11 to 15 registers.)
template <typename T>
hipError_t run_sample(Sample a, int64_t N, int compute_units, hipStream_t stream) {
    constexpr int64_t kMaxGrid = int64_t(1) << 21;      // a launch has less than 2^32 threads
    hipError_t e = hipSuccess;
    for (int64_t first = 0; first < N && e == hipSuccess; first += kMaxGrid) {
        a.first = first;
        const dim3 grid(static_cast<unsigned>(std::min(kMaxGrid, N - first)));
        if (a.K <= 8192)
            hipLaunchKernelGGL((sample_kernel<T, 256, 512, 256>), grid, dim3(256), 0, stream, a);
        else if (a.K <= 16384 && N > 2 * compute_units)
            hipLaunchKernelGGL((sample_kernel<T, 256, 1024, 256>), grid, dim3(256), 0, stream, a);
        else if (a.K <= 16384)
            hipLaunchKernelGGL((sample_kernel<T, 512, 1024, 256>), grid, dim3(512), 0, stream, a);
        else if (a.K <= 65536 || N > compute_units)
            hipLaunchKernelGGL((sample_kernel<T, 512, 2048, 512>), grid, dim3(512), 0, stream, a);
        else
            hipLaunchKernelGGL((sample_kernel<T, 1024, 2048, 512>), grid, dim3(1024), 0, stream, a);
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
