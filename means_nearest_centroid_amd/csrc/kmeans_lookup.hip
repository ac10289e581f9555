// kmeans_lookup.hip -- gfx950 kernels of the table lookup and of its gradient.
//
//     lookup     Y[i]  = scale * C[labels[i]]        (zero for a stray label)
//     gradient   dC[k] = scale * sum of dY[i] over labels[i] == k
//
// Both move rows and compute next to nothing: the bound is the bytes of the
// rows, read once and written once.
//
// Gradient.  Two paths, by a rule on N, K and the row's bytes.  In neither are there
// floating-point atomics: the order of every sum follows from the labels.
//
// Buckets (K up to 65536 and N up to 2^20, rows of 256 bytes or more, or 256
// buckets of at most 1024 positions on average): each tile of positions is
// sorted by bucket of up to 64 rows, as in the centroid update.
//  1. lookup_bucket_kernel: one workgroup per bucket gathers its positions,
//     sorts them by row in LDS (stably) and sums them; groups of lanes that
//     together hold one row's columns each take an equal share of the sorted
//     positions, and the sums of runs cut between groups meet in LDS.  The
//     workgroup owns its rows, so it zeroes those without a position too.
//  2. A bucket of more positions than one workgroup should sum (a frequent
//     label) is put on a list instead, in parts of `cap` positions.
//     lookup_part_kernel does the same for each part, leaving partial sums,
//     and lookup_part_join_kernel adds them in order: work per workgroup is
//     bounded whatever the frequencies.  Both end at once when the list is
//     empty (about 2 us each).  Workgroups of the first launch taking parts
//     themselves once done with their buckets, without further launches, was
//     700 us instead of 160 at 16384 x 4096 of 32768 tokens: the fences that
//     hand partial sums from one XCD to another inside a launch empty its L2.
// 262144 x 128 of 4096 rows: 25.5 us a call (16 of them lookup_bucket_kernel,
// 5 the binning; 68 MB); by the sort 61.  16384 x 4096 of 32768 tokens: 124 us
// (81 lookup_bucket_kernel, 26 + 9 the parts; 403 MB, 3.2 TB/s), by the sort
// 213.  What is above the bytes is the chain from directory to slots to rows,
// which a workgroup walks before its first row arrives; deeper batches of rows,
// smaller parts or stores past the caches change nothing.
//
// Sort (every other shape): the positions are sorted by label (the stable
// radix sort of the centroid update), so that a label's rows are one run of
// sorted positions.
//  1. lookup_sum_kernel walks fixed chunks of sorted positions; a group of
//     lanes owns one chunk and sums each run in position order.  A run inside
//     the chunk is finished there (one rounding); a run cut by a chunk edge
//     leaves its partial sum.  Further workgroups of the same launch zero the
//     rows that no label names.
//  2. lookup_join_kernel adds the partial sums of the runs that were cut, in
//     an order fixed by the chunks.
#include <stdint.h>

#include <algorithm>
#include <optional>

#include "kmeans_types.h"
#include "kmeans_update_internal.h"

namespace kmeans {
namespace {

constexpr int kRowThreads = 256;
// Workgroups across a grid: a launch takes less than 2^32 threads that way.
// More go to a second dimension (lookup) or are walked (zeroed rows).
constexpr int64_t kMaxGridX = int64_t(1) << 20;

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
// whose loads are in flight together; the rows are written past the caches
// (non-temporal), which leaves the table there.  262144 rows of 128 bf16 from
// a table of 4096: 11.8 us a call (5.9 TB/s); 14.0 with four pieces, 17.8 with
// eight, 15.4 with plain stores; 16384 rows of 4096 fp32 85 us instead of 98.
constexpr int kUnroll = 2;
template <typename T, int V, typename L>
__global__ __launch_bounds__(kRowThreads)
void lookup_kernel(const typename T::bits *__restrict__ C, int64_t ldc, const L *__restrict__ labels,
                   int64_t N, int D, int K, float scale, int pieces, uint32_t inv,
                   typename T::bits *__restrict__ Y, int64_t ldy) {
    typedef typename T::bits B;
    const int64_t wg = static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x;
    const int64_t first = wg * (kUnroll * kRowThreads);
    const int64_t row0 = first / pieces;
    const uint32_t rem0 = static_cast<uint32_t>(first - row0 * pieces);
    int64_t row[kUnroll];
    int col[kUnroll], from[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const uint32_t x = rem0 + u * kRowThreads + threadIdx.x;
        // x / pieces for x < pieces + 512: inv = ceil(2^32 / pieces), one
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
                __builtin_nontemporal_store(
                    __builtin_bit_cast(u32x4_any, narrow_run<T, V>(x)),
                    reinterpret_cast<u32x4_any *>(Y + row[u] * ldy + col[u]));
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

// The V columns that a lane holds in column slab `slab`.  The last lane of a
// row of D >= V columns that are no multiple of V starts at D - V, so that
// every load is a whole one; it shares its first `skip` columns with the lane
// before it and leaves them to that lane.  (D < V: V = 1.)
template <int V>
struct Columns {
    int first, skip;
    bool any;
    __device__ __forceinline__ Columns(int slab, int lanes, int l, int D) {
        const int c = (slab * lanes + l) * V;
        any = c < D;
        first = min(c, max(D - V, 0));
        skip = c - first;
    }
};

// A lane's columns of a row of dC (o), without the first `skip`.
template <typename O, int V>
__device__ __forceinline__ void store_columns(typename O::bits *o, int skip,
                                              const Packed<typename O::bits, V> &v) {
    if (skip == 0) {
        store_packed(o, v);
        return;
    }
#pragma unroll
    for (int e = 1; e < V; ++e)
        if (e >= skip)
            o[e] = v.v[e];
}

// A lane's columns of row k from the sums: scaled, added to the row where
// asked, rounded once.
template <typename O, int V>
__device__ __forceinline__ void finish_row(const GradArgs &g, int k, const Columns<V> &c,
                                           const float (&sum)[V]) {
    typedef typename O::bits B;
    B *o = static_cast<B *>(g.dC) + k * g.ldc + c.first;
    float v[V];
    if (g.accumulate) {
        const Packed<B, V> old = load_packed<B, V>(o);
#pragma unroll
        for (int e = 0; e < V; ++e)
            v[e] = fmaf(g.scale, sum[e], O::widen(old.v[e]));
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
            v[e] = g.scale * sum[e];
    }
    store_columns<O, V>(o, c.skip, narrow_run<O, V>(v));
}

// The same columns of a row that no label names.
template <typename O, int V>
__device__ __forceinline__ void zero_row(const GradArgs &g, int k, const Columns<V> &c) {
    if (!g.accumulate)
        store_columns<O, V>(static_cast<typename O::bits *>(g.dC) + k * g.ldc + c.first, c.skip,
                            Packed<typename O::bits, V>{});
}

// Partial sums are written whole: lanes that share columns hold the same sums.
template <int V>
__device__ __forceinline__ void store_partial(float *p, const float (&sum)[V]) {
    store_packed(p, narrow_run<Fp32, V>(sum));
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
        // Zero the rows that no label names: kFillRows at a time, this slab.
        __shared__ uint8_t named[kFillRows];
        const Columns<V> cols(blockIdx.y, lanes, l, g.D);
        const int64_t step = static_cast<int64_t>(gridDim.x - sum_wgs) * kFillRows;
        for (int64_t first = static_cast<int64_t>(blockIdx.x - sum_wgs) * kFillRows; first < g.K;
             first += step) {
            const int r0 = static_cast<int>(first), rows = min(kFillRows, g.K - r0);
            __syncthreads();
            if (tid < rows) {
                const int p = bound_of(g.keys, 0, g.N, r0 + tid, false);
                named[tid] = p < g.N && g.keys[p] == r0 + tid;
            }
            __syncthreads();
            if (cols.any)
                for (int r = tid >> g.lanes_log2; r < rows; r += kRowThreads >> g.lanes_log2)
                    if (!named[r])
                        zero_row<O, V>(g, r0 + r, cols);
        }
        return;
    }
    const int c = blockIdx.x * (kRowThreads >> g.lanes_log2) + (tid >> g.lanes_log2);
    const Columns<V> cols(blockIdx.y, lanes, l, g.D);
    if (c >= g.chunks || !cols.any)
        return;
    const int beg = c * g.chunk;
    const int end = static_cast<int>(min(static_cast<int64_t>(g.N),
                                         static_cast<int64_t>(beg) + g.chunk));
    const B *src = static_cast<const B *>(g.dY) + cols.first;
    float *part = g.partial + static_cast<int64_t>(c) * 2 * g.D + cols.first;
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
            row[u] = load_packed<B, V>(src + g.vals[p] * g.ldy);
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (key[u] < 0)
                continue;
            if (key[u] != cur) {
                if (cur < g.K) {
                    if (open_left)
                        store_partial<V>(part, sum);
                    else
                        finish_row<O, V>(g, cur, cols, sum);
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
        store_partial<V>(part, sum);
    else if (open_right)
        store_partial<V>(part + g.D, sum);
    else
        finish_row<O, V>(g, cur, cols, sum);
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
    const Columns<V> cols(blockIdx.y, lanes, l, g.D);
    for (int x = q; x < kJoinChunks; x += groups) {
        const int m = more[x];
        if (m == 0 || m >= kLongRun || !cols.any)
            continue;
        const float *p = g.partial + static_cast<int64_t>(first + x) * 2 * g.D + cols.first;
        const Packed<float, V> head = load_packed<float, V>(p + g.D);
        float sum[V];
#pragma unroll
        for (int e = 0; e < V; ++e)
            sum[e] = head.v[e];
        for (int s0 = 1; s0 <= m; s0 += 4) {
            Packed<float, V> w[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                w[u] = load_packed<float, V>(p + static_cast<int64_t>(min(s0 + u, m)) * 2 * g.D);
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int e = 0; e < V; ++e)
                    sum[e] += s0 + u <= m ? w[u].v[e] : 0.0f;
        }
        finish_row<O, V>(g, key_of[x], cols, sum);
    }
    for (int x = 0; x < kJoinChunks; ++x) {
        const int m = more[x];
        if (m < kLongRun)
            continue;
        const float *p = g.partial + static_cast<int64_t>(first + x) * 2 * g.D + cols.first;
        float sum[V] = {};
        if (cols.any)
            for (int s0 = q; s0 <= m; s0 += kBatch * groups) {
                Packed<float, V> w[kBatch];
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const int s = min(s0 + u * groups, m);
                    w[u] = load_packed<float, V>(
                        s == 0 ? p + g.D : p + static_cast<int64_t>(s) * 2 * g.D);
                }
#pragma unroll
                for (int u = 0; u < kBatch; ++u)
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        sum[e] += s0 + u * groups <= m ? w[u].v[e] : 0.0f;
            }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < V; ++e)
            sums[tid][e] = sum[e];
        __syncthreads();
        if (q == 0 && cols.any) {
            for (int r = 1; r < groups; ++r)
#pragma unroll
                for (int e = 0; e < V; ++e)
                    sum[e] += sums[r * lanes + l][e];
            finish_row<O, V>(g, key_of[x], cols, sum);
        }
    }
}

// ---- gradient by buckets ---------------------------------------------------

constexpr int kBucketCap = 2048;       // most positions one workgroup sorts and sums
constexpr int kMaxBucketRows = 64;
constexpr int kMaxTiles = 512;         // of positions (make_label_bins)
constexpr int kWaves = kRowThreads / 64;

// One bucket of more than `cap` positions.
struct Heavy {
    int bucket, first_part, parts;
};

struct BucketArgs {
    const int32_t *sidx, *dir;   // slot words and directory (launch_label_bins)
    int bucket_log2, buckets, tile_log2, tiles;
    int cap;                     // positions of a part; from more on a bucket is heavy
    int col_groups_log2;         // groups of lanes side by side on columns (the others
                                 // divide the positions)
    int *counts;                 // heavy buckets, parts
    Heavy *heavy;
    int *run_len;                // [parts][S]: positions of each row in the part
    float *partial;              // [parts][S][D]
};

struct BucketShared {
    int words[kBucketCap], sorted[kBucketCap];
    int off[kMaxTiles + 1], src[kMaxTiles];
    int cnt[kWaves][kMaxBucketRows], start[kMaxBucketRows + 1];
    int wave_total[kWaves];
    int found;                   // by one thread, for all
    float edge[2][kRowThreads * 8];
};

// Positions (slots, in tile order) of bucket b: their first slots per tile in
// sh.off, where each tile's lie in sidx in sh.src; returns their number.
__device__ __forceinline__ int find_segments(const BucketArgs &bk, int b, BucketShared &sh) {
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const size_t row = bk.buckets + 1;
    int len[2] = {0, 0}, base[2] = {0, 0};
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int t = min(2 * tid + u, bk.tiles - 1);
        const int32_t *d = bk.dir + t * row + b;
        const int lo = d[0], hi = d[1];
        len[u] = 2 * tid + u < bk.tiles ? hi - lo : 0;
        base[u] = (t << bk.tile_log2) + lo;
    }
    const int x = wave_inclusive_sum(len[0] + len[1]);
    if (lane == 63)
        sh.wave_total[w] = x;
    __syncthreads();
    int ex = x - len[0] - len[1], total = 0;
#pragma unroll
    for (int v = 0; v < kWaves; ++v) {
        ex += v < w ? sh.wave_total[v] : 0;
        total += sh.wave_total[v];
    }
    if (2 * tid < bk.tiles) {
        sh.off[2 * tid] = ex;
        sh.src[2 * tid] = base[0];
    }
    if (2 * tid + 1 < bk.tiles) {
        sh.off[2 * tid + 1] = ex + len[0];
        sh.src[2 * tid + 1] = base[1];
    }
    __syncthreads();
    return total;
}

// Slot words of slots [s0, s0 + n) into sh.words (n <= kBucketCap): each slot
// finds its tile by binary search.  Most buckets need one slot a thread; the
// loads of larger ones overlap four at a time.
__device__ __forceinline__ void gather_words(const BucketArgs &bk, int s0, int n,
                                             BucketShared &sh) {
    constexpr int kPer = 4;
    for (int p0 = threadIdx.x; p0 < n; p0 += kPer * kRowThreads) {
        int v[kPer];
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const int p = p0 + u * kRowThreads;
            if (p >= n)
                break;
            int lo = 0, hi = bk.tiles - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (sh.off[mid] <= s0 + p)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            v[u] = bk.sidx[sh.src[lo] + (s0 + p - sh.off[lo])];
        }
#pragma unroll
        for (int u = 0; u < kPer; ++u)
            if (p0 + u * kRowThreads < n)
                sh.words[p0 + u * kRowThreads] = v[u];
    }
}

__device__ __forceinline__ int row_of(int word) {
    return static_cast<int>(static_cast<uint32_t>(word) >> kSlotIdxBits);
}

// Stable sort of sh.words[0, n) by row in the bucket into sh.sorted, and the
// first position of each row in sh.start[0 .. S].  Each wave owns a quarter;
// lanes of equal row are found by one ballot per row bit.
__device__ __forceinline__ void sort_by_row(int n, int s_log2, BucketShared &sh) {
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int S = 1 << s_log2;
    const int quarter = (n + kRowThreads - 1) / kRowThreads * 64;
    const int beg = min(n, w * quarter), end = min(n, beg + quarter);
    for (int x = tid; x < kWaves * kMaxBucketRows; x += kRowThreads)
        sh.cnt[x / kMaxBucketRows][x % kMaxBucketRows] = 0;
    __syncthreads();
    for (int i = beg + lane; i < end; i += 64)
        atomicAdd(&sh.cnt[w][row_of(sh.words[i])], 1);
    __syncthreads();
    if (w == 0) {
        int c[kWaves], sum = 0;
#pragma unroll
        for (int v = 0; v < kWaves; ++v) {
            c[v] = sh.cnt[v][lane];
            sum += c[v];
        }
        int run = wave_inclusive_sum(sum) - sum;
        if (lane < S)
            sh.start[lane] = run;
        if (lane == 0)
            sh.start[S] = n;
#pragma unroll
        for (int v = 0; v < kWaves; ++v) {
            sh.cnt[v][lane] = run;
            run += c[v];
        }
    }
    __syncthreads();
    const uint64_t below = (uint64_t(1) << lane) - 1;
    for (int i0 = beg; i0 < end; i0 += 64) {
        const bool in = i0 + lane < end;
        const int word = in ? sh.words[i0 + lane] : 0;
        const int r = row_of(word);
        uint64_t same = __ballot(in);
        for (int b = 0; b < s_log2; ++b) {
            const bool bit = (r >> b) & 1;
            const uint64_t m = __ballot(in && bit);
            same &= bit ? m : ~m;
        }
        if (in) {
            const int at = sh.cnt[w][r] + __popcll(same & below);
            if ((same >> lane) == 1)     // the last lane of its row
                sh.cnt[w][r] = at + 1;
            sh.sorted[at] = word;
        }
    }
    __syncthreads();
}

// A thread's place: its lane in a group, the group's share of the positions
// (qp of gp) and its columns.
template <int V>
struct Place {
    int l, qp, gp;
    Columns<V> cols;
    __device__ __forceinline__ Place(const GradArgs &g, const BucketArgs &bk)
        : l(threadIdx.x & ((1 << g.lanes_log2) - 1)),
          qp(threadIdx.x >> (g.lanes_log2 + bk.col_groups_log2)),
          gp(kRowThreads >> (g.lanes_log2 + bk.col_groups_log2)),
          cols((blockIdx.y << bk.col_groups_log2) +
                   ((threadIdx.x >> g.lanes_log2) & ((1 << bk.col_groups_log2) - 1)),
               1 << g.lanes_log2, l, g.D) {}
};

// Sums sh.sorted[0, n) (rows of bucket b) over this workgroup's columns.  PART:
// into the partial sums of part `part`; else into dC, rows without a position
// zeroed.  Ends with a barrier.
template <typename T, typename O, int V, bool PART>
__device__ __forceinline__ void sum_sorted(const GradArgs &g, const BucketArgs &bk,
                                           const Place<V> &at, int b, int part, int n,
                                           BucketShared &sh) {
    typedef typename T::bits B;
    const int S = 1 << bk.bucket_log2;
    const int lo = n * at.qp / at.gp, hi = n * (at.qp + 1) / at.gp;
    const bool any = at.cols.any;
    auto edge = [&](int side, int thread) __attribute__((always_inline)) {
        return sh.edge[side] + thread * V;
    };
    auto put = [&](int r, const float (&sum)[V]) __attribute__((always_inline)) {
        if (PART)
            store_partial<V>(
                bk.partial + (static_cast<int64_t>(part) * S + r) * g.D + at.cols.first, sum);
        else
            finish_row<O, V>(g, (b << bk.bucket_log2) + r, at.cols, sum);
    };
    // The zeros need no positions: their stores go first and drain meanwhile.
    if (!PART && any)
        for (int r = at.qp; r < S; r += at.gp)
            if (sh.start[r] == sh.start[r + 1] && (b << bk.bucket_log2) + r < g.K)
                zero_row<O, V>(g, (b << bk.bucket_log2) + r, at.cols);
    if (any && lo < hi) {
        const B *src = static_cast<const B *>(g.dY) + at.cols.first;
        int row = row_of(sh.sorted[lo]), first = lo;
        float sum[V] = {};
        // The run [first, end) of `row` is over: finished if it is the whole
        // row, else an edge (0: it began in an earlier group).
        auto close = [&](int end) __attribute__((always_inline)) {
            if (first == sh.start[row] && end == sh.start[row + 1]) {
                put(row, sum);
            } else {
                float *e = edge(first == sh.start[row] ? 1 : 0, threadIdx.x);
#pragma unroll
                for (int x = 0; x < V; ++x)
                    e[x] = sum[x];
            }
        };
        int word[kBatch];
        Packed<B, V> val[kBatch];
        for (int p0 = lo; p0 < hi; p0 += kBatch) {
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                word[u] = sh.sorted[min(p0 + u, hi - 1)];
                const int64_t i = word[u] & ((1 << kSlotIdxBits) - 1);
                val[u] = load_packed<B, V>(src + i * g.ldy);
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                if (p0 + u >= hi)
                    break;
                const int r = row_of(word[u]);
                if (r != row) {
                    close(p0 + u);
                    row = r;
                    first = p0 + u;
#pragma unroll
                    for (int x = 0; x < V; ++x)
                        sum[x] = 0.0f;
                }
#pragma unroll
                for (int x = 0; x < V; ++x)
                    sum[x] += T::widen(val[u].v[x]);
            }
        }
        close(hi);
    }
    __syncthreads();
    // The group in which a cut run began adds its pieces, in order.
    if (any && lo < hi) {
        const int r = row_of(sh.sorted[hi - 1]);
        const int end = sh.start[r + 1];
        if (sh.start[r] >= lo && end > hi) {
            float sum[V];
#pragma unroll
            for (int x = 0; x < V; ++x)
                sum[x] = edge(1, threadIdx.x)[x];
            for (int o = at.qp + 1; o < at.gp && n * o / at.gp < end; ++o) {
                if (n * o / at.gp == n * (o + 1) / at.gp)
                    continue;
                const float *e =
                    edge(0, threadIdx.x + ((o - at.qp) << (g.lanes_log2 + bk.col_groups_log2)));
#pragma unroll
                for (int x = 0; x < V; ++x)
                    sum[x] += e[x];
            }
            put(r, sum);
        }
    }
    __syncthreads();
}

template <typename T, typename O, int V>
__global__ __launch_bounds__(kRowThreads, 4)
void lookup_bucket_kernel(const GradArgs g, const BucketArgs bk) {
    __shared__ BucketShared sh;
    // Each XCD takes a contiguous range of buckets: its directory entries and
    // slot words are neighbours in memory.
    const int b = xcd_contiguous(blockIdx.x, bk.buckets);
    const int n = find_segments(bk, b, sh);
    if (n > bk.cap) {
        if (blockIdx.y == 0 && threadIdx.x == 0) {
            const int parts = (n + bk.cap - 1) / bk.cap;
            bk.heavy[atomicAdd(&bk.counts[0], 1)] = {b, atomicAdd(&bk.counts[1], parts), parts};
        }
        return;
    }
    if (n > 0)
        gather_words(bk, 0, n, sh);
    __syncthreads();
    sort_by_row(n, bk.bucket_log2, sh);
    sum_sorted<T, O, V, false>(g, bk, Place<V>(g, bk), b, 0, n, sh);
}

template <typename T, typename O, int V>
__global__ __launch_bounds__(kRowThreads, 4)
void lookup_part_kernel(const GradArgs g, const BucketArgs bk) {
    __shared__ BucketShared sh;
    const int entries = bk.counts[0], parts = bk.counts[1];
    const int S = 1 << bk.bucket_log2;
    for (int t = blockIdx.x; t < parts; t += gridDim.x) {
        for (int e = threadIdx.x; e < entries; e += kRowThreads)
            if (t >= bk.heavy[e].first_part && t < bk.heavy[e].first_part + bk.heavy[e].parts)
                sh.found = e;                // exactly one
        __syncthreads();
        const Heavy h = bk.heavy[sh.found];
        const int s0 = (t - h.first_part) * bk.cap;
        const int n = min(find_segments(bk, h.bucket, sh) - s0, bk.cap);
        gather_words(bk, s0, n, sh);
        __syncthreads();
        sort_by_row(n, bk.bucket_log2, sh);
        if (blockIdx.y == 0 && static_cast<int>(threadIdx.x) < S)
            bk.run_len[t * S + threadIdx.x] = sh.start[threadIdx.x + 1] - sh.start[threadIdx.x];
        sum_sorted<T, O, V, true>(g, bk, Place<V>(g, bk), h.bucket, t, n, sh);
    }
}

// Rows of heavy buckets, one workgroup a row at a time: its groups of lanes
// take every groups-th part, and their sums are added in group order.
template <typename O, int V>
__global__ __launch_bounds__(kRowThreads)
void lookup_part_join_kernel(const GradArgs g, const BucketArgs bk) {
    __shared__ float sums[kRowThreads][V + 1];
    __shared__ int total[kRowThreads];
    const int S = 1 << bk.bucket_log2;
    const int items = bk.counts[0] << bk.bucket_log2;
    const Place<V> at(g, bk);
    for (int x = blockIdx.x; x < items; x += gridDim.x) {
        const Heavy h = bk.heavy[x >> bk.bucket_log2];
        const int r = x & (S - 1), k = (h.bucket << bk.bucket_log2) + r;
        float sum[V] = {};
        int positions = 0;
        for (int t0 = at.qp; t0 < h.parts; t0 += kBatch * at.gp) {
            int len[kBatch];
            Packed<float, V> v[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const bool in = t0 + u * at.gp < h.parts;
                len[u] = in ? bk.run_len[(h.first_part + t0 + u * at.gp) * S + r] : 0;
                v[u] = Packed<float, V>{};
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u)     // else nothing was written there
                if (len[u] > 0 && at.cols.any)
                    v[u] = load_packed<float, V>(
                        bk.partial + (static_cast<int64_t>(h.first_part + t0 + u * at.gp) * S + r) * g.D +
                        at.cols.first);
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                positions += len[u];
#pragma unroll
                for (int e = 0; e < V; ++e)
                    sum[e] += v[u].v[e];
            }
        }
#pragma unroll
        for (int e = 0; e < V; ++e)
            sums[threadIdx.x][e] = sum[e];
        total[threadIdx.x] = positions;
        __syncthreads();
        if (at.qp == 0 && at.cols.any && k < g.K) {
            for (int o = 1; o < at.gp; ++o) {
                const int other = threadIdx.x + (o << g.lanes_log2);
                positions += total[other];
#pragma unroll
                for (int e = 0; e < V; ++e)
                    sum[e] += sums[other][e];
            }
            if (positions > 0)
                finish_row<O, V>(g, k, at.cols, sum);
            else
                zero_row<O, V>(g, k, at.cols);
        }
        __syncthreads();
    }
}

// ---- launch ----------------------------------------------------------------

struct GradPlan {
    int lanes_log2, slabs;
    bool by_buckets;
    // buckets
    LabelBins bins;
    int cap, col_groups_log2, column_groups;
    int max_parts;
    size_t counts, heavy, run_len;
    // sort
    LabelSort sort;
    int chunk, chunks;
    size_t partial, bytes;
};

size_t align_up(size_t n) { return (n + 255) & ~size_t(255); }

// Buckets pay where a row is wide enough to hide the gathering of its position
// (256 bytes: 262144 x 1024 of 16 rows 129 us, sorted 210; 65536 x 128 of 255
// 20 and 30; 4096 x 128 of 128 16 and 19), or where most of them are summed by
// one workgroup and there are enough to fill the GPU (262144 x 32 of 250 rows
// 69 us, sorted 37; 1000000 x 16 of 300 135 and 108).
constexpr int64_t kWideRow = 256;                       // bytes
constexpr int64_t kMinBucketRows = 256;
constexpr int64_t kMaxMeanBucket = 1024;                // positions
constexpr int64_t kMaxBucketTable = int64_t(1024) * kMaxBucketRows;
constexpr int64_t kMaxBucketPositions = int64_t(1) << 20;
constexpr int64_t kMinCap = 128;

GradPlan make_grad_plan(int64_t N, int64_t D, int64_t K, int V, int compute_units) {
    GradPlan p{};
    while (p.lanes_log2 < 6 && (int64_t(V) << p.lanes_log2) < D)
        ++p.lanes_log2;
    const int64_t slab = int64_t(V) << p.lanes_log2;    // columns of one group of lanes
    p.slabs = static_cast<int>((D + slab - 1) / slab);
    if (N == 0)
        return p;
    if (K <= kMaxBucketTable && N <= kMaxBucketPositions) {
        p.bins = make_label_bins(N, K);
        p.by_buckets = D * (V == 8 ? 2 : 4) >= kWideRow ||
                       (K >= kMinBucketRows && N <= kMaxMeanBucket * p.bins.buckets);
    }
    if (p.by_buckets) {
        // Few positions per bucket and wide rows: the groups of a workgroup
        // take columns side by side, so that none waits for the others and
        // the gathering serves them all.  Else they divide the positions.
        if (N <= 64 * static_cast<int64_t>(p.bins.buckets))
            while ((1 << (p.lanes_log2 + p.col_groups_log2)) < kRowThreads &&
                   (1 << p.col_groups_log2) < p.slabs)
                ++p.col_groups_log2;
        p.column_groups = (p.slabs + (1 << p.col_groups_log2) - 1) >> p.col_groups_log2;
        // A part is 512 positions of 256 bytes, fewer for wider slabs, and
        // at least twice the mean bucket if there is one for every CU; larger
        // where the partial sums would take more than 256 MiB.  A heavy bucket
        // has more than `cap` positions, so its parts hold half of that each
        // on average at least.
        const int64_t bytes = std::min(D, slab) * (V == 8 ? 2 : 4);
        int64_t cap = (int64_t(1) << 25) / (bytes * bytes);
        if (p.bins.buckets >= compute_units)
            cap = std::max<int64_t>(cap, 2 * N / p.bins.buckets);
        cap = std::min<int64_t>(std::max(cap, kMinCap), kBucketCap);
        auto rows = [&] { return static_cast<size_t>(2 * N / cap + 1) << p.bins.bucket_log2; };
        while (cap < kBucketCap && rows() * D * sizeof(float) > (size_t(256) << 20))
            cap = std::min<int64_t>(2 * cap, kBucketCap);
        p.cap = static_cast<int>(cap);
        p.max_parts = static_cast<int>(2 * N / cap + 1);
        p.counts = align_up(p.bins.bytes);
        p.heavy = p.counts + 256;
        p.run_len = p.heavy + align_up((N / cap + 1) * sizeof(Heavy));
        p.partial = p.run_len + align_up(rows() * sizeof(int));
        p.bytes = p.partial + rows() * D * sizeof(float);
        return p;
    }
    // Chunks of at least 8 positions, more when that leaves eight waves or
    // more per CU (four: 3% slower at 200000 x 64 of 100 rows; two: 38%).
    const int64_t waves_at_1 = ((N << p.lanes_log2) + 63) / 64 * p.slabs;
    int64_t chunk = 8;
    while (chunk < 4096 && waves_at_1 / (2 * chunk) >= 8 * compute_units)
        chunk *= 2;
    p.chunk = static_cast<int>(chunk);
    p.chunks = static_cast<int>((N + chunk - 1) / chunk);
    p.sort = make_label_sort(N, K);
    p.partial = align_up(p.sort.bytes);
    p.bytes = p.partial + static_cast<size_t>(p.chunks) * 2 * D * sizeof(float);
    return p;
}

template <typename T, typename O, int V>
hipError_t launch_grad(const GradPlan &p, const GradArgs &g, const BucketArgs &bk,
                       int compute_units, hipStream_t stream) {
    if (p.by_buckets) {
        hipLaunchKernelGGL((lookup_bucket_kernel<T, O, V>),
                           dim3(p.bins.buckets, p.column_groups), dim3(kRowThreads), 0, stream, g,
                           bk);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess || g.N <= p.cap)            // no bucket can be heavy
            return e;
        BucketArgs pk = bk;
        pk.col_groups_log2 = 0;
        hipLaunchKernelGGL((lookup_part_kernel<T, O, V>),
                           dim3(std::min(p.max_parts, 2 * compute_units), p.slabs),
                           dim3(kRowThreads), 0, stream, g, pk);
        if ((e = hipGetLastError()) != hipSuccess)
            return e;
        hipLaunchKernelGGL((lookup_part_join_kernel<O, V>), dim3(compute_units, p.slabs),
                           dim3(kRowThreads), 0, stream, g, pk);
        return hipGetLastError();
    }
    const int per_wg = kRowThreads >> p.lanes_log2;
    const int sum_wgs = (p.chunks + per_wg - 1) / per_wg;
    const int fill_wgs =
        g.accumulate ? 0 : static_cast<int>(std::min<int64_t>((int64_t(g.K) + kFillRows - 1) / kFillRows,
                                                              kMaxGridX));
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
    const int64_t across = std::min(wgs, kMaxGridX);
    const dim3 grid(static_cast<unsigned>(across),
                    static_cast<unsigned>((wgs + across - 1) / across));
    hipLaunchKernelGGL((lookup_kernel<T, V, L>), grid, dim3(kRowThreads), 0, stream,
                       static_cast<const B *>(C), ldc, static_cast<const L *>(labels), N,
                       static_cast<int>(D), static_cast<int>(K), scale, static_cast<int>(pieces),
                       inv, static_cast<B *>(Y), ldy);
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
    // 16 bytes of a row per lane, single values where a row is shorter.
    const int V = D * static_cast<int64_t>(dtype_size(dtype)) >= 16
                      ? 16 / static_cast<int>(dtype_size(dtype)) : 1;
    const int cus = device_compute_units();
    const GradPlan p = make_grad_plan(N, D, K, V, cus);
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
    BucketArgs bk{};
    std::optional<WorkspaceLease> lease;
    hipError_t e = hipSuccess;
    if (N > 0) {
        lease.emplace(stream, p.bytes);
        if (lease->error() != hipSuccess)
            return fail(KMEANS_ERR_NO_MEMORY, "workspace of %zu bytes: %s", p.bytes,
                        hipGetErrorString(lease->error()));
        auto *ws = static_cast<char *>(lease->ptr());
        auto ints = [&](size_t at) { return reinterpret_cast<int *>(ws + at); };
        g.partial = reinterpret_cast<float *>(ws + p.partial);
        if (p.by_buckets) {
            bk = {ints(p.bins.sidx), ints(p.bins.dir), p.bins.bucket_log2, p.bins.buckets,
                  p.bins.tile_log2, p.bins.tiles, p.cap, p.col_groups_log2, ints(p.counts),
                  reinterpret_cast<Heavy *>(ws + p.heavy), ints(p.run_len), g.partial};
            e = launch_label_bins(p.bins, labels, label_type, g.N, g.K, ws, bk.counts, 2, stream);
        } else {
            e = launch_label_sort(p.sort, labels, label_type, g.N, g.K, ws, &g.keys, &g.vals,
                                  stream);
        }
    }
    if (e == hipSuccess) {
        auto launch = [&](auto type, auto out) {
            using T = decltype(type);
            using O = decltype(out);
            constexpr int kWide = 16 / sizeof(typename T::bits);
            return V == 1 ? launch_grad<T, O, 1>(p, g, bk, cus, stream)
                          : launch_grad<T, O, kWide>(p, g, bk, cus, stream);
        };
        if (dtype == KMEANS_BF16)
            e = out_dtype == dtype ? launch(Bf16{}, Bf16{}) : launch(Bf16{}, Fp32{});
        else if (dtype == KMEANS_FP16)
            e = out_dtype == dtype ? launch(Fp16{}, Fp16{}) : launch(Fp16{}, Fp32{});
        else
            e = launch(Fp32{}, Fp32{});
    }
    if (e != hipSuccess)
        return fail(KMEANS_ERR_HIP, "lookup gradient launch failed: %s", hipGetErrorString(e));
    return ok();
}
