// kmeans_update_internal.h -- launch plan of the centroid update (the step
// after assignment in a Lloyd iteration).  Not part of the public interface.
#pragma once

#include "kmeans_internal.h"

namespace kmeans {

// Workspace layout and launch shape of one stable radix sort of N labels in
// [0, K), stray ones last (the update's sort path, the lookup's gradient).
struct LabelSort {
    int passes;        // radix passes over the keys 0..K (K = stray label)
    int digit_bits;    // bits per pass (<= 8): the key bits split evenly
    int tile_log2;     // sort tile of 2^tile_log2 points (>= 1024)
    int tiles;         // sort tiles
    int stride;        // histogram row length: tiles rounded up to 4
    size_t keys[2], vals[2];   // byte offsets of the ping-pong sort buffers
    size_t hist;       // [passes][256][stride] int32
    size_t bytes;      // total workspace
};

// Requires 1 <= N < 2^31, 1 <= K < 2^31.
LabelSort make_label_sort(int64_t N, int64_t K);

// The sort's launches on `stream`, scratch of sort.bytes at ws; labels are
// int32 or int64 (kmeans_label_t).  *keys receives the sorted keys (the
// label, or K for one outside [0, K)) and *vals their positions, both in ws.
hipError_t launch_label_sort(const LabelSort &sort, const void *labels, int32_t label_type, int N,
                             int K, void *ws, const int32_t **keys, const int32_t **vals,
                             hipStream_t stream);

// Labels grouped into at most 1024 buckets of 2^bucket_log2 clusters: each tile
// of 2^tile_log2 points is sorted by bucket, stably, into slot words (the point
// index, its cluster in the bucket above bit kSlotIdxBits) at sidx, and its
// directory row holds the first slot of each bucket and, last, the number of
// points with a label in [0, K): dir[tile][buckets + 1].  Offsets are relative
// to the workspace.
struct LabelBins {
    int bucket_log2, buckets, tile_log2, tiles;
    size_t sidx, dir, bytes;
};
constexpr int kSlotIdxBits = 24;

// At most 2^24 points, 512 tiles, and buckets of at most 128 clusters
// (K <= 2^17).
LabelBins make_label_bins(int64_t N, int64_t K);

// The one launch; it also zeroes n_clear entries of clear.
hipError_t launch_label_bins(const LabelBins &bins, const void *labels, int32_t label_type, int N,
                             int K, void *ws, int32_t *clear, int n_clear, hipStream_t stream);

// A label as int32 (one outside its range as -1, a stray label too).
__device__ __forceinline__ int32_t label32(int32_t label) { return label; }
__device__ __forceinline__ int32_t label32(int64_t label) {
    return label < 0 || label > INT32_MAX ? -1 : static_cast<int32_t>(label);
}

// Inclusive prefix sum over the 64 lanes of a wave by DPP: shifts right by
// 1, 2, 4 and 8 lanes within each row of 16 (lanes shifted in from outside
// the row read 0), then each row adds the last lane of the rows before it
// (row_bcast:15 into rows 1 and 3, row_bcast:31 into rows 2 and 3).
__device__ __forceinline__ int wave_inclusive_sum(int x) {
    constexpr int kRowShr = 0x110, kRowBcast15 = 0x142, kRowBcast31 = 0x143;
    x += __builtin_amdgcn_update_dpp(0, x, kRowShr + 1, 0xf, 0xf, true);
    x += __builtin_amdgcn_update_dpp(0, x, kRowShr + 2, 0xf, 0xf, true);
    x += __builtin_amdgcn_update_dpp(0, x, kRowShr + 4, 0xf, 0xf, true);
    x += __builtin_amdgcn_update_dpp(0, x, kRowShr + 8, 0xf, 0xf, true);
    x += __builtin_amdgcn_update_dpp(0, x, kRowBcast15, 0xa, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, kRowBcast31, 0xc, 0xf, false);
    return x;
}

// Workgroups are dispatched to the eight XCDs in turn (workgroup i to XCD
// i mod 8), and each XCD has its own L2.  Mapping workgroup i to item
// start(x) + i / 8 (x = i mod 8, XCD x owning the contiguous items
// [start(x), start(x + 1))) gives each XCD a contiguous range of buckets, so
// the directory lines and sorted-index lines it reads are its own eighth of
// them instead of lines shared with every other XCD.  A bijection on
// [0, n) for any n.
__device__ __forceinline__ int xcd_contiguous(int i, int n) {
    constexpr int kXcds = 8;
    const int x = i % kXcds;
    const int q = n / kXcds;
    const int r = n % kXcds;
    return x * q + min(x, r) + i / kXcds;
}

// Workspace layout and launch shape of one kmeans_update call.
struct UpdatePlan {
    int path;          // 1: radix sort + chunked reduce + finish; 2: buckets
    // path 2 (bucket_path_fits): buckets of 2^bucket_log2 clusters, sort
    // tiles of 2^bin_tile_log2 points, workspace offsets of the sorted slot
    // words (point index, cluster in bucket) and the [bin_tiles][buckets + 1]
    // tile directory.
    int bucket_log2, buckets, bin_tile_log2, bin_tiles;
    size_t sidx, dir;
    // path 1
    LabelSort sort;    // its workspace comes first
    int chunk;         // sorted positions per reduce chunk (32 KiB of rows, <= 240)
    int chunks;        // reduce chunks
    size_t start, end; // [K] int32 each
    size_t partial;    // [chunks][2][D] fp32
    size_t bytes;      // total workspace (0 when N == 0)
    int compute_units; // reduce workgroups: four per CU
};

// Whether the bucket path supports the shape (N <= 2^24, K <= 16384).
bool bucket_path_fits(int64_t N, int64_t K);

// Requires 0 <= N < 2^31, valid D, 1 <= K < 2^31 (checked by the caller);
// compute_units <= 0 means 256; force_path 0 (automatic), 1 or 2 (2 only
// where bucket_path_fits).
UpdatePlan make_update_plan(int64_t N, int64_t D, int64_t K, int compute_units,
                            int force_path);

// All launches of one update on `stream`; ws holds plan.bytes bytes (may be
// null when N == 0).  means may be null.
hipError_t launch_update(const UpdatePlan &plan, const uint16_t *X, const int32_t *labels,
                         const uint16_t *C_old, int N, int D, int K, uint16_t *C_new,
                         float *norms, int32_t *counts, float *means, void *ws,
                         hipStream_t stream);

}  // namespace kmeans
