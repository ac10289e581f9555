// kmeans_linear_plan.h -- the arithmetic of kmeans_linear.hip that needs no
// GPU: which bytes of an operand its staging reads.  Plain C++, so that a test
// can follow it on the CPU.  Not part of the public interface.
#pragma once

#include <stdint.h>

#if defined(__HIPCC__)
#include <hip/hip_runtime.h>
#define KM_BOTH __host__ __device__ __forceinline__
#else
#define KM_BOTH inline
#endif

namespace kmeans {

constexpr int kTileK = 64;            // k extent of a staged tile: two MFMA k-steps of 32

// One operand's tile of kTileK values of k by R values of its own index, as
// it is staged in LDS.
//
//   own index contiguous == false: R rows of 64 k (128 bytes, 8 chunks of 16).
//     Chunk c of row r lies at chunk c ^ ((r >> 1) & 7): the 16 rows that a
//     ds_read_b128 group reads at one k cover all 64 banks once.
//   own index contiguous == true: 64 rows (k) of R values (R / 16 granules of
//     32 bytes).  Granule g of row k lies at g ^ f(k), f(k) = (k & 3) |
//     ((k >> 3) & 3) << 2 (as many bits as there are granules): the 16 rows
//     that one ds_read_b64_tr_b16 reads of one granule then lie in different
//     granules, so in different banks.
template <bool OWN, int R>
struct TileMap {
    static constexpr int kRows = OWN ? kTileK : R;
    static constexpr int kRowBytes = (OWN ? R : kTileK) * 2;
    static constexpr int kChunks = kRowBytes / 16;
    static constexpr int kBytes = kRows * kRowBytes;
    static constexpr int kGranules = R / 16;

    static KM_BOTH int spread(int k) {
        return ((k & 3) | (((k >> 3) & 3) << 2)) & (kGranules - 1);
    }
    // The chunk of row r that lies at chunk slot c (its own inverse).
    static KM_BOTH int chunk(int r, int c) {
        if (OWN)
            return (((c >> 1) ^ spread(r)) << 1) | (c & 1);
        return c ^ ((r >> 1) & 7);
    }
};

// The 16-byte pieces of a tile that THREADS threads stage together: piece u of
// thread tid is chunk c of row r.  With DMA a wave's pieces lie one after
// another in LDS.
template <bool OWN, int R, int THREADS, bool DMA>
struct TilePieces {
    typedef TileMap<OWN, R> Map;
    static constexpr int kCount = Map::kBytes / 16 / THREADS;
    static_assert(kCount >= 1 && Map::kBytes % (16 * THREADS) == 0, "whole pieces per thread");

    static KM_BOTH void at(int tid, int u, int &r, int &c) {
        const int o = DMA ? (((tid >> 6) * kCount + u) * 64 + (tid & 63)) : u * THREADS + tid;
        r = o / Map::kChunks;
        c = Map::chunk(r, o % Map::kChunks);
    }
};

// Whether 16-byte runs that start inside the rows of a whole tile end inside
// the operand: k_left values of k lie from the tile's first one to the end of
// the range, rows are ld values apart, and own_lim values of the own index
// exist from the tile's first one on.  k contiguous: a run stays in its row
// where k goes on.  Own index contiguous: the last row's last run goes past its
// row's end by what own_lim lacks to a multiple of 8, which the k_left - kTileK
// rows after it have to hold (rows of one to six values, that many rows or
// fewer before the end, do not).
KM_BOTH bool runs_stay_inside(bool own_contiguous, int k_left, int64_t ld, int own_lim) {
    return k_left > kTileK &&
           (!own_contiguous || (k_left - kTileK) * ld >= ((8 - (own_lim & 7)) & 7));
}

// Values by which run c of a row of `lim` values starts early to end with it.
KM_BOTH int values_cut(int c, int lim) { return c * 8 + 8 > lim ? c * 8 + 8 - lim : 0; }

}  // namespace kmeans
