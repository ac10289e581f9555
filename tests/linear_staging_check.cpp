// Follows, on the CPU, the addresses that the linear kernels' staging through
// registers reads, for operands whose own index is contiguous (the weight
// gradient's X, the input gradient's W) and for those whose k is.  Prints the
// first read outside an operand and exits with 1, else prints the number of
// runs followed.
#include <cstdio>
#include <initializer_list>

#include "kmeans_linear_plan.h"

using namespace kmeans;

namespace {

long runs = 0;

bool inside(long first, long size, const char *what, bool own, int k, int width, long ld, int t) {
    ++runs;
    if (first >= 0 && first + 8 <= size)
        return true;
    std::printf("%s: own=%d k=%d width=%d stride=%ld tile %d reads [%ld, %ld) of %ld\n", what, own,
                k, width, ld, t, first, first + 8, size);
    return false;
}

// `outer` rows of `width` values, ld apart; k is the rows' index (OWN) or the
// values' (else).  Tiles as a workgroup walks them, from every own offset.
template <bool OWN, int R, int THREADS>
bool follow(int k, int other, long ld) {
    typedef TilePieces<OWN, R, THREADS, false> Pieces;
    const int width = OWN ? other : k, rows = OWN ? k : other;
    const long size = static_cast<long>(rows - 1) * ld + width;
    const int tiles = (k + kTileK - 1) / kTileK;
    for (int own0 = 0; own0 < other; own0 += R) {
        const int own_lim = other - own0;
        const bool narrow = OWN ? own_lim < 8 && own0 == 0 : k < 8;
        for (int t = 0; t < tiles; ++t) {
            const int k_left = k - t * kTileK;
            const long base = OWN ? static_cast<long>(t) * kTileK * ld + own0
                                  : static_cast<long>(own0) * ld + t * kTileK;
            const bool whole = runs_stay_inside(OWN, k_left, ld, own_lim);
            if (!whole && t + 2 < tiles) {
                std::printf("tile %d of %d is not whole\n", t, tiles);   // cut_tiles() <= 2
                return false;
            }
            if (!whole && !narrow && t + 1 < tiles) {
                std::printf("tile %d of %d: no path for it\n", t, tiles);
                return false;
            }
            if (!whole && narrow)
                continue;                                // value by value
            for (int tid = 0; tid < THREADS; ++tid)
                for (int u = 0; u < Pieces::kCount; ++u) {
                    int r, c;
                    Pieces::at(tid, u, r, c);
                    const bool some = OWN ? c * 8 < own_lim && r < k_left : c * 8 < k_left;
                    if (!some)
                        continue;                        // offset out of range: zeros
                    const long row = OWN ? r : (r < own_lim ? r : own_lim - 1);
                    const long at = c * 8 - (whole ? 0 : values_cut(c, OWN ? own_lim : k_left));
                    if (!inside(base + row * ld + at, size, whole ? "whole" : "last", OWN, k,
                                width, ld, t))
                        return false;
                }
        }
    }
    return true;
}

}  // namespace

int main() {
    const int widths[] = {1, 2, 3, 4, 5, 6, 7, 8, 9, 15, 16, 17, 127, 128, 129, 135, 257};
    const int gaps[] = {0, 1, 2, 5, 8};
    for (int width : widths)
        for (int gap : gaps) {
            for (int k = 1; k <= 4 * kTileK + 8; ++k)
                if (!follow<true, 128, 512>(k, width, width + gap))
                    return 1;
            for (int rows : {1, 5, 128, 130})
                if (!follow<false, 128, 512>(width, rows, width + gap))
                    return 1;
        }
    // The rule is no wider than it has to be: with rows one after another,
    // exactly those runs are refused that would leave the operand.
    for (int width = 1; width <= 12; ++width)
        for (int k_left = 1; k_left <= 3 * kTileK; ++k_left) {
            const long size = static_cast<long>(k_left - 1) * width + width;
            const long end = static_cast<long>(kTileK - 1) * width + (width + 7) / 8 * 8;
            if (runs_stay_inside(true, k_left, width, width) !=
                (k_left > kTileK && end <= size)) {
                std::printf("width %d, %d rows left: %ld of %ld\n", width, k_left, end, size);
                return 1;
            }
        }
    std::printf("%ld runs inside\n", runs);
    return 0;
}
