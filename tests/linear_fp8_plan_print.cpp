// Prints how kmeans_linear_fp8 would tile and split shapes on a GPU of 256 compute
// units: for each "N D F" of the arguments a line "16-bit fp32" (outputs), each as
// shape:splits:blocks-of-128-per-split.
#include <cstdio>
#include <cstdlib>

#include "kmeans_linear_plan.h"

using namespace kmeans;

int main(int argc, char **argv) {
    static const char *const kNames[] = {"wide", "deep", "paired", "rows", "unaligned"};
    for (int i = 1; i + 2 < argc; i += 3)
        for (int wide = 1; wide >= 0; --wide) {
            const Product g = fp8_product(std::atoll(argv[i]), std::atoll(argv[i + 1]),
                                          std::atoll(argv[i + 2]), 256, wide != 0);
            std::printf("%s:%d:%d%s", kNames[g.shape], g.splits,
                        (std::min(g.K, g.k_chunk) + kTileK - 1) / kTileK, wide ? " " : "\n");
        }
    return 0;
}
