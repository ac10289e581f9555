// Prints how the linear operators would tile and split shapes on a GPU of 256
// compute units: for each "N D F extra" (extra: values between rows) of the
// arguments a line "forward dX dW", each as shape:splits:tiles-of-k-per-split,
// with a * where an operand is laid out anew.
#include <cstdio>
#include <cstdlib>

#include "kmeans_linear_plan.h"

using namespace kmeans;

namespace {

void print(const Product &g, bool moved, const char *end) {
    static const char *const kNames[] = {"wide", "deep", "paired", "rows", "unaligned"};
    const int k = std::min(g.K, g.k_chunk);
    std::printf("%s%s:%d:%d%s", kNames[g.shape], moved ? "*" : "", g.splits,
                (k + kTileK - 1) / kTileK, end);
}

}  // namespace

int main(int argc, char **argv) {
    for (int i = 1; i + 3 < argc; i += 4) {
        const int64_t N = std::atoll(argv[i]), D = std::atoll(argv[i + 1]),
                      F = std::atoll(argv[i + 2]), ld = D + std::atoll(argv[i + 3]);
        const void *at = reinterpret_cast<const void *>(0x1000);
        size_t bytes = 0;
        {
            Operand x{at, ld, N, D, false, 0}, w{at, ld, F, D, false, 0};
            const Product g = forward_product(x, w, 256, bytes);
            print(g, x.moved || w.moved, " ");
        }
        {
            Operand w{at, ld, F, D, false, 0};
            const Product g = input_grad_product(N, w, 256, bytes);
            print(g, w.moved, " ");
        }
        Operand x{at, ld, N, D, false, 0};
        const Product g = weight_grad_product(F, x, 256, bytes);
        print(g, x.moved, "\n");
    }
    return 0;
}
