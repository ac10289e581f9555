// kmeans_linear_plan.h -- the arithmetic of kmeans_linear.hip that needs no
// GPU: which bytes of an operand its staging reads, and how a product is tiled
// and split.  Plain C++, so that tests can follow it on the CPU.  Not part of
// the public interface.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <algorithm>

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

// ---- products ---------------------------------------------------------------

constexpr int64_t kMaxWidth = 1 << 20;   // D, F and row strides: 64 rows stay below 2^31 bytes
constexpr int kMaxKSplits = 64;
// linear_dz_kernel's threads, and rows in flight per lane.
constexpr int kDzThreads = 256;
constexpr int kDzRows = 4;

struct Epilogue {
    const void *bias;       // [J] or null
    const void *residual;   // [I][J] or null
    int64_t ldr;
    void *out;              // [I][J]
    int64_t ldo;
    void *pre;              // [I][J] or null
    int64_t ldp;
    int act;
};

struct Product {
    const void *P, *Q;
    int64_t ldp, ldq;       // elements between rows as they lie in memory
    int I, J, K;
    bool dma;               // both operands' rows are 16-byte aligned and of whole chunks of 8
    int shape;              // Shape
    int k_chunk;            // k per split, a multiple of kTileK
    int splits;
    int first_wg;           // of this launch
    float *partial;         // [splits][I][J] fp32 when splits > 1
    Epilogue epi;
};

inline size_t align_up(size_t n) { return (n + 255) & ~size_t(255); }

// Rows that DMA may read: 16-byte aligned base and stride.
inline bool rows_aligned(const void *p, int64_t ld) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0;
}

// A product's workspace: its partial sums.
inline size_t partial_bytes(const Product &g) {
    return g.splits > 1 ? static_cast<size_t>(g.splits) * g.I * g.J * sizeof(float) : 0;
}

// How one product is tiled and split.  Rates of the shapes on an MI355X, bf16,
// as the whole call (the library's product beside it):
//   8192 x 4096 x 4096   kWide 1310-1440 TFLOP/s by operand order, kPaired
//                        1110-1200, kDeep 1020-1100 (library 1440, 1260, 1140)
//   2048 x 2048 x 2048   kDeep 21.5 us, kPaired 24.6-27.4, kWide 45 (21.4-25.3)
//   65536 x 512 x 128    kPaired 18.1 us, kWide 22.6, kDeep 22.0 (18.6)
// kWide halves the LDS reads per flop; kDeep keeps three tiles on their way
// where one workgroup per CU is all there is; kPaired overlaps one workgroup's
// epilogue with the other's products where k is short.
enum Shape {
    kWide,      // 256 x 256 tiles, two stages, one workgroup of eight waves per CU
    kDeep,      // 128 x 128, four stages, one workgroup of eight waves per CU
    kPaired,    // 128 x 128, two stages, two workgroups of four waves per CU
    kRows,      // at most kMaxFewRows rows: weights straight into fragments (forward only)
    kUnaligned  // 128 x 128, two stages through registers, two of eight waves per CU
};

constexpr int kMaxFewRows = 16;

inline int64_t tiles_of(const Product &g, int side) {
    return ((static_cast<int64_t>(g.I) + side - 1) / side) *
           ((static_cast<int64_t>(g.J) + side - 1) / side);
}

// Chooses the shape and the splits of k with the least estimated time (us),
// which it returns.
inline double plan_product(Product &g, int compute_units) {
    const int64_t k_tiles = (g.K + kTileK - 1) / kTileK;
    struct Cost {
        Shape shape;
        int side, per_cu;
        double round;     // us per staged tile of a full round of workgroups
        double single;    // the same with one workgroup per CU
        double fixed;     // us per round: first copies, epilogue
    };
    static constexpr Cost kAligned[] = {{kWide, 256, 1, 1.50, 1.50, 4.0},
                                        {kDeep, 128, 1, 0.50, 0.50, 2.0},
                                        {kPaired, 128, 2, 0.92, 0.65, 1.5}};
    static constexpr Cost kOther[] = {{kUnaligned, 128, 2, 1.6, 1.1, 2.0}};
    const Cost *costs = g.dma ? kAligned : kOther;
    const int kinds = g.dma ? 3 : 1;
    double best = 1e30;
    for (int c = 0; c < kinds; ++c) {
        const Cost &k = costs[c];
        const int64_t tiles = tiles_of(g, k.side);
        for (int64_t s = 1; s <= std::min<int64_t>(kMaxKSplits, k_tiles); s *= 2) {
            const int64_t per = (k_tiles + s - 1) / s;
            const int64_t wgs = tiles * ((k_tiles + per - 1) / per);
            const int64_t slots = static_cast<int64_t>(compute_units) * k.per_cu;
            const int64_t rest = wgs % slots;       // workgroups of the last round
            double t = static_cast<double>(wgs / slots) * (per * k.round + k.fixed);
            if (rest > 0)
                t += per * (rest <= compute_units ? k.single : k.round) + k.fixed;
            if (s > 1)    // the join's launch, and the partial sums written and read
                t += 4.5 + static_cast<double>(s) * g.I * g.J * 8e-6 / 4.0;
            if (t < best) {
                best = t;
                g.shape = k.shape;
                g.k_chunk = static_cast<int>(per * kTileK);
                g.splits = static_cast<int>((k_tiles + per - 1) / per);
            }
        }
    }
    return best;
}

// How linear_dz_kernel divides N rows of F values.
struct RowPlan {
    int64_t ld;                 // values from one written row to the next
    int lanes_log2, rows_per_wg, row_wgs, col_wgs;
    RowPlan(int64_t N, int64_t F, int compute_units) : ld((F + 7) / 8 * 8), lanes_log2(0) {
        const int64_t col_groups = ld / 8;
        while (lanes_log2 < 6 && (1 << lanes_log2) < col_groups)
            ++lanes_log2;
        col_wgs = static_cast<int>((col_groups + (1 << lanes_log2) - 1) >> lanes_log2);
        // About eight workgroups per CU, each at least one round of rows; few
        // enough that the column partials stay small beside dY.
        const int64_t rows_round = kDzRows * (kDzThreads >> lanes_log2);
        int64_t wgs = std::min<int64_t>(512, std::max<int64_t>(1, 8 * compute_units / col_wgs));
        wgs = std::min<int64_t>(wgs, (N + rows_round - 1) / rows_round);
        rows_per_wg = static_cast<int>((N + wgs - 1) / wgs);
        row_wgs = static_cast<int>((N + rows_per_wg - 1) / rows_per_wg);
    }
    size_t bytes(int64_t N) const { return align_up(static_cast<size_t>(N) * ld * 2); }
};

// An operand as its caller has it, and whether and where in the workspace it
// is laid out anew, with rows that the global-to-LDS copies take.
struct Operand {
    const void *p;
    int64_t ld, rows, cols;
    bool moved;
    size_t at;
    bool fits() const { return rows_aligned(p, ld) && cols % 8 == 0; }
};

// Plans a product of operands, some of which may not fit the copies: as they
// lie through registers (kUnaligned), or laid out anew first where that costs
// less, at workspace offset `bytes` on (as it lies, moved: forward 4133 x 515 x
// 1001 24 us, 33; 8192 x 2001 x 2000 140 us, 114; gradients 263 us, 198).
inline void plan_operands(Product &g, Operand *const *ops, int n, int compute_units, size_t &bytes) {
    double moves = 0;
    g.dma = true;
    for (int i = 0; i < n; ++i)
        if (!ops[i]->fits()) {
            g.dma = false;
            moves += 5.0 + static_cast<double>(ops[i]->rows) * ops[i]->cols * 4e-6 / 2.5;
        }
    const double as_is = plan_product(g, compute_units);
    if (g.dma)
        return;
    Product moved = g;
    moved.dma = true;
    if (plan_product(moved, compute_units) + moves >= as_is)
        return;
    g = moved;
    for (int i = 0; i < n; ++i)
        if (!ops[i]->fits()) {
            ops[i]->moved = true;
            ops[i]->at = bytes;
            bytes += RowPlan(ops[i]->rows, ops[i]->cols, compute_units).bytes(ops[i]->rows);
        }
}

// The products of the entry points, for operands as the caller has them;
// `bytes` grows by the workspace of those laid out anew.  Pointers of the
// outputs and of dZ are the caller's to fill in.
inline Product forward_product(Operand &x, Operand &w, int compute_units, size_t &bytes) {
    Product g{};
    g.P = x.p;
    g.ldp = x.ld;
    g.Q = w.p;
    g.ldq = w.ld;
    g.I = static_cast<int>(x.rows);
    g.J = static_cast<int>(w.rows);
    g.K = static_cast<int>(x.cols);
    if (x.rows <= kMaxFewRows) {
        g.shape = kRows;
        g.splits = 1;
    } else {
        Operand *const ops[] = {&x, &w};
        plan_operands(g, ops, 2, compute_units, bytes);
    }
    return g;
}
inline Product input_grad_product(int64_t N, Operand &w, int compute_units, size_t &bytes) {
    Product g{};
    g.Q = w.p;
    g.ldq = w.ld;
    g.I = static_cast<int>(N);
    g.J = static_cast<int>(w.cols);
    g.K = static_cast<int>(w.rows);
    Operand *const ops[] = {&w};
    plan_operands(g, ops, 1, compute_units, bytes);
    return g;
}
inline Product weight_grad_product(int64_t F, Operand &x, int compute_units, size_t &bytes) {
    Product g{};
    g.Q = x.p;
    g.ldq = x.ld;
    g.I = static_cast<int>(F);
    g.J = static_cast<int>(x.cols);
    g.K = static_cast<int>(x.rows);
    Operand *const ops[] = {&x};
    plan_operands(g, ops, 1, compute_units, bytes);
    return g;
}

}  // namespace kmeans
