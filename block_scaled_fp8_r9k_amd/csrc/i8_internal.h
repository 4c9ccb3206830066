// Host-side interfaces between the C ABI (api_i8.hip) and the kernels of the 8-bit
// integer products and of the router's training operators.  Every launcher enqueues on
// `stream` and returns hipGetLastError().
#pragma once

#include "r9k_internal.h"

namespace r9k {

// ---- 8-bit integer products (i8_quant.hip, gemm_i8.hip) ----
hipError_t launch_quant_i8(const uint16_t *x, int64_t rows, int64_t K, int8_t *q, float *s, hipStream_t st);

struct I8Args {
    const int8_t *aq;        // activation codes [arows][K]
    const float *as;         // their scales [arows]
    const int8_t *wp;        // packed codes [E][N*K]
    const float *ws;         // channel scales [E][N]
    uint16_t *c;             // [M][N] bf16, or [M][N/2] with silu
    int64_t M, K, N;         // M: rows of c (expert products: the most that offsets cover)
    const int32_t *offsets;  // expert products: [E + 1] first rows; NULL for a dense product
    const int32_t *src;      // expert products: row r reads activation row src[r] / topk; NULL: row r
    int64_t E, topk, arows;
    int silu;                // 1: columns [0, N/2) gate, [N/2, N) up, c = silu(gate) * up
    int32_t *part;           // with a K split: sums [ksplit][M][N] (workspace)
    const uint16_t *a;       // bf16 activations that the streaming kernel quantises itself (aq and as are not read)
    // set by the launchers
    int nblk, nrow, ksplit;  // tiled kernel: column blocks, row blocks; CTAs along K
    int wnl, span, cps;      // streaming kernel: log2 of the waves along the columns; chunks a split, a wave's slice
    uint32_t tmagic;         // ceil(2^32 / topk), 0 for topk = 1
};
struct I8Cfg {       // the weight-streaming kernel
    int mt;          // row tiles of 16 a CTA
    int nt;          // column tiles a wave
    int wn, wk;      // waves along the columns, K slices
    int ksplit;      // CTAs along K (dense products only)
};
struct I8TiledCfg {  // the LDS-tiled kernel
    int shape;       // I8_TILES
    int ksplit;      // CTAs along K (dense products only)
};
struct I8Plan {
    bool tile;       // the tiled kernel takes it
    bool fused;      // bf16 activations are quantised in the streaming kernel
    I8Cfg cfg;
    I8TiledCfg tiled;
    int ksplit() const { return tile ? tiled.ksplit : cfg.ksplit; }
};
// the streaming kernel's shapes: row tiles, column tiles a wave, waves along the columns and along K
inline constexpr int I8_STREAMS[][4] = {{1, 1, 1, 4}, {1, 1, 1, 8}, {1, 1, 1, 16}, {1, 2, 1, 4}, {1, 2, 1, 8}, {1, 2, 2, 2}, {2, 1, 1, 4},
                                        {2, 1, 1, 8}, {2, 2, 1, 4}, {2, 2, 1, 8}, {2, 2, 2, 2}, {4, 2, 1, 4}, {4, 2, 1, 8}};
// the tiled kernel's: columns x rows of a CTA, CTAs that share a compute unit
enum { I8_256X256, I8_256X128, I8_128X128, I8_128X64, I8_64X128, I8_64X64, I8_SHAPES };
inline constexpr int I8_TILES[I8_SHAPES][3] = {{256, 256, 1}, {256, 128, 1}, {128, 128, 2}, {128, 64, 2}, {64, 128, 2}, {64, 64, 2}};
// r9k_set_i8_plan's choice: kernel 0 (the planner's), R9K_I8_STREAM or R9K_I8_TILED, the shape (0: the planner's), the split
struct I8Tuning {
    int kernel, a, b, c, rows, ksplit;
};
I8Tuning &i8_tuning();
// quant: from bf16 activations; wide: activations read through an index, 4 GiB of them or more, which the streaming
// kernel's 32-bit offsets do not reach
I8Plan i8_plan_new(int64_t M, int64_t K, int64_t N, int64_t E, bool silu, bool quant, bool wide);
hipError_t launch_gemm_i8(const I8Args &a, const I8Cfg &c, hipStream_t s);
hipError_t launch_gemm_i8_tiled(const I8Args &a, const I8TiledCfg &c, hipStream_t s);
hipError_t launch_i8_reduce(const I8Args &a, int ksplit, hipStream_t s);  // a split's sums, added and scaled

// ---- the router's training operators (router.hip) ----
struct BalanceArgs {
    const void *logits;     // [T][E], fp32 or bf16
    bool f32;
    int64_t T, E, topk;
    const int32_t *ids;     // [T][topk]
    const uint8_t *mask;    // [T], or NULL
    float *loss;            // [1]
    int32_t *counts;        // [E + 1]
    float *psum;            // [E]
    // set by the launcher, in the workspace
    float *part_p;          // the parts' sums
    int32_t *part_c, *part_n, *ticket;
    double *dots;
};
size_t balance_workspace(int64_t T, int64_t E);
hipError_t launch_balance_loss(BalanceArgs a, void *workspace, hipStream_t s);
struct RouterGradArgs {
    const float *gw;        // [T][topk], or NULL: the balance loss's part alone
    const int32_t *ids;
    const float *w;
    int64_t T, E, topk;
    const float *gloss;     // [1], or NULL: the routing weights' part alone
    const void *logits;
    bool f32;
    const int32_t *counts;
    const uint8_t *mask;
    void *g;                // [T][E] of the logits' type
};
hipError_t launch_router_backward(const RouterGradArgs &a, hipStream_t s);

}  // namespace r9k
