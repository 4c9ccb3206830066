// Host-side interfaces between the C ABI (api_w4.hip) and the kernels of the 4-bit
// weights and of the rows sorted by expert.  Every launcher enqueues on `stream` and
// returns hipGetLastError().
#pragma once

#include "r9k_internal.h"

namespace r9k {

// Tuning overrides: r9k_set_w4_plan's, before its first call the environment's, read
// once per process (as struct Tuning's):
//   R9K_W4=nt,wn,wk[,ks]            streaming kernel: column tiles a wave, waves along columns, K slices, K split
//   R9K_W4_TILED=on[,tn[,ks]]       tiled kernel: 0 never, 1 always; column tiles a wave, K split
struct W4Tuning {
    int stream[4];  // 0: the planner's
    int tiled[3];   // -1: the planner's
};
W4Tuning &w4_tuning();

// ---- 4-bit weights (w4_weight.hip, gemm_w4.hip) ----
// fmt: W4_INT or W4_MXFP4; grp: values a scale covers; the packed layout is in w4_device.h
hipError_t launch_quant_weight_w4(const uint16_t *w, int64_t N, int64_t K, int fmt, int grp, uint8_t *wq, void *s,
                                  uint8_t *z, hipStream_t st);
hipError_t launch_pack_weight_w4(const uint8_t *wq, const void *s, const uint8_t *z, int64_t N, int64_t K, int fmt,
                                 int grp, uint8_t *wp, void *sp, uint8_t *zp, hipStream_t st);
struct W4Args {
    const uint16_t *a;       // activations [arows][K] bf16
    const uint8_t *wp;       // packed codes [E][N*K/2]
    const void *sp;          // packed scales
    const uint8_t *zp;       // packed zeros, or NULL
    uint16_t *c;             // [M][N] bf16, or [M][N/2] with silu
    int64_t M, K, N;         // M: rows of c (expert products: the most that offsets cover)
    const int32_t *offsets;  // expert products: [E + 1] first rows; NULL for a dense product
    const int32_t *src;      // expert products: row r reads activation row src[r] / topk; NULL: row r
    int64_t E, topk, arows;
    int silu;                // 1: columns [0, N/2) gate, [N/2, N) up, c = silu(gate) * up
    float *part;             // with a K split: fp32 partials [ksplit][M][N] (workspace)
    // set by the launchers
    int nblk, nrow, ksplit;         // tiled kernel: column blocks, row blocks, K split
    int wnl, span, seg, cps;        // streaming kernel: log2 of the waves along the columns; chunks a split, a segment, a wave's slice
    uint32_t bmagic, tmagic, zfill; // ceil(2^20 / (64-piece blocks a row)), ceil(2^32 / topk), the zeros where none are given
};
struct W4Cfg {
    int mt;      // row tiles of 16 a CTA
    int nt;      // column tiles a wave
    int wn, wk;  // waves along the columns, K slices
    int ksplit;  // CTAs along K (dense products only)
    int seg;     // chunks of 128 K whose activation rows a CTA holds in LDS at a time
    double us;   // the planner's estimate
};
double w4_expert_blocks(int64_t M, int64_t E, int64_t RB);  // row blocks that uniform routing makes
W4Cfg w4_config(int64_t M, int64_t K, int64_t N, int64_t E, bool silu);
bool w4_stream_shape(int nt, int wn, int wk);  // one that the streaming kernel has
// segments in which a CTA's activation rows go through LDS; 0: slices loaded whole
int w4_segments(const W4Cfg &c, int64_t K, int fmt, int grp);
struct W4TiledCfg {
    bool on;     // false: the weight-streaming kernel takes the shape whatever the estimates
    int tn;      // column tiles a wave (4 waves along the columns)
    int ksplit;  // CTAs along K (dense products only)
    double us;   // the planner's estimate
};
W4TiledCfg w4_tiled_config(int64_t M, int64_t K, int64_t N, int64_t E, bool silu);
hipError_t launch_gemm_w4_tiled(const W4Args &a, int fmt, int grp, const W4TiledCfg &c, hipStream_t s);
hipError_t launch_gemm_w4(const W4Args &a, int fmt, int grp, const W4Cfg &c, hipStream_t s);

// ---- rows sorted by expert (moe_sort.hip) ----
struct SortArgs {
    const int32_t *ids;  // [T][topk]
    const void *x;       // [T] rows, or NULL: the sort alone
    void *xs;            // [T*topk] rows
    int32_t *src, *pos, *offsets, *count;
    int64_t T, topk, E, row_bytes;
};
size_t moe_sort_workspace(int64_t R, int64_t E);
hipError_t launch_moe_permute(const SortArgs &a, hipStream_t s);
hipError_t launch_moe_unpermute(const void *y, bool f32, int64_t row_bytes, int64_t T, int64_t topk,
                                const int32_t *pos, const float *w, void *out, hipStream_t s);
hipError_t launch_moe_unpermute_backward(const void *g, const void *y, bool f32, int64_t row_bytes, int64_t T,
                                         int64_t topk, const int32_t *pos, const float *w, void *gy, float *gw,
                                         hipStream_t s);

}  // namespace r9k
