// Products with 4-bit weights, few rows: the weight-streaming kernel.
//
//   C[m][n] = bf16( sum_g s[n][g] * ( sum_{k in g} a[m][k] q[n][k]  -  z[n][g] * sum_{k in g} a[m][k] ) )
//
// for int4 codes (a product of a bf16 and a code 0..15 is exact in fp32; z = 8
// where the weight has no zero points), and for mxfp4 the plain product with
// the converted weights, whose scale is a power of two and so rounds nothing.
// Neither the weights nor the sums are ever rounded to fewer than 32 bits; the
// output is rounded once.
//
// C^T = W A^T: a wave takes NT column tiles of 16 (rows of W) and MT row tiles
// of 16 (rows of A) and streams its K slice of the packed weights into
// registers, one 16-byte load a lane for a tile's 128 of K, D such chunks
// ahead; the codes become bf16 fragments of v_mfma_f32_16x16x32_bf16 there.
// The sums over a group's activations come out of the same instruction with a
// fragment of ones in place of the weights, in the register layout that the
// products have.  The CTA's waves hold consecutive K slices of the same tiles;
// their sums are added through LDS in ascending order.
//
// Bound by the packed weights' bytes, each read once (per 16 or 32 rows), and below a few
// MB by launch and latency.  In graphs, weights from memory: one row of 4096 x 14336 in
// int4 (groups of 128, zeros) 9.9 us (3.1 TB/s, 70 vector instructions a chunk and wave
// beside the loads; a plain read of as many bytes takes 6.0 us, with as many instructions
// 7.8; weights in the caches 8.1), in groups of 64 11.1, of 32 13.8, in mxfp4 8.3; 16 rows
// of 14336 x 4096 in mxfp4 13.6 us (2.3 TB/s, the reduce launch 4 of them); 16 tokens' top 8
// of 128 experts, 2048 -> 2 x 768 in int4, 34 us (3.9 TB/s).  K slices inside a CTA fill the chip where
// there are few columns without partials in memory; a persistent loop over tiles was
// slower than a CTA a tile (its prologue hides behind other CTAs' streams).
//
// For expert products the rows are ranges of `offsets`, one per expert; a CTA
// finds its expert and row block there (the grid covers the most blocks that R
// rows can make), and may read its activation rows through the sort's index.
// With silu the first half of a wave's tiles are gate columns, the second half
// the up columns that belong to them.
#include <algorithm>
#include <cmath>
#include <mutex>

#include "w4_internal.h"
#include "w4_device.h"

namespace r9k {

namespace {

// LDS of a CTA: its activation rows, then the K slices' sums in their place
constexpr int64_t W4_LDS = 150 * 1024;

// The lane's scales (and zeros) of one tile's chunk, as loaded.
template <int FMT, int NG>
struct W4Scale {
    uint32_t s[FMT == W4_MXFP4 ? 1 : 2 * NG];  // int4: 4 rows x NG groups of bf16; mxfp4: 4 bytes, one a group
    uint32_t z[FMT == W4_MXFP4 ? 1 : NG];      // int4: 4 rows x NG groups of bytes
};

}  // namespace

// LONG: the general form, for slices of more than D chunks and for activation rows
// that do not fit LDS at once.  Without it a slice is loaded whole before its first
// chunk is computed, in straight code: the waits are then exact, chunk by chunk.
template <int FMT, int GRP, int MT, int NT, int D, bool LONG>
__global__ __launch_bounds__(512) void k_gemm_w4(W4Args p) {
    constexpr int NG = 128 / GRP;  // groups a chunk
    constexpr int KPG = GRP / 32;  // MFMA steps a group
    extern __shared__ __align__(16) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, q = lane >> 4;
    const int nw = blockDim.x >> 6, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = 1 << p.wnl, ct = wave & (wn - 1), slice = wave >> p.wnl, wk = nw >> p.wnl;
    const int C = (int)(p.K / 128), tiles = (int)(p.N / 16);
    const int bx = blockIdx.x, item = blockIdx.y;

    // rows [r0, r1) of this CTA, of expert e
    int e = 0, r0, r1;
    if (p.offsets) {
        int a0, a1;
        if (!w4_find_block(p.offsets, (int)p.E, (int)p.M, 16 * MT, item, e, a0, a1)) return;
        r0 = a0;
        r1 = min(a1, a0 + 16 * MT);
    } else {
        r0 = item * 16 * MT;
        r1 = (int)min<int64_t>(p.M, (int64_t)r0 + 16 * MT);
    }
    e = __builtin_amdgcn_readfirstlane(e);
    r0 = __builtin_amdgcn_readfirstlane(r0);
    r1 = __builtin_amdgcn_readfirstlane(r1);
    const int rows = r1 - r0;

    // this CTA's chunks [kb, ke) of split blockIdx.z
    const int ks = blockIdx.z;
    const int kb = ks * p.span, ke = min(C, kb + p.span);

    // the wave's column tiles; those past the last repeat it and are not stored
    int tile[NT];
    const int u0 = bx * wn + ct;  // the wave's place among all column groups
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        tile[j] = min(u0 * NT + j, tiles - 1);
        if constexpr (NT > 1) {
            if (p.silu) tile[j] = min(u0 * (NT / 2) + j % (NT / 2), tiles / 2 - 1) + (j < NT / 2 ? 0 : tiles / 2);
        }
    }

    // the activation row of each row of the block, in lane r; an index that points
    // outside the activations means row 0
    uint32_t arow = r0 + min(lane, rows - 1);
    if (p.src) {
        arow = w4_div_topk((uint32_t)p.src[arow], (uint32_t)p.topk, p.tmagic);
        if (arow >= (uint32_t)p.arows) arow = 0;
    }

    v4f acc[NT][MT];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[j][m] = v4f{0.f, 0.f, 0.f, 0.f};

    constexpr int SB = FMT == W4_MXFP4 ? 64 : 32 * NG, ZB = 16 * NG;  // bytes of scales and zeros a tile's chunk
    uint4 wr[D][NT];
    W4Scale<FMT, NG> sc[D][NT];
    const uint8_t *al[MT];
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(w4_lds_addr(lds));

    auto compute = [&](int c, int d) {
        w4_v8bf af[MT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int k = 0; k < 4; ++k) af[m][k] = w4_frag(*(const uint4 *)(al[m] + c * 256 + 64 * k));
        if constexpr (FMT == W4_MXFP4) {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const uint32_t word[4] = {wr[d][j].x, wr[d][j].y, wr[d][j].z, wr[d][j].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float s = __uint_as_float(((sc[d][j].s[0] >> (8 * k)) & 255u) << 23);
                    const w4_v8bf wf = w4_fp4_frag(word[k], s);
#pragma unroll
                    for (int m = 0; m < MT; ++m) acc[j][m] = w4_mfma(wf, af[m][k], acc[j][m]);
                }
            }
        } else {
            const v4f zero = {0.f, 0.f, 0.f, 0.f};
            v4f sum[NG][MT];  // sums of a group's activations, the same in all four registers
#pragma unroll
            for (int i = 0; i < NG; ++i)
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    sum[i][m] = zero;
#pragma unroll
                    for (int k = 0; k < KPG; ++k) sum[i][m] = w4_mfma(w4_ones(), af[m][i * KPG + k], sum[i][m]);
                }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const uint32_t word[4] = {wr[d][j].x, wr[d][j].y, wr[d][j].z, wr[d][j].w};
#pragma unroll
                for (int i = 0; i < NG; ++i) {
                    v4f pr[MT];
#pragma unroll
                    for (int m = 0; m < MT; ++m) pr[m] = zero;
#pragma unroll
                    for (int k = 0; k < KPG; ++k) {
                        const w4_v8bf wf = w4_int_frag(word[i * KPG + k]);
#pragma unroll
                        for (int m = 0; m < MT; ++m) pr[m] = w4_mfma(wf, af[m][i * KPG + k], pr[m]);
                    }
                    const float s[4] = {bf16_lo(sc[d][j].s[2 * i]), bf16_hi(sc[d][j].s[2 * i]),
                                        bf16_lo(sc[d][j].s[2 * i + 1]), bf16_hi(sc[d][j].s[2 * i + 1])};
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float z = (float)(((sc[d][j].z[i] | p.zfill) >> (8 * r)) & 255u);
                            acc[j][m][r] = __builtin_fmaf(s[r], __builtin_fmaf(-z, sum[i][m][0], pr[m][r]), acc[j][m][r]);
                        }
                }
            }
        }
    };

    // The chunks [s0, s1): their activation rows go into LDS; the wave computes its
    // slice of them.
    auto segment = [&](int s0, int s1) {
        const int cb = min(s1, s0 + slice * p.cps), ce = min(s1, cb + p.cps);

        // 1. the rows into LDS, padded by 16 bytes so that the 16 rows of a fragment
        // read fall on distinct banks; a wave moves 64 16-byte pieces of a row at a
        // time, straight into LDS
        const int ppr = (s1 - s0) * 16;  // pieces a row
        const int bpr = (s1 - s0 + 3) >> 2, blocks = rows * bpr, pitch = ppr * 16 + 16;
        for (int i = wave; i < blocks; i += nw) {
            // bmagic = ceil(2^20 / bpr) of a whole segment
            const int r = !LONG || s1 - s0 == p.seg ? (int)((uint32_t)i * p.bmagic >> 20) : i / bpr;
            const int c0 = (i - r * bpr) * 64;
            const uint16_t *row = p.a + (int64_t)(uint32_t)__builtin_amdgcn_readlane((int)arow, r) * p.K + s0 * 128;
            w4_load16_first(row + 8 * (c0 + lane), lds0 + r * pitch + c0 * 16, ppr - c0);
        }
        __builtin_amdgcn_sched_barrier(0);

        // 2. the weight stream, through descriptors that end with the slice: loads past
        // the end return zeros and move nothing.  Without zero points theirs is empty.
        __amdgpu_buffer_rsrc_t wd[NT], sd[NT], zd[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int64_t t0 = ((int64_t)e * tiles + tile[j]) * C;  // the tile's first chunk
            wd[j] = __builtin_amdgcn_make_buffer_rsrc((void *)(p.wp + t0 * 1024), (short)0, ce * 1024, 0x00020000);
            sd[j] = __builtin_amdgcn_make_buffer_rsrc((void *)((const uint8_t *)p.sp + t0 * SB), (short)0, ce * SB, 0x00020000);
            if constexpr (FMT == W4_INT)
                zd[j] = __builtin_amdgcn_make_buffer_rsrc((void *)(p.zp + t0 * ZB), (short)0, p.zp ? ce * ZB : 0, 0x00020000);
        }
        const int wvo = 16 * lane, svo = FMT == W4_MXFP4 ? 4 * l16 : 8 * NG * q, zvo = 4 * NG * q;
        auto load_scales = [&](int c, int d) {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                if constexpr (FMT == W4_MXFP4) {
                    sc[d][j].s[0] = __builtin_amdgcn_raw_buffer_load_b32(sd[j], svo + c * SB, 0, 0);
                } else if constexpr (NG == 1) {
                    const auto v = __builtin_amdgcn_raw_buffer_load_b64(sd[j], svo + c * SB, 0, 0);
                    sc[d][j].s[0] = v[0];
                    sc[d][j].s[1] = v[1];
                    sc[d][j].z[0] = __builtin_amdgcn_raw_buffer_load_b32(zd[j], zvo + c * ZB, 0, 0);
                } else {
#pragma unroll
                    for (int i = 0; i < NG / 2; ++i) {
                        const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(sd[j], svo + c * SB + 16 * i, 0, 0);
#pragma unroll
                        for (int r = 0; r < 4; ++r) sc[d][j].s[4 * i + r] = v[r];
                    }
                    if constexpr (NG == 2) {
                        const auto v = __builtin_amdgcn_raw_buffer_load_b64(zd[j], zvo + c * ZB, 0, 0);
                        sc[d][j].z[0] = v[0];
                        sc[d][j].z[1] = v[1];
                    } else {
                        const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(zd[j], zvo + c * ZB, 0, 0);
#pragma unroll
                        for (int r = 0; r < 4; ++r) sc[d][j].z[r] = v[r];
                    }
                }
            }
        };
        auto load_codes = [&](int c, int d) {
#pragma unroll
            for (int j = 0; j < NT; ++j) wr[d][j] = load_buf_nt16(wd[j], wvo + c * 1024);
        };
#pragma unroll
        for (int d = 0; d < D; ++d) load_scales(cb + d, d);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int d = 0; d < D; ++d) {
            load_codes(cb + d, d);
            __builtin_amdgcn_sched_barrier(0);  // in the order of use
        }
        // the rows (and scales) have landed once at most the D * NT code loads behind them are in flight
        w4_wait_vm<D * NT>();
        __syncthreads();
#pragma unroll
        for (int m = 0; m < MT; ++m) al[m] = lds + min(16 * m + l16, rows - 1) * pitch + 16 * q;

        if constexpr (LONG) {
            for (int c = cb; c < ce; c += D) {
#pragma unroll
                for (int d = 0; d < D; ++d) {
                    if (c + d < ce) compute(c + d - s0, d);
                    if (c + d + D < ce) {
                        load_scales(c + d + D, d);
                        load_codes(c + d + D, d);
                    }
                }
            }
        } else {
#pragma unroll
            for (int d = 0; d < D; ++d)
                if (cb + d < ce) compute(cb + d - s0, d);
        }
    };
    if constexpr (LONG) {
        for (int s0 = kb; s0 < ke; s0 += p.seg) {
            if (s0 > kb) __syncthreads();  // every wave is done with the segment before
            segment(s0, min(ke, s0 + p.seg));
        }
    } else {
        segment(kb, ke);
    }

#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int m = 0; m < MT; ++m) pin_acc(acc[j][m]);  // the MFMAs run with every lane enabled

    // 3. sum the K slices in ascending order, in the LDS that held the rows; an item is
    // one output tile of the CTA (with silu, a gate tile and its up tile)
    v4f *red = (v4f *)lds;  // [wave][tile][row tile][lane]
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int m = 0; m < MT; ++m) red[((wave * NT + j) * MT + m) * 64 + lane] = acc[j][m];
    __syncthreads();
    const int64_t ldc = p.silu ? p.N / 2 : p.N;
    const int nt = p.silu ? NT / 2 : NT;  // output tiles a wave
    const int otiles = p.silu ? tiles / 2 : tiles;
    const int outs = wn * nt * MT;
    // the block's rows of c or of this split's partials: at most 32 rows of 2^24 columns, 2^31 bytes
    void *first = p.ksplit > 1 ? (void *)(p.part + ((int64_t)ks * p.M + r0) * p.N) : (void *)(p.c + r0 * ldc);
    const __amdgpu_buffer_rsrc_t out = __builtin_amdgcn_make_buffer_rsrc(
        first, (short)0, (int)((uint32_t)rows * (uint32_t)ldc * (p.ksplit > 1 ? 4u : 2u)), 0x00020000);
    for (int it = wave; it < outs; it += nw) {
        const int w = it & (wn - 1), j = (it >> p.wnl) / MT, m = (it >> p.wnl) % MT;
        auto total = [&](int jj) {
            v4f x = red[((w * NT + jj) * MT + m) * 64 + lane];
            for (int s = 1; s < wk; ++s) x += red[(((s * wn + w) * NT + jj) * MT + m) * 64 + lane];
            return x;
        };
        v4f x = total(j);
        const int t = (bx * wn + w) * nt + j;
        if (p.silu) {
            const v4f u = total(j + nt);
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] = w4_silu_mul(x[r], u[r]);
        }
        if (t >= otiles) continue;
        // a store past the last row falls behind the descriptor's end and is dropped (no lane is masked)
        const uint32_t at = (uint32_t)(16 * m + l16) * (uint32_t)ldc + 16 * t + 4 * q;
        if (p.ksplit > 1) __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), out, 4 * at, 0, 0);
        else __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(w4_v2u, w4_bf16x4(x)), out, 2 * at, 0, 0);
    }
}

// The launch of the least estimated time.  A compute unit's CTAs take turns for the
// LDS and registers they need; its busiest unit moves A (activations into LDS) and W
// (codes) and pays for each CTA and wave; a turn is as long as the longest slice; a K
// split adds its partials and the reduce launch.  Fitted to 30 dense shapes (M = 1, 4, 16; K
// and N from 1024 to 14336, int4 in groups of 128 with zeros), 10 launches each, in graphs with
// the weights out of the caches: the launch it picks takes 1% longer than the fastest of the
// ten on average (at most 8%).  Groups of 32, of which a wave loads half as many chunks
// ahead, were not fitted: over 12 other shapes 11% behind the fastest (at most 40%: 16 rows of
// 4096 x 4096 11.2 us, eight slices 8.0), the other formats within 1% (5%).  Experts, whose turns begin with the search for their rows
// and whose bytes hide behind other CTAs' starts: 15 shapes (8 to 128 experts, up to 8 rows each, int4 and mxfp4,
// 128 to 1536 wide), 11 launches each, 1% (at most 11%); over 48 other shapes, up to 8 rows an
// expert in every format, 9% (at most 47%: 64 rows of 8 experts, 4096 -> 2 x 1024).
// E.g. one row of 4096 x 4096 5.1 us with four slices of one tile a wave, 5.6 with eight;
// 16 rows of 14336 x 4096 16 us in the split it picks, 25 in one.  Up to 400 rows it
// also decides against the tiled kernel (figures there).
struct W4Shape {
    int nt, wn, wk;
};
static constexpr W4Shape W4_SHAPES[] = {{1, 1, 4}, {1, 1, 8}, {1, 2, 2}, {1, 2, 4}, {1, 4, 2}, {2, 1, 2},
                                        {2, 1, 4}, {2, 1, 8}, {2, 2, 2}, {2, 2, 4}, {2, 4, 2}};
bool w4_stream_shape(int nt, int wn, int wk) {
    for (const W4Shape &s : W4_SHAPES)
        if (s.nt == nt && s.wn == wn && s.wk == wk) return true;
    return false;
}
static double w4_cost(const W4Cfg &c, int64_t rows, int64_t C, int64_t M, int64_t N, int64_t E, double items) {
    const int waves = c.wn * c.wk;
    const int64_t span = (C + c.ksplit - 1) / c.ksplit, segs = (span + c.seg - 1) / c.seg;
    const int64_t tiles = N / 16, per = (int64_t)c.nt * c.wn;
    const double ctas = (double)((tiles + per - 1) / per * c.ksplit) * items;
    const double lds = (double)std::max<int64_t>(std::min<int64_t>(M, 16 * c.mt) * (c.seg * 256 + 16), (int64_t)waves * c.nt * c.mt * 1024);
    const double fit = std::max(1.0, std::min(std::floor(163840.0 / lds), std::floor(20.0 / waves)));
    const double rounds = std::ceil(ctas / 256.0), turns = std::ceil(rounds / fit);
    if (E)
        return 0.9 + 0.28 * waves + rounds * (0.0189 * 0.25 * (double)(rows * span) + 0.0108 * (double)(per * span) + 0.015 * waves) +
               turns * (0.22 * (double)((c.seg + c.wk - 1) / c.wk * segs * c.nt * c.mt) + 1.12 * (double)(segs - 1) + 3.55);
    double us = 1.5 + 0.2 * waves + rounds * (0.0176 * 0.25 * (double)(rows * span) + 0.0356 * (double)(per * span) + 0.175 + 0.03 * waves);
    us += turns * (0.13 * (double)((c.seg + c.wk - 1) / c.wk * segs * c.nt * c.mt) + 1.12 * (double)(segs - 1));
    if (c.ksplit > 1) us += 2.5 + 2.0e-6 * (double)(c.ksplit * M * N);
    return us;
}

// Row blocks of RB rows that uniform routing of M rows to E experts makes: the experts with
// more than 0, RB, 2 RB, ... rows, their counts taken as normal with the mean's variance.
// Counts four deviations and more below the mean are passed by every expert; where the
// deviation is a block or more, a last block is as likely to hold any number of rows
// (both within 2e-5 of the whole sum), so that no plan takes more than a few steps.
double w4_expert_blocks(int64_t M, int64_t E, int64_t RB) {
    const double mean = (double)M / (double)E, sd = std::sqrt(mean), rb = (double)RB;
    if (sd >= rb) return (double)E * (mean / rb + 0.5 - 0.5 / rb);
    const double sure = std::max(0.0, std::floor((mean - 4.0 * sd) / rb));
    double blocks = (double)E * (1.0 - std::pow(1.0 - 1.0 / (double)E, (double)M) + sure);
    for (double j = rb * (sure + 1.0); j < mean + 4.0 * sd + 1.0; j += rb)
        blocks += (double)E * 0.5 * std::erfc((j + 0.5 - mean) / std::sqrt(2.0 * mean));
    return blocks;
}

W4Cfg w4_config(int64_t M, int64_t K, int64_t N, int64_t E, bool silu) {
    const int64_t C = K / 128;
    W4Cfg best{};
    // one row tile up to 16 rows; experts up to 12 on average, where few have more than 16 (2048
    // -> 2 x 768 of 128 experts, int4, 8 rows an expert: 50 us, 78 with two; 4096 -> 1536 of 8,
    // 10 rows: 14.3 and 20.3; at 15 rows 23.0, at 20 rows 16.8 with two)
    best.mt = M <= (E ? 12 * E : 16) ? 1 : 2;
    const int64_t RB = 16 * best.mt, most = std::min<int64_t>(M, RB);
    const double items = E ? w4_expert_blocks(M, E, RB) : (double)((M + RB - 1) / RB);
    const int64_t rows = E ? std::min<int64_t>(most, (int64_t)std::ceil((double)M / items)) : most;
    const int64_t fit = std::max<int64_t>(1, (W4_LDS / most - 16) / 256);  // chunks whose rows fit LDS
    const int *tune = w4_tuning().stream;
    const W4Shape wish{std::max(tune[0], silu ? 2 : 1), tune[1], tune[2]};
    const bool force = tune[0] && w4_stream_shape(wish.nt, wish.wn, wish.wk);
    for (const W4Shape &sh : W4_SHAPES) {
        if (force && (sh.nt != wish.nt || sh.wn != wish.wn || sh.wk != wish.wk)) continue;
        if (silu && sh.nt == 1) continue;
        for (int ks = 1; ks <= (E ? 1 : 4); ks *= 2) {
            W4Cfg c = best;
            c.nt = sh.nt;
            c.wn = sh.wn;
            const int64_t want = force && tune[3] && !E ? tune[3] : ks;
            // a split where one CTA a compute unit is not reached without it
            if (!force && ks > 1 && (double)(N / 16) / (sh.nt * sh.wn) * items * (ks / 2) >= 256.0) break;
            const int64_t span = (C + std::min(want, C) - 1) / std::min(want, C);
            c.ksplit = (int)((C + span - 1) / span);  // no split without chunks
            const int64_t segs = (span + fit - 1) / fit;
            c.seg = (int)((span + segs - 1) / segs);
            c.wk = (int)std::min<int64_t>(sh.wk, c.seg);
            const double us = w4_cost(c, rows, C, M, N, E, items);
            if (best.us == 0.0 || us < best.us) {
                best = c;
                best.us = us;
            }
        }
    }
    return best;
}

// chunks ahead: as many registers as two waves a SIMD leave, scales included
constexpr int w4_ahead(int fmt, int grp, int nt) { return (grp == 32 && fmt == W4_INT ? 4 : 8) / nt; }

int w4_segments(const W4Cfg &c, int64_t K, int fmt, int grp) {
    // whole: one segment, the same in every split, and slices that are loaded whole
    const int64_t C = K / 128, span = (C + c.ksplit - 1) / c.ksplit;
    const bool whole = c.seg >= span && C % span == 0 && (c.seg + c.wk - 1) / c.wk <= w4_ahead(fmt, grp, c.nt);
    return whole ? 0 : (int)((span + c.seg - 1) / c.seg);
}

template <int FMT, int GRP, int MT, int NT, bool LONG>
static hipError_t launch_one(W4Args a, const W4Cfg &c, hipStream_t s) {
    auto kernel = k_gemm_w4<FMT, GRP, MT, NT, w4_ahead(FMT, GRP, NT), LONG>;
    // the dynamic LDS limit is a per-device function attribute: set it once per device
    static std::once_flag once[64];
    static hipError_t attr_err[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return hipErrorInvalidDevice;
    std::call_once(once[dev], [&] {
        attr_err[dev] = hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, W4_LDS);
    });
    if (attr_err[dev] != hipSuccess) return attr_err[dev];
    const int64_t per = (int64_t)c.wn * (a.silu ? NT / 2 : NT), tiles = a.N / 16 / (a.silu ? 2 : 1);
    const int64_t nblk = (tiles + per - 1) / per, RB = 16 * MT, C = a.K / 128;
    int64_t items = (a.M + RB - 1) / RB;
    if (a.offsets) items = (a.M + std::min(a.E, a.M) * (RB - 1)) / RB;
    a.wnl = __builtin_ctz((unsigned)c.wn);
    a.ksplit = c.ksplit;
    a.span = (int)((C + c.ksplit - 1) / c.ksplit);
    a.seg = std::min(c.seg, a.span);
    a.cps = (a.seg + c.wk - 1) / c.wk;
    const int bpr = (a.seg + 3) / 4;
    a.bmagic = (uint32_t)(((1 << 20) + bpr - 1) / bpr);
    a.tmagic = a.topk > 1 ? (uint32_t)(((uint64_t(1) << 32) + a.topk - 1) / a.topk) : 0;
    a.zfill = a.zp ? 0u : 0x08080808u;
    const size_t rows = (size_t)std::min<int64_t>(a.M, RB) * (size_t)(a.seg * 256 + 16);
    const size_t lds = std::max<size_t>(rows, (size_t)c.wn * c.wk * NT * MT * 1024);
    if (nblk > 0x7fffffff || items > 65535 || lds > (size_t)W4_LDS || c.wn * c.wk > 8) return hipErrorInvalidValue;
    hipLaunchKernelGGL(kernel, dim3((unsigned)nblk, (unsigned)items, (unsigned)c.ksplit), dim3(64 * c.wn * c.wk), lds,
                       s, a);
    return hipGetLastError();
}

template <int FMT, int GRP, int MT, int NT>
static hipError_t launch_nt(const W4Args &a, const W4Cfg &c, hipStream_t s) {
    return w4_segments(c, a.K, FMT, GRP) == 0 ? launch_one<FMT, GRP, MT, NT, false>(a, c, s)
                                              : launch_one<FMT, GRP, MT, NT, true>(a, c, s);
}

template <int FMT, int GRP, int MT>
static hipError_t launch_mt(const W4Args &a, const W4Cfg &c, hipStream_t s) {
    return c.nt == 1 ? launch_nt<FMT, GRP, MT, 1>(a, c, s) : launch_nt<FMT, GRP, MT, 2>(a, c, s);
}

template <int FMT, int GRP>
static hipError_t launch_fmt(const W4Args &a, const W4Cfg &c, hipStream_t s) {
    return c.mt == 1 ? launch_mt<FMT, GRP, 1>(a, c, s) : launch_mt<FMT, GRP, 2>(a, c, s);
}

hipError_t launch_gemm_w4(const W4Args &a, int fmt, int grp, const W4Cfg &c, hipStream_t s) {
    hipError_t err;
    if (fmt == W4_MXFP4) err = launch_fmt<W4_MXFP4, 32>(a, c, s);
    else if (grp == 32) err = launch_fmt<W4_INT, 32>(a, c, s);
    else if (grp == 64) err = launch_fmt<W4_INT, 64>(a, c, s);
    else err = launch_fmt<W4_INT, 128>(a, c, s);
    if (err != hipSuccess || c.ksplit == 1) return err;
    return launch_splitk_reduce(a.part, a.c, a.M, a.N, c.ksplit, s);
}

}  // namespace r9k
