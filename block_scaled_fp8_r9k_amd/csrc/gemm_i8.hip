// Products in 8-bit integers, few rows: the weight-streaming kernel.
//
//   c[m][n] = bf16( (sum_k aq[m][k] * wq[n][k]) * as[m] * ws[n] )
//
// with the sum in 32-bit integers, exact: no split of K and no order of the sum changes a
// bit of the output, which is rounded where the sum becomes fp32, at each scale and at the end.
//
// C^T = W A^T: a wave takes NT column tiles of 16 (rows of W) and MT row tiles of 16 (rows
// of A) and streams its K slice of both into registers as fragments of
// v_mfma_i32_16x16x64_i8, D chunks of 128 K ahead.  The CTA's waves hold consecutive K
// slices of the same tiles; their sums meet in LDS.  Rows of the block that are not there
// repeat its last row and are not stored.
//
// For expert products the rows are ranges of `offsets`, one per expert; a CTA finds its
// expert and row block there, and may read its activation rows through the sort's index.
// With silu the first half of a wave's tiles are gate columns, the second half the up
// columns that belong to them.
//
// Weight bytes bound it, read once: a launch has few rows to meet them, and matrix instructions take 6% of the cycles.
// Kernel trace, weights from memory: gate_up of 16 tokens, 2048 -> 2 x 768 of 128 experts, 41 us for 250 MB, 6 TB/s; 16 rows of
// 14336 x 4096 14.1 us for 59 MB, 4.2 TB/s, of which the launch, the first loads' way and the sums' way through LDS are 3 us;
// one row of 4096 x 14336 with its quantisation 11.8 us, 5.0 TB/s.
#include <algorithm>

#include "r9k.h"
#include "w4_internal.h"
#include "i8_device.h"
#include "i8_internal.h"

namespace r9k {

// 512-value units that a wave quantises, held in registers
static constexpr int I8_QA_UNITS = 4;

template <int MT, int NT, int D, bool LONG, bool QA>
__global__ __launch_bounds__(MT * NT == 1 ? 1024 : 512) void k_gemm_i8(I8Args p) {
    static_assert(!QA || MT == 1, "activations are quantised up to 16 rows");
    extern __shared__ __align__(16) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, q = lane >> 4;
    const int nw = blockDim.x >> 6, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = 1 << p.wnl, ct = wave & (wn - 1), slice = wave >> p.wnl, wk = nw >> p.wnl;
    const int C = (int)(p.K / 128), tiles = (int)(p.N / 16);
    const int bx = blockIdx.x, item = blockIdx.y, ks = blockIdx.z;

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

    // the wave's column tiles; those past the last repeat it and are not stored
    int tile[NT];
    const int u0 = bx * wn + ct;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        tile[j] = min(u0 * NT + j, tiles - 1);
        if constexpr (NT > 1) {
            if (p.silu) tile[j] = min(u0 * (NT / 2) + j % (NT / 2), tiles / 2 - 1) + (j < NT / 2 ? 0 : tiles / 2);
        }
    }

    // QA: the rows are quantised here, from bf16.  A unit is 512 values of a row, one 16-byte load of a
    // wave; the loads go out before the weights'.
    const int segs = (int)((p.K + 511) / 512), units = QA ? rows * segs : 0, K = (int)p.K;
    uint4 av[QA ? I8_QA_UNITS : 1];
    if constexpr (QA) {
#pragma unroll
        for (int i = 0; i < I8_QA_UNITS; ++i) {
            const int u = wave + i * nw, r = u / segs, k = (u - r * segs) * 512 + 8 * lane;
            av[i] = u < units && k < K ? *(const uint4 *)(p.a + (int64_t)(r0 + r) * K + k) : make_uint4(0, 0, 0, 0);
        }
    }
    // activation rows of the lane's row in each row tile; an index that points outside the
    // activations means row 0
    uint32_t aoff[MT];
    float as[MT];
    if constexpr (!QA) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int r = r0 + min(16 * m + l16, rows - 1);
            uint32_t row = r;
            if (p.src) {
                row = w4_div_topk((uint32_t)p.src[r], (uint32_t)p.topk, p.tmagic);
                if (row >= (uint32_t)p.arows) row = 0;
            }
            as[m] = p.as[row];
            aoff[m] = (p.src ? row : row - (uint32_t)r0) * (uint32_t)p.K + 16 * q;
        }
    }

    // this wave's chunks [cb, ce).  Weight loads past ce lie behind the descriptors' end, return
    // zeros and move nothing, and so make no difference whatever activations meet them.
    const int kb = ks * p.span, ke = min(C, kb + p.span);
    const int cb = kb + slice * p.cps, ce = __builtin_amdgcn_readfirstlane(min(ke, cb + p.cps));
    __amdgpu_buffer_rsrc_t wd[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j)
        wd[j] = __builtin_amdgcn_make_buffer_rsrc((void *)(p.wp + ((int64_t)e * tiles + tile[j]) * C * 2048), (short)0,
                                                  ce * 2048, 0x00020000);
    // (the block's rows, or with an index all of the activations, less than 2^32 bytes)
    const __amdgpu_buffer_rsrc_t ad = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(p.src ? p.aq : p.aq + (int64_t)r0 * p.K), (short)0,
        (int)((uint32_t)(p.src ? p.arows : rows) * (uint32_t)p.K), 0x00020000);

    v4i acc[NT][MT];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[j][m] = v4i{0, 0, 0, 0};
    v4i wr[D][NT][2], ar[QA ? 1 : D][MT][2];
    auto load = [&](int c, int d) {
        if constexpr (!QA) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    ar[d][m][h] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(ad, aoff[m] + c * 128 + 64 * h, 0, 0));
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                wr[d][j][h] = __builtin_bit_cast(v4i, load_buf_nt16(wd[j], 16 * lane + c * 2048 + 1024 * h));
    };
#pragma unroll
    for (int d = 0; d < D; ++d) {
        load(cb + d, d);
        __builtin_amdgcn_sched_barrier(0);  // in the order of use
    }
    // QA: [rows][K] codes, rows 16 bytes apart so that a fragment read's fall on distinct banks, then the units' maxima
    const uint8_t *al = lds;
    if constexpr (QA) {
        const int pitch = K + 16;
        uint32_t *top = (uint32_t *)(lds + rows * pitch);
        uint32_t *sums = top + units;  // the rows' scales
#pragma unroll
        for (int i = 0; i < I8_QA_UNITS; ++i) {
            const uint32_t m = max64(absmax8_bits(av[i]));
            if (wave + i * nw < units) top[wave + i * nw] = m;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < I8_QA_UNITS; ++i) {
            const int u = wave + i * nw, r = u / segs, k = (u - r * segs) * 512 + 8 * lane;
            if (u >= units) break;
            uint32_t m = 0;
            for (int s = lane; s < segs; s += 64) m = max(m, top[r * segs + s]);
            const I8Scale sc = i8_row_scale(max64(m));
            if (k < K) *(uint2 *)(lds + r * pitch + k) = i8_quant8(av[i], sc);
            if (u == r * segs) sums[r] = __float_as_uint(sc.s);
        }
        __syncthreads();
        as[0] = __uint_as_float(sums[min(l16, rows - 1)]);
        al = lds + min(l16, rows - 1) * pitch + 16 * q;
    }
    auto compute = [&](int c, int d) {
        if constexpr (QA) {
#pragma unroll
            for (int h = 0; h < 2; ++h) ar[0][0][h] = *(const v4i *)(al + c * 128 + 64 * h);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int m = 0; m < MT; ++m) acc[j][m] = i8_mfma(wr[d][j][h], ar[QA ? 0 : d][m][h], acc[j][m]);
    };
    if constexpr (LONG) {
        for (int c = cb; c < ce; c += D) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                if (c + d < ce) compute(c + d, d);
                if (c + d + D < ce) load(c + d + D, d);
            }
        }
    } else {
#pragma unroll
        for (int d = 0; d < D; ++d)
            if (cb + d < ce) compute(cb + d, d);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int m = 0; m < MT; ++m) i8_pin(acc[j][m]);

    // the K slices' sums, in LDS; an item is one output tile of the CTA (with silu, a gate
    // tile and its up tile)
    v4i *red = (v4i *)lds;  // [wave][tile][row tile][lane], where the codes were
    if constexpr (QA) __syncthreads();
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int m = 0; m < MT; ++m) red[((wave * NT + j) * MT + m) * 64 + lane] = acc[j][m];
    __syncthreads();
    const int64_t ldc = p.silu ? p.N / 2 : p.N;
    const int nt = p.silu ? NT / 2 : NT;
    const int otiles = p.silu ? tiles / 2 : tiles;
    const int outs = wn * nt * MT;
    // the block's rows of c or of this split's sums, less than 2^32 bytes; a store past the last
    // row falls behind the descriptor's end and is dropped (no lane is masked)
    void *first = p.ksplit > 1 ? (void *)(p.part + ((int64_t)ks * p.M + r0) * p.N) : (void *)(p.c + r0 * ldc);
    const __amdgpu_buffer_rsrc_t out = __builtin_amdgcn_make_buffer_rsrc(
        first, (short)0, (int)((uint32_t)rows * (uint32_t)ldc * (p.ksplit > 1 ? 4u : 2u)), 0x00020000);
    for (int it = wave; it < outs; it += nw) {
        const int w = it & (wn - 1), j = (it >> p.wnl) / MT, m = (it >> p.wnl) % MT;
        auto total = [&](int jj) {
            v4i x = red[((w * NT + jj) * MT + m) * 64 + lane];
            for (int s = 1; s < wk; ++s) x += red[(((s * wn + w) * NT + jj) * MT + m) * 64 + lane];
            return x;
        };
        const int t = (bx * wn + w) * nt + j;
        if (t >= otiles) continue;
        const v4i x = total(j);
        const uint32_t at = (uint32_t)(16 * m + l16) * (uint32_t)ldc + 16 * t + 4 * q;
        if (p.ksplit > 1) {
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), out, 4 * at, 0, 0);
            continue;
        }
        float a = as[0];
#pragma unroll
        for (int i = 1; i < MT; ++i) a = m == i ? as[i] : a;
        const float *ws = p.ws + (int64_t)e * p.N + 16 * t + 4 * q;
        v4f y = i8_scale(x, a, *(const float4 *)ws);
        if (p.silu) y = i8_silu_mul(y, i8_scale(total(j + nt), a, *(const float4 *)(ws + p.N / 2)));
        __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(w4_v2u, w4_bf16x4(y)), out, 2 * at, 0, 0);
    }
}

// The sums of a K split, added and scaled.
__global__ __launch_bounds__(256) void k_i8_reduce(const int32_t *__restrict__ part, const float *__restrict__ as,
                                                   const float *__restrict__ ws, uint16_t *__restrict__ c, int64_t M,
                                                   int64_t N, int ksplit) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= M * N) return;
    v4i x = *(const v4i *)(part + i);
    for (int k = 1; k < ksplit; ++k) x += *(const v4i *)(part + k * M * N + i);
    *(uint2 *)(c + i) = w4_bf16x4(i8_scale(x, as[i / N], *(const float4 *)(ws + i % N)));
}

hipError_t launch_i8_reduce(const I8Args &a, int ksplit, hipStream_t s) {
    hipLaunchKernelGGL(k_i8_reduce, dim3((unsigned)((a.M * a.N / 4 + 255) / 256)), dim3(256), 0, s, a.part, a.as, a.ws,
                       a.c, a.M, a.N, ksplit);
    return hipGetLastError();
}

// ---- the launch of the least estimated time ------------------------------------
//
// Times in us, fitted to every launch of 2492 dense shapes (1 to 1200 rows, K and N from 256 to 14336) and 10354 of
// experts (4 to 256 of them, up to 4096 tokens, 128 to 4096 wide), in graphs, weights from memory, so that the launch
// picked is as little as possible behind the fastest of all: on 738 and 3101 other shapes 1.7% on average dense (10% at
// the 90th percentile, at most 44%), 1.3% with experts (8%, at most 50%).
//
// Streaming: a compute unit's busiest CTAs move W (weight blocks of 2 KiB) and A (activation blocks as large), and each of
// its turns is as long as a wave's slice.  A split adds its sums and the reduce launch.  E.g. one row of 4096 x 14336: 11.9 us
// in eight slices, 12.7 in four; of 4096 x 4096 5.4 and 6.1; 16 rows of 14336 x 4096 14.4 whole, 17.7 in two.
static double stream_us(const I8Cfg &c, int64_t M, int64_t K, int64_t N, int64_t E, bool silu, double blocks) {
    const int64_t C = K / 128, span = (C + c.ksplit - 1) / c.ksplit, cps = (span + c.wk - 1) / c.wk, tiles = N / 16;
    const int waves = c.wn * c.wk, per = (int)cps * (c.nt + c.mt);
    const int vgprs = c.mt == 1 ? (c.nt == 1 ? 80 : 120) : c.mt == 2 ? (c.nt == 1 ? 120 : 160) : 248;
    const double fit = std::max(1, std::min(8, 512 / vgprs * 4 / waves));  // CTAs that share a compute unit
    const int64_t cols = (tiles + c.nt * c.wn - 1) / (c.nt * c.wn);
    const double W = (double)(c.nt * c.wn * span), A = (double)(c.wn * c.mt * span), ctas = (double)(cols * c.ksplit) * blocks;
    if (E) {
        const int64_t RB = 16 * c.mt, grid = cols * ((M + std::min(E, M) * (RB - 1)) / RB);
        const double rounds = std::max(1.0, ctas / 256.0), turns = std::max(1.0, ctas / 256.0 / fit);
        const double us = 3.65 + 0.113 * waves + rounds * (W * (c.mt == 1 ? 0.0234 : 0.0738) + 0.0004 * A + 0.0283 * waves) +
                          turns * (0.192 * per + 0.148) + 0.05 * std::max(0.0, (double)grid - ctas) / 256.0;
        return std::max(us, 3.65 + 0.000389 * blocks * (double)(tiles * C)) + 0.1 * us;
    }
    const double rounds = std::ceil(ctas / 256.0), turns = std::ceil(ctas / 256.0 / fit);
    double us = 2.11 + 0.0046 * waves + turns * 0.0516 * per +
                rounds * (W * (c.mt == 1 ? 0.0346 : c.mt == 2 ? 0.0572 : 0.1345) + 0.0245 * A + 0.19);
    if (c.mt == 4 && c.wk == 8) us += 0.069;
    if (c.ksplit > 1) us += 2.96 + 0.43e-6 * (double)(c.ksplit * M * N);
    return us;
}

// Tiled: a stage takes `alone` where its CTA has the compute unit to itself and `shared` for each of those that share
// it, each tile its start and its outputs.  E.g. from codes 4096 x 4096 x 12288: 168 us in tiles of 256 x 256, 219 in 256 x 128,
// 244 in 128 x 128; 2048 x 4096 x 4096 48, 35, 41; 256 x 4096 x 4096 12.4 in 64 x 64, 18.8 in 64 x 128, 22.9 in 128 x 128;
// 100 x 4096 x 4096 11.5 in 64 x 64, streaming 14.1, and 64 rows 12.6 and 8.5; gate_up of 64 tokens, eight of 128 experts, 72
// in 128 x 64, 74 in 64 x 64, of 2048 tokens 108 in 256 x 256, 130 in 256 x 128, 124 in 128 x 128.
static double tiled_us(const I8TiledCfg &c, int64_t M, int64_t K, int64_t N, int64_t E, bool silu, double blocks) {
    static constexpr double dense[][3] = {{0.341, 0.0385, 3.3}, {0.243, 0.349, 1.27}, {0.238, 0.201, 1.05},
                                     {0.281, 0.244, 0.148}, {0.211, 0.15, 1.14}, {0.0993, 0.122, 0.746}};
    static constexpr double moe[][3] = {{0.154, 0.785, 5.89}, {0.3, 0.338, 3.03}, {0.0466, 0.18, 2.24},
                                   {0.149, 0.0774, 0.582}, {0.46, 0.322, 1.59}, {0.0694, 0.133, 0.64}};
    const int *t = I8_TILES[c.shape];
    const double *u = E ? moe[c.shape] : dense[c.shape], fit = t[2];
    const int64_t C = K / 128, stages = 2 * ((C + c.ksplit - 1) / c.ksplit);
    const double load = (double)((N + t[0] - 1) / t[0] * c.ksplit) * blocks / 256.0;
    const double busy = std::min(fit, E ? std::max(1.0, load) : std::ceil(load));
    const double seq = load <= 2.0 * fit ? std::max(1.0, std::ceil(load / fit)) : load / fit + 0.5;
    const double us = seq * ((double)stages * std::max(u[0], u[1] * busy) + u[2]);
    if (E) return 4.96 + 0.141 * seq + 0.1 * us + std::max(us, 2.05e-7 * (blocks * (double)(N * K) + (double)(M * (silu ? N : 2 * N))));
    return 2.76 + us + (c.ksplit > 1 ? 3.08 + 2.88e-6 * (double)(c.ksplit * M * N) : 0.0);
}

// 512-value units of the rows that the streaming kernel quantises itself: as many as its waves hold
static bool quant_fits(const I8Cfg &c, int64_t M, int64_t K) {
    return c.mt == 1 && c.ksplit == 1 && M <= 16 && M * ((K + 511) / 512) <= I8_QA_UNITS * c.wn * c.wk;
}

I8Plan i8_plan_new(int64_t M, int64_t K, int64_t N, int64_t E, bool silu, bool quant, bool wide) {
    const I8Tuning f = i8_tuning();
    const int64_t C = K / 128;
    I8Plan best{};
    double least = 0.0;
    auto blocks = [&](int64_t RB) { return E ? w4_expert_blocks(M, E, RB) : (double)((M + RB - 1) / RB); };
    auto offer = [&](const I8Plan &p, double us) {
        if (least == 0.0 || us < least) {
            best = p;
            least = us;
        }
    };
    // a split's sums stay below 2^32 bytes a row block
    const int64_t splits = E || N >= int64_t(1) << 22 ? 1 : std::min<int64_t>(C, 8);
    const bool forced = f.kernel && f.a;
    if (f.kernel != R9K_I8_TILED && !wide)
        for (const auto &s : I8_STREAMS) {
            const int nt = forced && silu ? std::max(f.a, 2) : f.a;
            if (forced && (s[0] != f.rows || s[1] != nt || s[2] != f.b || s[3] != f.c)) continue;
            // dense: one row tile up to 16 rows, two up to 64 and four above; up to 256 rows
            if (!forced && (E ? s[0] == 4 : s[2] != 1 || (s[0] == 1) != (M <= 16) || (s[0] == 4 && M <= 32) || (s[0] == 2 && M > 256))) continue;
            if (!forced && !f.kernel && M > (E ? 100 * E : 256)) continue;
            if (silu && s[1] == 1) continue;
            if (((M + 16 * s[0] - 1) / (16 * s[0]) + (E ? std::min(E, M) : 0)) > 65535) continue;  // the grid's
            const double items = blocks(16 * s[0]);
            for (int64_t ks = 1; ks <= std::min<int64_t>(splits, 4); ks *= 2) {
                I8Plan p{};
                int64_t want = f.kernel && f.ksplit && !E ? std::min<int64_t>(f.ksplit, N >= int64_t(1) << 22 ? 1 : C) : ks;
                const int64_t span = (C + want - 1) / want;
                p.cfg = I8Cfg{s[0], s[1], s[2], s[3], (int)((C + span - 1) / span)};  // no split without chunks
                // a split where one CTA a compute unit is not reached without it
                if (ks > 1 && !(f.kernel && f.ksplit) && (double)((N / 16 + s[1] * s[2] - 1) / (s[1] * s[2])) * items * (double)ks >= 512.0) break;
                p.fused = quant && !E && quant_fits(p.cfg, M, K);
                offer(p, stream_us(p.cfg, M, K, N, E, silu, items) + (quant && !p.fused ? 2.5 : 0.0));
            }
        }
    if (f.kernel != R9K_I8_STREAM || least == 0.0)
        for (int sh = 0; sh < I8_SHAPES; ++sh) {
            const int *t = I8_TILES[sh];
            if (f.kernel == R9K_I8_TILED && f.a ? t[0] != f.a || t[1] != f.b : !f.kernel && !E && M <= 16 && least != 0.0) continue;
            if (!f.kernel && !E && t[1] >= 4 * M && least != 0.0) continue;  // mostly rows that are not there
            const double items = blocks(t[1]);
            for (int64_t ks = 1; ks <= splits; ks *= 2) {
                I8Plan p{};
                p.tile = true;
                p.tiled = I8TiledCfg{sh, (int)(f.kernel == R9K_I8_TILED && f.ksplit && !E ? std::min<int64_t>(f.ksplit, splits == 1 ? 1 : C) : ks)};
                if (ks > 1 && (double)((N + t[0] - 1) / t[0] * ks) * items > 600.0) break;
                offer(p, tiled_us(p.tiled, M, K, N, E, silu, items) + (quant ? 2.5 : 0.0));
            }
        }
    return best;
}

template <int MT, int NT, bool LONG, bool QA>
static hipError_t launch_one(I8Args a, const I8Cfg &c, hipStream_t s) {
    constexpr int D = 4;
    const int64_t C = a.K / 128, RB = 16 * MT;
    const int64_t per = (int64_t)c.wn * (a.silu ? NT / 2 : NT), tiles = a.N / 16 / (a.silu ? 2 : 1);
    const int64_t nblk = (tiles + per - 1) / per;
    int64_t items = (a.M + RB - 1) / RB;
    if (a.offsets) items = (a.M + std::min(a.E, a.M) * (RB - 1)) / RB;
    a.wnl = __builtin_ctz((unsigned)c.wn);
    a.ksplit = c.ksplit;
    a.span = (int)((C + c.ksplit - 1) / c.ksplit);
    a.cps = (a.span + c.wk - 1) / c.wk;
    a.tmagic = a.topk > 1 ? (uint32_t)(((uint64_t(1) << 32) + a.topk - 1) / a.topk) : 0;
    size_t lds = (size_t)c.wn * c.wk * NT * MT * 1024;
    if (QA) lds = std::max(lds, (size_t)(a.M * (a.K + 16) + a.M * ((a.K + 511) / 512) * 4 + a.M * 4));
    if (nblk > 0x7fffffff / 1024 || items > 65535 || lds > 64 * 1024) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_gemm_i8<MT, NT, D, LONG, QA>), dim3((unsigned)nblk, (unsigned)items, (unsigned)c.ksplit),
                       dim3(64 * c.wn * c.wk), lds, s, a);
    return hipGetLastError();
}
template <int MT, int NT>
static hipError_t launch_nt(const I8Args &a, const I8Cfg &c, hipStream_t s) {
    const int64_t C = a.K / 128, span = (C + c.ksplit - 1) / c.ksplit;
    const bool longer = (span + c.wk - 1) / c.wk > 4;
    if constexpr (MT == 1) {
        if (a.a) return longer ? launch_one<1, NT, true, true>(a, c, s) : launch_one<1, NT, false, true>(a, c, s);
    }
    return longer ? launch_one<MT, NT, true, false>(a, c, s) : launch_one<MT, NT, false, false>(a, c, s);
}
template <int MT>
static hipError_t launch_mt(const I8Args &a, const I8Cfg &c, hipStream_t s) {
    return c.nt == 1 ? launch_nt<MT, 1>(a, c, s) : launch_nt<MT, 2>(a, c, s);
}

hipError_t launch_gemm_i8(const I8Args &a, const I8Cfg &c, hipStream_t s) {
    const hipError_t err = c.mt == 1 ? launch_mt<1>(a, c, s) : c.mt == 2 ? launch_mt<2>(a, c, s) : launch_nt<4, 2>(a, c, s);
    if (err != hipSuccess || c.ksplit == 1) return err;
    return launch_i8_reduce(a, c.ksplit, s);
}

}  // namespace r9k
