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
// For expert products the rows are ranges of `offsets`, one per expert; a CTA
// finds its expert and row block there (the grid covers the most blocks that R
// rows can make), and may read its activation rows through the sort's index.
// With silu the first half of a wave's tiles are gate columns, the second half
// the up columns that belong to them.
#include <algorithm>
#include <mutex>

#include "r9k_internal.h"
#include "w4_device.h"

namespace r9k {

namespace {

// LDS that a CTA's activation rows may take
constexpr int64_t W4_LDS = 150 * 1024;

// The lane's scales (and zeros) of one tile's chunk, as loaded.
template <int FMT, int NG>
struct W4Scale {
    uint32_t s[FMT == W4_MXFP4 ? 1 : 2 * NG];  // int4: 4 rows x NG groups of bf16; mxfp4: 4 bytes, one a group
    uint32_t z[FMT == W4_MXFP4 ? 1 : NG];      // int4: 4 rows x NG groups of bytes
};

}  // namespace

template <int FMT, int GRP, int MT, int NT, int D, int NTHR>
__global__ __launch_bounds__(NTHR) void k_gemm_w4(W4Args p) {
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

    v4f acc[NT][MT];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[j][m] = v4f{0.f, 0.f, 0.f, 0.f};

    uint4 wr[D][NT];
    W4Scale<FMT, NG> sc[D][NT];
    const uint8_t *al[MT];
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(lds));

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
                            const float z = (float)((sc[d][j].z[i] >> (8 * r)) & 255u);
                            acc[j][m][r] = __builtin_fmaf(s[r], __builtin_fmaf(-z, sum[i][m][0], pr[m][r]), acc[j][m][r]);
                        }
                }
            }
        }
    };

    // Segments of p.seg chunks, whose activation rows fit LDS (all of the CTA's
    // chunks where they do); a wave takes its slice [cb, ce) of each.
    for (int s0 = kb; s0 < ke; s0 += p.seg) {
        const int s1 = min(ke, s0 + p.seg);
        const int cb = min(s1, s0 + slice * p.cps), ce = min(s1, cb + p.cps);

        // 1. the rows into LDS, padded by 16 bytes so that the 16 rows of a fragment
        // read fall on distinct banks; a wave moves 64 16-byte pieces of a row at a
        // time, straight into LDS.  A row index that points outside the activations
        // reads row 0.
        const int ppr = (s1 - s0) * 16;  // pieces a row
        const int bpr = (s1 - s0 + 3) >> 2, blocks = rows * bpr, pitch = ppr * 16 + 16;
        if (s0 > kb) __syncthreads();  // every wave is done with the segment before
        for (int i = wave; i < blocks; i += nw) {
            // bmagic = ceil(2^20 / bpr) of a whole segment
            const int r = s1 - s0 == p.seg ? (int)((uint32_t)i * p.bmagic >> 20) : i / bpr;
            const int c0 = (i - r * bpr) * 64;
            int64_t row = r0 + r;
            if (p.src) {
                const uint32_t t = w4_div_topk((uint32_t)p.src[row], (uint32_t)p.topk, p.tmagic);
                row = t < (uint32_t)p.arows ? t : 0;
            }
            if (c0 + lane < ppr) load_lds16(p.a + row * p.K + s0 * 128 + 8 * (c0 + lane), lds0 + r * pitch + c0 * 16);
        }
        __builtin_amdgcn_sched_barrier(0);

        // 2. the weight stream, through one descriptor a tile that ends with the
        // slice: loads past the end return zeros and move nothing
        __amdgpu_buffer_rsrc_t wd[NT];
        const uint8_t *sb[NT];
        const uint8_t *zb[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int64_t t0 = ((int64_t)e * tiles + tile[j]) * C;  // the tile's first chunk
            wd[j] = __builtin_amdgcn_make_buffer_rsrc((void *)(p.wp + t0 * 1024), (short)0, ce * 1024, 0x00020000);
            sb[j] = (const uint8_t *)p.sp + t0 * (FMT == W4_MXFP4 ? 64 : 32 * NG) +
                    (FMT == W4_MXFP4 ? 4 * l16 : 8 * NG * q);
            zb[j] = p.zp + t0 * 16 * NG + 4 * NG * q;
        }
        auto load = [&](int c, int d) {
            const int cc = max(min(c, ce - 1), 0);  // the scales' loads stay inside the weight
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                if constexpr (FMT == W4_MXFP4) {
                    sc[d][j].s[0] = *(const uint32_t *)(sb[j] + (int64_t)cc * 64);
                } else {
                    const uint2 *s2 = (const uint2 *)(sb[j] + (int64_t)cc * 32 * NG);
#pragma unroll
                    for (int i = 0; i < NG; ++i) {
                        sc[d][j].s[2 * i] = s2[i].x;
                        sc[d][j].s[2 * i + 1] = s2[i].y;
                    }
                    if (p.zp) {
#pragma unroll
                        for (int i = 0; i < NG; ++i)
                            sc[d][j].z[i] = *(const uint32_t *)(zb[j] + (int64_t)cc * 16 * NG + 4 * i);
                    } else {
#pragma unroll
                        for (int i = 0; i < NG; ++i) sc[d][j].z[i] = 0x08080808u;
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) wr[d][j] = load_buf_nt16(wd[j], 16 * lane + c * 1024);
        };
#pragma unroll
        for (int d = 0; d < D; ++d) load(cb + d, d);
        __builtin_amdgcn_sched_barrier(0);

        // the rows have landed once at most the D * NT code loads behind them are in flight
        wait_vm<D * NT>();
        __syncthreads();
#pragma unroll
        for (int m = 0; m < MT; ++m) al[m] = lds + min(16 * m + l16, rows - 1) * pitch + 16 * q;

        for (int c = cb; c < ce; c += D) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                if (c + d < ce) compute(c + d - s0, d);
                if (c + d + D < ce) load(c + d + D, d);
            }
        }
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
        const int r = 16 * m + l16;
        if (t < otiles && r < rows) {
            const int64_t at = (int64_t)(r0 + r) * ldc + 16 * t + 4 * q;
            if (p.ksplit > 1) *(v4f *)(p.part + (int64_t)ks * p.M * p.N + at) = x;
            else *(uint2 *)(p.c + at) = w4_bf16x4(x);
        }
    }
}

// [first version: one rule for every shape]
W4Cfg w4_config(int64_t M, int64_t K, int64_t N, int64_t E, bool silu) {
    W4Cfg c;
    const int64_t rows = E ? (M + E - 1) / E : M, C = K / 128;
    c.mt = rows <= 16 ? 1 : 2;
    c.nt = 2;
    c.wn = 1;
    c.wk = 8;
    c.ksplit = 1;
    const int *f = tuning().w4;
    if (f[0]) c.nt = f[0];
    if (f[1]) c.wn = f[1];
    if (f[2]) c.wk = f[2];
    if (f[3] && !E) c.ksplit = f[3];
    if (silu && c.nt == 1) c.nt = 2;
    c.ksplit = (int)std::min<int64_t>(c.ksplit, C);
    const int64_t most = std::min<int64_t>(M, 16 * c.mt), span = (C + c.ksplit - 1) / c.ksplit;
    const int64_t fit = std::max<int64_t>(1, (W4_LDS / most - 16) / 256);  // chunks of a segment
    c.seg = (int)(span <= fit ? span : (span + (span + fit - 1) / fit - 1) / ((span + fit - 1) / fit));
    c.ksplit = (int)((C + span - 1) / span);  // no split without chunks
    c.wk = (int)std::min<int64_t>(c.wk, c.seg);
    const int waves = c.mt == 1 ? 16 : 8;
    while (c.wn > waves || (c.wn & (c.wn - 1))) --c.wn;
    c.wk = std::min(c.wk, waves / c.wn);
    return c;
}

template <int FMT, int GRP, int MT, int NT, int NTHR>
static hipError_t launch_one(W4Args a, const W4Cfg &c, hipStream_t s) {
    // chunks ahead: as many registers as two waves a SIMD leave, scales included
    constexpr int D = (GRP == 32 && FMT == W4_INT ? 4 : 8) / NT;
    auto kernel = k_gemm_w4<FMT, GRP, MT, NT, D, NTHR>;
    static std::once_flag once[64];
    static hipError_t attr_err[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return hipErrorInvalidDevice;
    std::call_once(once[dev], [&] {
        attr_err[dev] = hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
    });
    if (attr_err[dev] != hipSuccess) return attr_err[dev];
    const int64_t per = (int64_t)c.wn * (a.silu ? NT / 2 : NT), tiles = a.N / 16 / (a.silu ? 2 : 1);
    const int64_t RB = 16 * MT;
    int64_t items = (a.M + RB - 1) / RB;
    if (a.offsets) items = (a.M + std::min(a.E, a.M) * (RB - 1)) / RB;
    const int64_t nblk = (tiles + per - 1) / per, C = a.K / 128;
    a.wnl = __builtin_ctz((unsigned)c.wn);
    a.ksplit = c.ksplit;
    a.span = (int)((C + c.ksplit - 1) / c.ksplit);
    a.seg = std::min(c.seg, a.span);
    a.cps = (a.seg + c.wk - 1) / c.wk;
    const int bpr = (a.seg + 3) / 4;
    a.bmagic = (uint32_t)(((1 << 20) + bpr - 1) / bpr);
    a.tmagic = a.topk > 1 ? (uint32_t)(((uint64_t(1) << 32) + a.topk - 1) / a.topk) : 0;
    const size_t rows = (size_t)std::min<int64_t>(a.M, RB) * (size_t)(c.seg * 256 + 16);
    const size_t lds = std::max<size_t>(rows, (size_t)c.wn * c.wk * NT * MT * 1024);
    if (nblk > 0x7fffffff || items > 65535 || lds > 160 * 1024 || 64 * c.wn * c.wk > NTHR) return hipErrorInvalidValue;
    hipLaunchKernelGGL(kernel, dim3((unsigned)nblk, (unsigned)items, (unsigned)c.ksplit), dim3(64 * c.wn * c.wk), lds, s, a);
    return hipGetLastError();
}

template <int FMT, int GRP, int MT>
static hipError_t launch_mt(const W4Args &a, const W4Cfg &c, hipStream_t s) {
    if constexpr (MT == 1)
        if (c.wn * c.wk > 8)
            return c.nt == 1 ? launch_one<FMT, GRP, MT, 1, 1024>(a, c, s) : launch_one<FMT, GRP, MT, 2, 1024>(a, c, s);
    return c.nt == 1 ? launch_one<FMT, GRP, MT, 1, 512>(a, c, s) : launch_one<FMT, GRP, MT, 2, 512>(a, c, s);
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
