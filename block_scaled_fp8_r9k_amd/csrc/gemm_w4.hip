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

#include "r9k_internal.h"
#include "w4_device.h"

namespace r9k {

namespace {

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
    const int C = (int)(p.K / 128), tiles = (int)(p.N / 16);
    const int bx = blockIdx.x % p.nblk, item = blockIdx.x / p.nblk;

    // rows [r0, r1) of this CTA, of expert e
    int64_t r0, r1;
    int e = 0;
    if (p.offsets) {
        int a0, a1;
        if (!w4_find_block(p.offsets, (int)p.E, (int)p.M, 16 * MT, item, e, a0, a1)) return;
        r0 = a0;
        r1 = min(a1, a0 + 16 * MT);
    } else {
        r0 = (int64_t)item * 16 * MT;
        r1 = min<int64_t>(p.M, r0 + 16 * MT);
    }
    r0 = __builtin_amdgcn_readfirstlane((int)r0);
    r1 = __builtin_amdgcn_readfirstlane((int)r1);
    e = __builtin_amdgcn_readfirstlane(e);

    // column tiles; those past the last repeat it and are not stored
    int tile[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        if (p.silu) {
            const int half = tiles / 2, u = bx * (NT / 2) + j % (NT / 2);
            tile[j] = min(u, half - 1) + (j < NT / 2 ? 0 : half);
        } else {
            tile[j] = min(bx * NT + j, tiles - 1);
        }
    }

    // the lane's activation rows (past the last: the last again, never stored).
    // A row index that points outside the activations reads row 0.
    const uint16_t *arow[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        int64_t r = min<int64_t>(r0 + 16 * m + l16, r1 - 1);
        if (p.src) {
            r = (int64_t)((uint32_t)p.src[r] / (uint32_t)p.topk);
            r = r < p.arows ? r : 0;
        }
        arow[m] = p.a + r * p.K + 8 * q;
    }

    const int cb = (int)((int64_t)wave * C / nw), ce = (int)((int64_t)(wave + 1) * C / nw);
    // Weights through one descriptor a tile, which ends with the wave's slice:
    // loads ahead of the end return zeros and move nothing.
    __amdgpu_buffer_rsrc_t wd[NT];
    const uint8_t *sb[NT];
    const uint8_t *zb[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int64_t t0 = ((int64_t)e * tiles + tile[j]) * C;  // the tile's first chunk
        wd[j] = __builtin_amdgcn_make_buffer_rsrc((void *)(p.wp + t0 * 1024), (short)0, ce * 1024, 0x00020000);
        sb[j] = (const uint8_t *)p.sp + t0 * (FMT == W4_MXFP4 ? 64 : 32 * NG) + (FMT == W4_MXFP4 ? 4 * l16 : 8 * NG * q);
        zb[j] = p.zp + t0 * 16 * NG + 4 * NG * q;
    }

    uint4 wr[D][NT], ar[D][MT][4];
    W4Scale<FMT, NG> sc[D][NT];
    auto load = [&](int c, int d) {
#pragma unroll
        for (int j = 0; j < NT; ++j) wr[d][j] = load_buf_nt16(wd[j], 16 * lane + c * 1024);
        const int cc = min(c, ce - 1);  // the other loads stay inside the slice
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
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int k = 0; k < 4; ++k) ar[d][m][k] = *(const uint4 *)(arow[m] + (int64_t)cc * 128 + 32 * k);
    };

    v4f acc[NT][MT];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[j][m] = v4f{0.f, 0.f, 0.f, 0.f};

    auto compute = [&](int d) {
        if constexpr (FMT == W4_MXFP4) {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const uint32_t word[4] = {wr[d][j].x, wr[d][j].y, wr[d][j].z, wr[d][j].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float s = __uint_as_float(((sc[d][j].s[0] >> (8 * k)) & 255u) << 23);
                    const w4_v8bf wf = w4_fp4_frag(word[k], s);
#pragma unroll
                    for (int m = 0; m < MT; ++m) acc[j][m] = w4_mfma(wf, w4_frag(ar[d][m][k]), acc[j][m]);
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
                    for (int k = 0; k < KPG; ++k) sum[i][m] = w4_mfma(w4_ones(), w4_frag(ar[d][m][i * KPG + k]), sum[i][m]);
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
                        for (int m = 0; m < MT; ++m) pr[m] = w4_mfma(wf, w4_frag(ar[d][m][i * KPG + k]), pr[m]);
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

    if (cb < ce) {
#pragma unroll
        for (int d = 0; d < D; ++d) load(cb + d, d);
        __builtin_amdgcn_sched_barrier(0);
        for (int c = cb; c < ce; c += D) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                if (c + d < ce) compute(d);
                if (c + d + D < ce) load(c + d + D, d);
            }
        }
    }

#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int m = 0; m < MT; ++m) pin_acc(acc[j][m]);  // the MFMAs run with every lane enabled

    // sum the K slices in ascending order; an item is a lane's four columns of a tile pair
    v4f *red = (v4f *)lds;  // [wave][tile][row tile][lane]
    if (nw > 1) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int m = 0; m < MT; ++m) red[((wave * NT + j) * MT + m) * 64 + lane] = acc[j][m];
        __syncthreads();
    }
    const int64_t ldc = p.silu ? p.N / 2 : p.N;
    const int outs = (p.silu ? NT / 2 : NT) * MT;
    for (int it = wave; it < outs; it += nw) {
        const int j = it / MT, m = it % MT;
        auto total = [&](int jj) {
            v4f x = {0.f, 0.f, 0.f, 0.f};
            if (nw > 1) {
                x = red[(jj * MT + m) * 64 + lane];
                for (int s = 1; s < nw; ++s) x += red[((s * NT + jj) * MT + m) * 64 + lane];
            } else {
#pragma unroll
                for (int a = 0; a < NT; ++a)
#pragma unroll
                    for (int b = 0; b < MT; ++b)
                        if (a == jj && b == m) x = acc[a][b];
            }
            return x;
        };
        v4f x = total(j);
        int t = bx * NT + j;
        bool live = t < tiles;
        if (p.silu) {
            const v4f u = total(j + NT / 2);
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] = w4_silu_mul(x[r], u[r]);
            t = bx * (NT / 2) + j;
            live = t < tiles / 2;
        }
        const int64_t r = r0 + 16 * m + l16;
        if (live && r < r1) *(uint2 *)(p.c + r * ldc + 16 * t + 4 * q) = w4_bf16x4(x);
    }
}

// Rows a block and tiles a wave.  [first version: one rule for every shape]
W4Cfg w4_config(const W4Args &a) {
    W4Cfg c;
    const int64_t rows = a.offsets ? (a.M + a.E - 1) / a.E : a.M;
    c.mt = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
    c.nt = 2;
    c.nw = (int)std::min<int64_t>(8, a.K / 128);
    return c;
}

template <int FMT, int GRP, int MT>
static hipError_t launch_mt(W4Args a, const W4Cfg &c, hipStream_t s) {
    constexpr int NT = 2;
    const int64_t tiles = a.N / 16;
    a.nblk = (int)(a.silu ? (tiles / 2 + NT / 2 - 1) / (NT / 2) : (tiles + NT - 1) / NT);
    const int64_t RB = 16 * MT;
    int64_t items = (a.M + RB - 1) / RB;
    if (a.offsets) items = (a.M + std::min(a.E, a.M) * (RB - 1)) / RB;
    if (items * a.nblk > 0x7fffffff) return hipErrorInvalidValue;
    const size_t lds = c.nw > 1 ? (size_t)c.nw * NT * MT * 1024 : 0;
    hipLaunchKernelGGL((k_gemm_w4<FMT, GRP, MT, NT, 2, 512>), dim3((unsigned)(items * a.nblk)), dim3(64 * c.nw), lds, s, a);
    return hipGetLastError();
}

template <int FMT, int GRP>
static hipError_t launch_fmt(const W4Args &a, hipStream_t s) {
    const W4Cfg c = w4_config(a);
    switch (c.mt) {
        case 1: return launch_mt<FMT, GRP, 1>(a, c, s);
        case 2: return launch_mt<FMT, GRP, 2>(a, c, s);
        default: return launch_mt<FMT, GRP, 4>(a, c, s);
    }
}

hipError_t launch_gemm_w4(const W4Args &a, int fmt, int grp, hipStream_t s) {
    if (fmt == W4_MXFP4) return launch_fmt<W4_MXFP4, 32>(a, s);
    switch (grp) {
        case 32: return launch_fmt<W4_INT, 32>(a, s);
        case 64: return launch_fmt<W4_INT, 64>(a, s);
        default: return launch_fmt<W4_INT, 128>(a, s);
    }
}

}  // namespace r9k
