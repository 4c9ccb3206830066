// Products with 4-bit weights, many rows: the LDS-tiled MFMA kernel.
//
// The same sums as the weight-streaming kernel (gemm_w4.hip), for row counts at
// which the matrix instructions and not the weight bytes set the time.  C^T = W
// A^T: each wave owns TN column tiles by four row tiles of 16; a CTA is 4 waves
// along the columns by WM along the rows, 64 TN columns by 64 WM rows.
//
// Per chunk of 128 K a stage in LDS holds the A tile (bf16), the packed codes of
// the column tiles and their scales, all moved there by global_load_lds, NST - 1
// chunks ahead.  A wave converts its codes to bf16 fragments once a chunk, in
// registers, and uses them for its four row tiles.
//   int4: a group's product P starts from zero and is promoted into the fp32 sum
//   by acc += s * P, so neither the weights nor the sums are rounded.  The zero
//   points are not in the loop: sum_g z s S_g (S_g the sum of a group's activations)
//   is itself a matrix product with K / group terms, and goes into the sums first,
//   on the matrix cores: s z holds 12 bits, two bf16; S_g, fp32, is three; the six
//   products are exact and take six of a lane quarter's eight K positions, four
//   groups to an instruction.  S_g comes from a launch of its own (k_w4_sums), one
//   pass over the activations.
//   mxfp4: the scale is in the converted fragment (a power of two, exact) and the
//   matrix instruction accumulates through all of K.
// A rows are 256 bytes in LDS; 16-byte piece p of row r lies at piece p ^ (r % 16),
// so that the 16 rows of a fragment read fall on distinct banks.
#include <algorithm>
#include <mutex>

#include "r9k_internal.h"
#include "w4_device.h"

namespace r9k {

// Sums of each group's activations, fp32: sums[row][g], rows padded with zeros to
// a multiple of four groups.
__global__ __launch_bounds__(256) void k_w4_sums(const uint4 *__restrict__ a, int64_t n8, int k8, int grp, int G,
                                                 int G4, float *__restrict__ sums) {
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= n8) return;  // whole rows of 16 lanes and more: a group's lanes leave together
    const uint4 v = a[id];
    float s = ((bf16_lo(v.x) + bf16_hi(v.x)) + (bf16_lo(v.y) + bf16_hi(v.y))) +
              ((bf16_lo(v.z) + bf16_hi(v.z)) + (bf16_lo(v.w) + bf16_hi(v.w)));
    const int lanes = grp / 8;
    for (int d = 1; d < lanes; d <<= 1) s += __shfl_xor(s, d, 64);
    if ((threadIdx.x & (lanes - 1)) == 0) {
        const int64_t row = id / k8;
        const int g = (int)(id % k8) * 8 / grp;
        sums[row * G4 + g] = s;
        if (g == G - 1)
            for (int p = G; p < G4; ++p) sums[row * G4 + p] = 0.0f;
    }
}

namespace {
template <int FMT, int GRP, int TN_, int WM_, int NST_>
struct W4Tile {
    static constexpr int TN = TN_, WM = WM_, NST = NST_, NW = 4 * WM, THREADS = 64 * NW;
    static constexpr int NG = 128 / GRP, KPG = GRP / 32;
    static constexpr int BM = 64 * WM;
    static constexpr int ABYTES = BM * 256, WBYTES = 4 * TN * 1024;
    static constexpr int SDW = FMT == W4_MXFP4 ? 16 * TN : 8 * NG * TN;  // dwords of a wave's scales
    static constexpr int SLOADS = (SDW + 63) / 64, SBYTES = SLOADS * 256;
    static constexpr int STAGE = ABYTES + WBYTES + NW * SBYTES;
    static constexpr int WLOADS = 4 * TN / NW, ALOADS = 4;
    static constexpr int LOADS = WLOADS + ALOADS + SLOADS;  // load instructions a wave and stage
    static constexpr int CPITCH = 64 * TN * 2 + 16;         // output tile rows in LDS
    static constexpr int SMEM = NST * STAGE > BM * CPITCH ? NST * STAGE : BM * CPITCH;
    static_assert(WLOADS * NW == 4 * TN, "loads split evenly");
    static_assert(SMEM <= 160 * 1024, "LDS");
};

__device__ __forceinline__ uint32_t hi16(float lo, float hi) {  // upper halves of two fp32
    return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}
}  // namespace

template <int FMT, int GRP, class T>
__global__ __launch_bounds__(T::THREADS, 2) void k_gemm_w4_tiled(W4Args p) {
    constexpr int TN = T::TN, NG = T::NG, KPG = T::KPG, NST = T::NST, BM = T::BM;
    extern __shared__ __align__(16) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave & 3, wm = wave >> 2;
    const int C = (int)(p.K / 128), tiles = (int)(p.N / 16);

    // block -> (column block, row block).  Blocks go round-robin to the 8 XCDs.
    // Dense: an XCD takes a contiguous range, walked eight row blocks at a time, so
    // that what runs together shares A and W in its L2.  Experts: an XCD takes
    // every eighth row block, with all its column blocks (the blocks past the last
    // are then spread over the XCDs).
    int bx, by;
    if (p.offsets) {
        const int j = blockIdx.x >> 3;
        by = (j / p.nblk) * 8 + (blockIdx.x & 7);
        bx = j % p.nblk;
    } else {
        const int total = p.nblk * p.nrow;
        int lid = blockIdx.x;
        if (total % 8 == 0) lid = (blockIdx.x & 7) * (total / 8) + (blockIdx.x >> 3);
        const int per = 8 * p.nblk, first = lid / per * 8, rows = min(8, p.nrow - first), in = lid % per;
        by = first + in % rows;
        bx = in / rows;
    }

    int e = 0, r0, r1;
    if (p.offsets) {
        int a0, a1;
        if (!w4_find_block(p.offsets, (int)p.E, (int)p.M, BM, by, e, a0, a1)) return;
        r0 = a0;
        r1 = min(a1, a0 + BM);
    } else {
        r0 = by * BM;
        r1 = (int)min<int64_t>(p.M, (int64_t)r0 + BM);
    }
    e = __builtin_amdgcn_readfirstlane(e);
    r0 = __builtin_amdgcn_readfirstlane(r0);
    r1 = __builtin_amdgcn_readfirstlane(r1);
    const int ks = blockIdx.y;
    const int cb = (int)((int64_t)ks * C / p.ksplit), ce = (int)((int64_t)(ks + 1) * C / p.ksplit);

    // column tile j of wave column w; those past the last repeat it and are not stored
    auto col_tile = [&](int w, int j) {
        if (p.silu) {
            if constexpr (TN > 1) {
                const int u = (bx * 4 + w) * (TN / 2) + j % (TN / 2);
                return min(u, tiles / 2 - 1) + (j < TN / 2 ? 0 : tiles / 2);
            }
        }
        return min((bx * 4 + w) * TN + j, tiles - 1);
    };
    auto source_row = [&](int r) -> int64_t {  // activation row of output row r (clamped to the block)
        const int rr = min(r, r1 - 1);
        if (!p.src) return rr;
        const uint32_t t = w4_div_topk((uint32_t)p.src[rr], (uint32_t)p.topk, p.tmagic);
        return t < (uint32_t)p.arows ? t : 0;
    };

    // this wave's share of a stage's loads
    const uint8_t *ap[T::ALOADS], *wp[T::WLOADS], *sp[T::SLOADS];
#pragma unroll
    for (int u = 0; u < T::ALOADS; ++u) {
        const int row = 4 * (T::ALOADS * wave + u) + q;  // 4 rows of 16 pieces an instruction
        ap[u] = (const uint8_t *)p.a + source_row(r0 + row) * p.K * 2 + cb * 256 + 16 * (l16 ^ (row & 15));
    }
#pragma unroll
    for (int u = 0; u < T::WLOADS; ++u) {
        const int idx = T::WLOADS * wave + u;
        wp[u] = p.wp + (((int64_t)e * tiles + col_tile(idx / TN, idx % TN)) * C + cb) * 1024 + 16 * lane;
    }
#pragma unroll
    for (int u = 0; u < T::SLOADS; ++u) {
        constexpr int DPT = T::SDW / TN;  // dwords a tile
        const int d = min(64 * u + lane, T::SDW - 1);
        sp[u] = (const uint8_t *)p.sp + (((int64_t)e * tiles + col_tile(wn, d / DPT)) * C + cb) * (4 * DPT) + 4 * (d % DPT);
    }
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(lds));
    auto issue = [&](int st) {
        const uint32_t base = lds0 + st * T::STAGE;
#pragma unroll
        for (int u = 0; u < T::WLOADS; ++u) {
            load_lds16(wp[u], base + T::ABYTES + (T::WLOADS * wave + u) * 1024);
            wp[u] += 1024;
        }
#pragma unroll
        for (int u = 0; u < T::ALOADS; ++u) {
            load_lds16(ap[u], base + (T::ALOADS * wave + u) * 1024);
            ap[u] += 256;
        }
#pragma unroll
        for (int u = 0; u < T::SLOADS; ++u) {
            load_lds4(sp[u], base + T::ABYTES + T::WBYTES + wave * T::SBYTES + u * 256);
            sp[u] += 4 * (T::SDW / TN);
        }
    };

    v4f acc[TN][4];
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int m = 0; m < 4; ++m) acc[j][m] = v4f{0.f, 0.f, 0.f, 0.f};

    if constexpr (FMT == W4_INT) {
        // acc -= sum_g (s z)[n][g] * S[m][g]; lane: row l16 of either operand, group 4 i + q
        const float *srow[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) srow[m] = p.sums + source_row(r0 + 64 * wm + 16 * m + l16) * p.g4 + q;
        const int g0 = cb * NG, g1 = ce * NG;
        for (int i = g0 / 4; 4 * i < g1; ++i) {
            const int g = 4 * i + q;
            const bool mine = g >= g0 && g < g1;
            w4_v8bf sf[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const float s = srow[m][4 * i];
                const float h = __uint_as_float(__float_as_uint(s) & 0xFFFF0000u), d = s - h;
                const float mm = __uint_as_float(__float_as_uint(d) & 0xFFFF0000u), l = d - mm;
                sf[m] = __builtin_bit_cast(w4_v8bf, w4_v4u{hi16(h, mm), hi16(l, h), hi16(mm, l), 0});
            }
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int64_t at = ((((int64_t)e * tiles + col_tile(wn, j)) * C + min(g / NG, C - 1)) * 4 + (l16 >> 2)) * NG * 4 +
                                   (g % NG) * 4 + (l16 & 3);
                const float s = __uint_as_float((uint32_t)((const uint16_t *)p.sp)[at] << 16);
                const float z = p.zp ? (float)p.zp[at] : 8.0f;
                const float f = mine ? -s * z : 0.0f;
                const float h = __uint_as_float(__float_as_uint(f) & 0xFFFF0000u), l = f - h;
                const w4_v8bf wf = __builtin_bit_cast(w4_v8bf, w4_v4u{hi16(h, h), hi16(h, l), hi16(l, l), 0});
#pragma unroll
                for (int m = 0; m < 4; ++m) acc[j][m] = w4_mfma(wf, sf[m], acc[j][m]);
            }
        }
    }

    // fragment addresses inside a stage: row tile m, step k at (aoff ^ 64 k) + 4096 m
    const int aoff = (64 * wm + l16) * 256 + ((q ^ l16) << 4);
    const int woff = T::ABYTES + wn * TN * 1024 + 16 * lane;
    const int soff = T::ABYTES + T::WBYTES + wave * T::SBYTES;

    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // from here on only the stages' loads are counted
#pragma unroll
    for (int k = 0; k < NST - 1; ++k)
        if (cb + k < ce) issue(k);
    int st = 0;
    for (int c = cb; c < ce; ++c) {
        // this chunk's stage has landed: the wave's loads issued after it are those of chunk c + 1 (three stages)
        if (NST == 3 && c + 1 < ce) wait_vm<T::LOADS>();
        else wait_vm<0>();
        __syncthreads();
        if (c + NST - 1 < ce) issue(st == 0 ? NST - 1 : st - 1);
        const uint8_t *sb = lds + st * T::STAGE;
        st = st + 1 == NST ? 0 : st + 1;

        if constexpr (FMT == W4_MXFP4) {
            uint4 code[TN];
            uint32_t sc[TN];
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                code[j] = *(const uint4 *)(sb + woff + 1024 * j);
                sc[j] = *(const uint32_t *)(sb + soff + 64 * j + 4 * l16);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                w4_v8bf af[4];
#pragma unroll
                for (int m = 0; m < 4; ++m) af[m] = w4_frag(*(const uint4 *)(sb + (aoff ^ (64 * k)) + 4096 * m));
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    const uint32_t word[4] = {code[j].x, code[j].y, code[j].z, code[j].w};
                    const w4_v8bf wf = w4_fp4_frag(word[k], __uint_as_float(((sc[j] >> (8 * k)) & 255u) << 23));
#pragma unroll
                    for (int m = 0; m < 4; ++m) acc[j][m] = w4_mfma(wf, af[m], acc[j][m]);
                }
            }
        } else {
            uint4 code[TN];
#pragma unroll
            for (int j = 0; j < TN; ++j) code[j] = *(const uint4 *)(sb + woff + 1024 * j);
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                w4_v8bf wf[TN][KPG];
                float s[TN][4];
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    const uint32_t word[4] = {code[j].x, code[j].y, code[j].z, code[j].w};
#pragma unroll
                    for (int k = 0; k < KPG; ++k) wf[j][k] = w4_int_frag(word[i * KPG + k]);
                    const uint2 s2 = *(const uint2 *)(sb + soff + 32 * NG * j + 8 * NG * q + 8 * i);
                    s[j][0] = bf16_lo(s2.x);
                    s[j][1] = bf16_hi(s2.x);
                    s[j][2] = bf16_lo(s2.y);
                    s[j][3] = bf16_hi(s2.y);
                }
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    w4_v8bf af[KPG];
#pragma unroll
                    for (int k = 0; k < KPG; ++k)
                        af[k] = w4_frag(*(const uint4 *)(sb + (aoff ^ (64 * (i * KPG + k))) + 4096 * m));
                    v4f pr[TN];
#pragma unroll
                    for (int j = 0; j < TN; ++j) pr[j] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int k = 0; k < KPG; ++k)
#pragma unroll
                        for (int j = 0; j < TN; ++j) pr[j] = w4_mfma(wf[j][k], af[k], pr[j]);
#pragma unroll
                    for (int j = 0; j < TN; ++j)
#pragma unroll
                        for (int r = 0; r < 4; ++r) acc[j][m][r] = __builtin_fmaf(s[j][r], pr[j][r], acc[j][m][r]);
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int m = 0; m < 4; ++m) pin_acc(acc[j][m]);  // the MFMAs run with every lane enabled

    // lane holds, per tile (j, m), row 64 wm + 16 m + l16 and columns 4 q .. +3 of tile j
    const int rows = r1 - r0;
    if (p.ksplit > 1) {
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int t = (bx * 4 + wn) * TN + j;
            if (t >= tiles) continue;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const int r = 64 * wm + 16 * m + l16;
                if (r < rows) *(v4f *)(p.part + ((int64_t)ks * p.M + r0 + r) * p.N + 16 * t + 4 * q) = acc[j][m];
            }
        }
        return;
    }
    // through LDS, so that every store instruction writes whole pieces of rows
    __syncthreads();
    int cols = 64 * TN;
    if constexpr (TN > 1) {
        if (p.silu) {
            cols /= 2;
#pragma unroll
            for (int j = 0; j < TN / 2; ++j)
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[j][m][r] = w4_silu_mul(acc[j][m][r], acc[j + TN / 2][m][r]);
        }
    }
    const int wcols = cols / 4;  // a wave's
#pragma unroll
    for (int j = 0; j < TN; ++j) {
        if (16 * j >= wcols) continue;
#pragma unroll
        for (int m = 0; m < 4; ++m)
            *(uint2 *)(lds + (64 * wm + 16 * m + l16) * T::CPITCH + 2 * (wn * wcols + 16 * j + 4 * q)) = w4_bf16x4(acc[j][m]);
    }
    __syncthreads();
    const int64_t ldc = p.silu ? p.N / 2 : p.N;
    const int ppr = cols / 8;  // 16-byte pieces a row
    const int64_t n0 = (int64_t)bx * cols;
    for (int id = tid; id < rows * ppr; id += T::THREADS) {
        const int r = id / ppr, cc = id % ppr;
        if (n0 + 8 * cc < ldc)
            *(uint4 *)(p.c + (int64_t)(r0 + r) * ldc + n0 + 8 * cc) = *(const uint4 *)(lds + r * T::CPITCH + 16 * cc);
    }
}

W4TiledCfg w4_tiled_config(int64_t M, int64_t K, int64_t N, int64_t E, bool silu) {
    W4TiledCfg c{0, 4, 1};
    const int64_t rows = E ? (M + E - 1) / E : M;
    if (rows > 32) c.wm = 1;  // [first version]
    const int *force = tuning().w4_tiled;
    if (force[0] >= 0) {
        c.wm = force[0];
        if (force[1]) c.tn = force[1];
        if (force[2] && !E) c.ksplit = (int)std::min<int64_t>(force[2], K / 128);
    }
    if (silu && c.tn == 1) c.tn = 2;
    return c;
}

static int64_t w4_g4(int64_t K, int grp) { return (K / grp + 3) / 4 * 4; }

size_t w4_sums_bytes(int64_t rows, int64_t K, int grp) {
    return align_up((size_t)rows * (size_t)w4_g4(K, grp) * 4, 256);
}

template <int FMT, int GRP, int TN, int WM, int NST>
static hipError_t launch_tile(W4Args a, const W4TiledCfg &c, hipStream_t s) {
    using T = W4Tile<FMT, GRP, TN, WM, NST>;
    // the dynamic LDS limit is a per-device function attribute: set it once per device
    static std::once_flag once[64];
    static hipError_t attr_err[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return hipErrorInvalidDevice;
    std::call_once(once[dev], [&] {
        attr_err[dev] = hipFuncSetAttribute((const void *)k_gemm_w4_tiled<FMT, GRP, T>,
                                            hipFuncAttributeMaxDynamicSharedMemorySize, T::SMEM);
    });
    if (attr_err[dev] != hipSuccess) return attr_err[dev];
    const int64_t cols = 64 * TN / (a.silu ? 2 : 1), n = a.silu ? a.N / 2 : a.N;
    const int64_t nblk = (n + cols - 1) / cols;
    int64_t nrow = (a.M + T::BM - 1) / T::BM;
    if (a.offsets) nrow = ((a.M + std::min(a.E, a.M) * (T::BM - 1)) / T::BM + 7) / 8 * 8;
    if (nblk * nrow > 0x7fffffff) return hipErrorInvalidValue;
    a.nblk = (int)nblk;
    a.nrow = (int)nrow;
    a.ksplit = c.ksplit;
    a.tmagic = a.topk > 1 ? (uint32_t)(((uint64_t(1) << 32) + a.topk - 1) / a.topk) : 0;
    hipLaunchKernelGGL((k_gemm_w4_tiled<FMT, GRP, T>), dim3((unsigned)(nblk * nrow), (unsigned)c.ksplit),
                       dim3(T::THREADS), T::SMEM, s, a);
    return hipGetLastError();
}

template <int FMT, int GRP>
static hipError_t launch_fmt(const W4Args &a, const W4TiledCfg &c, hipStream_t s) {
    if (c.wm == 2) return launch_tile<FMT, GRP, 4, 2, 3>(a, c, s);
    switch (c.tn) {
        case 1: return launch_tile<FMT, GRP, 1, 1, 3>(a, c, s);
        case 2: return launch_tile<FMT, GRP, 2, 1, 2>(a, c, s);
        default: return launch_tile<FMT, GRP, 4, 1, 2>(a, c, s);
    }
}

hipError_t launch_gemm_w4_tiled(W4Args a, int fmt, int grp, const W4TiledCfg &c, hipStream_t s) {
    hipError_t err;
    if (fmt == W4_INT) {
        a.g4 = (int)w4_g4(a.K, grp);
        const int64_t n8 = a.arows * (a.K / 8);
        hipLaunchKernelGGL(k_w4_sums, dim3((unsigned)((n8 + 255) / 256)), dim3(256), 0, s, (const uint4 *)a.a, n8,
                           (int)(a.K / 8), grp, (int)(a.K / grp), a.g4, a.sums);
        if ((err = hipGetLastError()) != hipSuccess) return err;
    }
    if (fmt == W4_MXFP4) err = launch_fmt<W4_MXFP4, 32>(a, c, s);
    else if (grp == 32) err = launch_fmt<W4_INT, 32>(a, c, s);
    else if (grp == 64) err = launch_fmt<W4_INT, 64>(a, c, s);
    else err = launch_fmt<W4_INT, 128>(a, c, s);
    if (err != hipSuccess || c.ksplit == 1) return err;
    return launch_splitk_reduce(a.part, a.c, a.M, a.N, c.ksplit, s);
}

}  // namespace r9k
