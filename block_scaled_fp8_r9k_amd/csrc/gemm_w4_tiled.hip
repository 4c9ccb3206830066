// Products with 4-bit weights, many rows: the LDS-tiled MFMA kernel.
//
// The same sums as the weight-streaming kernel (gemm_w4.hip), for row counts at
// which the matrix instructions and not the weight bytes set the time.  C^T = W
// A^T: four waves along the columns, each with TN column tiles by four row tiles of
// 16; a CTA is 64 TN columns by 64 rows, of which only the row tiles that hold rows are
// loaded and computed (32 rows an expert, 2048 -> 2 x 768 of 128 in int4: 68 us, 83 with all four).
//
// Per chunk of 128 K a stage in LDS holds the A tile (bf16), the packed codes of
// the column tiles, their scales and zeros, all moved there by global_load_lds, NST
// - 1 chunks ahead.  A wave converts its codes to bf16 fragments once a chunk, in
// registers, and uses them for its four row tiles.
//   int4: a group's product P starts from zero and is promoted into the fp32 sum
//   by acc += s * P, so neither the weights nor the sums are rounded.  The zero
//   points' share, sum_g z s S_g (S_g the sum of a group's activations), is a matrix
//   product with one term a group, and goes through the matrix cores too, every four
//   groups: s z holds 12 bits, two bf16; S_g, fp32, is three; the six products are
//   exact and take six of a lane quarter's eight K positions.  Wave w takes the sums of
//   row tile w (an MFMA with ones for weights) and leaves them, split, in LDS.
//   mxfp4: the scale is in the converted fragment (a power of two, exact) and the
//   matrix instruction accumulates through all of K.
// What bounds it, 4096 x 4096 x 12288: int4 in groups of 128 with zeros 412-444 us by the
// card's clock (928 to 1000 TFLOP/s; a bf16 library product 328 us) with the matrix cores
// busy 44% of the cycles and the vector units 50%: decoding is 7 instructions for 8 codes once per four row tiles,
// promotion 4 for every 16 x 16 x 128, and a 16 x 16 x 32 MFMA hides two vector
// instructions.  Where that takes 444 us, groups of 64 take 484, of 32 608 (the promotions
// double and quadruple); mxfp4, with nothing to promote, 322 us (1283 TFLOP/s).  Measured and not taken:
// 32 x 32 x 16 MFMA (492 us: two product chains a wave instead of sixteen), 128 rows a CTA
// (its registers leave one CTA a compute unit), the zero points' sums in a launch of their own.
// A rows are 256 bytes in LDS; 16-byte piece p of row r lies at piece p ^ (r % 16),
// so that the 16 rows of a fragment read fall on distinct banks.
#include <algorithm>
#include <mutex>

#include "w4_internal.h"
#include "w4_device.h"

namespace r9k {

namespace {
template <int FMT, int GRP, int TN_, int NST_>
struct W4Tile {
    static constexpr int TN = TN_, NST = NST_, THREADS = 256, BM = 64;
    static constexpr int NG = 128 / GRP, KPG = GRP / 32;
    static constexpr int ABYTES = BM * 256, WBYTES = 4 * TN * 1024;
    static constexpr int SDW = FMT == W4_MXFP4 ? 16 * TN : 8 * NG * TN;  // dwords of a wave's scales
    static constexpr int ZDW = FMT == W4_MXFP4 ? 0 : 4 * NG * TN;        // and zeros
    static constexpr int SLOADS = (SDW + 63) / 64, ZLOADS = (ZDW + 63) / 64;
    static constexpr int SBYTES = SLOADS * 256, ZBYTES = ZLOADS * 256;
    static constexpr int STAGE = ABYTES + WBYTES + 4 * (SBYTES + ZBYTES);
    static constexpr int LOADS = TN + 4 + SLOADS + ZLOADS;  // load instructions a wave and stage
    static constexpr int SUMS = FMT == W4_MXFP4 ? 0 : 2 * BM * 4 * 16;  // two steps of split sums, 4 groups each
    static constexpr int CPITCH = 64 * TN * 2 + 16;                     // output tile rows in LDS
    static constexpr int SMEM = NST * STAGE + SUMS > BM * CPITCH ? NST * STAGE + SUMS : BM * CPITCH;
    static_assert(SMEM <= 160 * 1024, "LDS");
    static_assert((NST - 2) * LOADS < 64, "vmcnt");
};

template <int V>
struct Const {
    static constexpr int value = V;
};
__device__ __forceinline__ uint32_t hi16(float lo, float hi) {  // upper halves of two fp32
    return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}
__device__ __forceinline__ float top16(float x) { return __uint_as_float(__float_as_uint(x) & 0xFFFF0000u); }
}  // namespace

template <int FMT, int GRP, class T>
__global__ __launch_bounds__(T::THREADS, 2) void k_gemm_w4_tiled(W4Args p) {
    constexpr int TN = T::TN, NG = T::NG, KPG = T::KPG, NST = T::NST, BM = T::BM;
    constexpr int CPS = 4 / NG;  // chunks of a zero point step (four groups)
    extern __shared__ __align__(16) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
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
    const int mt = (r1 - r0 + 15) >> 4;  // row tiles that hold rows
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

    // this wave's share of a stage's loads: a quarter of the rows, its own column
    // tiles with their scales and zeros (without zero points the scales again, unread)
    // (scalar bases with 32-bit lane offsets, so that going on to the next chunk costs no
    // vector instruction; activations of 4 GiB and more take 64-bit lane addresses)
    const uint8_t *abase, *wbase[TN], *sp[T::SLOADS], *zp[T::ZLOADS + 1];
    uint32_t aoffs[4];  // or the row, where the activations are wide
    const bool wide = p.src && (uint64_t)p.arows * (uint64_t)p.K >= (uint64_t(1) << 31);
    abase = (const uint8_t *)p.a + cb * 256 + (p.src ? 0 : (int64_t)r0 * p.K * 2);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int row = 4 * (4 * wave + u) + q;  // 4 rows of 16 pieces an instruction
        const uint32_t from = (uint32_t)source_row(r0 + row) - (p.src ? 0 : (uint32_t)r0);
        aoffs[u] = wide ? from : from * (uint32_t)(2 * p.K) + 16 * (l16 ^ (row & 15));
    }
#pragma unroll
    for (int u = 0; u < TN; ++u) wbase[u] = p.wp + (((int64_t)e * tiles + col_tile(wave, u)) * C + cb) * 1024;
    const uint32_t wlane = 16 * lane;
    constexpr int SPT = 4 * T::SDW / TN, ZPT = 4 * T::ZDW / TN;  // bytes a tile's chunk
#pragma unroll
    for (int u = 0; u < T::SLOADS; ++u) {
        const int d = min(64 * u + lane, T::SDW - 1) * 4;
        sp[u] = (const uint8_t *)p.sp + (((int64_t)e * tiles + col_tile(wave, d / SPT)) * C + cb) * SPT + d % SPT;
    }
    if constexpr (FMT == W4_INT) {
#pragma unroll
        for (int u = 0; u < T::ZLOADS; ++u) {
            const int d = min(64 * u + lane, T::ZDW - 1) * 4;
            const uint8_t *z = p.zp ? p.zp : (const uint8_t *)p.sp;
            zp[u] = z + (((int64_t)e * tiles + col_tile(wave, d / ZPT)) * C + cb) * ZPT + d % ZPT;
        }
    }
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(w4_lds_addr(lds));
    const int soff = T::ABYTES + T::WBYTES + wave * (T::SBYTES + T::ZBYTES), zoff = soff + T::SBYTES;
    auto issue = [&](int st) {
        const uint32_t base = lds0 + st * T::STAGE;
#pragma unroll
        for (int u = 0; u < TN; ++u) {
            w4_load16(wbase[u], wlane, base + T::ABYTES + (TN * wave + u) * 1024);
            wbase[u] += 1024;
        }
        if (NST == 2 && wave >= mt) {  // rows that are not there (with three stages every wave's loads are counted)
        } else if (!wide) {
#pragma unroll
            for (int u = 0; u < 4; ++u) w4_load16(abase, aoffs[u], base + (4 * wave + u) * 1024);
        } else {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int row = 4 * (4 * wave + u) + q;
                w4_load16(abase + (uint64_t)aoffs[u] * (uint64_t)(2 * p.K) + 16 * (l16 ^ (row & 15)), base + (4 * wave + u) * 1024);
            }
        }
        abase += 256;
#pragma unroll
        for (int u = 0; u < T::SLOADS; ++u) {
            w4_load4(sp[u], base + soff + u * 256);
            sp[u] += SPT;
        }
#pragma unroll
        for (int u = 0; u < T::ZLOADS; ++u) {
            w4_load4(zp[u], base + zoff + u * 256);
            zp[u] += ZPT;
        }
    };

    v4f acc[TN][4];
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int m = 0; m < 4; ++m) acc[j][m] = v4f{0.f, 0.f, 0.f, 0.f};

    // fragment addresses inside a stage: row tile m, step k at (aoff ^ 64 k) + 4096 m
    const int aoff = l16 * 256 + ((q ^ l16) << 4);
    const int woff = T::ABYTES + wave * TN * 1024 + 16 * lane;

    // Zero points.  sz: -s z of row l16 of each column tile, for the step's group q;
    // split sums of row r, group g of a step: 16 bytes at (r * 4 + g) * 16 of its half.
    float sz[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j) sz[j] = 0.0f;
    uint8_t *sums = lds + NST * T::STAGE;
    int cis = 0, half = 0;  // chunk in the step, the step's half
    auto zero_step = [&](auto row_tiles, int h, int groups) {  // acc += sz x sums over the step's groups
        constexpr int MT = decltype(row_tiles)::value;
        w4_v8bf sf[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            uint4 v = *(const uint4 *)(sums + h * (T::SUMS / 2) + ((16 * m + l16) * 4 + q) * 16);
            if (q >= groups) v = make_uint4(0, 0, 0, 0);
            sf[m] = w4_frag(v);
        }
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const float hi = top16(sz[j]), lo = sz[j] - hi;
            const w4_v8bf wf = __builtin_bit_cast(w4_v8bf, w4_v4u{hi16(hi, hi), hi16(hi, lo), hi16(lo, lo), 0});
#pragma unroll
            for (int m = 0; m < MT; ++m) acc[j][m] = w4_mfma(wf, sf[m], acc[j][m]);
            sz[j] = 0.0f;
        }
    };

    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // from here on only the stages' loads are counted
#pragma unroll
    for (int k = 0; k < NST - 1; ++k)
        if (cb + k < ce) issue(k);
    auto chunk = [&](auto row_tiles, int c, auto stage) {
        constexpr int MT = decltype(row_tiles)::value, st = decltype(stage)::value;
        // this chunk's stage has landed: the wave's loads issued after it are those of the NST - 2 chunks behind it
        // (fewer at the end: then wait for all)
        if (c + NST - 2 < ce) w4_wait_vm<(NST - 2) * T::LOADS>();
        else w4_wait_vm<0>();
        __syncthreads();
        if (c + NST - 1 < ce) issue((st + NST - 1) % NST);
        const uint8_t *sb = lds + st * T::STAGE;

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
                w4_v8bf af[MT];
#pragma unroll
                for (int m = 0; m < MT; ++m) af[m] = w4_frag(*(const uint4 *)(sb + (aoff ^ (64 * k)) + 4096 * m));
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    const uint32_t word[4] = {code[j].x, code[j].y, code[j].z, code[j].w};
                    const w4_v8bf wf = w4_fp4_frag(word[k], __uint_as_float(((sc[j] >> (8 * k)) & 255u) << 23));
#pragma unroll
                    for (int m = 0; m < MT; ++m) acc[j][m] = w4_mfma(wf, af[m], acc[j][m]);
                }
            }
        } else {
            // the step before is complete: its sums are in LDS since the barrier
            if (c > cb && cis == 0) zero_step(row_tiles, half ^ 1, 4);
            // the sums of row tile `wave`, as three bf16 pieces against the pieces of sz in zero_step
            if (MT == 4 || wave < MT) {
#pragma unroll
                for (int i = 0; i < NG; ++i) {
                    v4f sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int k = 0; k < KPG; ++k)
                        sum = w4_mfma(w4_ones(), w4_frag(*(const uint4 *)(sb + (aoff ^ (64 * (i * KPG + k))) + 4096 * wave)), sum);
                    const float h = top16(sum[0]), d = sum[0] - h, mid = top16(d), l = d - mid;
                    // the four lanes of row l16 hold the same sum and write the same bytes: no lane is masked
                    *(uint4 *)(sums + half * (T::SUMS / 2) + ((16 * wave + l16) * 4 + cis * NG + i) * 16) =
                        make_uint4(hi16(h, mid), hi16(l, h), hi16(mid, l), 0);
                }
            }
            uint4 code[TN];
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                code[j] = *(const uint4 *)(sb + woff + 1024 * j);
                const int at = ((l16 >> 2) * NG + q % NG) * 4 + (l16 & 3);
                const float s = __uint_as_float((uint32_t)*(const uint16_t *)(sb + soff + SPT * j + 2 * at) << 16);
                const uint32_t zb = *(sb + zoff + ZPT * j + at);  // (a scale's byte where there are no zeros)
                const float z = (float)(p.zp ? zb : 8u);
                float v = -s * z;
                asm volatile("" : "+v"(v));  // formed in every lane, so that the choice is a select and masks no lane
                sz[j] = q / NG == cis ? v : sz[j];
            }
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                w4_v8bf wf[TN][KPG];
                float s[TN][4];
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    const uint32_t word[4] = {code[j].x, code[j].y, code[j].z, code[j].w};
#pragma unroll
                    for (int k = 0; k < KPG; ++k) wf[j][k] = w4_int_frag(word[i * KPG + k]);
                    const uint2 s2 = *(const uint2 *)(sb + soff + SPT * j + 8 * NG * q + 8 * i);
                    s[j][0] = bf16_lo(s2.x);
                    s[j][1] = bf16_hi(s2.x);
                    s[j][2] = bf16_lo(s2.y);
                    s[j][3] = bf16_hi(s2.y);
                }
#pragma unroll
                for (int m = 0; m < MT; ++m) {
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
                // the sums are formed here, not moved past the next branch with their products held
#pragma unroll
                for (int j = 0; j < TN; ++j)
#pragma unroll
                    for (int m = 0; m < MT; ++m) pin_acc(acc[j][m]);
            }
            if (++cis == CPS) {
                cis = 0;
                half ^= 1;
            }
        }
    };
    // the stages in turn, each with its own code: LDS addresses are then constants
    auto chunks = [&](auto row_tiles) {
        for (int c = cb; c < ce; c += NST) {
            chunk(row_tiles, c, Const<0>{});
            if (c + 1 < ce) chunk(row_tiles, c + 1, Const<1>{});
            if constexpr (NST == 3)
                if (c + 2 < ce) chunk(row_tiles, c + 2, Const<2>{});
        }
        if constexpr (FMT == W4_INT) {
            __syncthreads();  // the last step's sums; it may hold fewer than four groups
            if (cis) zero_step(row_tiles, half, cis * NG);
            else zero_step(row_tiles, half ^ 1, 4);
        }
    };
    switch (mt) {  // only the row tiles that hold rows are computed
        case 1: chunks(Const<1>{}); break;
        case 2: chunks(Const<2>{}); break;
        case 3: chunks(Const<3>{}); break;
        default: chunks(Const<4>{});
    }
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int m = 0; m < 4; ++m) pin_acc(acc[j][m]);  // the MFMAs run with every lane enabled

    // lane holds, per tile (j, m), row 16 m + l16 and columns 4 q .. +3 of tile j
    const int rows = r1 - r0;
    if (p.ksplit > 1) {
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int t = (bx * 4 + wave) * TN + j;
            if (t >= tiles) continue;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const int r = 16 * m + l16;
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
            *(uint2 *)(lds + (16 * m + l16) * T::CPITCH + 2 * (wave * wcols + 16 * j + 4 * q)) = w4_bf16x4(acc[j][m]);
    }
    __syncthreads();
    const int64_t ldc = p.silu ? p.N / 2 : p.N;
    const int pl = __builtin_ctz(cols / 8);  // log2 of the 16-byte pieces a row
    const int64_t n0 = (int64_t)bx * cols;
    for (int id = tid; id < rows << pl; id += T::THREADS) {
        const int r = id >> pl, cc = id & ((1 << pl) - 1);
        if (n0 + 8 * cc < ldc)
            *(uint4 *)(p.c + (int64_t)(r0 + r) * ldc + n0 + 8 * cc) = *(const uint4 *)(lds + r * T::CPITCH + 16 * cc);
    }
}

// The column tiles a wave and the K split of the least estimated time.  A chunk of a CTA
// takes `alone` when it has the compute unit to itself and `shared` where the unit's CTAs
// keep it busy, less where not all four row tiles hold rows; experts' CTAs, which find
// their rows first and share less in the caches, a quarter more; a split adds the partials
// and the reduce launch.  Fitted to 16 shapes (48 to 400 rows, K and N from 1024 to 14336, int4 in
// groups of 128 with zeros, each of 12 launches) within 6% (rms).  E.g. 100 rows of 4096 x
// 4096: 18.2 us in 4 splits of 2 tiles a wave, 37 whole; 4096 x 4096 x 12288: 414 us with 4
// tiles, 514 with 2.
// The streaming kernel takes what it is estimated to do sooner, always up to 32 rows.  Both
// timed on 90 shapes (33 to 400 rows dense, 3 to 250 rows an expert, 8 to 128 experts), the
// pick was 2% behind the faster on average, 17% at most; against every launch of both, over 96
// dense shapes of 33 to 400 rows in every format 3% (at most 25%), over 64 of 16 to 128 rows an
// expert 4% (at most 46%).  E.g. (streaming, tiled; us)
//   64 rows, int4      1024 x 4096  5.7, 9.6   4096 x 4096  13.7, 14.6   4096 x 14336  24.1, 23.8
//   400 rows, int4     1024 x 4096  11.6, 12.5  4096 x 4096  43.6, 31.7
//   2048 -> 2 x 768 of 128 experts, int4, rows an expert   8: 50, 58   16: 82, 62   32: 120, 70
W4TiledCfg w4_tiled_config(int64_t M, int64_t K, int64_t N, int64_t E, bool silu) {
    static constexpr struct {
        int tn;
        double alone, shared;
    } costs[] = {{1, 0.77, 0.555}, {2, 1.03, 0.747}, {4, 1.615, 1.115}};
    W4TiledCfg best{false, 4, 1, 0.0};
    const int *force = w4_tuning().tiled;
    if (force[0] == 0 || (force[0] < 0 && !E && M <= 32)) return best;
    const int64_t C = K / 128, tiles = N / 16;
    const double blocks = E ? w4_expert_blocks(M, E, 64) : (double)((M + 63) / 64);
    const double fill = (E ? 1.25 : 1.0) * (0.65 + 0.35 * std::ceil(std::min(64.0, (double)M / blocks) / 16.0) / 4.0);
    for (const auto &t : costs) {
        if (E && t.tn == 1) continue;  // slower at every expert shape measured (down of 128: 45 us, 28 with 2)
        if (force[0] > 0 && force[1] && force[1] != t.tn) continue;
        for (int64_t ks = 1; ks <= (E ? 1 : 8) && ks <= C; ks *= 2) {
            const int64_t want = force[0] > 0 && force[2] && !E ? std::min<int64_t>(force[2], C) : ks;
            const double ctas = blocks * (double)((tiles + 4 * t.tn - 1) / (4 * t.tn) * want);
            double load = ctas / 256.0;
            if (load <= 2.0) load = std::ceil(load);
            double us = 3.6 + (double)((C + want - 1) / want) * std::max(t.alone, load * t.shared) * fill;
            if (want > 1) us += 2.8 + 1.7e-6 * (double)(want * M * N);
            if (best.us == 0.0 || us < best.us) best = W4TiledCfg{true, t.tn, (int)want, us};
        }
    }
    return best;
}

template <int FMT, int GRP, int TN, int NST>
static hipError_t launch_tile(W4Args a, const W4TiledCfg &c, hipStream_t s) {
    using T = W4Tile<FMT, GRP, TN, NST>;
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
    if (nblk * nrow >= 1 << 24) return hipErrorInvalidValue;  // 2^32 threads
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
    switch (c.tn) {
        case 1: return launch_tile<FMT, GRP, 1, 3>(a, c, s);
        case 2: return launch_tile<FMT, GRP, 2, 2>(a, c, s);
        default: return launch_tile<FMT, GRP, 4, 2>(a, c, s);
    }
}

hipError_t launch_gemm_w4_tiled(const W4Args &a, int fmt, int grp, const W4TiledCfg &c, hipStream_t s) {
    hipError_t err;
    if (fmt == W4_MXFP4) err = launch_fmt<W4_MXFP4, 32>(a, c, s);
    else if (grp == 32) err = launch_fmt<W4_INT, 32>(a, c, s);
    else if (grp == 64) err = launch_fmt<W4_INT, 64>(a, c, s);
    else err = launch_fmt<W4_INT, 128>(a, c, s);
    if (err != hipSuccess || c.ksplit == 1) return err;
    return launch_splitk_reduce(a.part, a.c, a.M, a.N, c.ksplit, s);
}

}  // namespace r9k
