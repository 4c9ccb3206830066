// Products in 8-bit integers, many rows: the LDS-tiled MFMA kernel.
//
// The same sums as the weight-streaming kernel (gemm_i8.hip), for row counts at which the
// matrix instructions and not the weight bytes set the time.  C^T = W A^T: WN x WM waves,
// each TN column tiles by TM row tiles of 16; per half chunk of 64 K a stage in LDS holds the W
// tile in packed order ([column tile][lane][16 bytes]) and the A tile (rows of 64
// bytes), moved there straight from memory, NST - 1 stages ahead.  Integer sums need no
// promotion, so between the matrix instructions there are only the fragments' LDS reads, in
// a fixed order: a step multiplies one W fragment with the stage's TM A fragments, and asks for the W
// fragment of two steps later and, spread over the stage, for the A fragments of the next.  The stage that
// these come from has landed for every wave since the barrier before, so that no step waits for LDS
// after a barrier.
// 16-byte piece c of row r of the A tile lies at piece c ^ ((r >> 2) & 3), so that the 16
// rows of a fragment read fall on distinct banks.
#include <algorithm>
#include <mutex>
#include <utility>

#include "i8_device.h"
#include "i8_internal.h"

namespace r9k {

namespace {
template <int WN_, int WM_, int TN_, int TM_, int NST_>
struct I8Tile {
    static constexpr int WN = WN_, WM = WM_, TN = TN_, TM = TM_, NST = NST_;
    static constexpr int NW = WN * WM, THREADS = 64 * NW;
    static constexpr int BN = WN * TN * 16, BM = WM * TM * 16;  // output columns and rows of a CTA
    static constexpr int WBYTES = BN * 64, ABYTES = BM * 64, STAGE = WBYTES + ABYTES;
    static constexpr int WLOADS = BN / 16 / NW, ALOADS = BM / 16 / NW, LOADS = WLOADS + ALOADS;  // 1 KiB loads a wave
    static constexpr int CPITCH = BN * 2 + 16;  // output tile rows in LDS
    static constexpr int SMEM = NST * STAGE > BM * CPITCH ? NST * STAGE : BM * CPITCH;
    static_assert(SMEM <= 160 * 1024, "LDS");
    static_assert(WLOADS * NW * 16 == BN && ALOADS * NW * 16 == BM, "loads split evenly");
    static_assert(NST >= 4 && NST <= 5 && TN % 2 == 0, "stages; a ring of W fragments whose places are constants");
};
template <int V>
struct Const {
    static constexpr int value = V;
};
// f(Const<0>) ... f(Const<N - 1>)
template <class F, int... I>
__device__ __forceinline__ void each(F &&f, std::integer_sequence<int, I...>) {
    (f(Const<I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void each(F &&f) {
    each(f, std::make_integer_sequence<int, N>{});
}
}  // namespace

template <class T>
__global__ __launch_bounds__(T::THREADS, 1) void k_gemm_i8_tiled(I8Args p) {
    constexpr int WN = T::WN, TN = T::TN, TM = T::TM, NST = T::NST, BM = T::BM;
    extern __shared__ __align__(16) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wn = wave % WN, wm = wave / WN;
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
    const int rows = r1 - r0;
    const int mt = min(TM, max(0, (rows - wm * TM * 16 + 15) >> 4));  // the wave's row tiles that hold rows
    const int ks = blockIdx.y;
    const int cb = (int)((int64_t)ks * C / p.ksplit), ce = (int)((int64_t)(ks + 1) * C / p.ksplit);
    const int n = 2 * (ce - cb);  // stages

    // column tile i of wave column w; those past the last repeat it and are not stored
    auto col_tile = [&](int w, int i) {
        if constexpr (TN > 1) {
            if (p.silu) return min((bx * WN + w) * (TN / 2) + i % (TN / 2), tiles / 2 - 1) + (i < TN / 2 ? 0 : tiles / 2);
        }
        return min((bx * WN + w) * TN + i, tiles - 1);
    };
    auto source_row = [&](int r) -> int64_t {  // activation row of output row r (clamped to the block)
        const int rr = min(r, r1 - 1);
        if (!p.src) return rr;
        const uint32_t t = w4_div_topk((uint32_t)p.src[rr], (uint32_t)p.topk, p.tmagic);
        return t < (uint32_t)p.arows ? t : 0;
    };

    // this wave's share of a stage's loads: W instructions WLOADS wave + u, one half of a
    // column tile's block each, and A instructions ALOADS wave + u, sixteen rows each
    const int8_t *wsrc[T::WLOADS], *asrc[T::ALOADS];
#pragma unroll
    for (int u = 0; u < T::WLOADS; ++u) {
        const int t = T::WLOADS * wave + u;
        wsrc[u] = p.wp + (((int64_t)e * tiles + col_tile(t / TN, t % TN)) * C + cb) * 2048 + 16 * lane;
    }
#pragma unroll
    for (int u = 0; u < T::ALOADS; ++u) {
        const int row = 16 * (T::ALOADS * wave + u) + (lane >> 2), piece = (lane & 3) ^ ((row >> 2) & 3);
        asrc[u] = p.aq + source_row(r0 + row) * p.K + cb * 128 + 16 * piece;
    }
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(w4_lds_addr(lds));
    auto issue = [&](int st, auto load) {  // the wave's load instruction `load` of a stage
        constexpr int u = decltype(load)::value, v = u - T::WLOADS;
        if constexpr (u < T::WLOADS) {
            w4_load16(wsrc[u], lds0 + st * T::STAGE + (T::WLOADS * wave + u) * 1024);
            wsrc[u] += 1024;
        } else if constexpr (u < T::LOADS) {
            w4_load16(asrc[v], lds0 + st * T::STAGE + T::WBYTES + (T::ALOADS * wave + v) * 1024);
            asrc[v] += 64;
        }
    };

    v4i acc[TN][TM];
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) acc[i][j] = v4i{0, 0, 0, 0};
    // the scales of the wave's columns and rows, on their way before the first stage
    float4 ws[TN];
    float as[TM];
    if (p.ksplit == 1) {
#pragma unroll
        for (int i = 0; i < TN; ++i) ws[i] = *(const float4 *)(p.ws + (int64_t)e * p.N + 16 * col_tile(wn, i) + 4 * q);
#pragma unroll
        for (int j = 0; j < TM; ++j) as[j] = p.as[source_row(r0 + wm * TM * 16 + l16 + 16 * j)];
    }

    // fragment addresses inside a stage: column tile i at wfo + 1024 i, row tile j at afo + 1024 j
    const int wfo = wn * TN * 1024 + 16 * lane;
    const int arow = wm * TM * 16 + l16;
    const int afo = T::WBYTES + arow * 64 + ((q ^ ((arow >> 2) & 3)) << 4);

    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // from here on only the stages' loads are counted
#pragma unroll
    for (int k = 0; k < NST - 1; ++k)
        if (k < n) each<T::LOADS>([&](auto u) { issue(k, u); });
    // W fragments in a ring of four, two steps ahead; A fragments of this stage and the next
    v4i wf[4], af[2][TM];
    // at most `stages` stages' loads of the wave are in flight
    auto wait = [&](int stages) {
        if (NST > 4 && stages >= 3) w4_wait_vm<3 * T::LOADS>();
        else if (stages >= 2) w4_wait_vm<2 * T::LOADS>();
        else if (stages == 1) w4_wait_vm<T::LOADS>();
        else w4_wait_vm<0>();
    };
    wait(min(NST - 2, n - 1));
    __syncthreads();
    int at = 0;  // the stage's place: c % NST
    auto steps = [&](auto row_tiles, int c, auto parity, auto more) {
        constexpr int MT = decltype(row_tiles)::value, odd = decltype(parity)::value, ahead = decltype(more)::value;
        // the next stage has landed: the wave's loads issued after it are those of the NST - 3 stages behind it, fewer at
        // the end
        if (ahead) w4_wait_vm<(NST - 3) * T::LOADS>();
        else wait(min(NST - 3, n - 2 - c));
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        const int next = at + 1 == NST ? 0 : at + 1, last = at == 0 ? NST - 1 : at - 1;
        const uint8_t *sb = lds + at * T::STAGE, *sx = lds + next * T::STAGE;
        each<TN>([&](auto step) {
            constexpr int i = decltype(step)::value, PER = (T::LOADS + TN - 1) / TN;
            if (ahead)  // the loads of the stage NST - 1 behind, spread over the steps
                each<PER>([&](auto u) { issue(last, Const<PER * i + decltype(u)::value>{}); });
            if constexpr (MT > 0) {
                wf[(TN * odd + i + 2) & 3] = *(const v4i *)((i + 2 < TN ? sb + 1024 * (i + 2) : sx + 1024 * (i + 2 - TN)) + wfo);
#pragma unroll
                for (int j = 0; j < MT; ++j)
                    if (j * TN / MT == i) af[odd ^ 1][j] = *(const v4i *)(sx + afo + 1024 * j);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = 0; j < MT; ++j) acc[i][j] = i8_mfma(wf[(TN * odd + i) & 3], af[odd][j], acc[i][j]);
                __builtin_amdgcn_sched_barrier(0);
            }
        });
        at = next;
    };
    auto run = [&](auto row_tiles) {
        constexpr int MT = decltype(row_tiles)::value;
#pragma unroll
        for (int j = 0; j < MT; ++j) af[0][j] = *(const v4i *)(lds + afo + 1024 * j);
        wf[0] = *(const v4i *)(lds + wfo);
        wf[1] = *(const v4i *)(lds + wfo + 1024);
        int c = 0;
        for (; c + NST < n; c += 2) {
            steps(row_tiles, c, Const<0>{}, Const<1>{});
            steps(row_tiles, c + 1, Const<1>{}, Const<1>{});
        }
        if (c + NST - 1 < n) {  // one more stage to ask for
            steps(row_tiles, c, Const<0>{}, Const<1>{});
            steps(row_tiles, c + 1, Const<1>{}, Const<0>{});
            c += 2;
        }
        for (; c < n; c += 2) {
            steps(row_tiles, c, Const<0>{}, Const<0>{});
            steps(row_tiles, c + 1, Const<1>{}, Const<0>{});
        }
    };
    switch (mt) {  // only the row tiles that hold rows are computed
        case 0: run(Const<0>{}); break;
        case 1: run(Const<1>{}); break;
        case 2: run(Const<(TM < 2 ? TM : 2)>{}); break;
        default: run(Const<TM>{});
    }
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) i8_pin(acc[i][j]);

    // lane holds, per tile (i, j), row 16 (wm TM + j) + l16 and columns 4 q .. +3 of tile i
    if (p.ksplit > 1) {
#pragma unroll
        for (int i = 0; i < TN; ++i) {
            const int t = (bx * WN + wn) * TN + i;
            if (t >= tiles) continue;
#pragma unroll
            for (int j = 0; j < TM; ++j) {
                const int r = arow + 16 * j;
                if (r < rows) *(v4i *)(p.part + ((int64_t)ks * p.M + r0 + r) * p.N + 16 * t + 4 * q) = acc[i][j];
            }
        }
        return;
    }
    // through LDS, so that every store instruction writes whole pieces of rows
    __syncthreads();
    const int nt = p.silu ? TN / 2 : TN, wcols = nt * 16, cols = WN * wcols;
#pragma unroll
    for (int i = 0; i < TN; ++i) {
        if (16 * i >= wcols) continue;
#pragma unroll
        for (int j = 0; j < TM; ++j) {
            v4f y = i8_scale(acc[i][j], as[j], ws[i]);
            if constexpr (TN > 1) {
                if (p.silu) {
                    const v4f u = i8_scale(acc[(i + TN / 2) % TN][j], as[j], ws[(i + TN / 2) % TN]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) y[r] = w4_silu_mul(y[r], u[r]);
                }
            }
            *(uint2 *)(lds + (arow + 16 * j) * T::CPITCH + 2 * (wn * wcols + 16 * i + 4 * q)) = w4_bf16x4(y);
        }
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

template <class T>
static hipError_t launch_tile(I8Args a, const I8TiledCfg &c, hipStream_t s) {
    // the dynamic LDS limit is a per-device function attribute: set it once per device
    static std::once_flag once[64];
    static hipError_t attr_err[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return hipErrorInvalidDevice;
    std::call_once(once[dev], [&] {
        attr_err[dev] = hipFuncSetAttribute((const void *)k_gemm_i8_tiled<T>, hipFuncAttributeMaxDynamicSharedMemorySize, T::SMEM);
    });
    if (attr_err[dev] != hipSuccess) return attr_err[dev];
    const int64_t cols = T::BN / (a.silu ? 2 : 1), n = a.silu ? a.N / 2 : a.N;
    const int64_t nblk = (n + cols - 1) / cols;
    int64_t nrow = (a.M + T::BM - 1) / T::BM;
    if (a.offsets) nrow = ((a.M + std::min(a.E, a.M) * (T::BM - 1)) / T::BM + 7) / 8 * 8;
    if (nblk * nrow >= (int64_t(1) << 32) / T::THREADS) return hipErrorInvalidValue;
    a.nblk = (int)nblk;
    a.nrow = (int)nrow;
    a.ksplit = c.ksplit;
    a.tmagic = a.topk > 1 ? (uint32_t)(((uint64_t(1) << 32) + a.topk - 1) / a.topk) : 0;
    hipLaunchKernelGGL((k_gemm_i8_tiled<T>), dim3((unsigned)(nblk * nrow), (unsigned)c.ksplit), dim3(T::THREADS),
                       T::SMEM, s, a);
    return hipGetLastError();
}

hipError_t launch_gemm_i8_tiled(const I8Args &a, const I8TiledCfg &c, hipStream_t s) {
    hipError_t err;
    switch (c.shape) {
        case I8_256X256: err = launch_tile<I8Tile<2, 4, 8, 4, 5>>(a, c, s); break;
        case I8_256X128: err = launch_tile<I8Tile<4, 2, 4, 4, 4>>(a, c, s); break;
        case I8_256X64: err = launch_tile<I8Tile<4, 1, 4, 4, 4>>(a, c, s); break;
        case I8_128X64: err = launch_tile<I8Tile<4, 1, 2, 4, 4>>(a, c, s); break;
        default: err = launch_tile<I8Tile<4, 2, 2, 4, 4>>(a, c, s); break;
    }
    if (err != hipSuccess || c.ksplit == 1) return err;
    return launch_i8_reduce(a, c.ksplit, s);
}

}  // namespace r9k
