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
// A CTA computes one output tile after another: the first stages of the next are asked for before the
// outputs of the last are scaled and stored, and the waits of its first stages let those stores
// be in flight (at 4096 x 4096 x 12288 175 -> 168 us).
//
// Measured: 4096 x 4096 x 12288 in 168 us, 2.45e15 operations a second.  The matrix instructions alone reach 4.0e15 on
// such values, at the 2.0 GHz that the card's power leaves them; its clock is the same, with MFMA in 57% of the cycles.
// Without the loads it takes 146 us, without LDS reads 143: neither alone is what is left.  32 x 32 x 32 instructions
// reach 3.5e15; one barrier for two stages changes nothing.
// Few rows are bound by what a compute unit takes in from L2 and by the way from the first load to the last store:
// 64 x 64 with two groups of waves, two CTAs of five stages each, 12.5 us at 256 x 4096 x 4096 (one group 14.5;
// eight stages, one CTA 13.2; four stages, two CTAs 14.0); 128 x 64 in six stages, two CTAs 19.0 (four, three CTAs 21.7).
#include <algorithm>
#include <mutex>
#include <utility>

#include "i8_device.h"
#include "i8_internal.h"

namespace r9k {

namespace {
template <int WN_, int WM_, int TN_, int TM_, int NST_, int CTAS_, int KG_ = 1>
struct I8Tile {
    static constexpr int WN = WN_, WM = WM_, TN = TN_, TM = TM_, NST = NST_, CTAS = CTAS_;  // CTAs a compute unit
    static constexpr int AHEAD = NST - 1;  // stages asked for before they are computed
    static constexpr int KG = KG_;         // groups of waves: with two each computes the whole tile over half of every chunk
    static constexpr int NW = WN * WM, THREADS = 64 * NW * KG;  // waves of a group
    static constexpr int BN = WN * TN * 16, BM = WM * TM * 16;  // output columns and rows of a CTA
    static constexpr int WBYTES = BN * 64, ABYTES = BM * 64, STAGE = WBYTES + ABYTES, RING = NST * STAGE, SMEM = KG * RING;
    static constexpr int WLOADS = BN / 16 / NW, ALOADS = BM / 16 / NW, LOADS = WLOADS + ALOADS;  // 1 KiB loads a wave
    static_assert(CTAS * SMEM <= 160 * 1024, "LDS");
    static_assert(WLOADS * NW * 16 == BN && ALOADS * NW * 16 == BM, "loads split evenly");
    static_assert(NST >= 4 && TN % 2 == 0, "stages; a ring of W fragments whose places are constants");
    static_assert(TM == 4 && NW * 512 * TN <= STAGE, "the outputs' way through one stage's LDS");
    static_assert(KG == 1 || (KG == 2 && NW * TN * TM * 512 <= RING), "half of a group's sums, on their way to the other");
    static_assert((NST - 2) * LOADS + TN * TM < 64, "vmcnt");
};
template <int V>
struct Const {
    static constexpr int value = V;
};
// at most min(stages, MOST) * LOADS + MORE of the wave's vector-memory instructions are in flight
template <int MOST, int LOADS, int MORE>
__device__ __forceinline__ void wait_stages(int stages) {
    if constexpr (MOST == 0) w4_wait_vm<MORE>();
    else if (stages >= MOST) w4_wait_vm<MOST * LOADS + MORE>();
    else wait_stages<MOST - 1, LOADS, MORE>(stages);
}
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

template <class T, bool SILU>
__global__ __launch_bounds__(T::THREADS, (T::CTAS * T::NW * T::KG + 3) / 4) void k_gemm_i8_tiled(I8Args p) {
    constexpr int WN = T::WN, TN = T::TN, TM = T::TM, NST = T::NST, BM = T::BM, AHEAD = T::AHEAD;
    constexpr int NT = SILU ? TN / 2 : TN;                    // output tiles a wave and row tile
    constexpr int PR = 2 * NT, READS = PR < 4 ? 1 : PR / 4;   // 16-byte pieces of an output row; stores a row tile
    constexpr int KG = T::KG, TMG = TM / KG;                  // row tiles that a wave scales and stores
    extern __shared__ __align__(16) uint8_t lds_all[];
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, q = lane >> 4;
    const int wid = __builtin_amdgcn_readfirstlane(tid >> 6), group = KG == 1 ? 0 : wid / T::NW;
    const int wave = wid - group * T::NW, wn = wave % WN, wm = wave / WN;
    uint8_t *const lds = lds_all + group * T::RING;  // the group's stages
    const int C = (int)(p.K / 128), tiles = (int)(p.N / 16);
    const int64_t ldc = SILU ? p.N / 2 : p.N;
    const int blocks = p.nblk * p.nrow, total = blocks * p.ksplit;

    // Tile v: column block bx, rows [r0, r0 + rows) of expert e, split ks.  Tiles go round-robin to the 8 XCDs.
    // Dense: an XCD takes a contiguous range, walked eight row blocks at a time, so
    // that what runs together shares A and W in its L2.  Experts: an XCD takes
    // every eighth row block, with all its column blocks (the blocks past the last
    // are then spread over the XCDs).
    struct Work {
        int bx, e, r0, rows, ks;
    };
    I8Blocks blks;
    if (p.offsets && p.E <= 256) blks.load(p.offsets, (int)p.E, (int)p.M, BM);
    auto find = [&](int v, Work &w) -> bool {
        if (v >= total) return false;
        int by;
        w.e = w.ks = 0;
        if (p.offsets) {
            const int j = v >> 3;
            by = (j / p.nblk) * 8 + (v & 7);
            w.bx = j % p.nblk;
            int a0, a1;
            if (!(p.E <= 256 ? blks.find(by, BM, w.e, a0, a1) : w4_find_block(p.offsets, (int)p.E, (int)p.M, BM, by, w.e, a0, a1)))
                return false;  // nor do later tiles exist
            w.r0 = a0;
            w.rows = min(a1 - a0, BM);
        } else {
            w.ks = v / blocks;
            int lid = v % blocks;
            if (blocks % 8 == 0) lid = (lid & 7) * (blocks / 8) + (lid >> 3);
            const int per = 8 * p.nblk, first = lid / per * 8, rows = min(8, p.nrow - first), in = lid % per;
            by = first + in % rows;
            w.bx = in / rows;
            w.r0 = by * BM;
            w.rows = (int)min<int64_t>(p.M - w.r0, BM);
        }
        w.e = __builtin_amdgcn_readfirstlane(w.e);
        w.r0 = __builtin_amdgcn_readfirstlane(w.r0);
        w.rows = __builtin_amdgcn_readfirstlane(w.rows);
        return true;
    };
    // column tile i of wave column w; those past the last repeat it and are not stored
    auto col_tile = [&](int bx, int w, int i) {
        if constexpr (SILU) return min((bx * WN + w) * (TN / 2) + i % (TN / 2), tiles / 2 - 1) + (i < TN / 2 ? 0 : tiles / 2);
        return min((bx * WN + w) * TN + i, tiles - 1);
    };
    // activation row of the block's row r (clamped to it): looked up, and later made of what was found there
    auto look_up = [&](const Work &w, int r) -> uint32_t {
        const int rr = w.r0 + min(r, w.rows - 1);
        return p.src ? (uint32_t)p.src[rr] : (uint32_t)rr;
    };
    auto source_row = [&](uint32_t x) -> uint32_t {
        if (!p.src) return x;
        const uint32_t t = w4_div_topk(x, (uint32_t)p.topk, p.tmagic);
        return t < (uint32_t)p.arows ? t : 0;
    };

    // The lane, forgotten: what is computed from it inside the loop over tiles is computed there, and takes no
    // registers in the loop over stages.
    auto fresh = [&] {
        int l = lane;
        asm volatile("" : "+v"(l));
        return l;
    };
    // this wave's share of its group's loads of a stage: W instructions WLOADS wave + u, one half of a
    // column tile's block each, and A instructions ALOADS wave + u, sixteen rows each
    const int8_t *wsrc[T::WLOADS], *asrc[T::ALOADS];
    uint32_t arow[T::ALOADS], srow;  // what look_up found for those, and for the wave's row `lane`
    auto rows_of = [&](const Work &w) {
        const int l = fresh();
#pragma unroll
        for (int u = 0; u < T::ALOADS; ++u) arow[u] = look_up(w, 16 * (T::ALOADS * wave + u) + (l >> 2));
        srow = look_up(w, wm * TM * 16 + l);
    };
    auto chunks = [&](const Work &w, int &cb) {
        cb = (int)((int64_t)w.ks * C / p.ksplit);
        return (int)((int64_t)(w.ks + 1) * C / p.ksplit) - cb;
    };
    auto pointers = [&](const Work &w) {
        int cb;
        chunks(w, cb);
        const int l = fresh();
#pragma unroll
        for (int u = 0; u < T::WLOADS; ++u) {
            const int t = T::WLOADS * wave + u;
            wsrc[u] = p.wp + (((int64_t)w.e * tiles + col_tile(w.bx, t / TN, t % TN)) * C + cb) * 2048 + 1024 * group + 16 * l;
        }
#pragma unroll
        for (int u = 0; u < T::ALOADS; ++u) {
            const int row = 16 * (T::ALOADS * wave + u) + (l >> 2), piece = (l & 3) ^ ((row >> 2) & 3);
            asrc[u] = p.aq + (int64_t)source_row(arow[u]) * p.K + cb * 128 + 64 * group + 16 * piece;
        }
    };
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(w4_lds_addr(lds));
    auto issue = [&](int st, auto load) {  // the wave's load instruction `load` of a stage
        constexpr int u = decltype(load)::value, v = u - T::WLOADS;
        if constexpr (u < T::WLOADS) {
            w4_load16(wsrc[u], lds0 + st * T::STAGE + (T::WLOADS * wave + u) * 1024);
            wsrc[u] += 1024 * KG;
        } else if constexpr (u < T::LOADS) {
            w4_load16(asrc[v], lds0 + st * T::STAGE + T::WBYTES + (T::ALOADS * wave + v) * 1024);
            asrc[v] += 64 * KG;
        }
    };
    int at = 0;  // place of the stage that is next to be computed
    auto start = [&](int n) {  // the first stages
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            if (k < n) each<T::LOADS>([&](auto u) { issue(at + k >= NST ? at + k - NST : at + k, u); });
    };

    // fragment addresses inside a stage: column tile i at wfo + 1024 i, row tile j at afo + 1024 j
    const int wfo = wn * TN * 1024 + 16 * lane;
    const int lrow = wm * TM * 16 + l16;
    const int afo = T::WBYTES + lrow * 64 + ((q ^ ((lrow >> 2) & 3)) << 4);

    Work cur, nxt;
    int v = blockIdx.x;
    if (!find(v, cur)) return;
    rows_of(cur);
    pointers(cur);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    int cb, n = 2 / KG * chunks(cur, cb);  // stages
    start(n);
    bool stored = false;  // the last tile's stores were issued behind this tile's first stages

    for (;;) {
        // at most the loads of `stages` stages and, behind the first stages, the last tile's stores are in
        // flight; other memory instructions of the wave only make the wait longer
        auto wait = [&](int stages, bool behind) {
            if (!stored || !behind) wait_stages<AHEAD - 1, T::LOADS, 0>(stages);
            else if (p.ksplit > 1) wait_stages<AHEAD - 1, T::LOADS, TN * TMG>(stages);
            else wait_stages<AHEAD - 1, T::LOADS, TMG * READS>(stages);
        };
        wait(min(AHEAD - 1, n - 1), true);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");

        const int mt = min(TM, max(0, (cur.rows - wm * TM * 16 + 15) >> 4));  // the wave's row tiles that hold rows
        v4i acc[TN][TM];
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int j = 0; j < TM; ++j) acc[i][j] = v4i{0, 0, 0, 0};
        // W fragments in a ring of four, two steps ahead; A fragments of this stage and the next
        v4i wf[4], af[2][TM];
        // the next tile's rows, looked up before this one's loop; its pointers once this one's loads are out
        const Work now = cur;
        const float *asp = p.as + source_row(srow);
        v += gridDim.x;
        const bool more = find(v, nxt);
        if (more) rows_of(nxt);
        constexpr int AS = (TN + 3) / 4 * 256;  // the rows' scales behind the columns'
        bool scales = false;
        int scale_at = 0;
        auto steps = [&](auto row_tiles, int c, auto parity, auto behind) {
            constexpr int MT = decltype(row_tiles)::value, odd = decltype(parity)::value, ahead = decltype(behind)::value;
            // The next stage has landed: the wave's loads issued after it are those of the stages behind, fewer at the end, and
            // behind the first ones the last tile's stores.
            wait(ahead ? AHEAD - 2 : min(AHEAD - 2, n - 2 - c), c + 1 < AHEAD);
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            const int next = at + 1 == NST ? 0 : at + 1, last = at == 0 ? NST - 1 : at - 1;
            if (!ahead && !scales) {  // no more stages: the scales of the wave's columns and rows, into the place that is free
                scales = true;
                scale_at = last * T::STAGE + wave * (512 * TN);
                const int l = fresh();
#pragma unroll
                for (int u = 0; u < (TN + 3) / 4; ++u) {
                    const int i = min(4 * u + (l >> 4), TN - 1);
                    w4_load4(p.ws + (int64_t)now.e * p.N + 16 * col_tile(now.bx, wn, i) + (l & 15), lds0 + scale_at + 256 * u);
                }
                w4_load4(asp, lds0 + scale_at + AS);
            }
            const uint8_t *sb = lds + at * T::STAGE, *sx = lds + next * T::STAGE;
            each<TN>([&](auto step) {
                constexpr int i = decltype(step)::value, PER = (T::LOADS + TN - 1) / TN;
                if (ahead)  // the loads of the stage AHEAD behind, spread over the steps
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
            const uint8_t *sb = lds + at * T::STAGE;
#pragma unroll
            for (int j = 0; j < MT; ++j) af[0][j] = *(const v4i *)(sb + afo + 1024 * j);
            wf[0] = *(const v4i *)(sb + wfo);
            wf[1] = *(const v4i *)(sb + wfo + 1024);
            int c = 0;
            for (; c + 1 + AHEAD < n; c += 2) {
                steps(row_tiles, c, Const<0>{}, Const<1>{});
                steps(row_tiles, c + 1, Const<1>{}, Const<1>{});
            }
            if (c + AHEAD < n) {  // one more stage to ask for (with AHEAD even there is none)
                steps(row_tiles, c, Const<0>{}, Const<1>{});
                steps(row_tiles, c + 1, Const<1>{}, Const<0>{});
                c += 2;
            }
            if (more) pointers(nxt);
            for (; c + 1 < n; c += 2) {
                steps(row_tiles, c, Const<0>{}, Const<0>{});
                steps(row_tiles, c + 1, Const<1>{}, Const<0>{});
            }
            if (KG > 1 && c < n) steps(row_tiles, c, Const<0>{}, Const<0>{});
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
        float4 ws[TN];
        float as[TMG];
        w4_wait_vm<0>();  // the scales (waited for already, but in tiles of few stages)
#pragma unroll
        for (int i = 0; i < TN; ++i) ws[i] = *(const float4 *)(lds + scale_at + 64 * i + 16 * q);
#pragma unroll
        for (int j = 0; j < TMG; ++j) as[j] = *(const float *)(lds + scale_at + AS + 64 * (group * TMG + j) + 4 * l16);
        __syncthreads();  // every wave is done with this tile's stages
        if constexpr (KG == 2) {  // each group gives the other the sums of half of its row tiles, and adds up the other half
            uint8_t *to = lds + wave * (TN * TMG * 1024), *from = lds_all + (1 - group) * T::RING + wave * (TN * TMG * 1024);
#pragma unroll
            for (int i = 0; i < TN; ++i)
#pragma unroll
                for (int j = 0; j < TMG; ++j) {
                    *(v4i *)(to + (TMG * i + j) * 1024 + 16 * lane) = group ? acc[i][j] : acc[i][TMG + j];
                    if (group) acc[i][j] = acc[i][TMG + j];
                }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < TN; ++i)
#pragma unroll
                for (int j = 0; j < TMG; ++j) acc[i][j] += *(const v4i *)(from + (TMG * i + j) * 1024 + 16 * lane);
            __syncthreads();
        }
        if (more) {
            n = 2 / KG * chunks(nxt, cb);
            start(n);
        }

        // lane holds, per tile (i, j), row 16 (wm TM + group TMG + j) + l16 and columns 4 q .. +3 of tile i.  Stores past the last row
        // or column fall behind their descriptor's end and are dropped, so that every wave issues as many.
        const int l = fresh(), l16 = l & 15, q = l >> 4;
        const int have = max(0, now.rows - wm * TM * 16);  // rows of the wave that exist (at most 64)
        const int64_t row0 = (int64_t)now.r0 + wm * TM * 16;
        if (p.ksplit > 1) {
            const __amdgpu_buffer_rsrc_t out = __builtin_amdgcn_make_buffer_rsrc(
                (void *)(p.part + ((int64_t)now.ks * p.M + row0) * p.N), (short)0,
                (int)((uint32_t)min(have, TM * 16) * (uint32_t)p.N * 4u), 0x00020000);
#pragma unroll
            for (int i = 0; i < TN; ++i) {
                const int t = (now.bx * WN + wn) * TN + i;
#pragma unroll
                for (int j = 0; j < TMG; ++j) {
                    const uint32_t off = ((uint32_t)(16 * (group * TMG + j) + l16) * (uint32_t)p.N + 16 * t + 4 * q) * 4u;
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[i][j]), out, t < tiles ? off : 0xC0000000u, 0, 0);
                }
            }
        } else {
            // through LDS, a row tile at a time in the wave's own share of the stage that was computed last: the pieces of
            // a row, whose order is turned as the A tile's, leave 64 to a store
            const __amdgpu_buffer_rsrc_t out = __builtin_amdgcn_make_buffer_rsrc(
                (void *)(p.c + row0 * ldc), (short)0, (int)((uint32_t)min(have, TM * 16) * (uint32_t)ldc * 2u), 0x00020000);
            uint8_t *mine = lds + (at == 0 ? NST - 1 : at - 1) * T::STAGE + wave * (512 * TN);
            const int64_t n0 = (int64_t)(now.bx * WN + wn) * NT * 16;
#pragma unroll
            for (int j = 0; j < TMG; ++j) {
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    v4f y = i8_scale(acc[i][j], as[j], ws[i]);
                    if constexpr (SILU) y = i8_silu_mul(y, i8_scale(acc[i + NT][j], as[j], ws[i + NT]));
                    const int piece = (2 * i + (q >> 1)) ^ ((l16 * PR >> 4) & (PR - 1));
                    *(uint2 *)(mine + (l16 * PR + piece) * 16 + 8 * (q & 1)) = w4_bf16x4(y);
                }
#pragma unroll
                for (int r = 0; r < READS; ++r) {
                    const int id = 64 * r + l, row = id / PR, piece = id % PR;
                    const uint4 x = *(const uint4 *)(mine + ((row & 15) * PR + (piece ^ ((row * PR >> 4) & (PR - 1)))) * 16);
                    const bool in = row < 16 && n0 + 8 * piece < ldc;
                    const uint32_t off = (uint32_t)(16 * (group * TMG + j) + row) * (uint32_t)ldc * 2u + (uint32_t)(n0 + 8 * piece) * 2u;
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), out, in ? off : 0xC0000000u, 0, 0);
                }
            }
        }
        if (!more) return;
        cur = nxt;
        stored = true;
    }
}

template <class T, bool SILU>
static hipError_t launch_as(I8Args a, const I8TiledCfg &c, hipStream_t s) {
    // the dynamic LDS limit is a per-device function attribute: set it once per device
    static std::once_flag once[64];
    static hipError_t attr_err[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return hipErrorInvalidDevice;
    std::call_once(once[dev], [&] {
        attr_err[dev] = hipFuncSetAttribute((const void *)k_gemm_i8_tiled<T, SILU>,
                                            hipFuncAttributeMaxDynamicSharedMemorySize, T::SMEM);
    });
    if (attr_err[dev] != hipSuccess) return attr_err[dev];
    const int64_t cols = T::BN / (SILU ? 2 : 1), n = SILU ? a.N / 2 : a.N;
    const int64_t nblk = (n + cols - 1) / cols;
    int64_t nrow = (a.M + T::BM - 1) / T::BM;
    if (a.offsets) nrow = ((a.M + std::min(a.E, a.M) * (T::BM - 1)) / T::BM + 7) / 8 * 8;
    const int64_t total = nblk * nrow * c.ksplit;
    if (total >= int64_t(1) << 30) return hipErrorInvalidValue;
    a.nblk = (int)nblk;
    a.nrow = (int)nrow;
    a.ksplit = c.ksplit;
    a.tmagic = a.topk > 1 ? (uint32_t)(((uint64_t(1) << 32) + a.topk - 1) / a.topk) : 0;
    hipLaunchKernelGGL((k_gemm_i8_tiled<T, SILU>), dim3((unsigned)std::min<int64_t>(total, 256 * T::CTAS)), dim3(T::THREADS),
                       T::SMEM, s, a);
    return hipGetLastError();
}
template <class T>
static hipError_t launch_tile(const I8Args &a, const I8TiledCfg &c, hipStream_t s) {
    return a.silu ? launch_as<T, true>(a, c, s) : launch_as<T, false>(a, c, s);
}

hipError_t launch_gemm_i8_tiled(const I8Args &a, const I8TiledCfg &c, hipStream_t s) {
    hipError_t err;
    switch (c.shape) {
        case I8_256X256: err = launch_tile<I8Tile<2, 4, 8, 4, 5, 1>>(a, c, s); break;
        case I8_256X128: err = launch_tile<I8Tile<4, 2, 4, 4, 5, 1>>(a, c, s); break;
        case I8_128X128: err = launch_tile<I8Tile<4, 2, 2, 4, 5, 2>>(a, c, s); break;
        case I8_64X128: err = launch_tile<I8Tile<2, 2, 2, 4, 6, 2>>(a, c, s); break;
        case I8_64X64: err = launch_tile<I8Tile<2, 1, 2, 4, 5, 2, 2>>(a, c, s); break;
        default: err = launch_tile<I8Tile<4, 1, 2, 4, 6, 2>>(a, c, s); break;
    }
    if (err != hipSuccess || c.ksplit == 1) return err;
    return launch_i8_reduce(a, c.ksplit, s);
}

}  // namespace r9k
