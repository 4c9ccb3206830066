// Token rows sorted by expert and back, and the gradients of both.
//
// A slot p = t * topk + j carries token t to expert ids[t][j].  The sort is
// stable: rows go expert by expert, slots of one expert in ascending p, slots
// whose id lies outside [0, E) nowhere.  Positions come from counts alone, with no
// atomic whose order could show, so the same ids always give the same rows.
//   permute              xs[pos[p]] = x[p / topk]
//   unpermute            out[t] = sum_j w[t][j] * y[pos[t][j]]        (also permute's gradient, with w = 1)
//   unpermute_backward   gy[pos[p]] = w[p] * g[t],  gw[p] = <g[t], y[pos[p]]>
// All of it is bound by the rows' bytes: each token row is read once, each sorted
// row read or written once, in 16-byte pieces.  A large copy reaches 4.99 TB/s here
// (reads from the caches count on top).  Rows of 2048 bf16, 8192 tokens, top 8 of 128:
// permute 63 us (4.8 TB/s; with a quarter of the slots dropped 59 us, 46 of them for the
// rows behind 13 of sorting), unpermute 46 us (6.6 TB/s), its gradient 114 us (5.0 TB/s); 4096 rows of 4096 fp32, top 2: 42, 31 and 61 us
// (4.8, 6.5, 5.5 TB/s).  16 tokens: 3.6, 3.3 and 6.6 us, a launch and the loads' latencies.
#include <algorithm>

#include "w4_internal.h"
#include "w4_device.h"

namespace r9k {

namespace {
constexpr int SORT_THREADS = 256;

// 16 bytes of a row as fp32 values, and back (one rounding)
template <bool F32>
struct Row16 {
    static constexpr int N = F32 ? 4 : 8;
    float v[N];
};
template <bool F32>
__device__ __forceinline__ Row16<F32> row_unpack(uint4 x) {
    Row16<F32> r;
    if constexpr (F32) {
        r.v[0] = __uint_as_float(x.x);
        r.v[1] = __uint_as_float(x.y);
        r.v[2] = __uint_as_float(x.z);
        r.v[3] = __uint_as_float(x.w);
    } else {
        r.v[0] = bf16_lo(x.x);
        r.v[1] = bf16_hi(x.x);
        r.v[2] = bf16_lo(x.y);
        r.v[3] = bf16_hi(x.y);
        r.v[4] = bf16_lo(x.z);
        r.v[5] = bf16_hi(x.z);
        r.v[6] = bf16_lo(x.w);
        r.v[7] = bf16_hi(x.w);
    }
    return r;
}
template <bool F32>
__device__ __forceinline__ uint4 row_pack(const Row16<F32> &r) {
    if constexpr (F32) {
        return make_uint4(__float_as_uint(r.v[0]), __float_as_uint(r.v[1]), __float_as_uint(r.v[2]), __float_as_uint(r.v[3]));
    } else {
        const uint2 a = w4_bf16x4(v4f{r.v[0], r.v[1], r.v[2], r.v[3]}), b = w4_bf16x4(v4f{r.v[4], r.v[5], r.v[6], r.v[7]});
        return make_uint4(a.x, a.y, b.x, b.y);
    }
}

// Inclusive sum over a CTA's threads (256), through LDS scratch of 4 ints.
__device__ __forceinline__ int block_scan256(int v, int *scratch) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(v, d, 64);
        if (lane >= d) v += o;
    }
    __syncthreads();
    if (lane == 63) scratch[wave] = v;
    __syncthreads();
    for (int w = 0; w < wave; ++w) v += scratch[w];
    return v;
}

// Lanes of the wave that hold the same key (0 .. 2^bits - 1), among the active ones
__device__ __forceinline__ unsigned long long match_key(int key, int bits) {
    unsigned long long m = __ballot(1);
    for (int b = 0; b < bits; ++b) {
        const unsigned long long one = __ballot((key >> b) & 1);
        m &= ((key >> b) & 1) ? one : ~one;
    }
    return m;
}
}  // namespace

// Slots of a CTA's part, expert by expert (4.6 us for 65536 slots: a launch, and one round
// trip to memory per 256 slots).
__global__ __launch_bounds__(SORT_THREADS) void k_sort_count(const int32_t *__restrict__ ids, int R, int E, int per,
                                                             int32_t *__restrict__ count) {
    extern __shared__ int32_t hist[];
    for (int e = threadIdx.x; e < E; e += SORT_THREADS) hist[e] = 0;
    __syncthreads();
    const int lo = blockIdx.x * per, hi = min(R, lo + per);
    for (int p = lo + (int)threadIdx.x; p < hi; p += SORT_THREADS) {
        const int e = ids[p];
        if (e >= 0 && e < E) atomicAdd(&hist[e], 1);  // whole numbers: the order does not show
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += SORT_THREADS) count[(int64_t)blockIdx.x * E + e] = hist[e];
}

// Every slot's row.  Each CTA adds up the counts of the parts before its own and
// of all parts, scans the experts' totals, counts its own part wave by wave
// (consecutive quarters of it), and ranks a wave's slots 64 at a time.  65536 slots, 128
// experts: 9 us, the chain of the parts' counts (64, 16 loads in flight), the scan and four
// rounds of ranking; it reads the counts again in every CTA rather than in a launch of its own.
__global__ __launch_bounds__(SORT_THREADS) void k_sort_place(const int32_t *__restrict__ ids, int R, int E, int per,
                                                             int bits, const int32_t *__restrict__ count,
                                                             int32_t *__restrict__ src, int32_t *__restrict__ pos,
                                                             int32_t *__restrict__ offsets) {
    extern __shared__ int32_t lds_i[];
    int32_t *next = lds_i;                     // [4][E]: the next row of expert e for wave w
    int32_t *scratch = lds_i + 4 * (int64_t)E; // [4], and the running total
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int part = blockIdx.x, parts = gridDim.x;

    int run = 0;  // rows of the experts before this step's 256
    for (int e0 = 0; e0 < E; e0 += SORT_THREADS) {
        const int e = e0 + tid;
        int before = 0, all = 0;
        if (e < E) {
#pragma unroll 16
            for (int b = 0; b < parts; ++b) {
                const int c = count[(int64_t)b * E + e];
                all += c;
                before += b < part ? c : 0;
            }
        }
        const int incl = block_scan256(all, scratch);
        if (tid == SORT_THREADS - 1) scratch[4] = incl;
        __syncthreads();
        const int first = run + incl - all;
        if (e < E) {
            next[e] = first + before;
            if (part == 0) offsets[e] = first;
        }
        run += scratch[4];
        __syncthreads();
    }
    if (part == 0) {
        if (tid == 0) offsets[E] = run;
        for (int r = run + tid; r < R; r += SORT_THREADS) src[r] = -1;  // rows that no slot fills
    }

    // wave w's slots: [lo, hi); first counts of the waves before it
    const int quarter = per / 4;
    const int lo = min(R, part * per + wave * quarter), hi = min(R, lo + quarter);
    for (int e = tid; e < 3 * E; e += SORT_THREADS) next[E + e] = 0;
    __syncthreads();
    if (wave < 3)
        for (int p = lo + lane; p < hi; p += 64) {
            const int e = ids[p];
            if (e >= 0 && e < E) atomicAdd(&next[(wave + 1) * (int64_t)E + e], 1);
        }
    __syncthreads();
    for (int e = tid; e < E; e += SORT_THREADS) {
        int x = next[e];
        for (int w = 1; w < 4; ++w) {
            x += next[w * (int64_t)E + e];
            next[w * (int64_t)E + e] = x;
        }
    }
    __syncthreads();
    int32_t *mine = next + wave * (int64_t)E;
    for (int p0 = lo; p0 < hi; p0 += 64) {
        const int p = p0 + lane;
        int e = p < hi ? ids[p] : -1;
        if (e < 0 || e >= E) e = -1;
        const unsigned long long same = match_key(e + 1, bits);
        if (e >= 0) {
            const int row = mine[e] + __popcll(same & ((1ull << lane) - 1));
            pos[p] = row;
            src[row] = p;
        } else if (p < hi) {
            pos[p] = -1;
        }
        __builtin_amdgcn_wave_barrier();
        if (e >= 0 && (same >> lane) == 1) mine[e] += __popcll(same);  // the key's last lane
        __builtin_amdgcn_wave_barrier();
    }
}

// Few slots: sort and rows in one launch.  CTA t counts, for each slot of token t, the
// slots before it in the order (those of lower experts, and earlier ones of its own),
// one slot a wave at a time, and copies the token's row; the last CTA adds up the
// experts' first rows and marks the rows that no slot fills.  R * R comparisons in all.
__global__ __launch_bounds__(SORT_THREADS) void k_sort_small(const int32_t *__restrict__ ids, int T, int topk, int E,
                                                             const uint4 *__restrict__ x, int64_t w16,
                                                             uint4 *__restrict__ xs, int32_t *__restrict__ src,
                                                             int32_t *__restrict__ pos, int32_t *__restrict__ offsets) {
    extern __shared__ int32_t lds_i[];  // [max(E, topk)] and 5 for the scan
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int R = T * topk, t = blockIdx.x;
    if (t == T) {
        int32_t *scratch = lds_i + max(E, topk);
        for (int e = tid; e < E; e += SORT_THREADS) lds_i[e] = 0;
        __syncthreads();
        for (int p = tid; p < R; p += SORT_THREADS) {
            const int e = ids[p];
            if (e >= 0 && e < E) atomicAdd(&lds_i[e], 1);  // whole numbers: the order does not show
        }
        __syncthreads();
        int run = 0;
        for (int e0 = 0; e0 < E; e0 += SORT_THREADS) {
            const int e = e0 + tid, n = e < E ? lds_i[e] : 0;
            const int incl = block_scan256(n, scratch);
            if (tid == SORT_THREADS - 1) scratch[4] = incl;
            __syncthreads();
            if (e < E) offsets[e] = run + incl - n;
            run += scratch[4];
            __syncthreads();
        }
        if (tid == 0) offsets[E] = run;
        for (int r = run + tid; r < R; r += SORT_THREADS) src[r] = -1;
        return;
    }
    // the row's pieces are on their way while the slots are counted
    uint4 v = make_uint4(0, 0, 0, 0);
    if (x && tid < w16) v = x[(int64_t)t * w16 + tid];
    for (int j = wave; j < topk; j += SORT_THREADS / 64) {
        const int p = t * topk + j, e = ids[p];
        int row = -1;
        if (e >= 0 && e < E) {
            int n = 0;
            for (int i = lane; i < R; i += 64) {
                const int o = ids[i];
                n += (o >= 0 && o < e) || (o == e && i < p);
            }
            row = __builtin_amdgcn_readlane(w4_wave_scan(n), 63);
        }
        if (lane == 0) {
            lds_i[j] = row;
            pos[p] = row;
            if (row >= 0) src[row] = p;
        }
    }
    if (!x) return;
    __syncthreads();
    for (int64_t i = tid; i < w16; i += SORT_THREADS) {
        if (i >= SORT_THREADS) v = x[(int64_t)t * w16 + i];
        for (int j = 0; j < topk; ++j) {
            const int64_t r = lds_i[j];
            if (r >= 0) xs[r * w16 + i] = v;
        }
    }
}

// Each token's row to the rows of its slots; 2^lpt threads a token, 256 >> lpt tokens a CTA
// (rows of 512 bytes, 16384 tokens, top 4: 18.3 us with the sort; a CTA a token 21.0).
__global__ __launch_bounds__(SORT_THREADS) void k_permute_rows(const uint4 *__restrict__ x, int64_t w16, int topk,
                                                               int64_t T, int lpt, const int32_t *__restrict__ pos,
                                                               uint4 *__restrict__ xs) {
    const int64_t t = ((int64_t)blockIdx.x << (8 - lpt)) + (threadIdx.x >> lpt), R = T * topk;
    if (t >= T) return;
    const int32_t *pt = pos + t * topk;
    for (int64_t i = threadIdx.x & ((1 << lpt) - 1); i < w16; i += 1 << lpt) {
        const uint4 v = x[t * w16 + i];
        for (int j = 0; j < topk; ++j) {
            const int64_t r = pt[j];
            if (r >= 0 && r < R) xs[r * w16 + i] = v;
        }
    }
}

// A token takes 2^lpt threads (as many as its row has 16-byte pieces, up to the CTA),
// a CTA 256 >> lpt tokens (rows of 512 bytes, 16384 tokens, top 4: 7.3 us, a CTA a token
// 11.0); WIDE: the CTA, so that its positions and weights are scalars (rows of 4096
// bytes, 8192 tokens, top 8: 45.9 us, 48.1 without; 16 tokens 3.3 and 3.8).
// Four rows are asked for at a time.  Dropped slots read row 0 and drop what they read.
template <bool F32, bool WIDE>
__global__ __launch_bounds__(SORT_THREADS) void k_unpermute(const uint4 *__restrict__ y, int64_t w16, int topk,
                                                            int64_t T, int lpt, const int32_t *__restrict__ pos,
                                                            const float *__restrict__ w, uint4 *__restrict__ out) {
    constexpr int B = 4, N = Row16<F32>::N;
    const int64_t t = WIDE ? (int64_t)blockIdx.x : ((int64_t)blockIdx.x << (8 - lpt)) + (threadIdx.x >> lpt), R = T * topk;
    const int64_t i = WIDE ? (int64_t)blockIdx.y * SORT_THREADS + threadIdx.x
                           : ((int64_t)blockIdx.y << lpt) + (threadIdx.x & ((1 << lpt) - 1));
    if (t >= T || i >= w16) return;
    Row16<F32> acc;
#pragma unroll
    for (int k = 0; k < N; ++k) acc.v[k] = 0.0f;
    for (int j0 = 0; j0 < topk; j0 += B) {
        uint4 v[B] = {};
        float g[B] = {};
        bool live[B];
#pragma unroll
        for (int b = 0; b < B; ++b) {
            live[b] = false;
            if (j0 + b < topk) {
                const int64_t r = pos[t * topk + j0 + b];
                live[b] = r >= 0 && r < R;
                g[b] = w ? w[t * topk + j0 + b] : 1.0f;
                v[b] = y[(live[b] ? r : 0) * w16 + i];
            }
        }
#pragma unroll
        for (int b = 0; b < B; ++b) {
            if (j0 + b >= topk) continue;
            const Row16<F32> x = row_unpack<F32>(v[b]);
#pragma unroll
            for (int k = 0; k < N; ++k) acc.v[k] = live[b] ? __builtin_fmaf(g[b], x.v[k], acc.v[k]) : acc.v[k];
        }
    }
    out[t * w16 + i] = row_pack<F32>(acc);
}

// Rows of up to 64 pieces (WIDE false): 2^lpt <= 64 threads a token, whose sums stay in
// the wave (rows of 512 bytes, 16384 tokens, top 4: 13.5 us; a CTA a token 35.7).  Longer
// ones: a CTA a token, sums through LDS.  The token's row is read once from memory and
// again from L1 for each slot.
template <bool F32, bool WIDE>
__global__ __launch_bounds__(SORT_THREADS) void k_unpermute_bwd(const uint4 *__restrict__ g, const uint4 *__restrict__ y,
                                                                int64_t w16, int topk, int64_t T, int lpt,
                                                                const int32_t *__restrict__ pos,
                                                                const float *__restrict__ w, uint4 *__restrict__ gy,
                                                                float *__restrict__ gw) {
    __shared__ float part[4];
    const int per = WIDE ? SORT_THREADS : 1 << lpt, me = WIDE ? threadIdx.x : threadIdx.x & (per - 1);
    const int64_t t = WIDE ? (int64_t)blockIdx.x : ((int64_t)blockIdx.x << (8 - lpt)) + (threadIdx.x >> lpt), R = T * topk;
    if (!WIDE && t >= T) return;  // a token's threads leave together
    for (int j = 0; j < topk; ++j) {
        const int64_t r = pos[t * topk + j];
        float dot = 0.0f;
        if (r >= 0 && r < R) {
            const float s = w[t * topk + j];
            for (int64_t i = me; i < w16; i += per) {
                const Row16<F32> a = row_unpack<F32>(g[t * w16 + i]), b = row_unpack<F32>(y[r * w16 + i]);
                Row16<F32> o;
#pragma unroll
                for (int k = 0; k < Row16<F32>::N; ++k) {
                    dot = __builtin_fmaf(a.v[k], b.v[k], dot);
                    o.v[k] = s * a.v[k];
                }
                gy[r * w16 + i] = row_pack<F32>(o);
            }
        }
        if (WIDE) {
#pragma unroll
            for (int d = 32; d; d >>= 1) dot += __shfl_xor(dot, d, 64);
            __syncthreads();
            if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = dot;
            __syncthreads();
            if (threadIdx.x == 0) gw[t * topk + j] = (part[0] + part[1]) + (part[2] + part[3]);
        } else {
            for (int d = per >> 1; d; d >>= 1) dot += __shfl_xor(dot, d, 64);
            if (me == 0) gw[t * topk + j] = dot;
        }
    }
}

// log2 of the threads a token's row takes: as many as it has 16-byte pieces, 4 to 256
static int row_lpt(int64_t w16) {
    int l = 2;
    while (l < 8 && (int64_t(1) << l) < w16) ++l;
    return l;
}

// Slots a part holds: a multiple of 256, parts few enough that adding up their
// counts stays short.
static int sort_part(int64_t R) { return (int)std::max<int64_t>(1024, ((R + 255) / 256 + 255) / 256 * 256); }

// Slots up to which one launch sorts them by comparing all pairs.  Rows of 2048 bf16,
// top 8 of 128, one launch and three: 512 slots 5.0 and 10.4 us, 1024 6.9 and 11.3,
// 2048 10.9 and 12.2, 4096 19.5 and 14.4.
constexpr int64_t SORT_SMALL = 2048;

size_t moe_sort_workspace(int64_t R, int64_t E) {
    if (R <= SORT_SMALL) return 0;
    const int64_t per = sort_part(R);
    return align_up((size_t)((R + per - 1) / per) * (size_t)E * 4, 256);
}

hipError_t launch_moe_permute(const SortArgs &a, hipStream_t s) {
    const int64_t R = a.T * a.topk;
    if (R <= SORT_SMALL) {
        hipLaunchKernelGGL(k_sort_small, dim3((unsigned)a.T + 1), dim3(SORT_THREADS),
                           (size_t)std::max(a.E, a.topk) * 4 + 32, s, a.ids, (int)a.T, (int)a.topk, (int)a.E,
                           (const uint4 *)a.x, a.row_bytes / 16, (uint4 *)a.xs, a.src, a.pos, a.offsets);
        return hipGetLastError();
    }
    const int per = sort_part(R);
    const unsigned parts = (unsigned)((R + per - 1) / per);
    const int lpt = row_lpt(a.row_bytes / 16), tpc = 256 >> lpt;
    int bits = 1;
    while ((1 << bits) < a.E + 1) ++bits;
    hipLaunchKernelGGL(k_sort_count, dim3(parts), dim3(SORT_THREADS), (size_t)a.E * 4, s, a.ids, (int)R, (int)a.E, per,
                       a.count);
    hipLaunchKernelGGL(k_sort_place, dim3(parts), dim3(SORT_THREADS), (size_t)a.E * 16 + 32, s, a.ids, (int)R,
                       (int)a.E, per, bits, a.count, a.src, a.pos, a.offsets);
    if (a.x)
        hipLaunchKernelGGL(k_permute_rows, dim3((unsigned)((a.T + tpc - 1) / tpc)), dim3(SORT_THREADS), 0, s,
                           (const uint4 *)a.x, a.row_bytes / 16, (int)a.topk, a.T, lpt, a.pos, (uint4 *)a.xs);
    return hipGetLastError();
}

hipError_t launch_moe_unpermute(const void *y, bool f32, int64_t row_bytes, int64_t T, int64_t topk,
                                const int32_t *pos, const float *w, void *out, hipStream_t s) {
    const int64_t w16 = row_bytes / 16;
    const int lpt = row_lpt(w16), tpc = 256 >> lpt;
    const dim3 grid((unsigned)((T + tpc - 1) / tpc), (unsigned)((w16 + (1 << lpt) - 1) >> lpt));
    const bool wide = lpt == 8;
    auto kernel = f32 ? (wide ? k_unpermute<true, true> : k_unpermute<true, false>)
                      : (wide ? k_unpermute<false, true> : k_unpermute<false, false>);
    hipLaunchKernelGGL(kernel, grid, dim3(SORT_THREADS), 0, s, (const uint4 *)y, w16, (int)topk, T, lpt, pos, w,
                       (uint4 *)out);
    return hipGetLastError();
}

hipError_t launch_moe_unpermute_backward(const void *g, const void *y, bool f32, int64_t row_bytes, int64_t T,
                                         int64_t topk, const int32_t *pos, const float *w, void *gy, float *gw,
                                         hipStream_t s) {
    const int64_t w16 = row_bytes / 16;
    const bool wide = w16 > 64;
    const int lpt = row_lpt(w16), tpc = wide ? 1 : 256 >> lpt;
    auto kernel = f32 ? (wide ? k_unpermute_bwd<true, true> : k_unpermute_bwd<true, false>)
                      : (wide ? k_unpermute_bwd<false, true> : k_unpermute_bwd<false, false>);
    hipLaunchKernelGGL(kernel, dim3((unsigned)((T + tpc - 1) / tpc)), dim3(SORT_THREADS), 0, s, (const uint4 *)g,
                       (const uint4 *)y, w16, (int)topk, T, lpt, pos, w, (uint4 *)gy, gw);
    return hipGetLastError();
}

}  // namespace r9k
