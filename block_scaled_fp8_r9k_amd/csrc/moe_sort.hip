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
// row read or written once, in 16-byte pieces.
#include <algorithm>

#include "r9k_internal.h"
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

// Slots of a CTA's part, expert by expert.
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
// (consecutive quarters of it), and ranks a wave's slots 64 at a time.
__global__ __launch_bounds__(SORT_THREADS) void k_sort_place(const int32_t *__restrict__ ids, int R, int E, int per,
                                                             int bits, int parts, const int32_t *__restrict__ count,
                                                             int32_t *__restrict__ src, int32_t *__restrict__ pos,
                                                             int32_t *__restrict__ offsets) {
    extern __shared__ int32_t lds_i[];
    int32_t *next = lds_i;                     // [4][E]: the next row of expert e for wave w
    int32_t *scratch = lds_i + 4 * (int64_t)E; // [4], and the running total
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int part = blockIdx.x;

    int run = 0;  // rows of the experts before this step's 256
    for (int e0 = 0; e0 < E; e0 += SORT_THREADS) {
        const int e = e0 + tid;
        int before = 0, all = 0;
        if (e < E) {
            for (int b = 0; b < parts; ++b) {
                const int c = count[(int64_t)b * E + e];
                all += c;
                if (b < part) before += c;
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

// Each token's row to the rows of its slots; one CTA a token.
__global__ __launch_bounds__(SORT_THREADS) void k_permute_rows(const uint4 *__restrict__ x, int64_t w16, int topk,
                                                               int64_t R, const int32_t *__restrict__ pos,
                                                               uint4 *__restrict__ xs) {
    const int64_t t = blockIdx.x;
    const int32_t *pt = pos + t * topk;
    for (int64_t i = threadIdx.x; i < w16; i += SORT_THREADS) {
        const uint4 v = x[t * w16 + i];
        for (int j = 0; j < topk; ++j) {
            const int64_t r = pt[j];
            if (r >= 0 && r < R) xs[r * w16 + i] = v;
        }
    }
}

template <bool F32>
__global__ __launch_bounds__(SORT_THREADS) void k_unpermute(const uint4 *__restrict__ y, int64_t w16, int topk,
                                                            int64_t R, const int32_t *__restrict__ pos,
                                                            const float *__restrict__ w, uint4 *__restrict__ out) {
    const int64_t t = blockIdx.x;
    const int64_t i = (int64_t)blockIdx.y * SORT_THREADS + threadIdx.x;
    if (i >= w16) return;
    Row16<F32> acc;
#pragma unroll
    for (int k = 0; k < Row16<F32>::N; ++k) acc.v[k] = 0.0f;
    for (int j = 0; j < topk; ++j) {
        const int64_t r = pos[t * topk + j];
        if (r < 0 || r >= R) continue;
        const float g = w ? w[t * topk + j] : 1.0f;
        const Row16<F32> v = row_unpack<F32>(y[r * w16 + i]);
#pragma unroll
        for (int k = 0; k < Row16<F32>::N; ++k) acc.v[k] = __builtin_fmaf(g, v.v[k], acc.v[k]);
    }
    out[t * w16 + i] = row_pack<F32>(acc);
}

template <bool F32>
__global__ __launch_bounds__(SORT_THREADS) void k_unpermute_bwd(const uint4 *__restrict__ g, const uint4 *__restrict__ y,
                                                                int64_t w16, int topk, int64_t R,
                                                                const int32_t *__restrict__ pos,
                                                                const float *__restrict__ w, uint4 *__restrict__ gy,
                                                                float *__restrict__ gw) {
    __shared__ float part[4];
    const int64_t t = blockIdx.x;
    for (int j = 0; j < topk; ++j) {
        const int64_t r = pos[t * topk + j];
        float dot = 0.0f;
        if (r >= 0 && r < R) {
            const float s = w[t * topk + j];
            for (int64_t i = threadIdx.x; i < w16; i += SORT_THREADS) {
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
#pragma unroll
        for (int d = 32; d; d >>= 1) dot += __shfl_xor(dot, d, 64);
        __syncthreads();
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = dot;
        __syncthreads();
        if (threadIdx.x == 0) gw[t * topk + j] = (part[0] + part[1]) + (part[2] + part[3]);
    }
}

// Slots a part holds: a multiple of 256, parts few enough that adding up their
// counts stays short.
static int sort_part(int64_t R) { return (int)std::max<int64_t>(1024, ((R + 255) / 256 + 255) / 256 * 256); }

size_t moe_sort_workspace(int64_t R, int64_t E) {
    const int64_t per = sort_part(R);
    return align_up((size_t)((R + per - 1) / per) * (size_t)E * 4, 256);
}

hipError_t launch_moe_permute(const SortArgs &a, hipStream_t s) {
    const int64_t R = a.T * a.topk;
    const int per = sort_part(R);
    const unsigned parts = (unsigned)((R + per - 1) / per);
    int bits = 1;
    while ((1 << bits) < a.E + 1) ++bits;
    if (R)
        hipLaunchKernelGGL(k_sort_count, dim3(parts), dim3(SORT_THREADS), (size_t)a.E * 4, s, a.ids, (int)R, (int)a.E,
                           per, a.count);
    hipLaunchKernelGGL(k_sort_place, dim3(std::max(parts, 1u)), dim3(SORT_THREADS), (size_t)a.E * 16 + 32, s, a.ids, (int)R,
                       (int)a.E, per, bits, (int)parts, a.count, a.src, a.pos, a.offsets);
    if (a.x && R)
        hipLaunchKernelGGL(k_permute_rows, dim3((unsigned)a.T), dim3(SORT_THREADS), 0, s, (const uint4 *)a.x,
                           a.row_bytes / 16, (int)a.topk, R, a.pos, (uint4 *)a.xs);
    return hipGetLastError();
}

hipError_t launch_moe_unpermute(const void *y, bool f32, int64_t row_bytes, int64_t T, int64_t topk,
                                const int32_t *pos, const float *w, void *out, hipStream_t s) {
    const int64_t w16 = row_bytes / 16;
    const dim3 grid((unsigned)T, (unsigned)((w16 + SORT_THREADS - 1) / SORT_THREADS));
    if (f32)
        hipLaunchKernelGGL(k_unpermute<true>, grid, dim3(SORT_THREADS), 0, s, (const uint4 *)y, w16, (int)topk, T * topk,
                           pos, w, (uint4 *)out);
    else
        hipLaunchKernelGGL(k_unpermute<false>, grid, dim3(SORT_THREADS), 0, s, (const uint4 *)y, w16, (int)topk,
                           T * topk, pos, w, (uint4 *)out);
    return hipGetLastError();
}

hipError_t launch_moe_unpermute_backward(const void *g, const void *y, bool f32, int64_t row_bytes, int64_t T,
                                         int64_t topk, const int32_t *pos, const float *w, void *gy, float *gw,
                                         hipStream_t s) {
    const int64_t w16 = row_bytes / 16;
    if (f32)
        hipLaunchKernelGGL(k_unpermute_bwd<true>, dim3((unsigned)T), dim3(SORT_THREADS), 0, s, (const uint4 *)g,
                           (const uint4 *)y, w16, (int)topk, T * topk, pos, w, (uint4 *)gy, gw);
    else
        hipLaunchKernelGGL(k_unpermute_bwd<false>, dim3((unsigned)T), dim3(SORT_THREADS), 0, s, (const uint4 *)g,
                           (const uint4 *)y, w16, (int)topk, T * topk, pos, w, (uint4 *)gy, gw);
    return hipGetLastError();
}

}  // namespace r9k
