// The router's training operators: the load balance loss with the experts' counts, and the
// gradient of the router's logits.
//
//   counts[e] = slots of kept tokens with id e, n = kept tokens, psum[e] = sum_t p[t][e],
//   loss      = E / (topk n^2) * sum_e counts[e] psum[e]                (0 where n = 0)
//   g[t][i]   = gloss / n * p[t][i] * (f[i] - sum_e f[e] p[t][e]),  f[e] = E counts[e] / (topk n),
//               0 for a token that is not kept,
//             + sum over j with ids[t][j] = i of w[t][j] (gw[t][j] - sum_i w[t][i] gw[t][i])
//
// p is the softmax of a token's logits over all experts, in fp32; a logit of -inf has p = 0,
// also where every logit of the token is.
//
// A token takes 2^LPT neighbouring lanes (8 to 64), a lane NV pieces of VEC consecutive
// experts, 16 bytes where the rows allow it; a wave walks over tokens 64 >> LPT at a time
// and asks for U such steps before it computes the first.
#include <algorithm>

#include "i8_device.h"
#include "i8_internal.h"

namespace r9k {

namespace {

// A piece as it lies in memory
template <bool F32, int VEC>
struct Piece {
    typedef typename std::conditional<VEC == 1, typename std::conditional<F32, uint32_t, uint16_t>::type, uint4>::type type;
};
template <bool F32, int VEC>
__device__ __forceinline__ void unpack(typename Piece<F32, VEC>::type v, float (&x)[VEC]) {
    if constexpr (VEC == 1) {
        x[0] = __uint_as_float((uint32_t)v << (F32 ? 0 : 16));
    } else if constexpr (F32) {
        x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
    } else {
        x[0] = bf16_lo(v.x), x[1] = bf16_hi(v.x), x[2] = bf16_lo(v.y), x[3] = bf16_hi(v.y);
        x[4] = bf16_lo(v.z), x[5] = bf16_hi(v.z), x[6] = bf16_lo(v.w), x[7] = bf16_hi(v.w);
    }
}
template <bool F32, int VEC>
__device__ __forceinline__ void store_piece(void *row, int at, const float (&x)[VEC]) {
    if constexpr (F32 && VEC == 4) {
        *(float4 *)((float *)row + at) = make_float4(x[0], x[1], x[2], x[3]);
    } else if constexpr (F32) {
        ((float *)row)[at] = x[0];
    } else if constexpr (VEC == 8) {
        const uint2 a = w4_bf16x4(v4f{x[0], x[1], x[2], x[3]}), b = w4_bf16x4(v4f{x[4], x[5], x[6], x[7]});
        *(uint4 *)((uint16_t *)row + at) = make_uint4(a.x, a.y, b.x, b.y);
    } else {
        ((uint16_t *)row)[at] = (uint16_t)w4_bf16x4(v4f{x[0], 0.0f, 0.0f, 0.0f}).x;
    }
}

// The lane's pieces of row t of the logits, as they lie there (lanes past the row's end read its first piece),
// and whether the mask keeps the token.  Nothing here waits for what it loads; finish_row does.
template <bool F32, int VEC, int NV, int L>
struct Row {
    typename Piece<F32, VEC>::type v[NV];
    uint8_t keep;
    __device__ __forceinline__ void load(const void *logits, const uint8_t *mask, int64_t t, int E, int me) {
        typedef typename Piece<F32, VEC>::type P;
        const P *row = (const P *)((const uint8_t *)logits + t * E * (F32 ? 4 : 2));
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = row[(i * L + me) * VEC < E ? i * L + me : 0];
        keep = mask ? mask[t] : 1;
    }
    // -inf past the row's end, and everywhere in a row that does not count, whatever it holds
    __device__ __forceinline__ void finish(bool live, int E, int me, float (&x)[NV][VEC]) const {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            unpack<F32, VEC>(v[i], x[i]);
            const bool in = live && (i * L + me) * VEC < E;
#pragma unroll
            for (int k = 0; k < VEC; ++k) x[i][k] = in ? x[i][k] : -__builtin_inff();
        }
    }
};

// A lane's piece of a row in LDS, read and written in the order of the program
template <int VEC>
__device__ __forceinline__ void lds_clear(volatile float *at) {
    if constexpr (VEC == 1) *at = 0.0f;
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) ((volatile v4f *)at)[i] = v4f{0.f, 0.f, 0.f, 0.f};
}
template <int VEC>
__device__ __forceinline__ void lds_add(volatile float *at, float (&x)[VEC]) {
    if constexpr (VEC == 1) x[0] += *at;
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
        const v4f y = ((volatile v4f *)at)[i];
        x[4 * i] += y[0], x[4 * i + 1] += y[1], x[4 * i + 2] += y[2], x[4 * i + 3] += y[3];
    }
}

// op over the token's 2^LPT lanes (8 to 64), the same in all of them: DPP within a row of 16
// (quad_perm [1,0,3,2], [2,3,0,1], row_half_mirror, row_mirror), then swaps of rows and of
// halves.  Every lane must be active.
template <int LPT, class OP>
__device__ __forceinline__ float over_lanes(float v, OP op) {
    auto dpp = [&](auto ctrl) {
        return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), decltype(ctrl)::value, 0xF, 0xF, false));
    };
    v = op(v, dpp(std::integral_constant<int, 0xB1>{}));
    v = op(v, dpp(std::integral_constant<int, 0x4E>{}));
    v = op(v, dpp(std::integral_constant<int, 0x141>{}));
    if constexpr (LPT > 3) v = op(v, dpp(std::integral_constant<int, 0x140>{}));
    if constexpr (LPT > 4) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = op(__uint_as_float(r[0]), __uint_as_float(r[1]));
    }
    if constexpr (LPT > 5) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = op(__uint_as_float(r[0]), __uint_as_float(r[1]));
    }
    return v;
}
// v added over the wave's 64 >> LPT tokens, the same in all of them
template <int LPT>
__device__ __forceinline__ float over_tokens(float v) {
    if constexpr (LPT < 4) v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x128, 0xF, 0xF, false));  // row_ror 8
    if constexpr (LPT < 5) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    if constexpr (LPT < 6) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    return v;
}
struct Add {
    __device__ float operator()(float a, float b) const { return a + b; }
};
struct Max {
    __device__ float operator()(float a, float b) const { return fmaxf(a, b); }
};

// exp(x - max) in place of the token's logits (experts past E as -inf); returns 1 / their sum, 0 where
// every logit is -inf.  exp is v_exp_f32 of the difference d to the maximum times log2 e: d, the product and the constant each
// round once, which moves the result by up to 2.2 d 2^-24 of itself (7 units of 2^-24 at d = 3, 66 at 30, where the
// probability is 1e-13), and v_exp_f32 by one unit more; 0 below 2^-126; the reciprocal v_rcp_f32's, one rounding off.
template <int LPT, int VEC, int NV>
__device__ __forceinline__ float softmax(float (&x)[NV][VEC]) {
    float mx = -__builtin_inff(), sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int v = 0; v < VEC; ++v) mx = fmaxf(mx, x[i][v]);
    mx = over_lanes<LPT>(mx, Max{});
    mx = mx == -__builtin_inff() ? 0.0f : mx;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            x[i][v] = __builtin_amdgcn_exp2f((x[i][v] - mx) * 1.44269504f);
            sum += x[i][v];
        }
    sum = over_lanes<LPT>(sum, Add{});
    return sum == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(sum);
}

// a part's sums and counts: E of each, padded to whole 16 bytes
__host__ __device__ constexpr int part_pitch(int E) { return (E + 3) & ~3; }
}  // namespace

// Waves of a CTA, at most: 16 where a lane holds few values, 4 where its registers and the sums in LDS are many
__host__ __device__ constexpr int balance_waves(int values) { return values > 16 ? 4 : 16; }

// The loss from the sum of counts[e] psum[e] over the wave's lanes, in one order.
__device__ __forceinline__ void put_loss(const BalanceArgs &p, double dot, int kept) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) dot += __shfl_xor(dot, d, 64);
    const double n = (double)kept;
    if ((threadIdx.x & 63) == 0) p.loss[0] = kept > 0 ? (float)(dot * (double)p.E / ((double)p.topk * n * n)) : 0.0f;
}

// A CTA's tokens, consecutive ones: their probabilities and counts, into its part of the
// workspace, or with one CTA the outputs.  Kernel trace, medians: 65536 tokens of 256 experts in bf16 12.8 us for 36 MB,
// 2.8 TB/s, in fp32 17.1 us for 69 MB, 4 TB/s; each of the 256 CTAs, one a compute unit, asks for its rows in about eight (16)
// steps, and its start, the histogram and its waves' sums are not hidden behind them.  1023 tokens of 128 in fp32: 5.2 us.
template <bool F32, int VEC, int NV, int LPT>
__global__ __launch_bounds__(64 * balance_waves(NV * VEC)) void k_balance(BalanceArgs p, int64_t per) {
    constexpr int U = NV == 1 ? 4 : 1, L = 1 << LPT, TPW = 64 >> LPT;
    extern __shared__ __align__(16) uint8_t lds[];
    const int E = (int)p.E, topk = (int)p.topk, pitch = part_pitch(E);
    double *red = (double *)lds;                   // [16]
    int32_t *kept = (int32_t *)lds + 32;           // [1], padded to 16 bytes
    int32_t *hist = kept + 4;                      // [pitch]
    float *sums = (float *)hist + pitch;           // [waves][pitch]
    const uint32_t tid = threadIdx.x, nt = blockDim.x;
    const int nw = nt >> 6, lane = tid & 63, wave = tid >> 6, me = lane & (L - 1);
    const int64_t lo = min(p.T, blockIdx.x * per), hi = min(p.T, lo + per);

    for (int e = tid; e < pitch; e += (int)nt) hist[e] = 0;
    if (tid == 0) *kept = p.mask ? 0 : (int32_t)(hi - lo);
    __syncthreads();

    Row<F32, VEC, NV, L> row[U];
    auto load = [&](int64_t t0) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            row[u].load(p.logits, p.mask, min(t0 + (int64_t)u * nw * TPW + (lane >> LPT), p.T - 1), E, me);
    };
    int64_t t0 = lo + wave * TPW;
    if (p.T > 0) load(t0);
    // the first slots of the thread and their tokens' masks, on their way meanwhile
    constexpr int S = 4;
    const uint32_t slots = (uint32_t)((hi - lo) * topk);  // a CTA's, below 2^32
    int id[S];
    uint8_t keep[S];
    if (slots)
#pragma unroll
        for (int k = 0; k < S; ++k) {
            const uint32_t i = min(tid + k * nt, slots - 1);
            id[k] = p.ids[lo * topk + i];
            keep[k] = p.mask ? p.mask[lo + i / (uint32_t)topk] : 1;
        }
    float acc[NV][VEC] = {};
    while (t0 < hi) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float x[NV][VEC];
            row[u].finish(t0 + (int64_t)u * nw * TPW + (lane >> LPT) < hi && row[u].keep, E, me, x);
            const float inv = softmax<LPT, VEC, NV>(x);
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int v = 0; v < VEC; ++v) acc[i][v] = __builtin_fmaf(x[i][v], inv, acc[i][v]);
        }
        t0 += nw * TPW * U;
        if (t0 < hi) load(t0);
    }
    // the slots' counts: whole numbers, so that the order of these additions does not show
    auto count = [&](int e, bool counts) {
        if (e >= 0 && e < E && counts) atomicAdd(&hist[e], 1);
    };
#pragma unroll
    for (int k = 0; k < S; ++k)
        if (tid + k * nt < slots) count(id[k], keep[k]);
    for (uint32_t i = tid + S * nt; i < slots; i += nt) count(p.ids[lo * topk + i], !p.mask || p.mask[lo + i / (uint32_t)topk]);
    if (p.mask)
        for (int64_t t = lo + tid; t < hi; t += nt)
            if (p.mask[t]) atomicAdd(kept, 1);
    // the wave's tokens, then the waves, in one order
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = (i * L + me) * VEC;
#pragma unroll
        for (int v = 0; v < VEC; ++v) acc[i][v] = over_tokens<LPT>(acc[i][v]);
        if (lane >= L || e >= E) continue;
        if constexpr (VEC == 1) sums[wave * pitch + e] = acc[i][0];
#pragma unroll
        for (int v = 0; v < VEC / 4; ++v)
            *(v4f *)(sums + wave * pitch + e + 4 * v) = v4f{acc[i][4 * v], acc[i][4 * v + 1], acc[i][4 * v + 2], acc[i][4 * v + 3]};
    }
    __syncthreads();
    const bool only = gridDim.x == 1;
    double dot = 0.0;
    for (int e = tid; e < E; e += (int)nt) {
        float s = 0.0f;
#pragma unroll 4
        for (int w = 0; w < nw; ++w) s += sums[w * pitch + e];  // 1, 4, 8 or 16
        (only ? p.psum : p.part_p + (int64_t)blockIdx.x * pitch)[e] = s;
        (only ? p.counts : p.part_c + (int64_t)blockIdx.x * pitch)[e] = hist[e];
        dot += (double)hist[e] * (double)s;
    }
    if (tid == 0) (only ? p.counts + E : p.part_n + blockIdx.x)[0] = *kept;
    if (blockIdx.x == 0 && tid == 0 && !only) *p.ticket = 0;  // for the next launch
    if (!only) return;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) dot += __shfl_xor(dot, d, 64);
    if (lane == 0) red[wave] = dot;
    __syncthreads();
    if (wave == 0) put_loss(p, lane < nw ? red[lane] : 0.0, *kept);
}

// The parts, added up, and the loss.  A CTA takes 32 columns: a thread four of them, every 32nd part.  With more
// than one CTA each leaves its share of the loss in the workspace, and the last to arrive (the ticket starts at 0
// in the launch before) adds them in their order, so that the order of arrival does not show.  Kernel trace, medians: 256
// parts of 256 columns 6.3 us, 16 of 128 4.6, the launch, a load of other CTAs' sums and the ticket in turn.
__global__ __launch_bounds__(256) void k_balance_end(BalanceArgs p, int parts) {
    __shared__ __align__(16) v4f sp[4][8];
    __shared__ __align__(16) v4i sc[4][8];
    __shared__ int kept;
    const int E = (int)p.E, pitch = part_pitch(E), tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int g = tid >> 3, col = blockIdx.x * 32 + 4 * (tid & 7);
    v4f s = {0.f, 0.f, 0.f, 0.f};
    v4i c = {0, 0, 0, 0};
    if (tid == 0) kept = 0;
    const int n = tid < parts ? p.part_n[tid] : 0;  // at most 256 parts
    for (int b0 = g; b0 < parts; b0 += 256) {       // eight parts asked for at a time
        v4f x[8];
        v4i y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (32 * i >= parts) break;  // uniform
            const int64_t at = (int64_t)min(b0 + 32 * i, parts - 1) * pitch + min(col, pitch - 4);
            x[i] = *(const v4f *)(p.part_p + at);
            y[i] = *(const v4i *)(p.part_c + at);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (b0 + 32 * i >= parts) continue;
            s += x[i];
            c += y[i];
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // the wave's eight groups of parts
        s[i] = over_tokens<3>(s[i]);
        c[i] += __builtin_amdgcn_mov_dpp(c[i], 0x128, 0xF, 0xF, false);
        const auto r = __builtin_amdgcn_permlane16_swap((uint32_t)c[i], (uint32_t)c[i], false, false);
        c[i] = (int)(r[0] + r[1]);
        const auto q = __builtin_amdgcn_permlane32_swap((uint32_t)c[i], (uint32_t)c[i], false, false);
        c[i] = (int)(q[0] + q[1]);
    }
    if (lane < 8) {
        sp[wave][lane] = s;
        sc[wave][lane] = c;
    }
    __syncthreads();
    if (n) atomicAdd(&kept, n);
    double dot = 0.0;
    const int e = blockIdx.x * 32 + tid;
    if (tid < 32 && e < E) {
        const float *fs = (const float *)sp + tid;
        const int *fc = (const int *)sc + tid;
        const float t = (fs[0] + fs[32]) + (fs[64] + fs[96]);
        const int k = (fc[0] + fc[32]) + (fc[64] + fc[96]);
        p.counts[e] = k;
        p.psum[e] = t;
        dot = (double)k * (double)t;
    }
    __syncthreads();
    if (blockIdx.x == 0 && tid == 0) p.counts[E] = kept;
    if (gridDim.x > 1) {
        if (tid >= 64) return;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) dot += __shfl_xor(dot, d, 64);
        int last = 0;
        if (tid == 0) {
            __hip_atomic_store(p.dots + blockIdx.x, dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            last = __hip_atomic_fetch_add(p.ticket, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == (int)gridDim.x - 1;
        }
        if (!__builtin_amdgcn_readfirstlane(last)) return;
        dot = tid < (int)gridDim.x ? __hip_atomic_load(p.dots + tid, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0.0;  // at most 64 CTAs
    }
    if (tid < 64) put_loss(p, dot, kept);
}

// The gradient of the logits: with gloss the balance loss's part, with gw the routing weights'.  The
// latter goes through the wave's own LDS: the token's row is cleared there, its slots put
// their terms in, and the lanes take their experts' back.  Slots that share an expert (seen by a tag that each slot
// leaves and reads again) add theirs one after another, in ascending order.  Bytes bound it where tokens are many: kernel trace,
// medians, 65536 tokens of 256 in fp32, both parts, 30.1 us for 140 MB, 4.7 TB/s; 8191 of 128 6.1 us for 9 MB, the counts'
// way and one step's, whose second half lies past the last token as long as the grid covers them all; 512 of 8 2.8, a launch.
template <bool F32, int VEC, int NV, int LPT>
__global__ __launch_bounds__(256) void k_router_bwd(RouterGradArgs p) {
    constexpr int U = NV == 1 ? 2 : 1, L = 1 << LPT, TPW = 64 >> LPT, ROW = L * NV * VEC;
    extern __shared__ __align__(16) uint8_t lds[];
    const int E = (int)p.E, topk = (int)p.topk;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, me = lane & (L - 1);
    const bool bal = p.gloss != nullptr, route = p.gw != nullptr;
    volatile float *mine = (volatile float *)lds + (wave * TPW + (lane >> LPT)) * ROW;  // the token's row
    float f[NV][VEC] = {};
    float scale = 0.0f;
    if (bal) {
        const float n = (float)p.counts[E];
        const float share = n > 0.0f ? (float)E / ((float)topk * n) : 0.0f;
        scale = n > 0.0f ? p.gloss[0] / n : 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const int e = (i * L + me) * VEC + v;
                f[i][v] = e < E ? (float)p.counts[e] * share : 0.0f;
            }
    }
    const int64_t step = (int64_t)gridDim.x * 4 * TPW;
    for (int64_t t0 = ((int64_t)blockIdx.x * 4 + wave) * TPW; t0 < p.T; t0 += step * U) {
        Row<F32, VEC, NV, L> row[U];
        float gw[U], w[U];
        int id[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t t = t0 + u * step + (lane >> LPT);
            if (bal) row[u].load(p.logits, p.mask, min(t, p.T - 1), E, me);
            gw[u] = w[u] = 0.0f;
            id[u] = -1;
            if (route && t < p.T && me < topk) {
                gw[u] = p.gw[t * topk + me];
                w[u] = p.w[t * topk + me];
                id[u] = p.ids[t * topk + me];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t t = t0 + u * step + (lane >> LPT);
            float x[NV][VEC];
            if (bal) {
                const bool live = t < p.T && row[u].keep;
                row[u].finish(live, E, me, x);
                const float inv = softmax<LPT, VEC, NV>(x);
                float mean = 0.0f;
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int v = 0; v < VEC; ++v) mean = __builtin_fmaf(f[i][v], x[i][v], mean);
                mean = over_lanes<LPT>(mean, Add{}) * inv;
                const float some = live ? scale : 0.0f;
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int v = 0; v < VEC; ++v) x[i][v] = x[i][v] * inv * some * (f[i][v] - mean);
            } else {
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int v = 0; v < VEC; ++v) x[i][v] = 0.0f;
            }
            if (route) {
                const float dot = over_lanes<LPT>(w[u] * gw[u], Add{});
                const float d = w[u] * (gw[u] - dot);
                const bool in = id[u] >= 0 && id[u] < E;
                // (LDS accesses of a wave take place in order; volatile keeps them so here)
#pragma unroll
                for (int i = 0; i < NV; ++i) lds_clear<VEC>(mine + (i * L + me) * VEC);
                if (in) ((volatile int *)mine)[id[u]] = me;
                const bool shared = in && ((volatile int *)mine)[id[u]] != me;
                if (__ballot(shared)) {
                    if (in) mine[id[u]] = 0.0f;
                    for (int j = 0; j < topk; ++j)
                        if (me == j && in) mine[id[u]] = mine[id[u]] + d;
                } else if (in) {
                    mine[id[u]] = d;
                }
#pragma unroll
                for (int i = 0; i < NV; ++i) lds_add<VEC>(mine + (i * L + me) * VEC, x[i]);
            }
            if (t >= p.T) continue;
            uint8_t *out = (uint8_t *)p.g + t * E * (F32 ? 4 : 2);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int e = (i * L + me) * VEC;
                if (e < E) store_piece<F32, VEC>(out, e, x[i]);
            }
        }
    }
}

// The routing weights' part alone, of more experts than a wave's registers hold.
__global__ __launch_bounds__(256) void k_route_bwd_wide(RouterGradArgs p) {
    const int64_t E = p.E, t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int topk = (int)p.topk, lane = threadIdx.x & 63;
    if (t >= p.T) return;  // uniform across the wave
    const float w = lane < topk ? p.w[t * topk + lane] : 0.0f, gw = lane < topk ? p.gw[t * topk + lane] : 0.0f;
    const int id = lane < topk ? p.ids[t * topk + lane] : -1;
    const float dot = over_lanes<6>(w * gw, Add{}), d = w * (gw - dot);
    for (int64_t e0 = 0; e0 < E; e0 += 64) {
        float x = 0.0f;
        for (int j = 0; j < topk; ++j) {
            const int ij = __builtin_amdgcn_readlane(id, j);
            if (ij >= e0 && ij < e0 + 64)  // uniform
                x += ij == e0 + lane ? __int_as_float(__builtin_amdgcn_readlane(__float_as_int(d), j)) : 0.0f;
        }
        if (e0 + lane < E) ((float *)p.g)[t * E + e0 + lane] = x;
    }
}

// The instance for E experts and at least `lanes` lanes a token: 16-byte pieces where every row begins on
// 16 bytes.  Past 64 pieces a row there are two lengths only, so that a row of 65 single experts costs one of 512: loss and both
// gradients of 65536 tokens in fp32, in graphs, 13.9 and 13.8 us at 64 experts, 17.1 and 18.6 at 100, 27.1 and 40.6 at 65.
template <class GO>
static hipError_t by_shape(int64_t E, int64_t lanes, bool f32, GO go) {
    auto sized = [&](auto F, auto V) {
        constexpr bool F32 = decltype(F)::value;
        constexpr int VEC = decltype(V)::value, ONE = 64 * VEC, MOST = 2048 / ONE;
        const int64_t need = std::max((E + VEC - 1) / VEC, lanes);
        if (need <= 8) return go.template run<F32, VEC, 1, 3>();
        if (need <= 16) return go.template run<F32, VEC, 1, 4>();
        if (need <= 32) return go.template run<F32, VEC, 1, 5>();
        if (need <= 64) return go.template run<F32, VEC, 1, 6>();
        return E <= ONE * MOST / 4 ? go.template run<F32, VEC, MOST / 4, 6>() : go.template run<F32, VEC, MOST, 6>();
    };
    if (f32) return E % 4 == 0 ? sized(std::true_type{}, std::integral_constant<int, 4>{}) : sized(std::true_type{}, std::integral_constant<int, 1>{});
    return E % 8 == 0 ? sized(std::false_type{}, std::integral_constant<int, 8>{}) : sized(std::false_type{}, std::integral_constant<int, 1>{});
}

// CTAs of the loss's first launch, each a part of the workspace (one: the outputs come from it)
// One launch of one CTA and two launches, in graphs: 512 tokens of 8 experts 5.6 and 6.4 us, of 64 7.5 and 8.0, of 128
// 12.2 and 8.2, 2048 of 8 11.5 and 7.3; a call of one launch takes the host 3 us less besides.
static int balance_parts(int64_t T, int64_t E) {
    if (T <= 512 && T * E <= 32768) return 1;
    return (int)std::max<int64_t>(1, std::min<int64_t>(256, (T + 63) / 64));
}
// The parts' sums, their counts, their kept tokens (256), the ticket, the end's CTAs' shares of the loss (64)
size_t balance_workspace(int64_t T, int64_t E) {
    const int parts = balance_parts(T, E);
    return parts == 1 ? 0 : align_up((size_t)parts * part_pitch((int)E) * 8 + 256 * 4 + 16 + 64 * 8, 256);
}

struct GoBalance {
    const BalanceArgs &a;
    hipStream_t s;
    template <bool F32, int VEC, int NV, int LPT>
    hipError_t run() const {
        const int64_t parts = balance_parts(a.T, a.E), per = (a.T + parts - 1) / parts;
        int waves = balance_waves(NV * VEC);  // as many as the part's tokens fill
        while (waves > 4 && per <= (waves / 2) * (64 >> LPT) * 4) waves /= 2;
        const size_t lds = (size_t)part_pitch((int)a.E) * 4 * (waves + 1) + 144;
        hipLaunchKernelGGL((k_balance<F32, VEC, NV, LPT>), dim3((unsigned)parts), dim3(64 * waves), lds, s, a, per);
        return hipGetLastError();
    }
};
hipError_t launch_balance_loss(BalanceArgs a, void *workspace, hipStream_t s) {
    const int parts = balance_parts(a.T, a.E), pitch = part_pitch((int)a.E);
    a.part_p = (float *)workspace;
    a.part_c = (int32_t *)(a.part_p + (size_t)parts * pitch);
    a.part_n = a.part_c + (size_t)parts * pitch;
    a.ticket = a.part_n + 256;
    a.dots = (double *)(a.ticket + 4);
    const hipError_t err = by_shape(a.E, 1, a.f32, GoBalance{a, s});
    if (err != hipSuccess || parts == 1) return err;
    hipLaunchKernelGGL(k_balance_end, dim3((unsigned)((pitch + 31) / 32)), dim3(256), 0, s, a, parts);
    return hipGetLastError();
}

struct GoGrad {
    const RouterGradArgs &a;
    hipStream_t s;
    template <bool F32, int VEC, int NV, int LPT>
    hipError_t run() const {
        const int64_t per = 4 * (64 >> LPT), blocks = std::min<int64_t>((a.T + per - 1) / per, 2048);
        const size_t lds = a.gw ? (size_t)4 * 64 * NV * VEC * 4 : 0;
        hipLaunchKernelGGL((k_router_bwd<F32, VEC, NV, LPT>), dim3((unsigned)blocks), dim3(256), lds, s, a);
        return hipGetLastError();
    }
};
hipError_t launch_router_backward(const RouterGradArgs &a, hipStream_t s) {
    if (a.E <= 2048) return by_shape(a.E, a.gw ? a.topk : 1, a.f32, GoGrad{a, s});
    hipLaunchKernelGGL(k_route_bwd_wide, dim3((unsigned)((a.T + 3) / 4)), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace r9k
