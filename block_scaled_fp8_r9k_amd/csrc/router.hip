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
// A token takes 2^lpt neighbouring lanes, a lane NV pieces of VEC consecutive experts; a
// wave walks over tokens 64 >> lpt at a time.
#include <algorithm>

#include "i8_device.h"
#include "i8_internal.h"

namespace r9k {

namespace {

template <bool F32, int VEC>
__device__ __forceinline__ void load_piece(const void *row, int at, float (&x)[VEC]) {
    if constexpr (F32 && VEC == 4) {
        const float4 v = *(const float4 *)((const float *)row + at);
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else if constexpr (F32) {
        x[0] = ((const float *)row)[at];
    } else if constexpr (VEC == 4) {
        const uint2 v = *(const uint2 *)((const uint16_t *)row + at);
        x[0] = bf16_lo(v.x), x[1] = bf16_hi(v.x), x[2] = bf16_lo(v.y), x[3] = bf16_hi(v.y);
    } else {
        x[0] = __uint_as_float((uint32_t)((const uint16_t *)row)[at] << 16);
    }
}

// over the token's lanes
__device__ __forceinline__ float group_sum(float v, int lpt) {
    for (int d = 0; d < lpt; ++d) v += __shfl_xor(v, 1 << d, 64);
    return v;
}
__device__ __forceinline__ float group_max(float v, int lpt) {
    for (int d = 0; d < lpt; ++d) v = fmaxf(v, __shfl_xor(v, 1 << d, 64));
    return v;
}

// The token's probabilities in place of its logits (experts past E as -inf)
template <int VEC, int NV>
__device__ __forceinline__ void softmax(float (&x)[NV][VEC], int lpt) {
    constexpr float ninf = -__builtin_inff();
    float mx = ninf, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int v = 0; v < VEC; ++v) mx = fmaxf(mx, x[i][v]);
    mx = group_max(mx, lpt);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            x[i][v] = x[i][v] == ninf ? 0.0f : expf(x[i][v] - mx);
            sum += x[i][v];
        }
    sum = group_sum(sum, lpt);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int v = 0; v < VEC; ++v) x[i][v] *= inv;
}
}  // namespace

// A CTA's tokens: its probabilities and counts, into its part of the workspace.
template <bool F32, int VEC, int NV>
__global__ __launch_bounds__(256) void k_balance(BalanceArgs p, int lpt) {
    extern __shared__ __align__(16) uint8_t lds[];
    const int E = (int)p.E, topk = (int)p.topk;
    int32_t *hist = (int32_t *)lds;                // [E + 1]
    float *sums = (float *)lds + ((E + 4) & ~3);   // [4][E]
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int L = 1 << lpt, me = lane & (L - 1), per = 64 >> lpt;
    for (int e = tid; e <= E; e += 256) hist[e] = 0;
    __syncthreads();
    float acc[NV][VEC] = {};
    const int64_t step = (int64_t)gridDim.x * 4 * per;
    for (int64_t t0 = ((int64_t)blockIdx.x * 4 + wave) * per; t0 < p.T; t0 += step) {
        const int64_t t = t0 + (lane >> lpt);
        const bool live = t < p.T && (!p.mask || p.mask[t]);
        const uint8_t *row = (const uint8_t *)p.logits + (live ? t : 0) * E * (F32 ? 4 : 2);
        float x[NV][VEC];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = (i * L + me) * VEC;
#pragma unroll
            for (int v = 0; v < VEC; ++v) x[i][v] = -__builtin_inff();
            if (live && e < E) load_piece<F32, VEC>(row, e, x[i]);
        }
        softmax<VEC, NV>(x, lpt);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int v = 0; v < VEC; ++v) acc[i][v] += x[i][v];
        if (live) {
            for (int j = me; j < topk; j += L) {
                const int e = p.ids[t * topk + j];
                if (e >= 0 && e < E) atomicAdd(&hist[e], 1);  // whole numbers: the order does not show
            }
            if (me == 0) atomicAdd(&hist[E], 1);
        }
    }
    // the wave's groups of lanes, then the waves, in one order
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            for (int d = lpt; d < 6; ++d) acc[i][v] += __shfl_xor(acc[i][v], 1 << d, 64);
            const int e = (i * L + me) * VEC + v;
            if (lane < L && e < E) sums[wave * E + e] = acc[i][v];
        }
    __syncthreads();
    for (int e = tid; e < E; e += 256)
        p.part_p[(int64_t)blockIdx.x * E + e] = (sums[e] + sums[E + e]) + (sums[2 * E + e] + sums[3 * E + e]);
    for (int e = tid; e <= E; e += 256) p.part_c[(int64_t)blockIdx.x * (E + 1) + e] = hist[e];
}

// The parts, added up, and the loss.
__global__ __launch_bounds__(256) void k_balance_end(BalanceArgs p, int parts) {
    __shared__ double red[4];
    const int E = (int)p.E, tid = threadIdx.x;
    double dot = 0.0;
    for (int e = tid; e <= E; e += 256) {
        int64_t c = 0;
        double s = 0.0;
        for (int b = 0; b < parts; ++b) {
            c += p.part_c[(int64_t)b * (E + 1) + e];
            if (e < E) s += p.part_p[(int64_t)b * E + e];
        }
        p.counts[e] = (int32_t)c;
        if (e < E) p.psum[e] = (float)s;
        dot += (double)c * s;
    }
    for (int d = 1; d < 64; d <<= 1) dot += __shfl_xor(dot, d, 64);
    if ((tid & 63) == 0) red[tid >> 6] = dot;
    __syncthreads();
    if (tid == 0) {
        double n = 0.0;
        for (int b = 0; b < parts; ++b) n += (double)p.part_c[(int64_t)b * (E + 1) + E];
        dot = (red[0] + red[1]) + (red[2] + red[3]);
        p.loss[0] = n > 0.0 ? (float)(dot * (double)E / ((double)p.topk * n * n)) : 0.0f;
    }
}

// The gradient of the logits: the balance loss's part, and with gw the routing weights'.
template <bool F32, int VEC, int NV>
__global__ __launch_bounds__(256) void k_router_bwd(RouterGradArgs p, int lpt) {
    const int E = (int)p.E, topk = (int)p.topk;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int L = 1 << lpt, me = lane & (L - 1), per = 64 >> lpt;
    const float n = (float)p.counts[E];
    const float scale = n > 0.0f ? p.gloss[0] / n : 0.0f, share = n > 0.0f ? (float)E / ((float)topk * n) : 0.0f;
    float f[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const int e = (i * L + me) * VEC + v;
            f[i][v] = e < E ? (float)p.counts[e] * share : 0.0f;
        }
    const int64_t step = (int64_t)gridDim.x * 4 * per;
    for (int64_t t0 = ((int64_t)blockIdx.x * 4 + wave) * per; t0 < p.T; t0 += step) {
        const int64_t t = t0 + (lane >> lpt);
        const bool here = t < p.T, live = here && (!p.mask || p.mask[t]);
        const uint8_t *row = (const uint8_t *)p.logits + (live ? t : 0) * E * (F32 ? 4 : 2);
        float x[NV][VEC];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = (i * L + me) * VEC;
#pragma unroll
            for (int v = 0; v < VEC; ++v) x[i][v] = -__builtin_inff();
            if (live && e < E) load_piece<F32, VEC>(row, e, x[i]);
        }
        softmax<VEC, NV>(x, lpt);
        float mean = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int v = 0; v < VEC; ++v) mean = __builtin_fmaf(f[i][v], x[i][v], mean);
        mean = group_sum(mean, lpt);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int v = 0; v < VEC; ++v) x[i][v] = live ? scale * x[i][v] * (f[i][v] - mean) : 0.0f;
        if (p.gw && here) {
            const float *w = p.w + t * topk, *gw = p.gw + t * topk;
            float dot = 0.0f;
            for (int j = 0; j < topk; ++j) dot = __builtin_fmaf(w[j], gw[j], dot);
            for (int j = 0; j < topk; ++j) {
                const int id = p.ids[t * topk + j];
                const float d = w[j] * (gw[j] - dot);
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int v = 0; v < VEC; ++v) x[i][v] += id == (i * L + me) * VEC + v ? d : 0.0f;
            }
        }
        if (!here) continue;
        uint8_t *out = (uint8_t *)p.g + t * E * (F32 ? 4 : 2);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = (i * L + me) * VEC;
            if (e >= E) continue;
            if constexpr (F32 && VEC == 4) *(float4 *)((float *)out + e) = make_float4(x[i][0], x[i][1], x[i][2], x[i][3]);
            else if constexpr (F32) ((float *)out)[e] = x[i][0];
            else if constexpr (VEC == 4) *(uint2 *)((uint16_t *)out + e) = w4_bf16x4(v4f{x[i][0], x[i][1], x[i][2], x[i][3]});
            else ((uint16_t *)out)[e] = (uint16_t)w4_bf16x4(v4f{x[i][0], 0.0f, 0.0f, 0.0f}).x;
        }
    }
}

// The routing weights' part alone: any number of experts.
__global__ __launch_bounds__(256) void k_route_bwd(RouterGradArgs p, int lpt) {
    const int64_t E = p.E;
    const int topk = (int)p.topk, L = 1 << lpt;
    const int64_t t = ((int64_t)blockIdx.x << (8 - lpt)) + (threadIdx.x >> lpt);
    if (t >= p.T) return;
    const float *w = p.w + t * topk, *gw = p.gw + t * topk;
    float dot = 0.0f;
    for (int j = 0; j < topk; ++j) dot = __builtin_fmaf(w[j], gw[j], dot);
    for (int64_t e = threadIdx.x & (L - 1); e < E; e += L) {
        float x = 0.0f;
        for (int j = 0; j < topk; ++j) x += p.ids[t * topk + j] == e ? w[j] * (gw[j] - dot) : 0.0f;
        ((float *)p.g)[t * E + e] = x;
    }
}

// lanes a token, and the kernel of its pieces
static int token_lanes(int64_t pieces) {
    int l = 0;
    while (l < 6 && (int64_t(1) << l) < pieces) ++l;
    return l;
}
template <class GO>
static hipError_t by_shape(int64_t E, bool f32, GO go) {
    const bool vec = E % 4 == 0;
    const int64_t pieces = vec ? E / 4 : E, nv = (pieces + 63) / 64;
    auto typed = [&](auto F) {
        constexpr bool F32 = decltype(F)::value;
        if (vec) return nv == 1 ? go.template run<F32, 4, 1>() : nv == 2 ? go.template run<F32, 4, 2>() : go.template run<F32, 4, 8>();
        return nv == 1 ? go.template run<F32, 1, 1>() : nv <= 8 ? go.template run<F32, 1, 8>() : go.template run<F32, 1, 32>();
    };
    return f32 ? typed(std::true_type{}) : typed(std::false_type{});
}

// CTAs of the first launch, each a part of the workspace: enough for the chip, at least 16 tokens a wave
int balance_parts(int64_t T, int64_t E) {
    (void)E;
    return (int)std::max<int64_t>(1, std::min<int64_t>(512, (T + 63) / 64));
}

struct GoBalance {
    const BalanceArgs &a;
    hipStream_t s;
    template <bool F32, int VEC, int NV>
    hipError_t run() const {
        const size_t lds = (size_t)((a.E + 4) / 4 * 4 + 4 * a.E) * 4;
        hipLaunchKernelGGL((k_balance<F32, VEC, NV>), dim3((unsigned)balance_parts(a.T, a.E)), dim3(256), lds, s, a,
                           token_lanes(VEC == 4 ? a.E / 4 : a.E));
        return hipGetLastError();
    }
};
hipError_t launch_balance_loss(const BalanceArgs &a, hipStream_t s) {
    const hipError_t err = by_shape(a.E, a.f32, GoBalance{a, s});
    if (err != hipSuccess) return err;
    hipLaunchKernelGGL(k_balance_end, dim3(1), dim3(256), 0, s, a, balance_parts(a.T, a.E));
    return hipGetLastError();
}

struct GoGrad {
    const RouterGradArgs &a;
    hipStream_t s;
    template <bool F32, int VEC, int NV>
    hipError_t run() const {
        const int lpt = token_lanes(VEC == 4 ? a.E / 4 : a.E), per = 4 * (64 >> lpt);
        const int64_t blocks = std::min<int64_t>((a.T + per - 1) / per, 2048);
        hipLaunchKernelGGL((k_router_bwd<F32, VEC, NV>), dim3((unsigned)blocks), dim3(256), 0, s, a, lpt);
        return hipGetLastError();
    }
};
hipError_t launch_router_backward(const RouterGradArgs &a, hipStream_t s) {
    if (a.gloss) return by_shape(a.E, a.f32, GoGrad{a, s});
    const int lpt = token_lanes(a.E);
    const int64_t per = 256 >> lpt;
    hipLaunchKernelGGL(k_route_bwd, dim3((unsigned)((a.T + per - 1) / per)), dim3(256), 0, s, a, lpt);
    return hipGetLastError();
}

}  // namespace r9k
