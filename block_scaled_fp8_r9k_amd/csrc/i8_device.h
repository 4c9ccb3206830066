// Device helpers of the 8-bit integer kernels.
//
// Codes are signed bytes, -128 to 127; a row of activations has one fp32 scale, an
// output channel (a row of W) one.  Packed weights (r9k_pack_weight_i8): for 16-row tile
// t = n / 16 and chunk c = k / 128 (C = K / 128 chunks) the 2 KiB block at (t * C + c) * 2048
// holds, at h * 1024 + 16 * l (h = 0, 1; l = 0..63), the 16 bytes that MFMA lane l
// feeds to v_mfma_i32_16x16x64_i8 as half h of the chunk: row 16 t + l % 16, columns 128 c +
// 64 h + 16 (l / 16) .. +15.
#pragma once

#include "r9k_device.h"
#include "w4_device.h"

namespace r9k {

typedef int v4i __attribute__((ext_vector_type(4)));

// D = W(16x64) * A(64x16) + C in 32-bit integers.  Lane l supplies row l % 16 of W and column
// l % 16 of A (row l % 16 of the activations), K bytes 16 (l / 16) .. +15 of both; D's lane l
// holds rows 4 (l / 16) .. +3 of column l % 16.  Sums are exact: K < 2^17 products of at most
// 2^14 stay below 2^31.
__device__ __forceinline__ v4i i8_mfma(v4i w, v4i a, v4i c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(w, a, c, 0, 0, 0);
}

// Computed where it stands, with the whole wave enabled (as pin_acc of fp32 sums)
__device__ __forceinline__ void i8_pin(v4i &x) { asm volatile("" : "+v"(x)); }

// Four sums of one row and four channels -> fp32: one rounding when the sum becomes fp32 (above
// 2^24), one for each scale.
__device__ __forceinline__ v4f i8_scale(v4i x, float as, float4 ws) {
    return v4f{(float)x[0] * as * ws.x, (float)x[1] * as * ws.y, (float)x[2] * as * ws.z, (float)x[3] * as * ws.w};
}

// silu(g) * u = g sigma(g) u, sigma from e = exp(-|g|): 1 / (1 + e), or e / (1 + e) where g < 0.  The exponent's
// product with log2 e is taken in two parts, so that e is v_exp_f32's result to its last place; 1 + e, v_rcp_f32
// (one unit) and three products round: 8 * 2^-24 in all.  Below 2^-126, from g = -87.34 on, v_exp_f32 gives 0: such gates
// are i8_silu_far's.  (The division and expf of the fp32 library cost twice as many instructions; with them a tile of
// 256 x 256 spent 9.8 us on its outputs, without silu 4.1.)
struct I8Log2 {  // x log2 e = hi + lo; log2 e = 1.44269502f + 1.92596299e-8f
    float hi, lo;
};
__device__ __forceinline__ I8Log2 i8_log2e(float x) {
    const float hi = x * 1.44269502f;
    return {hi, __builtin_fmaf(x, 1.92596299e-8f, __builtin_fmaf(x, 1.44269502f, -hi))};
}
__device__ __forceinline__ float i8_silu_near(float g, float u) {
    const I8Log2 p = i8_log2e(fmaxf(-fabsf(g), -200.0f));
    const float e0 = __builtin_amdgcn_exp2f(p.hi), e = __builtin_fmaf(e0, p.lo * 0.693147182f, e0);
    const float s = (g < 0.0f ? e : 1.0f) * __builtin_amdgcn_rcpf(1.0f + e);
    return g * s * u;
}
// g < -87.3: 1 + e is 1, and u takes the whole powers of two of e before the rest of it, which is near 1, and g
// follow.  Where u becomes subnormal it loses at most 2^-150, the output 2^-141 (bf16's smallest step is 2^-133).  At
// g = -300 the output of the largest u is 0.
__device__ __forceinline__ float i8_silu_far(float g, float u) {
    const I8Log2 p = i8_log2e(fmaxf(g, -300.0f));
    const float n = __builtin_rintf(p.hi), m0 = __builtin_amdgcn_exp2f(p.hi - n), m = __builtin_fmaf(m0, p.lo * 0.693147182f, m0);
    return __builtin_amdgcn_ldexpf(u, (int)n) * m * g;
}
// Four of them.  Far gates are rare: the wave looks once for its 256 whether there is one (the branch is the wave's, no
// lane is masked, and what it skips lies behind the kernel).  The look costs 0.3 to 1%: gate_up of 2048 tokens 101.5 us, 100.7
// without; with every gate far-proof by itself it would be seven instructions an output.
__device__ __forceinline__ v4f i8_silu_mul(v4f g, v4f u) {
    constexpr float far = -87.3f;
    v4f y;
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = i8_silu_near(g[i], u[i]);
    if (__builtin_expect(__ballot(fminf(fminf(g[0], g[1]), fminf(g[2], g[3])) < far) != 0, 0)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = g[i] < far ? i8_silu_far(g[i], u[i]) : y[i];
    }
    return y;
}

// A row's quantisation: b = max(amax, 1e-10) from the largest bf16 bit pattern; with an infinity
// or a NaN in the row (patterns from 0x7F80 on) the scale is NaN and the codes are 0.
struct I8Scale {
    float s, inv;
    bool bad;
};
__device__ __forceinline__ I8Scale i8_row_scale(uint32_t amax_bits) {
    I8Scale r;
    r.bad = amax_bits >= 0x7F80u;
    const float b = fmaxf(r.bad ? 0.0f : __uint_as_float(amax_bits << 16), 1e-10f);
    r.s = r.bad ? __uint_as_float(0x7FC00000u) : b / 127.0f;
    r.inv = r.bad ? 0.0f : 127.0f / b;
    return r;
}

// rint(x * inv) of eight bf16, |x * inv| <= 127 (1 + 2^-23): adding 1.5 * 2^23 rounds to the
// nearest integer, ties to even, and leaves its two's complement in the low byte.
__device__ __forceinline__ uint32_t i8x4(float a, float b, float c, float d, float inv) {
    const float m = 12582912.0f;
    const uint32_t x = __float_as_uint(a * inv + m), y = __float_as_uint(b * inv + m);
    const uint32_t z = __float_as_uint(c * inv + m), w = __float_as_uint(d * inv + m);
    const uint32_t lo = __builtin_amdgcn_perm(y, x, 0x0C0C0400u), hi = __builtin_amdgcn_perm(w, z, 0x04000C0Cu);
    return lo | hi;
}
__device__ __forceinline__ uint2 i8_quant8(uint4 v, const I8Scale &r) {
    const uint2 o = make_uint2(i8x4(bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y), r.inv),
                               i8x4(bf16_lo(v.z), bf16_hi(v.z), bf16_lo(v.w), bf16_hi(v.w), r.inv));
    return r.bad ? make_uint2(0, 0) : o;
}

// The experts' row blocks for a CTA that looks for several: up to 256 experts stay in the wave's registers, four a
// lane, and only the first search goes to memory; with more, each does (w4_find_block, whose blocks these are).
struct I8Blocks {
    int o[5], incl;
    __device__ __forceinline__ void load(const int32_t *offsets, int E, int R, int RB) {
        const int e = 4 * (threadIdx.x & 63), sh = __builtin_ctz(RB);
        int n = 0;
#pragma unroll
        for (int i = 0; i < 5; ++i) o[i] = offsets[min(e + i, E)];
#pragma unroll
        for (int i = 0; i < 5; ++i) o[i] = min(max(o[i], 0), R);
#pragma unroll
        for (int i = 0; i < 4; ++i) n += w4_row_blocks(o[i], o[i + 1], sh);
        incl = w4_wave_scan(n);
    }
    __device__ __forceinline__ bool find(int item, int RB, int &e, int &r0, int &r1) const {
        if (item >= __builtin_amdgcn_readlane(incl, 63)) return false;
        const int sh = __builtin_ctz(RB), l = __builtin_ctzll(__ballot(incl > item));
        if (l > 0) item -= __builtin_amdgcn_readlane(incl, l - 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int a = __builtin_amdgcn_readlane(o[i], l), z = __builtin_amdgcn_readlane(o[i + 1], l);
            const int b = w4_row_blocks(a, z, sh);
            if (item < b) {
                e = 4 * l + i;
                r0 = a + (item << sh);
                r1 = z;
                return true;
            }
            item -= b;
        }
        return false;
    }
};

// Maximum over the wave, the same in every lane.  Every lane must be active.
__device__ __forceinline__ uint32_t max64(uint32_t v) {
    v = max16_dpp(v);
    const uint32_t a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16);
    const uint32_t c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
    return max(max(a, b), max(c, d));
}

}  // namespace r9k
