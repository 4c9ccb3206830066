// 4-bit weights at load time: the group quantiser and the packed layout.
// Not on any hot path: each reads its input once and writes its output once.
#include "w4_internal.h"
#include "w4_device.h"

namespace r9k {

// One thread quantises 8 consecutive values; the GRP / 8 threads of a group are
// neighbouring lanes and agree on its range by shuffles.
//   int4   without zeros: s = bf16(max(amax, 1e-10) / 7), q = clamp(rint(w / s), -8, 7) + 8
//          with zeros: lo = min(0, min w), hi = max(0, max w),
//          s = bf16(max(hi - lo, 1e-10) / 15), z = clamp(rint(-lo / s), 0, 15),
//          q = clamp(rint(w / s) + z, 0, 15)
//   mxfp4  e = clamp(exponent of amax - 2, 2^-126 .. 2^127) biased by 127 in a byte,
//          q = e2m1(w / 2^e), ties to the even code, saturating at 6
// A group with an infinity or a NaN takes the scale NaN (255 in mxfp4), so that it shows.
// fp32 arithmetic, ties to even in rint; s is bf16 because that is how 4-bit
// checkpoints hold it, and the codes are taken against the rounded s.
template <int FMT>
__global__ __launch_bounds__(256) void k_quant_weight_w4(const uint16_t *__restrict__ w, int64_t n8, int grp,
                                                         uint8_t *__restrict__ wq, void *__restrict__ s_out,
                                                         uint8_t *__restrict__ z_out) {
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const bool live = id < n8;
    const uint4 v = live ? ((const uint4 *)w)[id] : make_uint4(0, 0, 0, 0);
    const float f[8] = {bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y),
                        bf16_lo(v.z), bf16_hi(v.z), bf16_lo(v.w), bf16_hi(v.w)};
    float lo = 0.0f, hi = 0.0f;  // the range always holds 0
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo = fminf(lo, f[i]);
        hi = fmaxf(hi, f[i]);
        bad |= (__float_as_uint(f[i]) & 0x7F800000u) == 0x7F800000u;
    }
    if (bad) hi = __uint_as_float(0x7F800000u);  // fmaxf passes over a NaN
    const int lanes = grp / 8;  // 4, 8 or 16
    for (int d = 1; d < lanes; d <<= 1) {
        lo = fminf(lo, __shfl_xor(lo, d, 64));
        hi = fmaxf(hi, __shfl_xor(hi, d, 64));
    }
    const float amax = fmaxf(-lo, hi);
    bad = amax == __uint_as_float(0x7F800000u);  // any of the group
    const bool first = live && (threadIdx.x & (lanes - 1)) == 0;
    const int64_t g = id * 8 / grp;
    uint32_t code[8];
    if (FMT == W4_INT) {
        // (the range of the halves: hi - lo may pass fp32's largest value)
        const float num = z_out ? fmaxf(0.5f * hi - 0.5f * lo, 0.5e-10f) / 15.0f * 2.0f : fmaxf(amax, 1e-10f) / 7.0f;
        const uint32_t sb = bad ? 0x7FC0u : bf16_rne(num);
        const float s = __uint_as_float(sb << 16);
        const float z = z_out ? fminf(fmaxf(rintf(-lo / s), 0.0f), 15.0f) : 8.0f;
        if (first) {
            ((uint16_t *)s_out)[g] = (uint16_t)sb;
            if (z_out) z_out[g] = (uint8_t)z;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) code[i] = (uint32_t)fminf(fmaxf(rintf(f[i] / s) + z, 0.0f), 15.0f);
    } else {
        const int ex = (int)(__float_as_uint(amax) >> 23);  // biased exponent; 0 for zero and subnormals
        const int e = bad ? 255 : min(max(ex - 2, 1), 254);
        if (first) ((uint8_t *)s_out)[g] = (uint8_t)e;
        // 2^(127 - e) as two factors, each a normal number
        const float r1 = __uint_as_float((uint32_t)(127 + (127 - e) / 2) << 23);
        const float r2 = __uint_as_float((uint32_t)(127 + (127 - e) - (127 - e) / 2) << 23);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float a = fabsf(f[i]) * r1 * r2;
            const uint32_t m = (a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) + (a >= 3.5f) +
                               (a > 5.0f);
            code[i] = m | (__float_as_uint(f[i]) >> 31) << 3;
        }
    }
    uint32_t out = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) out |= code[i] << (4 * i);
    if (live) ((uint32_t *)wq)[id] = out;
}

hipError_t launch_quant_weight_w4(const uint16_t *w, int64_t N, int64_t K, int fmt, int grp, uint8_t *wq, void *s,
                                  uint8_t *z, hipStream_t st) {
    const int64_t n8 = N * K / 8;
    const dim3 grid((unsigned)((n8 + 255) / 256));
    if (fmt == W4_INT) hipLaunchKernelGGL((k_quant_weight_w4<W4_INT>), grid, dim3(256), 0, st, w, n8, grp, wq, s, z);
    else hipLaunchKernelGGL((k_quant_weight_w4<W4_MXFP4>), grid, dim3(256), 0, st, w, n8, grp, wq, s, z);
    return hipGetLastError();
}

// One thread per (tile, chunk, lane): its 16 bytes of codes, and in the first
// 16 or so lanes the scales and zeros (layout: w4_device.h).
__global__ __launch_bounds__(256) void k_pack_weight_w4(const uint8_t *__restrict__ wq, const void *__restrict__ s,
                                                        const uint8_t *__restrict__ z, int64_t tiles, int64_t C,
                                                        int fmt, int grp, uint8_t *__restrict__ wp,
                                                        void *__restrict__ sp, uint8_t *__restrict__ zp) {
    const int64_t blk = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);  // tile * C + chunk
    if (blk >= tiles * C) return;
    const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
    const int64_t t = blk / C, c = blk % C;
    const int ng = 128 / grp;
    const int64_t gpr = C * ng;  // groups a row
    const uint8_t *row = wq + (16 * t + l16) * (C * 64) + c * 64 + 4 * q;
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t x = *(const uint32_t *)(row + 16 * j);  // element i in bits 4 i
        uint32_t y = x;
        if (fmt == W4_INT) {
            y = 0;
#pragma unroll
            for (int b = 0; b < 4; ++b) y |= ((x >> (4 * b)) & 15u) << (8 * b) | ((x >> (4 * b + 16)) & 15u) << (8 * b + 4);
        }
        o[j] = y;
    }
    ((uint4 *)wp)[blk * 64 + lane] = make_uint4(o[0], o[1], o[2], o[3]);
    if (lane < 16 * ng) {
        if (fmt == W4_INT) {
            // lane = ((q' * ng) + i) * 4 + r
            const int r = lane & 3, i = (lane >> 2) % ng, qq = (lane >> 2) / ng;
            const int64_t from = (16 * t + 4 * qq + r) * gpr + c * ng + i;
            ((uint16_t *)sp)[blk * 16 * ng + lane] = ((const uint16_t *)s)[from];
            if (z) zp[blk * 16 * ng + lane] = z[from] & 15;
        } else {
            const int64_t from = (16 * t + (lane >> 2)) * gpr + c * 4 + (lane & 3);
            ((uint8_t *)sp)[blk * 64 + lane] = ((const uint8_t *)s)[from];
        }
    }
}

hipError_t launch_pack_weight_w4(const uint8_t *wq, const void *s, const uint8_t *z, int64_t N, int64_t K, int fmt,
                                 int grp, uint8_t *wp, void *sp, uint8_t *zp, hipStream_t st) {
    const int64_t tiles = N / 16, C = K / 128;
    hipLaunchKernelGGL(k_pack_weight_w4, dim3((unsigned)((tiles * C + 3) / 4)), dim3(256), 0, st, wq, s, z, tiles, C,
                       fmt, grp, wp, sp, zp);
    return hipGetLastError();
}

}  // namespace r9k
