// Device helpers of the 4-bit weight kernels: formats, layout, decoding.
//
// Two formats of group-scaled 4-bit weights:
//   int4   codes q = 0..15, value (q - z) * s: s bf16 per group of 32, 64 or 128
//          along K, z a zero point 0..15 per group (8 where none are given);
//   mxfp4  codes e2m1 (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives), value
//          v * 2^(e - 127), e a byte per group of 32 (255: NaN).
// Packed layout (r9k_pack_weight_w4), for 16-row tile t = n / 16 and chunk
// c = k / 128 (C = K / 128 chunks): the 1 KiB block at (t * C + c) * 1024 holds
// at 16 * l the 16 bytes that MFMA lane l (row l % 16, quarter q = l / 16)
// feeds to the chunk's four v_mfma_f32_16x16x32_bf16: word j holds k = 128 c +
// 32 j + 8 q + 0..7.  int4: byte b of a word holds k + b in its low half and
// k + b + 4 in its high half, so that a mask and a shift leave four codes in
// four bytes; mxfp4: byte b holds k + 2 b and k + 2 b + 1, as the converter
// takes them.
// int4 scales and zeros, ng = 128 / group: element (((t * C + c) * 4 + q) * ng + i) * 4 + r
// is row 16 t + 4 q + r, group i of the chunk: the rows whose sums lane l holds
// after an MFMA.  mxfp4 scales: byte ((t * C + c) * 16 + r) * 4 + i is row 16 t + r,
// group i: the row whose codes lane l % 16 = r converts.
#pragma once

#include "r9k_device.h"

namespace r9k {

typedef __bf16 w4_v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 w4_v2bf __attribute__((ext_vector_type(2)));
typedef unsigned int w4_v2u __attribute__((ext_vector_type(2)));
typedef unsigned int w4_v4u __attribute__((ext_vector_type(4)));

enum { W4_INT = 0, W4_MXFP4 = 1 };

// Eight int4 codes (one packed word) -> eight bf16 of the values 0..15, exact.
// A code in the low half of a byte is the e4m3 number q * 2^-9 (subnormal up to
// 7, and the first binade continues with the same step up to 15), so the
// fp8 converter with scale 2^9 gives q: seven instructions for eight codes.
__device__ __forceinline__ w4_v8bf w4_int_frag(uint32_t x) {
    const int lo = (int)(x & 0x0F0F0F0Fu), hi = (int)((x >> 4) & 0x0F0F0F0Fu);
    const w4_v4u u = {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, false)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, true)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, false)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, true))};
    return __builtin_bit_cast(w4_v8bf, u);
}

// Eight e2m1 codes (one packed word) times the group's scale -> eight bf16.
// Two significant bits times a power of two: exact in bf16, infinite from 2^128 on.  The
// converter takes the scale's exponent field alone: e = 0, 0.0f here, is 2^-127, and 255 NaN.
__device__ __forceinline__ w4_v8bf w4_fp4_frag(uint32_t x, float scale) {
    const w4_v4u u = {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, scale, 0)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, scale, 1)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, scale, 2)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, scale, 3))};
    return __builtin_bit_cast(w4_v8bf, u);
}

__device__ __forceinline__ w4_v8bf w4_frag(uint4 v) { return __builtin_bit_cast(w4_v8bf, w4_v4u{v.x, v.y, v.z, v.w}); }

__device__ __forceinline__ w4_v8bf w4_ones() {
    return __builtin_bit_cast(w4_v8bf, w4_v4u{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});
}

__device__ __forceinline__ v4f w4_mfma(w4_v8bf w, w4_v8bf a, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, a, c, 0, 0, 0);
}

// Four fp32 -> four bf16, round to nearest even (hardware converter; infinities
// and NaN stay what they are).
__device__ __forceinline__ uint2 w4_bf16x4(v4f x) {
    const w4_v2bf lo = {(__bf16)x[0], (__bf16)x[1]}, hi = {(__bf16)x[2], (__bf16)x[3]};
    return make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
}

// silu(g) * u in fp32
__device__ __forceinline__ float w4_silu_mul(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// Inclusive sum over the wave's 64 lanes (DPP row shifts, then the row ends
// carried on).  Every lane must be active.
__device__ __forceinline__ int w4_wave_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // row_shr 1, 2, 4, 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast 15 into rows 1 and 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast 31 into rows 2 and 3
    return v;
}

// Blocks of 2^sh rows that rows [a, z) make; up to 2^31 - 1 rows, which a block's more would carry past int.
__device__ __forceinline__ int w4_row_blocks(int a, int z, int sh) {
    return (int)(((uint32_t)(max(z, a) - a) + (1u << sh) - 1) >> sh);
}

// Row block `item` of the experts' row ranges [offsets[e], offsets[e+1]), RB
// rows (a power of two) to a block, blocks counted expert by expert: the expert, and
// its rows from the block's first on; false if there are fewer blocks.  Every wave
// finds it by itself, four experts a lane and 256 a round, in one round trip to memory
// for up to 256 experts.  Offsets are held to [0, R], so that wrong ones cannot lead
// out of the rows.
__device__ __forceinline__ bool w4_find_block(const int32_t *offsets, int E, int R, int RB, int item, int &e_out,
                                              int &r0, int &r1) {
    const int lane = threadIdx.x & 63, sh = __builtin_ctz(RB);
    for (int e0 = 0; e0 < E; e0 += 256) {
        const int e = e0 + 4 * lane;
        int o[5], nb[4], n = 0;
#pragma unroll
        for (int i = 0; i < 5; ++i) o[i] = offsets[min(e + i, E)];
#pragma unroll
        for (int i = 0; i < 5; ++i) o[i] = min(max(o[i], 0), R);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            nb[i] = w4_row_blocks(o[i], o[i + 1], sh);  // none past the last expert
            n += nb[i];
        }
        const int incl = w4_wave_scan(n), total = __builtin_amdgcn_readlane(incl, 63);
        if (item >= total) {
            item -= total;
            continue;
        }
        const int l = __builtin_ctzll(__ballot(incl > item));
        item -= __builtin_amdgcn_readlane(incl, l) - __builtin_amdgcn_readlane(n, l);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int b = __builtin_amdgcn_readlane(nb[i], l);
            if (item < b) {
                e_out = e0 + 4 * l + i;
                r0 = __builtin_amdgcn_readlane(o[i], l) + (item << sh);
                r1 = __builtin_amdgcn_readlane(o[i + 1], l);
                return true;
            }
            item -= b;
        }
    }
    return false;
}

// p / topk for p < 2^31, with magic = ceil(2^32 / topk) (0 for topk = 1): at most one too large
__device__ __forceinline__ uint32_t w4_div_topk(uint32_t p, uint32_t topk, uint32_t magic) {
    if (magic == 0) return p;
    const uint32_t d = __umulhi(p, magic);
    return d - (d * topk > p);
}

// ---- loads straight into LDS --------------------------------------------------

// Global -> LDS loads (lane l's bytes land at LDS address `l_addr` + size * l,
// the address taken from M0).  Issued from inline asm so that the compiler
// neither waits for them at every barrier nor before every LDS read (it cannot
// tell that the reads touch another stage); the kernel waits for them itself
// with w4_wait_vm, counting this wave's load instructions.
__device__ __forceinline__ uint32_t w4_lds_addr(const uint8_t *p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t *)p;
}
// The global address is a wave-uniform base (SGPRs) plus a 32-bit lane offset;
// the LDS address goes in M0, which the compiler sets from the operand.  A load needs one
// wait state after the write of M0, which the compiler does not keep for inline asm: each
// load brings its own.
__device__ __forceinline__ void w4_load16(const void *base, uint32_t off, uint32_t l_addr) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "{m0}"(l_addr) : "memory");
}
// The same with a 64-bit address in each lane.
__device__ __forceinline__ void w4_load16(const void *p, uint32_t l_addr) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(p), "{m0}"(l_addr) : "memory");
}
// The same for the first n lanes (n >= 1, the same in all lanes).  Called where the whole
// wave is enabled; the mask is set and lifted here and not by a branch, so that no later
// MFMA can be moved under it.  (Setting the mask is the wait state after the write of M0.)
__device__ __forceinline__ void w4_load16_first(const void *p, uint32_t l_addr, int n) {
    const uint64_t mask = n >= 64 ? ~0ull : (1ull << n) - 1;
    asm volatile("s_mov_b64 exec, %1\n\tglobal_load_lds_dwordx4 %0, off\n\ts_mov_b64 exec, -1" ::"v"(p), "s"(mask), "{m0}"(l_addr)
                 : "memory");
}
__device__ __forceinline__ void w4_load4(const void *p, uint32_t l_addr) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(p), "{m0}"(l_addr) : "memory");
}

// wait until at most VM of this wave's vector-memory instructions are in flight
template <int VM>
__device__ __forceinline__ void w4_wait_vm() {
    static_assert(VM >= 0 && VM < 64, "vmcnt");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(VM) : "memory");
}

}  // namespace r9k
