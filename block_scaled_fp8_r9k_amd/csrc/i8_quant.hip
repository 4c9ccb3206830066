// Rows of bf16 to signed bytes, one scale a row: activations per token, weights per
// output channel.
//
//   b = max(max_k |x[k]|, 1e-10),  s = b / 127,  q[k] = rint(x[k] * (127 / b))
//
// every step in fp32.  The product with 127 / b, and not a division by s, costs one
// multiplication an element; the two rules give the same code except next to a tie.
// One pass: a row's values stay in registers between its maximum and its codes (rows past
// 16384 values are read again, from the caches).  Bytes bound it: 16384
// rows of 768 in 8.9 us for 38 MB, 4.2 TB/s, in a kernel trace with the rows from memory; 100 rows of 4096 2.7 us, most of it
// the launch.
#include "i8_device.h"
#include "i8_internal.h"

namespace r9k {

// TPR threads a row, NV 16-byte pieces a thread; NV = 0: any length, read twice.
template <int TPR, int NV>
__global__ __launch_bounds__(256) void k_quant_i8(const uint4 *__restrict__ x, int64_t rows, int K,
                                                  uint2 *__restrict__ q, float *__restrict__ s) {
    __shared__ uint32_t red[4];
    const int tid = threadIdx.x, n8 = K / 8, me = tid & (TPR - 1);
    for (int64_t row = (int64_t)blockIdx.x * (256 / TPR) + tid / TPR; row < rows; row += (int64_t)gridDim.x * (256 / TPR)) {
        const uint4 *xr = x + row * n8;
        uint4 v[NV ? NV : 1];
        uint32_t m = 0;
        if constexpr (NV > 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i) v[i] = me + i * TPR < n8 ? xr[me + i * TPR] : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < NV; ++i) m = max(m, absmax8_bits(v[i]));
        } else {
            for (int i = me; i < n8; i += TPR) m = max(m, absmax8_bits(xr[i]));
        }
        m = max64(m);  // (a wave's rows end together: row is the same in all its lanes)
        if constexpr (TPR == 256) {
            __syncthreads();  // the row before is done with red
            if ((tid & 63) == 0) red[tid >> 6] = m;
            __syncthreads();
            m = max(max(red[0], red[1]), max(red[2], red[3]));
        }
        const I8Scale r = i8_row_scale(m);
        uint2 *qr = q + row * n8;
        if constexpr (NV > 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (me + i * TPR < n8) qr[me + i * TPR] = i8_quant8(v[i], r);
        } else {
            for (int i = me; i < n8; i += TPR) qr[i] = i8_quant8(xr[i], r);
        }
        if (me == 0) s[row] = r.s;
    }
}

hipError_t launch_quant_i8(const uint16_t *x, int64_t rows, int64_t K, int8_t *q, float *s, hipStream_t st) {
    // A wave a row, else a CTA a row.  In graphs, the rows partly from the caches: 16384 x 768 7.1 and 13.3 us; 4096 x 4096 8.8
    // and 9.8; 512 x 4096 3.3 and 2.9, few rows having too few waves.
    const bool wave = K <= 4096 && rows >= 1024;
    const int64_t blocks = std::min<int64_t>(wave ? (rows + 3) / 4 : rows, 1 << 20);
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(256), 0, st, (const uint4 *)x, rows, (int)K, (uint2 *)q, s);
        return hipGetLastError();
    };
    if (wave) return K <= 1024 ? go(k_quant_i8<64, 2>) : K <= 2048 ? go(k_quant_i8<64, 4>) : go(k_quant_i8<64, 8>);
    if (K <= 4096) return go(k_quant_i8<256, 2>);
    return K <= 16384 ? go(k_quant_i8<256, 8>) : go(k_quant_i8<256, 0>);
}

}  // namespace r9k
