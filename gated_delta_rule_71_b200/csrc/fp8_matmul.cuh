// fp8_matmul.cuh -- matrix product of e4m3 operands with fp32 scales: one per row
// and block of 128 of the activations, one per 128 x 128 block of the weights.
//
//     out[m, n] = sum_b as[m, b] ws[n / 128, b] sum_{k in block b} a[m, k] w[n, k]
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace gdn {
namespace mm8 {

struct Args {
    const uint8_t* a;    // [M, K] e4m3, row stride lda
    const float* as;     // [M, ceil(K / 128)]
    const uint8_t* w;    // [N, K] e4m3, row stride ldw
    const float* ws;     // [ceil(N / 128), ceil(K / 128)]
    int64_t lda, ldw;
    int M, N, K;
    void* out;           // [M, N]
};

__device__ __forceinline__ float e4m3_f32(uint8_t v) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(v, __NV_E4M3);
    return __half2float(__half(h));
}

// Any K and any alignment, fp32 FMAs: 64 x 64 tiles, 256 threads of 4 x 4
// outputs, 32 columns of K through shared memory at a time.
template <typename TOut>
__global__ void __launch_bounds__(256) fp8_matmul_simt_kernel(const Args g) {
    __shared__ float sa[32][65], sw[32][65];
    const int m0 = 64 * blockIdx.y, n0 = 64 * blockIdx.x;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int kb_all = (g.K + 127) / 128;
    float acc[4][4] = {};
    for (int kb = 0; kb < kb_all; ++kb) {
        float part[4][4] = {};
        const int kend = g.K < 128 * (kb + 1) ? g.K : 128 * (kb + 1);
        for (int k0 = 128 * kb; k0 < kend; k0 += 32) {
            __syncthreads();
            for (int i = threadIdx.x; i < 64 * 32; i += 256) {
                const int r = i >> 5, k = i & 31;
                const bool in = k0 + k < kend;
                sa[k][r] = in && m0 + r < g.M ? e4m3_f32(g.a[(int64_t)(m0 + r) * g.lda + k0 + k]) : 0.f;
                sw[k][r] = in && n0 + r < g.N ? e4m3_f32(g.w[(int64_t)(n0 + r) * g.ldw + k0 + k]) : 0.f;
            }
            __syncthreads();
            for (int k = 0; k < 32; ++k) {
                float av[4], wv[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    av[i] = sa[k][ty + 16 * i];
                    wv[i] = sw[k][tx + 16 * i];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) part[i][j] = fmaf(av[i], wv[j], part[i][j]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int m = m0 + ty + 16 * i;
            const float s = (m < g.M ? g.as[(int64_t)m * kb_all + kb] : 0.f) *
                            g.ws[(int64_t)(n0 / 128) * kb_all + kb];
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(s, part[i][j], acc[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (m < g.M && n < g.N)
                static_cast<TOut*>(g.out)[(int64_t)m * g.N + n] = from_f32<TOut>(acc[i][j]);
        }
}

}  // namespace mm8
}  // namespace gdn
