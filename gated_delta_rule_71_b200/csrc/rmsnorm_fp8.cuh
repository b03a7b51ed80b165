// rmsnorm_fp8.cuh -- root-mean-square norm behind the residual's addition, with
// an 8-bit output and a scale for each block of 128 elements.
//
//     s = x + r,  r <- s                   (r optional; s kept in fp32)
//     y = s * rsqrt(mean(s^2) + eps) * w
//     per block of 128 of a row:  scale = max|y| / 448 (1 where that is 0),
//                                 q = e4m3(y / scale), round to nearest even
//
// One block per row, the row in registers between the two passes, so HBM sees
// each input once and each output once.  A thread owns units of eight
// consecutive elements; sixteen neighbouring threads hold one block of 128, so
// its maximum is four shuffles.  Bound by HBM.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace gdn {
namespace nrm {

struct Args {
    const void* x;
    void* r;          // residual, read and written, or null
    const float* w;
    int64_t rows;
    int D;
    int64_t xs, rs;   // row strides, in elements
    float eps;
    uint8_t* q;       // [rows, D]
    float* scale;     // [rows, ceil(D / 128)]
};

// max that keeps a NaN (so a NaN in a block shows in its scale too)
__device__ __forceinline__ float max_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}

// Eight consecutive elements.  VEC: 16-byte accesses, all eight in the row.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, int left, float (&v)[8]) {
    if constexpr (VEC) {
        constexpr int NU = sizeof(T) / 2;  // 16-byte units
        uint4 u[NU];
#pragma unroll
        for (int i = 0; i < NU; ++i) u[i] = reinterpret_cast<const uint4*>(p)[i];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_f32(reinterpret_cast<const T*>(u)[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < left ? to_f32(p[i]) : 0.f;
    }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* p, int left, const float (&v)[8]) {
    if constexpr (VEC) {
        constexpr int NU = sizeof(T) / 2;
        uint4 u[NU];
#pragma unroll
        for (int i = 0; i < 8; ++i) reinterpret_cast<T*>(u)[i] = from_f32<T>(v[i]);
#pragma unroll
        for (int i = 0; i < NU; ++i) reinterpret_cast<uint4*>(p)[i] = u[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) p[i] = from_f32<T>(v[i]);
    }
}

// Grid-stride over rows; blockDim.x * U units of 8 cover the row.
template <typename T, int U, bool VEC>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(const Args a) {
    __shared__ float part[32];
    const int D = a.D, nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nblk = (D + 127) / 128;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        float v[U][8];
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int e = 8 * (tid + i * nt), left = D - e;
            if (left > 0) {
                load8<T, VEC>(static_cast<const T*>(a.x) + row * a.xs + e, left, v[i]);
                if (a.r) {
                    float t[8];
                    T* rp = static_cast<T*>(a.r) + row * a.rs + e;
                    load8<T, VEC>(rp, left, t);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[i][j] += t[j];
                    store8<T, VEC>(rp, left, v[i]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (lane == 0) part[warp] = ss;
        __syncthreads();
        float sum = lane < (nt >> 5) ? part[lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float rstd = 1.0f / sqrtf(sum / (float)D + a.eps);
        __syncthreads();  // part is rewritten by the next row
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int e = 8 * (tid + i * nt), left = D - e;
            float m = 0.f;
            if (left > 0) {
                float w[8];
                load8<float, VEC>(a.w + e, left, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[i][j] = v[i][j] * rstd * w[j];
                    m = max_nan(m, fabsf(v[i][j]));
                }
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (left <= 0) continue;
            const float sc = (m > 0.f || m != m) ? m / 448.f : 1.f;
            if ((tid & 15) == 0) a.scale[row * nblk + e / 128] = sc;
            uint32_t b[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t lo = __nv_cvt_float2_to_fp8x2(
                    make_float2(v[i][4 * k] / sc, v[i][4 * k + 1] / sc), __NV_SATFINITE, __NV_E4M3);
                const uint32_t hi = __nv_cvt_float2_to_fp8x2(
                    make_float2(v[i][4 * k + 2] / sc, v[i][4 * k + 3] / sc), __NV_SATFINITE, __NV_E4M3);
                b[k] = lo | (hi << 16);
            }
            uint8_t* qp = a.q + row * D + e;
            if constexpr (VEC) {
                *reinterpret_cast<uint2*>(qp) = make_uint2(b[0], b[1]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j < left) qp[j] = (uint8_t)(b[j >> 2] >> (8 * (j & 3)));
            }
        }
    }
}

}  // namespace nrm
}  // namespace gdn
