// rmsnorm_fp8.cuh -- root-mean-square norm behind the residual's addition, with
// an 8-bit output and a scale for each block of 128 elements.
//
//     s = x + r,  r <- s                   (r optional; s kept in fp32)
//     y = s * rsqrt(mean(s^2) + eps) * w
//     per block of 128 of a row:  scale = max|y| / 448 (1 where that is 0),
//                                 q = e4m3(y / scale), round to nearest even
//
// A block works on a row at a time and holds it in registers between the two
// passes, so HBM sees each input once and each output once.  A thread owns units of
// eight elements, consecutive ones where rows allow 16-byte accesses: sixteen neighbouring
// threads hold one block of 128, so its maximum is four shuffles.  Three forms: a row a block in
// registers (few rows, any alignment and width), rows streamed through shared memory
// (many rows), and a row a warp (many narrow rows).
//
// Many rows are bound by HBM: 16384 x 4096 bf16 with a residual, 84 us, 5.6 TB/s (85 %
// of a copy's rate).  Few rows are bound by latency: 32 x 2048 2.6 us, of which an
// empty launch is most; 1111 x 1000 fp32 3.5 us.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"
#include "tc_ptx.cuh"

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

// A thread's units of eight elements: unit i starts at first<VEC>(i).  VEC: eight consecutive
// ones by 16-byte accesses, all in the row.  Else every 32nd of the 256 that the warp's unit
// covers, so that element by element a warp still touches consecutive ones (bf16, with a
// residual: 90511 x 241 71 us, 8000 x 2050 69; consecutive ones a thread: 91 and 73).
template <bool VEC>
__device__ __forceinline__ int first(int i, int tid, int nt) {
    return VEC ? 8 * (tid + i * nt) : 256 * ((tid >> 5) + i * (nt >> 5)) + (tid & 31);
}
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
        for (int i = 0; i < 8; ++i) v[i] = 32 * i < left ? to_f32(p[32 * i]) : 0.f;
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
            if (32 * i < left) p[32 * i] = from_f32<T>(v[i]);
    }
}

// The second pass of a row: v holds s; its normed values in 8 bits, and their scales.
template <int U, bool VEC>
__device__ __forceinline__ void write_row(const Args& a, int64_t row, float (&v)[U][8], float rstd, int tid, int nt) {
    const int D = a.D, nblk = (D + 127) / 128;
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int e = first<VEC>(i, tid, nt), left = D - e;
        float m[2] = {0.f, 0.f};  // of the unit's block; else of its two
        if (left > 0) {
            float w[8];
            load8<float, VEC>(a.w + e, left, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] = v[i][j] * rstd * w[j];
                m[VEC ? 0 : j / 4] = max_nan(m[VEC ? 0 : j / 4], fabsf(v[i][j]));
            }
        }
#pragma unroll
        for (int o = VEC ? 8 : 16; o > 0; o >>= 1) {
            m[0] = max_nan(m[0], __shfl_xor_sync(0xffffffffu, m[0], o));
            if (!VEC) m[1] = max_nan(m[1], __shfl_xor_sync(0xffffffffu, m[1], o));
        }
        if (left <= 0) continue;
        uint32_t b[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float mk = m[VEC ? 0 : k];
            const float mx = mk / 448.f;
            const float sc = (mx > 0.f || mx != mx) ? mx : 1.f;  // 0: no value of the block is above 2^-141
            // y / scale as y (1 / scale): one rounding more, far below half a step of e4m3;
            // where 1 / scale overflows (a block below 2^-117) y is divided
            const float inv = 1.0f / sc;
            const bool tiny = !(inv < 3.0e38f);
            if (VEC ? k == 0 && (tid & 15) == 0 : (tid & 31) == 0 && 128 * k < left)
                a.scale[row * nblk + e / 128 + (VEC ? 0 : k)] = sc;
            float q[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) q[j] = tiny ? v[i][4 * k + j] / sc : v[i][4 * k + j] * inv;
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(q[0], q[1]), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(q[2], q[3]), __NV_SATFINITE, __NV_E4M3);
            b[k] = lo | (hi << 16);
        }
        uint8_t* qp = a.q + row * D + e;
        if constexpr (VEC) {
            *reinterpret_cast<uint2*>(qp) = make_uint2(b[0], b[1]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (32 * j < left) qp[32 * j] = (uint8_t)(b[j >> 2] >> (8 * (j & 3)));
        }
    }
}

// Eight consecutive elements of shared memory.
template <typename T>
__device__ __forceinline__ void lds8(const T* p, float (&v)[8]) {
    constexpr int NU = sizeof(T) / 2;
    uint4 u[NU];
#pragma unroll
    for (int i = 0; i < NU; ++i) u[i] = reinterpret_cast<const uint4*>(p)[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(reinterpret_cast<const T*>(u)[i]);
}

// Grid-stride over rows; blockDim.x * U units of 8 cover the row.  Every load of a row
// is issued before its first store (the residual may lie anywhere, so the compiler would
// keep a later load behind an earlier store), and the sums of two rows alternate between
// two buffers, so a row costs one barrier.
template <typename T, int U, bool VEC>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(const Args a) {
    __shared__ float part[2][32];
    const int D = a.D, nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int flip = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
        float v[U][8];
        const T* xp = static_cast<const T*>(a.x) + row * a.xs;
        T* rp = static_cast<T*>(a.r) + row * a.rs;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int e = first<VEC>(i, tid, nt);
            if (e < D) {
                load8<T, VEC>(xp + e, D - e, v[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
            }
        }
        if (a.r) {
            float t[U][8];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int e = first<VEC>(i, tid, nt);
                if (e < D) load8<T, VEC>(rp + e, D - e, t[i]);
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int e = first<VEC>(i, tid, nt);
                if (e < D) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[i][j] += t[i][j];
                    store8<T, VEC>(rp + e, D - e, v[i]);
                }
            }
        }
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (lane == 0) part[flip][warp] = ss;
        __syncthreads();
        float sum = lane < (nt >> 5) ? part[flip][lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        write_row<U, VEC>(a, row, v, 1.0f / sqrtf(sum / (float)D + a.eps), tid, nt);
    }
}

// Many narrow rows: a row a warp, so no barriers and no thread without a unit but the last.
template <typename T, int U>
__global__ void __launch_bounds__(256) rmsnorm_warp_kernel(const Args a) {
    const int D = a.D, lane = threadIdx.x & 31;
    for (int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); row < a.rows; row += (int64_t)gridDim.x * 8) {
        float v[U][8];
        const T* xp = static_cast<const T*>(a.x) + row * a.xs;
        T* rp = static_cast<T*>(a.r) + row * a.rs;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int e = 8 * (lane + 32 * i);
            if (e < D) {
                load8<T, true>(xp + e, D - e, v[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
            }
        }
        if (a.r) {
            float t[U][8];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int e = 8 * (lane + 32 * i);
                if (e < D) load8<T, true>(rp + e, D - e, t[i]);
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int e = 8 * (lane + 32 * i);
                if (e < D) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[i][j] += t[i][j];
                    store8<T, true>(rp + e, D - e, v[i]);
                }
            }
        }
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        write_row<U, true>(a, row, v, 1.0f / sqrtf(ss / (float)D + a.eps), lane, 32);
    }
}

// The same over many rows of moderate width, with the rows streamed through shared memory
// by bulk copies: a block keeps two rows in flight behind the one it works on, whatever
// its warps are doing, which the register form cannot (16384 x 4096 bf16 with a residual:
// 109 us there at its best, 84 here).  Each thread reads its own units from the stage; the barrier
// of the row's sum is also the one after which the stage is refilled.
constexpr int kStages = 3;
template <typename T, int U>
__global__ void __launch_bounds__(256) rmsnorm_stream_kernel(const Args a) {
    extern __shared__ __align__(128) uint8_t stage[];
    __shared__ __align__(8) uint64_t full[kStages];
    __shared__ float part[2][8];
    __shared__ uint32_t abort_word;
    volatile uint32_t* abort_flag = &abort_word;
    const int D = a.D, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t bytes = (uint32_t)D * sizeof(T);
    const uint32_t step = a.r ? 2 * bytes : bytes;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(&full[i], 1);
        abort_word = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    auto load = [&](int64_t row, int st) {
        tc::mbar_arrive_expect_tx(&full[st], step);
        tc::bulk_g2s(smem_u32(stage + st * step), static_cast<const T*>(a.x) + row * a.xs, bytes, &full[st]);
        if (a.r)
            tc::bulk_g2s(smem_u32(stage + st * step + bytes), static_cast<const T*>(a.r) + row * a.rs, bytes, &full[st]);
    };
    if (tid == 0)
        for (int i = 0; i < kStages; ++i)
            if (blockIdx.x + (int64_t)i * gridDim.x < a.rows) load(blockIdx.x + (int64_t)i * gridDim.x, i);
    int it = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, ++it) {
        const int st = it % kStages;
        nap_wait(&full[st], (it / kStages) & 1, abort_flag);
        const T* xs = reinterpret_cast<const T*>(stage + st * step);
        const T* rs = reinterpret_cast<const T*>(stage + st * step + bytes);
        T* rp = static_cast<T*>(a.r) + row * a.rs;
        float v[U][8];
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int e = 8 * (tid + i * 256);
            if (e < D) {
                lds8(xs + e, v[i]);
                if (a.r) {
                    float t[8];
                    lds8(rs + e, t);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[i][j] += t[j];
                    store8<T, true>(rp + e, 8, v[i]);
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
        if (lane == 0) part[it & 1][warp] = ss;
        __syncthreads();
        if (tid == 0 && row + (int64_t)kStages * gridDim.x < a.rows && !*abort_flag)
            load(row + (int64_t)kStages * gridDim.x, st);
        float sum = part[it & 1][lane & 7];
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        write_row<U, true>(a, row, v, 1.0f / sqrtf(sum / (float)D + a.eps), tid, 256);
    }
    if (tid == 0 && *abort_flag) {
        record_status(GDN_ERR_TIMEOUT);
        for (int i = 0; i < kStages; ++i)  // never leave with a copy in flight
            for (int n = 0; n < 1000 && !try_wait_ns(smem_u32(&full[(it + i) % kStages]), ((it + i) / kStages) & 1, kNap); ++n) {
            }
    }
}

}  // namespace nrm
}  // namespace gdn
