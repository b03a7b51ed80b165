// ssm_decode.cuh -- one token of a state space layer: the short-convolution
// update of the projected row [x H*P | B G*N | C G*N], then the state update.
//
//     v     = silu(conv_bias + conv_w . [window, row])        window shifted in place
//     dt    = softplus(dt_raw + dt_bias),  a = exp(-exp(A_log) dt)
//     h     = a h + dt B x^T              h [N, P] fp32 of the request's slot, in place
//     y     = (h^T C + D x) silu(z)
//
// Two launches.  The first convolves every channel once into an fp32 row in the
// caller's workspace (unrounded: the step's result is rounded once, at y); it
// stays in L2.  The second streams the states; it is a programmatic dependent
// launch, so its first blocks hold their state slabs in registers before the
// convolution is done.  Fusing the convolution into the state blocks instead
// would make every block of a group convolve the group's B and C again.
//
// The state kernel is bound by HBM: 2*N*P*4 bytes per (request, head).  A block
// owns 64 state columns (32 at P = 32): warp w holds the rows [w*N/8, (w+1)*N/8),
// lane l two columns, so each row is one coalesced 256-byte access, loaded and
// stored with streaming hints (touched once a step).  256 requests, H 32, G 16, P = N =
// 128: 183 us, 6.0 TB/s (92 % of a copy's rate, the convolution's launch included); one
// request, H 32, P 64, N 128: 4.5 us, two launches' latency.
#pragma once

#include "common.cuh"
#include "ssm_scan.cuh"

namespace gdn {
namespace ssm {

struct DecodeArgs {
    const __nv_bfloat16* row;   // [n, *] before the convolution
    const __nv_bfloat16* dt;    // [n, *]
    const __nv_bfloat16* z;     // [n, *] or null
    int64_t rs, dts, zs;        // row strides, in elements
    const float* w;             // [C, W]
    const float* bias;          // [C] or null
    __nv_bfloat16* cstate;      // [n_slots, C, W-1]
    const int32_t* idx;         // [n] or null
    int W, act, n, n_slots, C;
    const float *A_log, *dt_bias, *D;
    int H, G;
    float* state;               // [n_slots, H, N, P]
    float* v;                   // [n, C] workspace
    __nv_bfloat16* y;           // [n, H, P]
};

constexpr int kDecReqs = 8;  // requests of one convolution thread (its taps are loaded once)

// Grid: x over channels (128 per block), y over runs of kDecReqs requests.  A
// slot >= n_slots is reported by the state kernel.
template <int W>
__global__ void __launch_bounds__(128) decode_conv_kernel(const DecodeArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int c = blockIdx.x * 128 + threadIdx.x;
    if (c >= a.C) return;
    float w[W];
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = a.w[(int64_t)c * W + i];
    const float b = a.bias ? a.bias[c] : 0.f;
    const int r0 = blockIdx.y * kDecReqs;
    const int r1 = r0 + kDecReqs < a.n ? r0 + kDecReqs : a.n;
#pragma unroll 4
    for (int r = r0; r < r1; ++r) {
        const int slot = a.idx ? a.idx[r] : r;
        if (slot < 0 || slot >= a.n_slots) continue;
        __nv_bfloat16* win = a.cstate + ((int64_t)slot * a.C + c) * (W - 1);
        __nv_bfloat16 t[W];
#pragma unroll
        for (int i = 0; i + 1 < W; ++i) t[i] = win[i];
        t[W - 1] = a.row[(int64_t)r * a.rs + c];
        float acc = b;
#pragma unroll
        for (int i = 0; i < W; ++i) acc = fmaf(w[i], __bfloat162float(t[i]), acc);
        a.v[(int64_t)r * a.C + c] = a.act ? silu_f32(acc) : acc;
#pragma unroll
        for (int i = 0; i + 1 < W; ++i) win[i] = t[i + 1];
    }
}

// The same for rows, windows and taps on 16 bytes (C is a multiple of 32): eight channels a thread,
// so a window is W - 1 loads of 16 bytes, and the windows of four requests are in flight.
// Grid: x over units of eight channels (128 per block), y over runs of kDecVecReqs requests.
constexpr int kDecVecReqs = 4;
template <int W>
__global__ void __launch_bounds__(128) decode_conv_vec_kernel(const DecodeArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int c = 8 * (blockIdx.x * 128 + threadIdx.x);
    if (c >= a.C) return;
    const int r0 = blockIdx.y * kDecVecReqs;
    uint4 win[kDecVecReqs][W > 1 ? W - 1 : 1], in[kDecVecReqs];
    int64_t at[kDecVecReqs];  // of the window, or -1
#pragma unroll
    for (int k = 0; k < kDecVecReqs; ++k) {
        const int r = r0 + k, slot = r < a.n ? (a.idx ? a.idx[r] : r) : -1;
        at[k] = slot < 0 || slot >= a.n_slots ? -1 : ((int64_t)slot * a.C + c) * (W - 1);
        if (at[k] < 0) continue;
        in[k] = *reinterpret_cast<const uint4*>(a.row + (int64_t)r * a.rs + c);
#pragma unroll
        for (int i = 0; i + 1 < W; ++i) win[k][i] = reinterpret_cast<const uint4*>(a.cstate + at[k])[i];
    }
    float4 wv[2 * W];
    float b[8];
    const float* w = reinterpret_cast<const float*>(wv);
#pragma unroll
    for (int i = 0; i < 2 * W; ++i) wv[i] = reinterpret_cast<const float4*>(a.w + (int64_t)c * W)[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = a.bias ? a.bias[c + i] : 0.f;
#pragma unroll
    for (int k = 0; k < kDecVecReqs; ++k) {
        if (at[k] < 0) continue;
        const __nv_bfloat16* t = reinterpret_cast<const __nv_bfloat16*>(win[k]);
        const __nv_bfloat16* x = reinterpret_cast<const __nv_bfloat16*>(&in[k]);
        uint4 next[W > 1 ? W - 1 : 1];
        __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(next);
        float4 v[2];
        float* vf = reinterpret_cast<float*>(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float acc = b[j];
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const __nv_bfloat16 e = i + 1 < W ? t[j * (W - 1) + i] : x[j];
                acc = fmaf(w[j * W + i], __bfloat162float(e), acc);
                if (i > 0) o[j * (W - 1) + i - 1] = e;
            }
            vf[j] = a.act ? silu_f32(acc) : acc;
        }
        float4* vo = reinterpret_cast<float4*>(a.v + (int64_t)(r0 + k) * a.C + c);
        vo[0] = v[0];
        vo[1] = v[1];
#pragma unroll
        for (int i = 0; i + 1 < W; ++i) reinterpret_cast<uint4*>(a.cstate + at[k])[i] = next[i];
    }
}

// Grid: n * H * (P / PB) blocks of 256 threads.
template <int N, int P>
__global__ void __launch_bounds__(256, 5) decode_state_kernel(const DecodeArgs a) {
    constexpr int PB = P >= 64 ? 64 : 32;
    constexpr int RPW = N / 8, CPL = PB / 32, NPART = P / PB;
    __shared__ float sB[N], sC[N], red[8][PB];
    const int rh = blockIdx.x / NPART, p0 = (blockIdx.x - rh * NPART) * PB;
    const int r = rh / a.H, h = rh - r * a.H, g = h / (a.H / a.G);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __nv_bfloat16* y = a.y + (int64_t)rh * P + p0;
    const int slot = a.idx ? a.idx[r] : r;
    if (slot < 0 || slot >= a.n_slots) {  // padding (uniform across the block)
        if (slot >= a.n_slots && threadIdx.x == 0) record_status(GDN_ERR_INVALID_ARG);
        // A grid whose blocks are all padding would else be done before the convolution, and what
        // comes next in the stream could change the slots under it.
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (threadIdx.x < PB) y[threadIdx.x] = __float2bfloat16_rn(0.f);
        return;
    }
    float* st = a.state + ((int64_t)slot * a.H + h) * N * P + (int64_t)warp * RPW * P + p0 + lane * CPL;
    float s[RPW][CPL];
#pragma unroll
    for (int i = 0; i < RPW; ++i) {
        if constexpr (CPL == 2) {
            const float2 t = __ldcs(reinterpret_cast<const float2*>(st + (int64_t)i * P));
            s[i][0] = t.x;
            s[i][1] = t.y;
        } else {
            s[i][0] = __ldcs(st + (int64_t)i * P);
        }
    }
    const float dt = softplus_f32(__bfloat162float(a.dt[(int64_t)r * a.dts + h]) + a.dt_bias[h]);
    const float at = expf(-expf(a.A_log[h]) * dt);
    // the convolved row is there once the first kernel's writes are visible
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const float* v = a.v + (int64_t)r * a.C;
    const int64_t boff = (int64_t)a.H * P + (int64_t)g * N, coff = boff + (int64_t)a.G * N;
    if (threadIdx.x < N)
        sB[threadIdx.x] = v[boff + threadIdx.x];
    else if (threadIdx.x < 2 * N)
        sC[threadIdx.x - N] = v[coff + threadIdx.x - N];
    float x[CPL], u[CPL], acc[CPL];
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
        x[c] = v[(int64_t)h * P + p0 + lane * CPL + c];
        u[c] = dt * x[c];
        acc[c] = 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < RPW; ++i) {
        const float b = sB[warp * RPW + i], cc = sC[warp * RPW + i];
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            s[i][c] = fmaf(at, s[i][c], u[c] * b);
            acc[c] = fmaf(s[i][c], cc, acc[c]);
        }
        if constexpr (CPL == 2)
            __stcs(reinterpret_cast<float2*>(st + (int64_t)i * P), make_float2(s[i][0], s[i][1]));
        else
            __stcs(st + (int64_t)i * P, s[i][0]);
    }
#pragma unroll
    for (int c = 0; c < CPL; ++c) red[warp][lane * CPL + c] = acc[c];
    __syncthreads();
    if (threadIdx.x < PB) {
        const int c = threadIdx.x;
        float o = a.D ? a.D[h] * v[(int64_t)h * P + p0 + c] : 0.f;
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) sum += red[w][c];
        o += sum;
        if (a.z) o *= silu_f32(__bfloat162float(a.z[(int64_t)r * a.zs + (int64_t)h * P + p0 + c]));
        y[c] = __float2bfloat16_rn(o);
    }
}

}  // namespace ssm
}  // namespace gdn
