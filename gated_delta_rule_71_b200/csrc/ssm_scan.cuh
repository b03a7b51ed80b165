// ssm_scan.cuh -- the selective state space scan in IEEE fp32, token by token.
//
// Per sequence and head (B, C of group h / (H/G)):
//     dt_t = softplus(dt_raw_t + dt_bias)      a_t = exp(-exp(A_log) dt_t)
//     h_t  = a_t h_{t-1} + dt_t B_t x_t^T      h [N, P] fp32, key-major
//     y_t  = (h_t^T C_t + D x_t) silu(z_t)     D and z optional
// This kernel serves fp32 inputs, rows that TMA cannot address and a few tokens;
// other bf16 rows run on the chunked tensor-core kernel (ssm_scan_tc.cuh).
//
// Columns p of the state never interact, so a block owns 32 of them: thread
// (p, s) = (tid / 4, tid % 4) keeps the rows n = 16 j + 4 s + i (i < 4) of
// column p in registers, and y needs one sum over 4 neighbouring lanes.  The
// interleaving makes a warp's B and C reads 64 contiguous bytes (no bank
// conflict).  Tokens are staged 32 at a time through shared memory, the next 32
// on their way in registers meanwhile.  The kernel is bound by the serial walk over
// the tokens (3 N/4 fp32 operations and two shuffles a thread and token), not by
// memory: 717 fp32 tokens in three sequences at H = 8, P = N = 32 take 51 us (112
// with the loads in line, 55 at 16 tokens a batch).
#pragma once

#include "common.cuh"

namespace gdn {
namespace ssm {

struct ScanArgs {
    const void *x, *Bm, *Cm, *dt, *z;    // z may be null
    int64_t xs, bs, cs, dts, zs;         // token strides, in elements
    const float *A_log, *dt_bias, *D;    // D may be null
    const float* h0;                     // [n_seq, H, N, P] or null
    const int32_t* cu;                   // [n_seq + 1] or null (n_seq sequences of T rows)
    int n_seq;
    int64_t T;
    int H, G, P, N;
    void* y;                             // [rows, H, P] contiguous
    float* hT;                           // [n_seq, H, N, P] or null
};

__device__ __forceinline__ float softplus_f32(float v) { return v > 20.f ? v : log1pf(expf(v)); }
// v * sigmoid(v), accurate to a few fp32 ulp (division and expf, no fast forms:
// fp32 outputs keep fp32 accuracy)
__device__ __forceinline__ float silu_f32(float v) { return v / (1.f + expf(-v)); }

__device__ __forceinline__ void seq_rows(const ScanArgs& a, int s, int64_t& r0, int64_t& r1) {
    if (a.cu) {
        r0 = a.cu[s];
        r1 = a.cu[s + 1];
        if (r1 < r0) r1 = r0;  // offsets out of order: no tokens
    } else {
        r0 = (int64_t)s * a.T;
        r1 = r0 + a.T;
    }
}

constexpr int kTok = 32;  // tokens staged at a time

// Grid: n_seq * H * (P / 32) blocks of 128 threads.
template <int N, typename TIn>
__global__ void __launch_bounds__(128) scan_kernel(const ScanArgs a) {
    constexpr int J = N / 16;  // float4 rows of one thread
    __shared__ __align__(16) float sB[kTok][N], sC[kTok][N];
    __shared__ float sx[kTok][32], sy[kTok][32], sdt[kTok], sa[kTok];
    const int slabs = a.P / 32;
    const int p0 = 32 * (int)(blockIdx.x % slabs);
    const int sh = (int)(blockIdx.x / slabs);
    const int h = sh % a.H, seq = sh / a.H, g = h / (a.H / a.G);
    const int tid = threadIdx.x, p = tid >> 2, s = tid & 3;
    int64_t r0, r1;
    seq_rows(a, seq, r0, r1);
    const TIn* x = static_cast<const TIn*>(a.x) + (int64_t)h * a.P + p0;
    const TIn* Bm = static_cast<const TIn*>(a.Bm) + (int64_t)g * N;
    const TIn* Cm = static_cast<const TIn*>(a.Cm) + (int64_t)g * N;
    const TIn* dt = static_cast<const TIn*>(a.dt) + h;
    const TIn* z = a.z ? static_cast<const TIn*>(a.z) + (int64_t)h * a.P + p0 : nullptr;
    TIn* y = static_cast<TIn*>(a.y) + (int64_t)h * a.P + p0;
    const float A = -expf(a.A_log[h]), bias = a.dt_bias[h], Dh = a.D ? a.D[h] : 0.f;
    const int64_t hbase = ((int64_t)seq * a.H + h) * N * a.P + p0 + p;
    float st[J][4];
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            st[j][i] = a.h0 ? a.h0[hbase + (int64_t)(16 * j + 4 * s + i) * a.P] : 0.f;

    // one batch of tokens, loaded while the one before it is walked
    constexpr int NL = kTok * N / 128, XL = kTok * 32 / 128;
    float rb[NL], rc[NL], rx[XL], rz[XL], rdt = 0.f;
    auto load = [&](int64_t t0) {
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const int e = tid + 128 * i, t = e / N, n = e - t * N;
            const bool in = t0 + t < r1;
            rb[i] = in ? to_f32(Bm[(t0 + t) * a.bs + n]) : 0.f;
            rc[i] = in ? to_f32(Cm[(t0 + t) * a.cs + n]) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < XL; ++i) {
            const int64_t t = t0 + (tid >> 5) + 4 * i;
            rx[i] = t < r1 ? to_f32(x[t * a.xs + (tid & 31)]) : 0.f;
            rz[i] = z && t < r1 ? to_f32(z[t * a.zs + (tid & 31)]) : 0.f;
        }
        if (tid < kTok && t0 + tid < r1) rdt = to_f32(dt[(t0 + tid) * a.dts]);
    };
    load(r0);
    for (int64_t t0 = r0; t0 < r1; t0 += kTok) {
        const int nt = (int)(r1 - t0 < kTok ? r1 - t0 : kTok);
        float gate[XL];
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const int e = tid + 128 * i;
            (&sB[0][0])[e] = rb[i];
            (&sC[0][0])[e] = rc[i];
        }
#pragma unroll
        for (int i = 0; i < XL; ++i) {
            sx[(tid >> 5) + 4 * i][tid & 31] = rx[i];
            gate[i] = z ? silu_f32(rz[i]) : 1.f;
        }
        if (tid < nt) {
            const float d = softplus_f32(rdt + bias);
            sdt[tid] = d;
            sa[tid] = expf(A * d);
        }
        __syncthreads();
        if (t0 + kTok < r1) load(t0 + kTok);
#pragma unroll 4
        for (int t = 0; t < nt; ++t) {
            const float at = sa[t], u = sdt[t] * sx[t][p];
            float acc0 = 0.f, acc1 = 0.f;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const float4 b = *reinterpret_cast<const float4*>(&sB[t][16 * j + 4 * s]);
                const float4 c = *reinterpret_cast<const float4*>(&sC[t][16 * j + 4 * s]);
                st[j][0] = fmaf(at, st[j][0], u * b.x);
                st[j][1] = fmaf(at, st[j][1], u * b.y);
                st[j][2] = fmaf(at, st[j][2], u * b.z);
                st[j][3] = fmaf(at, st[j][3], u * b.w);
                acc0 = fmaf(st[j][0], c.x, fmaf(st[j][1], c.y, acc0));
                acc1 = fmaf(st[j][2], c.z, fmaf(st[j][3], c.w, acc1));
            }
            float acc = acc0 + acc1;
            acc += __shfl_xor_sync(0xffffffffu, acc, 1);
            acc += __shfl_xor_sync(0xffffffffu, acc, 2);
            if (s == 0) sy[t][p] = fmaf(Dh, sx[t][p], acc);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < XL; ++i) {
            const int t = (tid >> 5) + 4 * i;
            if (t < nt) {
                const float v = sy[t][tid & 31];
                y[(t0 + t) * a.H * a.P + (tid & 31)] = from_f32<TIn>(z ? v * gate[i] : v);
            }
        }
        // the next batch writes sB, sC, sx, sdt, sa only, and those were last read
        // before the barrier above; sy is rewritten after the next one
    }
    if (a.hT) {
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) a.hT[hbase + (int64_t)(16 * j + 4 * s + i) * a.P] = st[j][i];
    }
}

}  // namespace ssm
}  // namespace gdn
