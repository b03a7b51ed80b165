// ssm_scan_tc.cuh -- the selective state space scan on the tensor cores (bf16
// rows that TMA can address; fp32 states).
//
// Chunks of 128 tokens.  With g_t = -exp(A_log) dt_t (<= 0), G the inclusive sum
// of g over a chunk, R_s = sum of g behind s, and h the state entering the chunk:
//     y_r = sum_{s <= r} (C_r . B_s) e^{G_r - G_s} dt_s x_s  +  e^{G_r} h^T C_r
//     h  <- e^{G_last} h + sum_s B_s (e^{R_s} dt_s x_s)^T
// Four products a chunk on tcgen05 (M = 128, fp32 accumulation):
//   CB  = C B^T                     tokens x tokens, shared by the CTA's heads
//   Y2  = C h                       h in bf16 from shared memory
//   Y1  = W x                       W = the decayed, masked CB in bf16, in tensor
//                                   memory in place of CB; x as it came
//   S  += (w x)^T B                 S = h^T, or where decays are slow what its bf16 copy lacks,
//                                   accumulates in tensor memory in fp32 (kSlow)
// The weights e^{R_s} dt_s are fp32, so w x is split into three bf16 terms (24
// bits): states keep fp32 accuracy (an infinity does not survive the split: it becomes a
// NaN).  W and the copy of h that multiplies C are rounded to bf16 once each, since the
// tensor cores take W x and C h as bf16, as y itself is; where a segment is one chunk (short
// sequences, whose y is mostly the entering state's) that copy has a second term.  The skip
// D x rides on W's diagonal and so shares W's rounding: added in fp32 behind the products it
// would take the Y warps a second reading of x's tile.
//
// Decays are factored so that every exponent is <= 0 (nothing overflows) and is a
// sum of same-signed terms or a difference within 32 tokens: for s in an earlier
// block of 32 than r, e^{G_r - G_s} = rowfac(r, block) * colfac(s), one exponential
// per row and block; inside a block it is taken per pair.
//
// A CTA owns 128 value lanes (two heads of 64 or 32 value columns of one group, or
// one head of 128) of one segment of a sequence.  28 warps, each with one job:
//   X (4)  reads x, writes the split (w x)^T to tensor memory, 32 tokens at a time
//   M (8)  turns CB into W          S (4)  makes the gates two chunks ahead; decays S,
//                                          hands its bf16 copy to C h (at N = 128 X takes half)
//   Y (8)  e^G Y2, then y = Y1 + that (the skip D x rides on W's diagonal), gate
//   MMA (2): CB, C h, W x; and the state's products   TMA (2): x, B, C; and z, y tiles
// x, B, C and z come in and y goes out by TMA tiles; x^T reaches tensor memory by
// transposing 8 x 8 loads (ldmatrix.trans, st.16x128b).
//
// What bounds it: the latency of the chain of hand-overs in a chunk (CB, W, W x; S, C h, y), of
// which a CTA has one in flight; no unit is full.  A chunk takes 5900 cycles an SM at N = 64,
// some 8500 at N = 128 with a gate; there the warps' work on CB, x, S and y is some 4800 warp
// instructions a scheduler (57 % of the issue slots), the products are 3400 cycles
// (36 % of the tensor pipe), HBM runs at a third of its rate.  Where P is 64 or 32 and H / G odd,
// one CTA of a group has half its lanes empty; P = 32 fills half of each half, and N = 32 runs
// as 64.
// Measured: 4 x 4096 tokens, H 32, G 8, P 64, N 128, gate: 121 us; 8 packed sequences of
// 32768 tokens in all, H 32, G 16, P = N = 128: 380 to 420 us; one of 131072, H 32, P = N = 64: 565 us
// in short runs, 600 over seconds, where the power cap holds the clock at 1.7 GHz
// (token by token: 4131, 10462 and 58698 us).  Steps that gave most, on the first: z
// and y through tiles, not a row a thread, 197 to 163; x transposed by its loads and two
// warpgroups on W, 163 to 153; gates on the S warps and two MMA warps, 143 to 135.
//
// Long sequences with few heads are cut into segments: a first launch (STATES)
// sums each segment's own contribution to the state, a small one chains them, and
// the main launch starts each segment from the state that enters it.
#pragma once

#include "chunk_tc.cuh"
#include "ssm_scan.cuh"

namespace gdn {
namespace ssm {

constexpr int L = 128;          // tokens of a chunk
constexpr int kScanThreads = 896;
constexpr int NGR = 3;          // gate ring
// A product truncates the sum in tensor memory that it is added to, half a step off it on average and
// always towards zero, so a chunk's 24 products take some 12 x 2^-24 of a state S that stays there whole.
// Where a state keeps the share e of itself over a chunk that adds up to 12 / (1 - e): 50 x 2^-24 at 3/4;
// where nothing decays to 1.2e-5 of S after 32 chunks, 1.3e-4 after 512.  Above 3/4, therefore, S holds only
// what the bf16 copy of the state lacks, 2^-9 of it, and the copy is added back in fp32 for the next chunk
// (3.5e-7 after 32 chunks, 8e-6, the rounding of e, after 512).  Slow heads take 7 to 11 % longer by it.
constexpr float kSlow = 0.75f;
// The first pass has no copy, and no decay between chunks: the sums of kGroup chunks at a time are added up
// in fp32 in shared memory (37 us for 64 segments of 16 chunks, 35 left in tensor memory; groups of 4: 42).
constexpr int kGroup = 8;
constexpr float kMinG2 = -160.f;  // 2^-160 is 0 in fp32: more decay changes nothing

struct Gates {                  // of one chunk and head; sums in log2 units
    float pre[L];               // inclusive sum within the token's block of 32
    float col[L];               // dt 2^(sum behind the token within its block)
    float w[L];                 // dt 2^(sum behind the token within the chunk)
    float prd[L];               // log2(dt) - pre
    float tot[4];               // block sums
    float last;                 // 2^(sum of the chunk)
    float pad[3];
};

struct ScanTcArgs {
    CUtensorMap x, b, c, z, y;  // (P, H, rows), (N, G, rows), boxes 64 x 1 x 128
    ScanArgs a;
    int pairs;                  // CTAs' worth of value lanes of a group
    int units;                  // of all groups
    int per;                    // heads of a group
    int seg_chunks;             // chunks of a segment
    float* part;                // [slots, units, N, 128] segment states
    float* part_g;              // [slots, units, 2] segment sums of g (log2)
};

template <int NP>
struct ScanCfg {
    static constexpr int NH = NP / 64;
    // tiles in flight: shared memory holds two of B and C at N <= 64, one at N = 128
    // (refilled, from L2, under the products that do not need it)
    static constexpr int NBC = NP == 128 ? 1 : 2;
    static constexpr int NXB = NP == 128 ? 5 : 6;       // half-tiles of x
    // state columns of the S warps; the rest are the X warps', whose buffers are full when the state is
    // due (slow decays: 94 us of the main pass of 4 x 4096 against 101; at 64 columns the X warps are
    // the ones waited for, 426 us of one of 131072 against 405)
    static constexpr int NS = 64;
    static constexpr uint32_t TILE = 16384;             // 128 rows of 128 bytes
    static constexpr uint32_t BT = NH * TILE;
    static constexpr uint32_t OFF_B = 0;                // [NBC]
    static constexpr uint32_t OFF_C = OFF_B + NBC * BT; // [NBC]
    static constexpr uint32_t OFF_X = OFF_C + NBC * BT; // [NXB]
    static constexpr uint32_t OFF_Z = OFF_X + NXB * TILE;  // [2 halves] z, then y in its place
    static constexpr uint32_t OFF_H = OFF_Z + 2 * TILE;
    static constexpr uint32_t OFF_G = OFF_H + BT;       // [NGR][2] Gates
    static constexpr uint32_t OFF_BAR = OFF_G + NGR * 2 * (uint32_t)sizeof(Gates);
    static constexpr uint32_t SMEM = OFF_BAR + 60 * 8 + 16 + 1024;
    static constexpr uint32_t OFF_SUM = OFF_Z;          // first pass: [NP][128] fp32, over z and h
    static_assert(OFF_SUM + NP * 512 <= OFF_G, "the sums fit");
    static_assert(SMEM <= 232448, "shared memory budget");
    // tensor memory columns
    static constexpr uint32_t COL_CB = 0;               // fp32 CB, then W of both heads
    static constexpr uint32_t COL_S = 128;              // S, lane = value lane, NP columns
    static constexpr uint32_t COL_Y = COL_S + NP;       // [2 halves] x 64
    static constexpr uint32_t COL_WX = COL_Y + 128;     // [2] x 48: three terms of 32 tokens
    static constexpr uint32_t COL_WX1 = COL_Y;          // [4] x 48 in the first pass
    static_assert(COL_WX + 96 <= 512 && COL_WX1 + 192 <= 512, "tensor memory budget");
    // first pass: two accumulators, of NP columns each
    static __device__ __forceinline__ uint32_t col_acc(int group) { return group & 1 ? COL_S : COL_CB; }
};

enum : int {
    B_FULL = 0, B_FREE = B_FULL + 4, C_FULL_ = B_FREE + 4, C_FREE_ = C_FULL_ + 2, X_FULL = C_FREE_ + 2,
    X_DONE = X_FULL + 6, Z_FULL = X_DONE + 6, Y_OUT = Z_FULL + 2, G_FULL = Y_OUT + 2, G_FREE = G_FULL + NGR, CB_FULL = G_FREE + NGR, M_FULL, W_FREE,
    XQ_FULL, XQ_FREE = XQ_FULL + 4, S_READY = XQ_FREE + 4, DS_DONE, H_FREE, Y_FULL, Y_FREE = Y_FULL + 2,
    CLEAN = Y_FREE + 2, S_DRAIN, N_SCAN_BARS = S_DRAIN + 2,
    // of the first pass's two accumulators, in place of barriers of what it does not have
    ACC_FULL = DS_DONE, ACC_FREE = Y_FREE
};
static_assert(H_FREE == ACC_FULL + 1, "two barriers of one arrival");
static_assert(N_SCAN_BARS <= 60, "barrier slots");

// 3-D tiled load of one box (x innermost), completing on `bar`.
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z,
                                            uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}
// Bounded wait for what is still in flight on the way out (no abort flag).
__device__ __forceinline__ void drain(uint64_t* bar, uint32_t phase) {
    const uint32_t at = smem_u32(bar);
#pragma unroll 1
    for (uint32_t i = 0; i < tcf::kPolls && !mbar_try_wait(at, phase); ++i) {
    }
}
__device__ __forceinline__ float ex2_approx(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(z), "r"(src)
                 : "memory");
}
// Four 8 x 8 matrices of 16-bit elements, transposed: thread t of the warp gets rows
// 2 (t % 4), + 1 (low, high half) of column t / 4.  Row addresses of matrix i from lanes 8 i ...
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// 16 lanes x 16 columns of tensor memory: r[2 i] is lane t / 4, r[2 i + 1] lane 8 + t / 4, both
// column 4 i + t % 4.
__device__ __forceinline__ void tmem_st_16x128(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap* map, int x, int y, int z) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(z)
                 : "memory");
}
__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// Segments of a sequence of `len` tokens: every one but the last is full.
__device__ __forceinline__ int64_t seq_segments(int64_t len, int64_t seg) {
    return len <= seg ? 1 : (len + seg - 1) / seg;
}

// Where segment k of the batch lies: its sequence, its place j in it, how many the
// sequence has, and the first slot of the sequence's segment states (its segments
// but the last, counted over the sequences before it).  STATES counts those
// segments only.  Called by one whole warp; false when there is no segment k.
struct Segment { int seq; int j; int n; int slot; };
template <bool STATES>
__device__ __noinline__ bool find_segment(const ScanArgs& a, int64_t k, int64_t seg, int lane, Segment& o) {
    if (a.cu && seg >= a.T) {  // one segment a sequence (many short ones: no search)
        if (STATES || k >= a.n_seq) return false;
        o.seq = (int)k;
        o.j = o.slot = 0;
        o.n = 1;
        return true;
    }
    if (!a.cu) {
        const int64_t n = seq_segments(a.T, seg), per = STATES ? n - 1 : n;
        if (per == 0 || k >= per * a.n_seq) return false;
        o.seq = (int)(k / per);
        o.j = (int)(k - o.seq * per);
        o.n = (int)n;
        o.slot = (int)(o.seq * (n - 1));
        return true;
    }
    int64_t before = 0, slots = 0;
    for (int s0 = 0; s0 < a.n_seq; s0 += 32) {
        const int s = s0 + lane;
        const int64_t n = s < a.n_seq ? seq_segments((int64_t)a.cu[s + 1] - a.cu[s], seg) : 0;
        const int64_t full = s < a.n_seq ? n - 1 : 0, own = STATES ? full : n;
        int64_t inc = own, fin = full;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, inc, d), v = __shfl_up_sync(0xffffffffu, fin, d);
            if (lane >= d) {
                inc += u;
                fin += v;
            }
        }
        const int64_t first = before + inc - own;
        const uint32_t hit = __ballot_sync(0xffffffffu, k >= first && k < first + own);
        if (hit) {
            const int src = __ffs(hit) - 1;
            o.seq = s0 + src;
            o.j = (int)(k - __shfl_sync(0xffffffffu, first, src));
            o.n = (int)__shfl_sync(0xffffffffu, n, src);
            o.slot = (int)(slots + __shfl_sync(0xffffffffu, fin - full, src));
            return true;
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
        slots += __shfl_sync(0xffffffffu, fin, 31);
    }
    return false;
}

// The value lanes of a unit: half j is 64 lanes of one head.
struct Half { int head; int col; int width; };  // width 0: no such head
__device__ __forceinline__ Half half_of(const ScanTcArgs& p, int unit, int j) {
    const int g = unit / p.pairs, u = unit - g * p.pairs;
    if (p.a.P == 128) return Half{g * p.per + u, 64 * j, 64};
    const int h = 2 * u + j;
    return Half{g * p.per + h, 0, h < p.per ? p.a.P : 0};
}

// Grid: segments * units.  ONE: the 128 lanes are one head (P = 128).
template <int NP, bool STATES, bool ONE>
__global__ void __launch_bounds__(kScanThreads, 1) scan_tc_kernel(const __grid_constant__ ScanTcArgs p) {
    using K = ScanCfg<NP>;
    constexpr int NH = K::NH, NXB = K::NXB, NBC = K::NBC;
    constexpr int NS = K::NS;
    constexpr int NB = STATES ? 2 * NBC : NBC;  // the first pass has no C: its room is for B
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_u32 = smem_u32(smem_raw);
    const uint32_t sbase = (raw_u32 + 1023u) & ~1023u;
    uint8_t* base = smem_raw + (sbase - raw_u32);
    uint64_t* bars = reinterpret_cast<uint64_t*>(base + K::OFF_BAR);
    uint32_t* misc = reinterpret_cast<uint32_t*>(bars + 60);
    volatile uint32_t* abort_flag = misc + 1;
    Gates* gates = reinterpret_cast<Gates*>(base + K::OFF_G);
    const ScanArgs& a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int unit = blockIdx.x % p.units;
    const int64_t seg_tokens = (int64_t)p.seg_chunks * L;
    Segment sg;
    if (!find_segment<STATES>(a, blockIdx.x / p.units, seg_tokens, lane, sg)) return;  // all warps alike
    int64_t r0, r1;
    seq_rows(a, sg.seq, r0, r1);
    r0 += sg.j * seg_tokens;
    if (r1 > r0 + seg_tokens) r1 = r0 + seg_tokens;
    r0 = __shfl_sync(0xffffffffu, r0, 0);
    const int rows = __shfl_sync(0xffffffffu, (int)(r1 - r0), 0);
    const int nch = (int)__reduce_max_sync(0xffffffffu, (uint32_t)((rows + L - 1) / L));
    const int tail = rows - (nch - 1) * L;  // rows of the last chunk
    const int grp = unit / p.pairs;
    // the two halves (as half_of, without its division)
    auto half = [&](int j) {
        const int u = unit - grp * p.pairs, h = 2 * u + j;
        return ONE ? Half{grp * p.per + u, 64 * j, 64} : Half{grp * p.per + h, 0, h < p.per ? a.P : 0};
    };

    if (threadIdx.x == 0) {
        for (int i = 0; i < N_SCAN_BARS; ++i) {
            uint32_t n = 1;
            if (i >= X_DONE && i < X_DONE + NXB) n = STATES ? 8 : 3;  // X warps (, the product)
            if (i >= B_FREE && i < B_FREE + 4) n = STATES ? 1 : 2;  // the products of two warps
            if (i >= G_FULL && i < G_FULL + NGR) n = 4;
            if (i >= G_FREE && i < G_FREE + NGR) n = STATES ? 16 : 20;
            if (i == M_FULL) n = 8;
            if (i == S_READY) n = NS < NP ? 8 : 4;
            if ((i >= XQ_FULL && i < XQ_FULL + 4) || i == Y_OUT || i == Y_OUT + 1 || i == Y_FREE ||
                i == Y_FREE + 1 || i == CLEAN)
                n = 4;
            mbar_init(&bars[i], n);
        }
        misc[1] = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) tc::tmem_alloc(&misc[0], 512);
    tc::tc_before_sync();
    __syncthreads();
    tc::tc_after_sync();
    const uint32_t tmem = __reduce_max_sync(0xffffffffu, misc[0]);
    auto wait = [&](int b, int phase) { nap_wait(&bars[b], (uint32_t)phase & 1u, abort_flag); };
    auto arrive = [&](int b) {  // one arrival a warp
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars[b]);
    };

    // The first pass walks a segment from its end, so that each token's weight reaches to
    // the segment's end and the sum needs no decay between chunks: step c is chunk_of(c).
    auto chunk_of = [&](int c) { return STATES ? nch - 1 - c : c; };
    const int q = warp & 3, ln = 32 * q + lane;  // tensor-memory lane of the four-warp jobs
    const uint32_t lane_base = tmem + ((uint32_t)(32 * q) << 16);

    // The state between the chunks, its columns n_lo .. n_hi, by the S warps and (at 128 columns) the X warps.
    auto enter = [&](int n_lo, int n_hi) {  // the state that enters the segment
        const Half hf = half(q >> 1);
        const float* src = nullptr;
        int64_t step = 0;
        if ((ln & 63) < hf.width) {
            if (sg.j > 0) {
                src = p.part + ((int64_t)(sg.slot + sg.j - 1) * p.units + unit) * a.N * 128 + ln;
                step = 128;
            } else if (a.h0) {
                src = a.h0 + (((int64_t)sg.seq * a.H + hf.head) * a.N) * a.P + hf.col + (ln & 63);
                step = a.P;
            }
            src += n_lo * step;
        }
#pragma unroll 1
        for (int n0 = n_lo; n0 < n_hi; n0 += 16) {
            uint32_t u[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                u[i] = step && n0 + i < a.N ? __float_as_uint(__ldg(src)) : 0u;
                src += step;
            }
            tc::tmem_st16(lane_base + K::COL_S + n0, u);
        }
        tc::tmem_wait_st();
    };
    // Sixteen columns of it: S, and e times the last copy where that is not in S (e is 0 where it is).
    auto state16 = [&](int n0, float e, float (&v)[16]) {
        tc::tmem_ld16(lane_base + K::COL_S + n0, v);
        if (e != 0.f) {
            const uint32_t at = sbase + K::OFF_H + (n0 / 64) * K::TILE;
            const uint4 h0 = tc::ld_shared_v4(at + tc::sw128_off(ln, (n0 / 8) & 7));
            const uint4 h1 = tc::ld_shared_v4(at + tc::sw128_off(ln, (n0 / 8 + 1) & 7));
            const uint32_t w[8] = {h0.x, h0.y, h0.z, h0.w, h1.x, h1.y, h1.z, h1.w};
            tc::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 t = __ffma2_rn(make_float2(bf16_lo(w[i]), bf16_hi(w[i])), make_float2(e, e),
                                            make_float2(v[2 * i], v[2 * i + 1]));
                v[2 * i] = t.x;
                v[2 * i + 1] = t.y;
            }
        } else {
            tc::tmem_wait_ld();
        }
    };
    // The state that enters chunk c: its bf16 copy to shared memory, and e times it, or, where the copy
    // stays apart, e times what the copy lacks, to S.  ep: what this returned for the chunk before.
    auto advance = [&](int c, int n_lo, int n_hi, float ep) {
        const float e = gates[2 * (c % NGR) + (ONE ? 0 : q >> 1)].last;
        const bool apart = e > kSlow || nch == 1;
        if (c > 0) wait(DS_DONE, c - 1);
        if (c > 0) wait(H_FREE, c - 1);
        __syncwarp();
        tc::tc_after_sync();
        const uint32_t hrow = sbase + K::OFF_H;
        if (!apart && ep == 0.f) {  // (a loop of its own: 6 % of the main pass)
#pragma unroll 1
            for (int n0 = n_lo; n0 < n_hi; n0 += 16) {
                float v[16];
                uint32_t u[16];
                tc::tmem_ld16(lane_base + K::COL_S + n0, v);
                tc::tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    tc::st_shared_v4(hrow + (n0 / 64) * K::TILE + tc::sw128_off(ln, (n0 / 8 + i) & 7),
                                     tc::pack_bf16(v[8 * i], v[8 * i + 1]), tc::pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                                     tc::pack_bf16(v[8 * i + 4], v[8 * i + 5]), tc::pack_bf16(v[8 * i + 6], v[8 * i + 7]));
#pragma unroll
                for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(v[i] * e);
                tc::tmem_st16(lane_base + K::COL_S + n0, u);
            }
        } else {
            const float2 part = apart ? make_float2(-1.f, -1.f) : make_float2(0.f, 0.f);
#pragma unroll 1
            for (int n0 = n_lo; n0 < n_hi; n0 += 16) {
                float v[16];
                uint32_t u[16];
                state16(n0, ep, v);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t off = (n0 / 64) * K::TILE + tc::sw128_off(ln, (n0 / 8 + i) & 7);
                    uint32_t h[4], rest[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int at = 8 * i + 2 * k;
                        h[k] = tc::pack_bf16(v[at], v[at + 1]);
                        const float2 t = __ffma2_rn(make_float2(bf16_lo(h[k]), bf16_hi(h[k])), part, make_float2(v[at], v[at + 1]));
                        rest[k] = tc::pack_bf16(t.x, t.y);
                        u[at] = __float_as_uint(t.x * e);
                        u[at + 1] = __float_as_uint(t.y * e);
                    }
                    tc::st_shared_v4(hrow + off, h[0], h[1], h[2], h[3]);
                    if (nch == 1)  // the rest in bf16, into a tile of x that one chunk leaves free
                        tc::st_shared_v4(sbase + K::OFF_X + 2 * K::TILE + off, rest[0], rest[1], rest[2], rest[3]);
                }
                tc::tmem_st16(lane_base + K::COL_S + n0, u);
            }
        }
        tc::tmem_wait_st();
        tc::fence_async_smem();
        tc::tc_before_sync();
        arrive(S_READY);
        return apart ? e : 0.f;
    };
    auto leave = [&](int n_lo, int n_hi, float ep) {  // the state that leaves the sequence
        if (nch > 0) wait(DS_DONE, nch - 1);
        __syncwarp();
        tc::tc_after_sync();
        const Half hf = half(q >> 1);
        const bool live = a.hT && sg.j == sg.n - 1 && (ln & 63) < hf.width;
        float* dst = live ? a.hT + (((int64_t)sg.seq * a.H + hf.head) * a.N + n_lo) * a.P + hf.col + (ln & 63) : nullptr;
#pragma unroll 1
        for (int n0 = n_lo; n0 < n_hi; n0 += 16) {
            float v[16];
            state16(n0, ep, v);
            if (live)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (n0 + i < a.N) dst[(int64_t)(n0 - n_lo + i) * a.P] = v[i];
        }
    };

    if (warp < 4 || (STATES && (warp < 12 || (warp >= 16 && warp < 20)))) {
        // =============================================================== X warps
        // A chunk goes through in quarters of 32 tokens and two buffers of tensor memory
        // (the first pass has a warpgroup and a buffer for each quarter).  x^T comes out of
        // shared memory by transposing 8 x 8 loads: a thread gets two tokens of a value
        // column, the layout in which 16 lanes x 4 columns go to tensor memory.
        constexpr int SETS = STATES ? 4 : 1;
        const int set = STATES ? (warp < 12 ? warp >> 2 : 3) : 0;
        const int j = q >> 1;                  // half
        const int tr = lane & 7, tm = lane >> 3;
        uint32_t off[2];                       // of the loads of value columns 16 hb .. + 16
#pragma unroll
        for (int hb = 0; hb < 2; ++hb)
            off[hb] = (tm >> 1) * 1024 + tr * 128 + (((uint32_t)(4 * (q & 1) + 2 * hb + (tm & 1)) ^ tr) << 4);
        float ep = 0.f;
        if constexpr (!STATES && NS < NP) enter(NS, NP);
        for (int c = 0; c < nch; ++c) {
            const int gs = c % NGR, xi = 2 * c + j, xb = xi % NXB;
            if (c == nch - 1 && tail < L) {
                // rows behind the sequence's end belong to another one: x and B to zero
                // (a zero weight would still carry a NaN through the products)
                for (int h = 0; h < 2; ++h) wait(X_FULL + (2 * c + h) % NXB, (2 * c + h) / NXB);
                wait(B_FULL + c % NB, c / NB);
                if (ln >= tail) {
                    const uint32_t row = (uint32_t)ln * 128u;
#pragma unroll 1
                    for (int i = 0; i < 8; ++i) {
                        for (int h = 0; h < 2; ++h)
                            tc::st_shared_v4(sbase + K::OFF_X + ((2 * c + h) % NXB) * K::TILE + row + 16 * i, 0, 0, 0, 0);
                        for (int h = 0; h < NH; ++h)
                            tc::st_shared_v4(sbase + K::OFF_B + (c % NB) * K::BT + h * K::TILE + row + 16 * i, 0, 0, 0, 0);
                    }
                }
                tc::fence_async_smem();
                tc::named_bar(1, 128);  // (a segment that is not a sequence's last has no tail)
                arrive(CLEAN);
            }
            wait(X_FULL + xb, xi / NXB);
            wait(G_FULL + gs, c / NGR);
            const float* w = gates[2 * gs + (ONE ? 0 : j)].w + 2 * (lane & 3);
            const uint32_t xt = sbase + K::OFF_X + xb * K::TILE;
#pragma unroll 1
            for (int k = set; k < 4; k += SETS) {
                const int buf = STATES ? k : k & 1, use = STATES ? c : 2 * c + (k >> 1);
                const uint32_t col = lane_base + (STATES ? K::COL_WX1 : K::COL_WX) + 48 * buf;
                float2 wv[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) wv[i] = *reinterpret_cast<const float2*>(&w[32 * k + 8 * i]);
                if (use > 0) wait(XQ_FREE + buf, use - 1);
                __syncwarp();
                tc::tc_after_sync();
#pragma unroll 1
                for (int hb = 0; hb < 2; ++hb) {
                    uint32_t x[8], hi[8], mi[8], lo[8];
                    ldmatrix4_trans(xt + 4096 * k + (hb ? off[1] : off[0]), x);
                    ldmatrix4_trans(xt + 4096 * k + 2048 + (hb ? off[1] : off[0]), x + 4);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        // 24 bits in three truncated terms of 8: the last is exact
                        const float2 v = __fmul2_rn(make_float2(bf16_lo(x[i]), bf16_hi(x[i])), wv[i >> 1]);
                        const float2 m = __fadd2_rn(v, make_float2(-bf16_hi(__float_as_uint(v.x)), -bf16_hi(__float_as_uint(v.y))));
                        const float2 l = __fadd2_rn(m, make_float2(-bf16_hi(__float_as_uint(m.x)), -bf16_hi(__float_as_uint(m.y))));
                        hi[i] = __byte_perm(__float_as_uint(v.x), __float_as_uint(v.y), 0x7632);
                        mi[i] = __byte_perm(__float_as_uint(m.x), __float_as_uint(m.y), 0x7632);
                        lo[i] = __byte_perm(__float_as_uint(l.x), __float_as_uint(l.y), 0x7632);
                    }
                    const uint32_t at = col + ((uint32_t)(16 * hb) << 16);
                    tmem_st_16x128(at, hi);
                    tmem_st_16x128(at + 16, mi);
                    tmem_st_16x128(at + 32, lo);
                }
                tc::tmem_wait_st();
                tc::tc_before_sync();
                arrive(XQ_FULL + buf);
                // the next buffer is free once the last chunk's state is summed
                if (!STATES && NS < NP && k == 0) ep = advance(c, NS, NP, ep);
            }
            arrive(X_DONE + xb);
            arrive(G_FREE + gs);
        }
        if constexpr (!STATES && NS < NP) leave(NS, NP, ep);
    } else if (warp < 12) {
        // =============================================================== M warps
        if constexpr (!STATES) {
            const uint32_t zero[16] = {};
            constexpr int HEADS = ONE ? 1 : 2;
            const int kb0 = (warp >> 2) - 1;  // this warpgroup's blocks of 16 tokens: kb0, kb0 + 2, ...
            float Dh[HEADS];
#pragma unroll
            for (int h = 0; h < HEADS; ++h) {
                const Half hf = half(h);
                Dh[h] = a.D && hf.width ? a.D[hf.head] : 0.f;
            }
            for (int c = 0; c < nch; ++c) {
                const int gs = c % NGR;
                const Gates* G = &gates[2 * gs];
                wait(G_FULL + gs, c / NGR);
                float pr[HEADS], e[HEADS];
#pragma unroll
                for (int h = 0; h < HEADS; ++h) e[h] = pr[h] = G[h].pre[ln];
                wait(CB_FULL, c);
                __syncwarp();
                tc::tc_after_sync();
                // 16 columns of CB become 8 of each head's W: earlier blocks of 32 by factors
#pragma unroll 1
                for (int b = q - 1; b >= 0; --b) {
                    const int kb = 2 * b + kb0;
                    const uint32_t col = lane_base + K::COL_CB + 16 * kb;
                    float v[16];
                    tc::tmem_ld16(col, v);
                    float2 rf[HEADS];
#pragma unroll
                    for (int h = 0; h < HEADS; ++h) {
                        const float f = ex2_approx(e[h]);
                        rf[h] = make_float2(f, f);
                        e[h] += G[h].tot[b];
                    }
                    tc::tmem_wait_ld();
                    uint32_t o[HEADS][8];
#pragma unroll
                    for (int s = 0; s < 16; s += 4)
#pragma unroll
                        for (int h = 0; h < HEADS; ++h) {
                            const float4 f = *reinterpret_cast<const float4*>(&G[h].col[16 * kb + s]);
                            const float2 m = __fmul2_rn(make_float2(v[s], v[s + 1]), __fmul2_rn(rf[h], make_float2(f.x, f.y)));
                            const float2 n = __fmul2_rn(make_float2(v[s + 2], v[s + 3]), __fmul2_rn(rf[h], make_float2(f.z, f.w)));
                            o[h][s / 2] = tc::pack_bf16(m.x, m.y);
                            o[h][s / 2 + 1] = tc::pack_bf16(n.x, n.y);
                        }
#pragma unroll
                    for (int h = 0; h < HEADS; ++h) tc::tmem_st8(col + 8 * h, o[h]);
                }
                {  // the block on the diagonal, which is at s == r
                    const int kb = 2 * q + kb0, r = ln - 16 * kb;
                    const uint32_t col = lane_base + K::COL_CB + 16 * kb;
                    float v[16];
                    tc::tmem_ld16(col, v);
                    tc::tmem_wait_ld();
                    uint32_t o[HEADS][8];
#pragma unroll
                    for (int s = 0; s < 16; s += 4)
#pragma unroll
                        for (int h = 0; h < HEADS; ++h) {
                            // 2^(pre_r - pre_s) dt_s with dt in the exponent
                            const float4 f = *reinterpret_cast<const float4*>(&G[h].prd[16 * kb + s]);
                            float m[4] = {v[s] * ex2_approx(pr[h] + f.x), v[s + 1] * ex2_approx(pr[h] + f.y),
                                          v[s + 2] * ex2_approx(pr[h] + f.z), v[s + 3] * ex2_approx(pr[h] + f.w)};
#pragma unroll
                            for (int i = 0; i < 4; ++i)  // the skip D x rides on the diagonal
                                m[i] = s + i < r ? m[i] : (s + i == r ? m[i] + Dh[h] : 0.f);
                            o[h][s / 2] = tc::pack_bf16(m[0], m[1]);
                            o[h][s / 2 + 1] = tc::pack_bf16(m[2], m[3]);
                        }
#pragma unroll
                    for (int h = 0; h < HEADS; ++h) tc::tmem_st8(col + 8 * h, o[h]);
                }
#pragma unroll 1
                for (int b = q + 1; b < 4; ++b)  // above it
                    tc::tmem_st16(lane_base + K::COL_CB + 16 * (2 * b + kb0), zero);
                tc::tmem_wait_st();
                tc::tc_before_sync();
                arrive(M_FULL);
                arrive(G_FREE + gs);
            }
        }
    } else if (warp < 16) {
        // =============================================================== S warps
        if constexpr (!STATES) enter(0, NS);
        // The gates are made here too, two chunks ahead, while the products run: a token a
        // thread, a block of 32 tokens a warp.
        constexpr int HEADS = ONE ? 1 : 2;
        bool on[HEADS];
        float A2[HEADS], bias[HEADS];
        uint16_t raw[HEADS];
        float run[HEADS];  // first pass: sums of the chunks behind, which are made first
#pragma unroll
        for (int h = 0; h < HEADS; ++h) {
            const Half f = half(h);
            on[h] = f.width > 0;
            A2[h] = on[h] ? -expf(a.A_log[f.head]) * tcf::kLog2e : 0.f;
            bias[h] = on[h] ? a.dt_bias[f.head] : 0.f;
            raw[h] = 0;
            run[h] = 0.f;
        }
        const uint16_t* dtp = static_cast<const uint16_t*>(a.dt) + (r0 + ln) * a.dts + half(0).head;
        auto fetch = [&](int c) {
#pragma unroll
            for (int h = 0; h < HEADS; ++h)
                if (on[h] && chunk_of(c) * L + ln < rows) raw[h] = dtp[(int64_t)chunk_of(c) * L * a.dts + h];
        };
        auto make_gates = [&](int c) {
            const int gs = c % NGR;
            Gates* G = &gates[2 * gs];
            float d[HEADS], left[HEADS], right[HEADS], behind[HEADS];
#pragma unroll
            for (int h = 0; h < HEADS; ++h) {
                const float v = __uint_as_float((uint32_t)raw[h] << 16) + bias[h];
                d[h] = on[h] && chunk_of(c) * L + ln < rows ? softplus_f32(v) : 0.f;
                float g = d[h] * A2[h];
                g = g < kMinG2 ? kMinG2 : g;  // (written so that a NaN stays one)
                left[h] = right[h] = g;
            }
            if (c + 1 < nch) fetch(c + 1);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1)  // sums within the block, from both ends
#pragma unroll
                for (int h = 0; h < HEADS; ++h) {
                    const float u = __shfl_up_sync(0xffffffffu, left[h], o), v = __shfl_down_sync(0xffffffffu, right[h], o);
                    if (lane >= o) left[h] += u;
                    if (lane + o < 32) right[h] += v;
                }
            if (c >= NGR) wait(G_FREE + gs, c / NGR - 1);
#pragma unroll
            for (int h = 0; h < HEADS; ++h) {
                behind[h] = __shfl_down_sync(0xffffffffu, right[h], 1);
                if (lane == 31) {
                    behind[h] = 0.f;
                    G[h].tot[q] = left[h];
                }
                if (STATES) continue;
                G[h].pre[ln] = left[h];
                // (the weights of W are rounded to bf16: approximate exponentials do)
                G[h].prd[ln] = __log2f(d[h]) - left[h];
                G[h].col[ln] = d[h] * ex2_approx(behind[h]);
            }
            tc::named_bar(4, 128);
#pragma unroll
            for (int h = 0; h < HEADS; ++h) {
                float later = 0.f;
                for (int b = 3; b > q; --b) later += G[h].tot[b];
                G[h].w[ln] = d[h] * exp2f(behind[h] + (later + run[h]));
                if (STATES) {
                    for (int b = q; b >= 0; --b) later += G[h].tot[b];
                    run[h] += later;
                } else if (ln == 0) {
                    G[h].last = exp2f(later + G[h].tot[0]);
                }
            }
            arrive(G_FULL + gs);
        };
        if (nch > 0) fetch(0);
        if constexpr (STATES) {
            // The groups' sums, added up in shared memory, a group's once the next one's first half has
            // its gates (the products are done by then); the last one's on its way out.
            const int ng = (nch + kGroup - 1) / kGroup;
            float* dst = p.part + ((int64_t)(sg.slot + sg.j) * p.units + unit) * a.N * 128 + ln;
            const uint32_t row = sbase + K::OFF_SUM + ln * NP * 4;  // in 16-byte units, swizzled
#pragma unroll 1
            for (int hg = 0; hg <= 2 * ng; ++hg) {  // half groups
                const int end = (hg + 1) * (kGroup / 2) < nch ? (hg + 1) * (kGroup / 2) : nch;
#pragma unroll 1
                for (int c = hg * (kGroup / 2); c < end; ++c) make_gates(c);
                const int g = (hg >> 1) - 1;
                if ((hg & 1) || g < 0) continue;
                wait(ACC_FULL + (g & 1), g >> 1);
                __syncwarp();
                tc::tc_after_sync();
#pragma unroll 1
                for (int n0 = 0; n0 < NP; n0 += 16) {
                    float v[16];
                    tc::tmem_ld16(lane_base + K::col_acc(g) + n0, v);
                    tc::tmem_wait_ld();
                    if (g > 0)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint4 o = tc::ld_shared_v4(row + (((n0 / 4 + i) ^ (ln & 7)) << 4));
                            v[4 * i] += __uint_as_float(o.x);
                            v[4 * i + 1] += __uint_as_float(o.y);
                            v[4 * i + 2] += __uint_as_float(o.z);
                            v[4 * i + 3] += __uint_as_float(o.w);
                        }
                    if (g < ng - 1)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            tc::st_shared_v4(row + (((n0 / 4 + i) ^ (ln & 7)) << 4), __float_as_uint(v[4 * i]),
                                             __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                                             __float_as_uint(v[4 * i + 3]));
                    else
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (n0 + i < a.N) dst[(n0 + i) * 128] = v[i];
                }
                tc::tc_before_sync();
                arrive(ACC_FREE + (g & 1));
            }
            if ((ln & 63) == 0) p.part_g[((int64_t)(sg.slot + sg.j) * p.units + unit) * 2 + (ln >> 6)] = run[ONE ? 0 : ln >> 6];
        } else {
            float ep = 0.f;
#pragma unroll 1
            for (int c = -2; c < nch; ++c) {
                if (c + 2 < nch) make_gates(c + 2);
                if (c < 0) continue;
                wait(G_FULL + c % NGR, c / NGR);
                ep = advance(c, 0, NS, ep);
            }
            leave(0, NS, ep);
        }
    } else if (warp < 24) {
        // =============================================================== Y warps
        // warpgroup j: half j, one token a thread
        if constexpr (!STATES) {
            const int j = (warp >> 2) & 1;
            const uint32_t ycol = lane_base + K::COL_Y + 64 * j;
            const uint32_t tile = sbase + K::OFF_Z + j * K::TILE;
            for (int c = 0; c < nch; ++c) {
                const int gs = c % NGR;
                wait(G_FULL + gs, c / NGR);
                const Gates& G = gates[2 * gs + (ONE ? 0 : j)];
                float e = G.pre[ln];
                for (int b = 0; b < q; ++b) e += G.tot[b];
                const float eg = ex2_approx(e);
                arrive(G_FREE + gs);
                wait(Y_FULL + j, 0);  // C h: times e^G, for W x to add to
                __syncwarp();
                tc::tc_after_sync();
#pragma unroll 1
                for (int n0 = 0; n0 < 64; n0 += 32) {
                    float v[32];
                    tc::tmem_ld32(ycol + n0, v);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 32; k += 8) {
                        uint32_t u[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) u[i] = __float_as_uint(eg * v[k + i]);
                        tc::tmem_st8(ycol + n0 + k, u);
                    }
                }
                tc::tmem_wait_st();
                tc::tc_before_sync();
                arrive(Y_FREE + j);
                wait(Y_FULL + j, 1);
                wait(Z_FULL + j, c);
                __syncwarp();
                tc::tc_after_sync();
                // y takes z's place, each thread in its own row
#pragma unroll 1
                for (int n0 = 0; n0 < 64; n0 += 16) {
                    float v[16];
                    tc::tmem_ld16(ycol + n0, v);
                    const uint32_t at[2] = {tile + tc::sw128_off(ln, n0 / 8), tile + tc::sw128_off(ln, n0 / 8 + 1)};
                    if (a.z) {
                        const uint4 z0 = tc::ld_shared_v4(at[0]), z1 = tc::ld_shared_v4(at[1]);
                        const uint32_t zw[8] = {z0.x, z0.y, z0.z, z0.w, z1.x, z1.y, z1.z, z1.w};
                        float2 g[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) g[i] = conv_silu2(make_float2(bf16_lo(zw[i]), bf16_hi(zw[i])));
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            v[2 * i] *= g[i].x;
                            v[2 * i + 1] *= g[i].y;
                        }
                    }
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int u = 0; u < 2; ++u)
                        tc::st_shared_v4(at[u], tc::pack_bf16(v[8 * u], v[8 * u + 1]), tc::pack_bf16(v[8 * u + 2], v[8 * u + 3]),
                                         tc::pack_bf16(v[8 * u + 4], v[8 * u + 5]), tc::pack_bf16(v[8 * u + 6], v[8 * u + 7]));
                }
                tc::tc_before_sync();
                arrive(Y_FREE + j);
                tc::fence_async_smem();
                arrive(Y_OUT + j);
            }
        }
    } else if (warp == 27) {
        // ======================================================= z and y tiles warp
        if constexpr (!STATES) {
#pragma unroll 1
            for (int c = 0; c <= nch; ++c)
#pragma unroll 1
                for (int j = 0; j < 2; ++j) {
                    const Half hf = half(j);
                    const uint32_t tile = sbase + K::OFF_Z + j * K::TILE;
                    if (c > 0) {  // y of the chunk before out of the tile
                        wait(Y_OUT + j, c - 1);
                        __syncwarp();
                        if (hf.width && !*abort_flag) {
                            if (c * L <= rows) {
                                if (lane == 0) {
                                    tma_store_3d(&p.y, tile, hf.col, hf.head, (int)r0 + (c - 1) * L);
                                    tc::bulk_commit();
                                    tc::bulk_wait_read0();
                                }
                            } else {  // the rows behind the sequence's end belong to another one
                                __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.y) +
                                                   ((r0 + (c - 1) * L) * a.H + hf.head) * a.P + hf.col;
#pragma unroll 1
                                for (int i = lane; i < tail * 8; i += 32)
                                    if (8 * (i & 7) < hf.width)
                                        *reinterpret_cast<uint4*>(y + (int64_t)(i >> 3) * a.H * a.P + 8 * (i & 7)) =
                                            tc::ld_shared_v4(tile + tc::sw128_off(i >> 3, i & 7));
                            }
                        }
                    }
                    if (c == nch || lane != 0) continue;
                    if (a.z && hf.width && !*abort_flag) {
                        tc::mbar_arrive_expect_tx(&bars[Z_FULL + j], K::TILE);
                        tma_load_3d(base + K::OFF_Z + j * K::TILE, &p.z, hf.col, hf.head, (int)r0 + c * L, &bars[Z_FULL + j]);
                    } else {
                        tc::mbar_arrive(&bars[Z_FULL + j]);
                    }
                }
            if (lane == 0) tc::bulk_wait0();  // y is in global memory before the CTA leaves, no load in flight
#pragma unroll 1
            for (int j = 0; nch > 0 && j < 2; ++j) drain(&bars[Z_FULL + j], (uint32_t)(nch - 1) & 1u);
            __syncwarp();
        }
    } else if (warp == 26) {
        // ============================================================== TMA warp
        if (lane == 0) {
            Half hf[2] = {half(0), half(1)};
            // a missing second head reads the first one's columns: nothing uses them
            if (hf[1].width == 0) hf[1] = hf[0];
            int done = 0;
#pragma unroll 1
            for (int c = 0; c < nch && !*abort_flag; ++c) {
                const int r = (int)r0 + chunk_of(c) * L;
                for (int j = 0; j < 2; ++j) {
                    const int xi = 2 * c + j, xb = xi % NXB;
                    if (xi >= NXB) wait(X_DONE + xb, xi / NXB - 1);
                    tc::mbar_arrive_expect_tx(&bars[X_FULL + xb], K::TILE);
                    tma_load_3d(base + K::OFF_X + xb * K::TILE, &p.x, hf[j].col, hf[j].head, r, &bars[X_FULL + xb]);
                }
                const int bc = c % NBC;
                if (!STATES) {
                    if (c >= NBC) wait(C_FREE_ + bc, c / NBC - 1);
                    tc::mbar_arrive_expect_tx(&bars[C_FULL_ + bc], K::BT);
                    for (int h = 0; h < NH; ++h)
                        tma_load_3d(base + K::OFF_C + bc * K::BT + h * K::TILE, &p.c, 64 * h, grp, r, &bars[C_FULL_ + bc]);
                }
                const int bb = c % NB;
                if (c >= NB) wait(B_FREE + bb, c / NB - 1);
                tc::mbar_arrive_expect_tx(&bars[B_FULL + bb], K::BT);
                for (int h = 0; h < NH; ++h)
                    tma_load_3d(base + K::OFF_B + bb * K::BT + h * K::TILE, &p.b, 64 * h, grp, r, &bars[B_FULL + bb]);
                if (NB == 1 && c + 1 < nch)
                    for (int h = 0; h < NH; ++h) {
                        tma_prefetch_3d(&p.b, 64 * h, grp, (int)r0 + chunk_of(c + 1) * L);
                        tma_prefetch_3d(&p.c, 64 * h, grp, (int)r0 + chunk_of(c + 1) * L);
                    }
                done = c + 1;
            }
            // never leave with a copy in flight
#pragma unroll 1
            for (int c = done >= NB ? done - NB : 0; c < done; ++c) {
                drain(&bars[B_FULL + c % NB], (c / NB) & 1);
                if (!STATES) drain(&bars[C_FULL_ + c % NBC], (c / NBC) & 1);
            }
#pragma unroll 1
            for (int i = 2 * done >= NXB ? 2 * done - NXB : 0; i < 2 * done; ++i)
                drain(&bars[X_FULL + i % NXB], (i / NXB) & 1);
        }
    } else if (warp < 26) {
        // ============================================================= MMA warps
        // Warp 25 the state's products; warp 24 C B^T, C h and W x.  Two warps, since one
        // would issue a chunk's 50 products slower than the tensor cores run them.
        constexpr uint32_t idCB = tc::idesc_bf16(128, 128, 0, 0), idY1 = tc::idesc_bf16(128, 64, 0, 1),
                           idS = tc::idesc_bf16(128, NP, 0, 1);
        auto ready = [&](int b, int phase) { nap_wait(&bars[b], (uint32_t)phase & 1u, abort_flag); };
        auto go = [&]() {
            __syncwarp();
            tc::tc_after_sync();
        };
        if (warp == 25) {
            for (int c = 0; c < nch; ++c) {
                const uint32_t lb0 = tc::desc_lo(sbase + K::OFF_B + (c % NB) * K::BT, K::TILE);
                ready(B_FULL + c % NB, c / NB);
                if (c == nch - 1 && tail < L) ready(CLEAN, 0);
                const int g = STATES ? c / kGroup : 0;
                const bool first = STATES && c == g * kGroup;  // of a group, whose sum starts anew
                if (!STATES) ready(S_READY, c);
                if (first && g > 1) ready(ACC_FREE + (g & 1), (g >> 1) - 1);
                const uint32_t acc = tmem + (STATES ? K::col_acc(g) : K::COL_S);
#pragma unroll 1
                for (int k = 0; k < 4; ++k) {  // S += (w x)^T B, 32 tokens
                    const int buf = STATES ? k : k & 1;
                    ready(XQ_FULL + buf, STATES ? c : 2 * c + (k >> 1));
                    go();
                    if (tc::elect_one()) {
                        const uint32_t wx = tmem + (STATES ? K::COL_WX1 : K::COL_WX) + 48 * buf, lb = lb0 + 256 * k;
                        if (first && k == 0) tc::mma_ts<0>(acc, wx, tc::desc(lb), idS);
                        else tc::mma_ts<1>(acc, wx, tc::desc(lb), idS);
                        tc::mma_ts<1>(acc, wx + 8, tc::desc(lb + 128), idS);
#pragma unroll 1
                        for (int s = 1; s < 3; ++s)
#pragma unroll
                            for (int ks = 0; ks < 2; ++ks)
                                tc::mma_ts<1>(acc, wx + 16 * s + 8 * ks, tc::desc(lb + 128 * ks), idS);
                        tc::mma_commit(&bars[XQ_FREE + buf]);
                        if (k == 3) {
                            if (!STATES) tc::mma_commit(&bars[DS_DONE]);
                            else if (c == nch - 1 || c == (g + 1) * kGroup - 1) tc::mma_commit(&bars[ACC_FULL + (g & 1)]);
                            tc::mma_commit(&bars[B_FREE + c % NB]);
                        }
                    }
                    __syncwarp();
                }
            }
        } else if constexpr (!STATES) {
            for (int c = 0; c < nch; ++c) {
                const int bc = c % NBC;
                const uint32_t lc = tc::desc_lo(sbase + K::OFF_C + bc * K::BT, 16),
                               lbk = tc::desc_lo(sbase + K::OFF_B + bc * K::BT, 16);
                ready(B_FULL + bc, c / NBC);
                if (c == nch - 1 && tail < L) ready(CLEAN, 0);
                ready(C_FULL_ + bc, c / NBC);
                if (c > 0) ready(W_FREE, c - 1);  // the last chunk's W has been read
                go();
                if (tc::elect_one()) {
#pragma unroll 1
                    for (int k = 0; k < NP / 16; ++k) {
                        const uint32_t o = (k >> 2) * (K::TILE / 16) + (k & 3) * 2;
                        tc::mma_bf16(tmem + K::COL_CB, tc::desc(lc + o), tc::desc(lbk + o), idCB, k > 0);
                    }
                    tc::mma_commit(&bars[CB_FULL]);
                    tc::mma_commit(&bars[B_FREE + bc]);
                }
                __syncwarp();
                ready(S_READY, c);
                if (c > 0) {
                    ready(Y_FREE, 1);
                    ready(Y_FREE + 1, 1);
                }
                go();
                if (tc::elect_one()) {  // C h, both halves
                    const uint32_t lh = tc::desc_lo(sbase + K::OFF_H, 16);
#pragma unroll 1
                    for (int k = 0; k < NP / 16; ++k) {
                        const uint32_t o = (k >> 2) * (K::TILE / 16) + (k & 3) * 2;
                        tc::mma_bf16(tmem + K::COL_Y, tc::desc(lc + o), tc::desc(lh + o), idCB, k > 0);
                    }
                    if (nch == 1) {  // its second term
                        const uint32_t lr = tc::desc_lo(sbase + K::OFF_X + 2 * K::TILE, 16);
#pragma unroll 1
                        for (int k = 0; k < NP / 16; ++k) {
                            const uint32_t o = (k >> 2) * (K::TILE / 16) + (k & 3) * 2;
                            tc::mma_bf16(tmem + K::COL_Y, tc::desc(lc + o), tc::desc(lr + o), idCB, 1);
                        }
                    }
                    tc::mma_commit(&bars[Y_FULL]);
                    tc::mma_commit(&bars[Y_FULL + 1]);
                    tc::mma_commit(&bars[H_FREE]);
                    tc::mma_commit(&bars[C_FREE_ + bc]);
                }
                __syncwarp();
                ready(M_FULL, c);
#pragma unroll 1
                for (int j = 0; j < 2; ++j) {  // W x, onto e^G C h
                    const int xi = 2 * c + j, xb = xi % NXB;
                    ready(X_FULL + xb, xi / NXB);
                    ready(Y_FREE + j, 0);
                    go();
                    if (tc::elect_one()) {
                        const uint32_t lx = tc::desc_lo(sbase + K::OFF_X + xb * K::TILE, K::TILE);
                        const uint32_t w = tmem + K::COL_CB + (ONE ? 0 : 8 * j), d = tmem + K::COL_Y + 64 * j;
#pragma unroll 1
                        for (int k = 0; k < 8; ++k) tc::mma_ts<1>(d, w + 16 * k, tc::desc(lx + 128 * k), idY1);
                        tc::mma_commit(&bars[Y_FULL + j]);
                        tc::mma_commit(&bars[X_DONE + xb]);
                        if (j == 1) tc::mma_commit(&bars[W_FREE]);
                    }
                    __syncwarp();
                }
            }
        }
        if (tc::elect_one()) {  // never leave with a product in flight
            uint64_t* bar = &bars[S_DRAIN + (warp & 1)];
            tc::mma_commit(bar);
            drain(bar, 0);
        }
        __syncwarp();
    }
    tc::tc_before_sync();
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) record_status(GDN_ERR_TIMEOUT);
    tc::tc_after_sync();
    if (warp == 0) tc::tmem_dealloc(tmem, 512);
}

// Chains the segment states of each sequence: slot j becomes the state behind
// segment j.  Grid: (element blocks, units, sequences) of 256 threads.
__global__ void __launch_bounds__(256) scan_chain_kernel(const __grid_constant__ ScanTcArgs p) {
    const ScanArgs& a = p.a;
    __shared__ int s_slot, s_n;
    const int unit = blockIdx.y, seq = blockIdx.z;
    const int64_t seg = (int64_t)p.seg_chunks * L;
    if (threadIdx.x < 32) {
        int64_t n, slot = 0;
        if (!a.cu) {
            n = seq_segments(a.T, seg);
            slot = seq * (n - 1);
        } else {
            n = seq_segments((int64_t)a.cu[seq + 1] - a.cu[seq], seg);
            if (n > 1)
                for (int s = threadIdx.x; s < seq; s += 32) slot += seq_segments((int64_t)a.cu[s + 1] - a.cu[s], seg) - 1;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) slot += __shfl_xor_sync(0xffffffffu, slot, o);
        }
        if (threadIdx.x == 0) {
            s_slot = (int)slot;
            s_n = (int)n;
        }
    }
    __syncthreads();
    if (s_n < 2) return;
    const int e = blockIdx.x * 256 + threadIdx.x;  // n * 128 + value lane
    if (e >= a.N * 128) return;
    const int n = e >> 7, ln = e & 127, j = ln >> 6;
    const Half hf = half_of(p, unit, j);
    float run = 0.f;
    if (a.h0 && (ln & 63) < hf.width)
        run = a.h0[(((int64_t)seq * a.H + hf.head) * a.N + n) * a.P + hf.col + (ln & 63)];
    const int64_t step = (int64_t)p.units * a.N * 128;
    float* s = p.part + ((int64_t)s_slot * p.units + unit) * a.N * 128 + e;
    const float* g = p.part_g + ((int64_t)s_slot * p.units + unit) * 2 + (a.P == 128 ? 0 : j);
    for (int i0 = 0; i0 + 1 < s_n; i0 += 8) {  // eight loads in flight
        float v[8], d[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i0 + i + 1 < s_n) {
                v[i] = s[(i0 + i) * step];
                d[i] = g[(int64_t)(i0 + i) * p.units * 2];
            }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i0 + i + 1 < s_n) {
                run = fmaf(run, exp2f(d[i]), v[i]);
                s[(i0 + i) * step] = run;
            }
    }
}

// ------------------------------------------------------------------------ host

inline bool make_map3(CUtensorMap* m, const void* ptr, int inner, int mid, int64_t rows, int64_t row_stride) {
    tcf::EncodeTiled enc = tcf::get_encode();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)mid, (cuuint64_t)rows};
    cuuint64_t strides[2] = {(cuuint64_t)inner * 2, (cuuint64_t)row_stride * 2};
    cuuint32_t box[3] = {64u, 1u, (cuuint32_t)L};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct ScanPlan {
    int pairs, units;
    int seg_chunks;   // chunks of a segment
    int64_t segments; // at most
    int64_t slots;    // segment states: full segments that are not a sequence's last, at most
};

// How long the segments are: the cheapest cut, in times of one chunk of the main pass (3 us).
// A CTA costs its chunks and about 2 more to start and end; a chunk of the first pass
// costs 0.3 and a CTA of it 1.5; the two more launches 3.  One segment a sequence is the
// plan when there are sequences and units enough for the SMs; a lone long sequence is cut
// into as many segments as fill them.  Packed lengths are not known here: the longest of
// n is taken as the mean of the longest of n random parts, and the segments as balanced
// by the order of the blocks.
inline ScanPlan plan_scan(int n_seq, int64_t T_total, bool packed, int H, int G, int P, int sms) {
    ScanPlan r;
    r.pairs = P == 128 ? H / G : (H / G + 1) / 2;
    r.units = G * r.pairs;
    const int64_t len = packed ? T_total : T_total / n_seq;
    const int64_t chunks = (len + L - 1) / L;
    double share = 0;  // of the longest packed sequence
    for (int i = 1; i <= n_seq && i <= 64; ++i) share += 1.0 / i / n_seq;
    const double longest = packed && n_seq > 1 ? chunks * (share < 1 ? share : 1) : (double)chunks;
    double best = 0;
    r.seg_chunks = 0x400000;
    for (int cut = 1; cut <= 160 && (cut == 1 || cut * 4 <= chunks); ++cut) {
        const int64_t sc = (chunks + cut - 1) / cut;
        const int64_t nseg = chunks ? (chunks + sc - 1) / sc : 1;
        double cost;
        if (packed) {
            const double u = (double)r.units / sms, part = longest > sc ? 1.0 - (double)sc / (2 * longest) : 0.0;
            const double tail = sc < longest ? (double)sc : longest;
            cost = u * chunks + 0.5 * tail + 2.0 * u * (nseg + n_seq);
            if (cost < tail) cost = tail;
            if (cut > 1) cost += part * (0.3 * u * chunks + 1.5 * u * nseg) + 3.0;
        } else {
            const int64_t main = n_seq * nseg * r.units, first = n_seq * (nseg - 1) * r.units;
            cost = (double)((main + sms - 1) / sms) * (sc + 2);
            if (nseg > 1) cost += (double)((first + sms - 1) / sms) * (0.3 * sc + 1.5) + 3.0;
        }
        if (cut == 1 || cost < best) {
            best = cost;
            r.seg_chunks = (int)(sc > 0 ? sc : 1);
        }
    }
    const int64_t seg = (int64_t)r.seg_chunks * L;
    if (packed) {
        r.slots = T_total > seg ? T_total / seg : 0;
        r.segments = r.slots + n_seq;
    } else {
        const int64_t n = len <= seg ? 1 : (len + seg - 1) / seg;
        r.slots = (n - 1) * n_seq;
        r.segments = n * n_seq;
    }
    return r;
}

inline size_t scan_part_bytes(const ScanPlan& r, int N) {
    return ((size_t)r.slots * r.units * ((size_t)N * 128 + 2) * 4 + 255) / 256 * 256;
}

// Whether TMA can address the rows of t.
inline bool tma_rows(const void* t, int64_t stride) {
    return (reinterpret_cast<uintptr_t>(t) & 15u) == 0 && stride % 8 == 0;
}

template <int NP>
inline cudaError_t launch_scan_np(const ScanTcArgs& p, const ScanPlan& r, cudaStream_t st) {
    using K = ScanCfg<NP>;
    auto main = p.a.P == 128 ? scan_tc_kernel<NP, false, true> : scan_tc_kernel<NP, false, false>;
    auto states = p.a.P == 128 ? scan_tc_kernel<NP, true, true> : scan_tc_kernel<NP, true, false>;
    cudaError_t e = cudaFuncSetAttribute(main, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)K::SMEM);
    if (e != cudaSuccess) return e;
    if (r.slots > 0) {
        e = cudaFuncSetAttribute(states, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)K::SMEM);
        if (e != cudaSuccess) return e;
        states<<<(unsigned)(r.slots * r.units), kScanThreads, K::SMEM, st>>>(p);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        scan_chain_kernel<<<dim3((unsigned)(p.a.N / 2), (unsigned)r.units, (unsigned)p.a.n_seq), 256, 0, st>>>(p);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    main<<<(unsigned)(r.segments * r.units), kScanThreads, K::SMEM, st>>>(p);
    return cudaGetLastError();
}

inline cudaError_t launch_scan_tc(const ScanArgs& a, int64_t rows, const ScanPlan& r, void* workspace, cudaStream_t st) {
    ScanTcArgs p;
    memset(&p, 0, sizeof(p));
    if (!make_map3(&p.x, a.x, a.P, a.H, rows, a.xs) || !make_map3(&p.b, a.Bm, a.N, a.G, rows, a.bs) ||
        !make_map3(&p.c, a.Cm, a.N, a.G, rows, a.cs) || (a.z && !make_map3(&p.z, a.z, a.P, a.H, rows, a.zs)) ||
        !make_map3(&p.y, a.y, a.P, a.H, rows, (int64_t)a.H * a.P))
        return cudaErrorInvalidValue;
    p.a = a;
    p.pairs = r.pairs;
    p.units = r.units;
    p.per = a.H / a.G;
    p.seg_chunks = r.seg_chunks;
    p.part = static_cast<float*>(workspace);
    p.part_g = p.part + r.slots * r.units * a.N * 128;
    return a.N == 128 ? launch_scan_np<128>(p, r, st) : launch_scan_np<64>(p, r, st);
}

}  // namespace ssm
}  // namespace gdn
