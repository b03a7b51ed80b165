// fp8_matmul_tc.cuh -- the block-scaled 8-bit product on the tensor cores.
//
//     out[m, n] = sum_b as[m, b] ws[n / 128, b] (sum_{k in block b} a[m, k] w[n, k])
//
// The scales change every 128 of K, so the tensor core accumulates one block of
// K at a time into tensor memory (four K = 32 products, kind::f8f6f4) and the
// promotion warps add it, scaled, to fp32 sums in registers.  Two accumulators
// alternate, so the products of block b + 1 run while block b is promoted.
//
// One operand's rows are the 128 tensor-memory lanes, the other's the TN columns:
//  * TOKENS = true, TN = 256: lanes are tokens.  A thread's scale is one number a
//    block (its columns lie in one 128-block of n).  The form of prompts.
//  * TOKENS = false, TN = 16..128: lanes are rows of w, columns are tokens, so a
//    few tokens fill whole tiles and w streams through once.  The K range may be
//    split over a cluster of up to 8 CTAs; each leaves its partial sums in
//    shared memory and the cluster adds them in rank order (no atomics).
// Warps: promotion (4 or 8), then a TMA warp and an MMA warp.  A CTA walks its
// tiles (blockIdx.x, + gridDim.x, ...): loads and products of the next tile run
// while the last one is written out.
//
// What bounds it and what it measured.
//  * 4096 x 14336 x 4096, bf16 out: 230 us (2.1 PFLOP/s) with the operands in L2, 255 to 270
//    (1.8) with other ones each time; the power cap holds the clock at 1.5 to 1.6 GHz.  A K
//    block takes about 900 cycles an SM, of which the products are 522 (4 x 131; the tensor
//    pipe is 60 % busy) and reading 128 x 256 sums from tensor memory and adding them some
//    500.  The two accumulators would let those overlap whole; what the rest of the 900 waits
//    for is not known (issue slots 41 %, L2 47 %, HBM 8 %).  1792 tiles are 12.1 rounds of 148
//    SMs, taken as 13.  The promotion warps have 168 registers for 128 sums and 32 loaded
//    ones (ten warps are three on some scheduler), so a few more live values cost a tenth.
//    Tried: 16 promotion warps of 64 columns 318 us (8 of 128: 292), an accumulator's
//    loads not ahead of its sums 292 (ahead: 267), rows written a thread each 267 (through
//    shared memory: 245), accumulators in halves of 128 columns 245 (whole: 232).
//  * 77 x 6176 x 2064: 11.2 us, 1 x 8192 x 4096: 8.3 us (10.0 with w from HBM), 64 x 8192 x 4096: 11.8 us: launch, the
//    ring's first fill and the cluster's barriers, then w's bytes at the rate that two CTAs
//    an SM sustain (one an SM, 17.7 us for the last).  1 x 65536 x 4096: 44 us, 6.1 TB/s.
#pragma once

#include "chunk_tc.cuh"
#include "fp8_matmul.cuh"

namespace gdn {
namespace mm8 {

constexpr uint32_t kLaneTile = 128 * 128;  // bytes of one 128-row tile of a K block

template <bool TOKENS, int TN>
struct Cfg {
    static constexpr int NPW = TN >= 128 ? 8 : 4;         // promotion warps: 16 to 128 columns a thread
    static constexpr int CPT = TN / (NPW / 4);            // columns of one promotion thread
    static constexpr int THREADS = 32 * (NPW + 2);
    static constexpr uint32_t STAGE = kLaneTile + TN * 128;
    static constexpr int NS = TN == 256 ? 4 : (TN == 128 ? 3 : (TN == 64 ? 4 : 5));  // ring stages
    static constexpr int PER_SM = TN == 256 ? 1 : 2;      // CTAs of an SM
    static constexpr uint32_t OFF_SC = NS * STAGE;        // [2][TN] column scales (columns = tokens)
    static constexpr uint32_t OFF_OUT = NS * STAGE;       // per-warp tiles of the result (lanes = tokens)
    static constexpr uint32_t OFF_BAR = NS * STAGE + (TOKENS ? NPW * 4096 : 2 * TN * 4);
    static constexpr uint32_t SMEM = OFF_BAR + (2 * NS + 5) * 8 + 16 + 1024;
    static constexpr uint32_t COLS = 2 * TN < 32 ? 32 : 2 * TN;
    static_assert(TOKENS || TN * 512 <= NS * STAGE, "partial sums fit in the ring");
    static_assert(SMEM <= (PER_SM == 1 ? 232448 : 115712), "shared memory budget");
};

struct TcArgs {
    CUtensorMap lanes, cols;  // [rows, K] e4m3, boxes of 128 bytes x 128 (TN) rows, 128-byte swizzle
    CUtensorMap out;          // [M, N], boxes of 128 bytes x 32 rows (MAP)
    Args g;
    int tiles_l, tiles;       // tiles along the lane operand, tiles in all
    int split;                // CTAs of a cluster, each with its part of K
};

// kind::f8f6f4: e4m3 x e4m3 -> fp32, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// The products of one K block (four of K = 32; operands at a, b in shared memory, 32 bytes
// apart) into d, then the arrivals on two barriers when they are done.  Called by a whole
// converged warp, issued by one elected lane in one sequence.
__device__ __forceinline__ void mma_block_e4m3(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t done0,
                                               uint32_t done1) {
    asm volatile(
        "{\n .reg .pred e, z;\n .reg .b32 t;\n .reg .b64 a0, a1, a2, a3, b0, b1, b2, b3;\n"
        " mov.b64 a0, {%1, %4};\n mov.b64 b0, {%2, %4};\n"
        " add.u32 t, %1, 2;\n mov.b64 a1, {t, %4};\n add.u32 t, %2, 2;\n mov.b64 b1, {t, %4};\n"
        " add.u32 t, %1, 4;\n mov.b64 a2, {t, %4};\n add.u32 t, %2, 4;\n mov.b64 b2, {t, %4};\n"
        " add.u32 t, %1, 6;\n mov.b64 a3, {t, %4};\n add.u32 t, %2, 6;\n mov.b64 b3, {t, %4};\n"
        " setp.ne.b32 z, 0, 0;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a0, b0, %3, z;\n"
        " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, 1;\n"
        " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a2, b2, %3, 1;\n"
        " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a3, b3, %3, 1;\n"
        " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n"
        " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%6];\n}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(tc::desc_hi_sw128()), "r"(done0), "r"(done1)
        : "memory");
}
// Waits for the loads from tensor memory; the values pass through, so no use of them moves
// before it.
__device__ __forceinline__ void wait_ld16(float (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
                 :
                 : "memory");
}
__device__ __forceinline__ float4 ld_cluster_v4(uint32_t caddr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(caddr)
                 : "memory");
    return v;
}

// MAP: the result's rows start on 16 bytes, and its tiles leave by TMA (lanes = tokens; with
// both ways in one kernel the sums spill: 228 to 241 us).
template <bool TOKENS, int TN, typename TOut, bool MAP>
__global__ void __launch_bounds__((Cfg<TOKENS, TN>::THREADS), (Cfg<TOKENS, TN>::PER_SM)) fp8_matmul_tc_kernel(
    const __grid_constant__ TcArgs p) {
    using C = Cfg<TOKENS, TN>;
    constexpr int NS = C::NS, NPW = C::NPW, CPT = C::CPT;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_u32 = smem_u32(smem_raw);
    const uint32_t sbase = (raw_u32 + 1023u) & ~1023u;
    uint8_t* base = smem_raw + (sbase - raw_u32);
    uint64_t* bars = reinterpret_cast<uint64_t*>(base + C::OFF_BAR);
    uint64_t *full = bars, *empty = bars + NS, *acc_full = bars + 2 * NS, *acc_free = acc_full + 2,
             *drain = acc_full + 4;
    uint32_t* misc = reinterpret_cast<uint32_t*>(drain + 1);
    volatile uint32_t* abort_flag = misc + 1;
    const Args& g = p.g;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kb_all = (g.K + 127) / 128;
    const int split = p.split;
    const int rank = split > 1 ? (int)tc::cluster_ctarank() : 0;
    const int kb0 = (int)((int64_t)kb_all * rank / split);
    const int kb1 = (int)((int64_t)kb_all * (rank + 1) / split);
    const int tile0 = blockIdx.x / split, tile_step = gridDim.x / split;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], TOKENS ? 1 : 2);  // the products (, their scales)
            mbar_init(&acc_free[i], NPW);
        }
        mbar_init(drain, 1);
        misc[1] = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) tc::tmem_alloc(&misc[0], C::COLS);
    tc::tc_before_sync();
    __syncthreads();
    tc::tc_after_sync();
    const uint32_t tmem = __reduce_max_sync(0xffffffffu, misc[0]);

    if (warp == NPW) {
        // ---------------------------------------------------------- TMA warp
        if (lane == 0) {
            tc::prefetch_tmap(&p.lanes);
            tc::prefetch_tmap(&p.cols);
            int it = 0;
            for (int t = tile0; t < p.tiles && !*abort_flag; t += tile_step) {
                const int lrow = 128 * (t % p.tiles_l), crow = TN * (t / p.tiles_l);
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    const int s = it % NS;
                    if (it >= NS) nap_wait(&empty[s], ((it / NS) - 1) & 1, abort_flag);
                    if (*abort_flag) break;
                    uint8_t* st = base + s * C::STAGE;
                    tc::mbar_arrive_expect_tx(&full[s], C::STAGE);
                    tc::tma_load_2d(st, &p.lanes, 128 * kb, lrow, &full[s]);
                    tc::tma_load_2d(st + kLaneTile, &p.cols, 128 * kb, crow, &full[s]);
                }
            }
            // never leave with a copy in flight
            for (int i = it > NS ? it - NS : 0; i < it; ++i) tcf::drain_wait(&full[i % NS], (i / NS) & 1);
        }
    } else if (warp == NPW + 1) {
        // ---------------------------------------------------------- MMA warp
        constexpr uint32_t id = idesc_e4m3(128, TN);
        const uint32_t la0 = tc::desc_lo(sbase, 16), lb0 = tc::desc_lo(sbase + kLaneTile, 16);
        auto products = [&](int it) {
            const int s = it % NS, b = it & 1;
            nap_wait(&full[s], (it / NS) & 1, abort_flag);
            if (it >= 2) nap_wait(&acc_free[b], ((it >> 1) - 1) & 1, abort_flag);
            __syncwarp();
            tc::tc_after_sync();
            mma_block_e4m3(tmem + b * TN, la0 + s * (C::STAGE / 16), lb0 + s * (C::STAGE / 16), id,
                           smem_u32(&empty[s]), smem_u32(&acc_full[b]));
        };
        int it = 0;
        if constexpr (TOKENS) {
            for (int t = tile0; t < p.tiles; t += tile_step)
                for (int kb = kb0; kb < kb1; ++kb, ++it) products(it);
        } else {
            // This warp also hands out the scales of a block's columns (ws as), behind its
            // products: loaded two blocks ahead, in place of those of two blocks ago, whose
            // sums are done.  (In the promotion warps, one block ahead, the loads cost 128
            // tokens their registers and their time.)
            constexpr int NC = (TN + 31) / 32;
            float* sc = reinterpret_cast<float*>(base + C::OFF_SC);
            for (int t = tile0; t < p.tiles; t += tile_step) {
                const int nb = t % p.tiles_l, m0 = TN * (t / p.tiles_l) + lane;
                const float* pw = g.ws + (int64_t)nb * kb_all;
                const float* pa = g.as + (int64_t)m0 * kb_all;
                float nw[2], na[2][NC];
                auto fetch = [&](int kb, int u) {
                    nw[u] = kb < kb1 ? __ldg(pw + kb) : 0.f;
#pragma unroll
                    for (int i = 0; i < NC; ++i)
                        na[u][i] = kb < kb1 && m0 + 32 * i < g.M && lane + 32 * i < TN
                                       ? __ldg(pa + (int64_t)32 * i * kb_all + kb) : 0.f;
                };
                fetch(kb0, 0);
                fetch(kb0 + 1, 1);
                for (int kbu = kb0; kbu < kb1; kbu += 2)
#pragma unroll
                    for (int u = 0; u < 2; ++u)
                        if (kbu + u < kb1) {
                            products(it);
#pragma unroll
                            for (int i = 0; i < NC; ++i)
                                if (lane + 32 * i < TN) sc[(it & 1) * TN + lane + 32 * i] = nw[u] * na[u][i];
                            __syncwarp();
                            if (lane == 0) tc::mbar_arrive(&acc_full[it & 1]);
                            fetch(kbu + u + 2, u);
                            ++it;
                        }
            }
        }
        if (tc::elect_one()) {  // never leave with a product in flight
            tc::mma_commit(drain);
            tcf::drain_wait(drain, 0);
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------- promotion warps
        const int q = warp & 3;                    // lane quarter of tensor memory
        const int c0 = CPT * (warp >> 2);          // first column of this thread
        const int ln = 32 * q + lane;
        const uint32_t taddr = tmem + ((uint32_t)(32 * q) << 16) + c0;
        const float* sc = reinterpret_cast<const float*>(base + C::OFF_SC) + c0;
        int it = 0;
        for (int t = tile0; t < p.tiles; t += tile_step) {
            const int lrow = 128 * (t % p.tiles_l) + ln, crow = TN * (t / p.tiles_l) + c0;
            float2 acc[CPT / 2];
#pragma unroll
            for (int j = 0; j < CPT / 2; ++j) acc[j] = make_float2(0.f, 0.f);
            // Lanes are tokens: this token's scale of a block is fetched a block ahead and multiplied
            // where it is used (a product here would wait for the loads).  Rows behind M and N
            // take the first one's: nothing of theirs is stored.
            const float* pw = g.ws + (int64_t)(TOKENS && crow < g.N ? crow / 128 : 0) * kb_all;
            const float* pa = g.as + (int64_t)(TOKENS && lrow < g.M ? lrow : 0) * kb_all;
            float nw = 0.f, na = 0.f;
            auto fetch = [&](int kb) {
                if constexpr (TOKENS) {
                    nw = __ldg(pw + kb);
                    na = __ldg(pa + kb);
                }
            };
            fetch(kb0);
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int b = it & 1;
                const float s = nw * na;
                const float* scb = sc + b * TN;
                if (kb + 1 < kb1) fetch(kb + 1);
                nap_wait(&acc_full[b], (it >> 1) & 1, abort_flag);
                __syncwarp();
                tc::tc_after_sync();
                // 16 columns at a time, the next ones under way while these are added
                float v[2][16];
                tc::tmem_ld16(taddr + b * TN, v[0]);
#pragma unroll
                for (int j = 0; j < CPT; j += 16) {
                    wait_ld16(v[(j / 16) & 1]);
                    if (j + 16 < CPT) tc::tmem_ld16(taddr + b * TN + j + 16, v[(j / 16 + 1) & 1]);
                    const float* u = v[(j / 16) & 1];
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        float2 f;
                        if constexpr (TOKENS)
                            f = make_float2(s, s);
                        else
                            f = *reinterpret_cast<const float2*>(&scb[j + i]);
                        acc[(j + i) / 2] = __ffma2_rn(make_float2(u[i], u[i + 1]), f, acc[(j + i) / 2]);
                    }
                }
                tc::tc_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&acc_free[b]);
            }
            TOut* out = static_cast<TOut*>(g.out);
            if constexpr (TOKENS) {
                // 32 rows x 128 bytes at a time through this warp's tile: a row a thread would
                // write 16 bytes (or one element) of 32 lines with every store
                constexpr int V = 16 / sizeof(TOut), CV = 128 / sizeof(TOut);
                uint8_t* stg = base + C::OFF_OUT + warp * 4096;
#pragma unroll
                for (int j = 0; j < CPT; j += CV) {
                    if (MAP && lane == 0) tc::bulk_wait_read0();
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        uint4 u;
                        TOut* e = reinterpret_cast<TOut*>(&u);
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            const int c = j + k * V + i;
                            e[i] = from_f32<TOut>((c & 1) ? acc[c / 2].y : acc[c / 2].x);
                        }
                        *reinterpret_cast<uint4*>(stg + lane * 128 + ((k ^ (lane & 7)) << 4)) = u;
                    }
                    if constexpr (MAP) {
                        tc::fence_async_smem();
                        __syncwarp();
                        if (lane == 0 && lrow < g.M && crow + j < g.N) {
                            tc::tma_store_2d(&p.out, smem_u32(stg), crow + j, lrow);
                            tc::bulk_commit();
                        }
                    } else {  // rows that do not start on 16 bytes: a row of the tile a warp's store
                        __syncwarp();
                        const int rows = g.M - (lrow - lane), left = g.N - crow - j;
#pragma unroll 4
                        for (int r = 0; r < 32; ++r)
#pragma unroll
                            for (int c = 0; c < CV; c += 32)
                                if (r < rows && c + lane < left)
                                    out[(int64_t)(lrow - lane + r) * g.N + crow + j + c + lane] =
                                        reinterpret_cast<const TOut*>(stg + r * 128 + ((((c + lane) / V) ^ (r & 7)) << 4))[lane % V];
                    }
                }
            } else if (split == 1) {
                if (lrow < g.N) {
#pragma unroll
                    for (int j = 0; j < CPT; ++j)
                        if (crow + j < g.M)
                            out[(int64_t)(crow + j) * g.N + lrow] = from_f32<TOut>((j & 1) ? acc[j / 2].y : acc[j / 2].x);
                }
            } else {
                // this CTA's part of the sums, [token][n], over the spent ring (one
                // tile a cluster, every load and product of it done)
                float* red = reinterpret_cast<float*>(base);
#pragma unroll
                for (int j = 0; j < CPT; ++j) red[(c0 + j) * 128 + ln] = (j & 1) ? acc[j / 2].y : acc[j / 2].x;
            }
        }
        if (MAP && lane == 0) tc::bulk_wait_read0();
    }
    tc::tc_before_sync();
    __syncthreads();
    if constexpr (!TOKENS) {
        if (split > 1) {
            tc::cluster_sync();
            // four neighbouring n a thread, every part's loads in flight together
            const int n0 = 128 * (tile0 % p.tiles_l), m0 = TN * (tile0 / p.tiles_l);
            const int toks = g.M - m0 < TN ? g.M - m0 : TN;
            TOut* out = static_cast<TOut*>(g.out);
            const bool whole = n0 + 128 <= g.N && g.N % 4 == 0 && (reinterpret_cast<uintptr_t>(out) & 15u) == 0;
            for (int e = rank * C::THREADS + threadIdx.x; e < toks * 32; e += split * C::THREADS) {
                const int j = e >> 5, n = n0 + 4 * (e & 31);
                float4 part[8];
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (r < split) part[r] = ld_cluster_v4(tc::mapa(sbase + 16 * e, (uint32_t)r));
                float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (r < split) {
                        v[0] += part[r].x;
                        v[1] += part[r].y;
                        v[2] += part[r].z;
                        v[3] += part[r].w;
                    }
                TOut* o = out + (int64_t)(m0 + j) * g.N + n;
                if (whole) {
                    if constexpr (sizeof(TOut) == 2)
                        *reinterpret_cast<uint2*>(o) = make_uint2(tc::pack_bf16(v[0], v[1]), tc::pack_bf16(v[2], v[3]));
                    else
                        *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (n + i < g.N) o[i] = from_f32<TOut>(v[i]);
                }
            }
            tc::cluster_sync();  // no CTA leaves while another reads its sums
        }
    }
    if (threadIdx.x == 0 && *abort_flag) record_status(GDN_ERR_TIMEOUT);
    tc::tc_after_sync();
    if (warp == 0) tc::tmem_dealloc(tmem, C::COLS);
}

// [rows, K] bytes, boxes of 128 bytes x box_rows rows; behind K and the rows, zeros.
inline bool make_map8(CUtensorMap* m, const void* ptr, int64_t rows, int64_t K, int64_t ld, int box_rows) {
    tcf::EncodeTiled enc = tcf::get_encode();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)ld};
    cuuint32_t box[2] = {128u, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The result: boxes of 128 bytes x 32 rows.
template <typename TOut>
inline bool make_map_out(CUtensorMap* m, void* ptr, int64_t rows, int64_t N) {
    tcf::EncodeTiled enc = tcf::get_encode();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)N, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)N * sizeof(TOut)};
    cuuint32_t box[2] = {128u / sizeof(TOut), 32u};
    cuuint32_t estr[2] = {1, 1};
    return enc(m, sizeof(TOut) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, ptr, dims,
               strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool TOKENS, int TN, typename TOut, bool MAP = false>
inline cudaError_t launch_tc(const Args& g, int split, int sms, cudaStream_t st) {
    using C = Cfg<TOKENS, TN>;
    TcArgs p;
    memset(&p, 0, sizeof(p));
    const bool ok = TOKENS ? make_map8(&p.lanes, g.a, g.M, g.K, g.lda, 128) &&
                                 make_map8(&p.cols, g.w, g.N, g.K, g.ldw, TN)
                           : make_map8(&p.lanes, g.w, g.N, g.K, g.ldw, 128) &&
                                 make_map8(&p.cols, g.a, g.M, g.K, g.lda, TN);
    if (!ok) return cudaErrorInvalidValue;
    if (MAP && !make_map_out<TOut>(&p.out, g.out, g.M, g.N)) return cudaErrorInvalidValue;
    p.g = g;
    const int64_t lanes = TOKENS ? g.M : g.N, cols = TOKENS ? g.N : g.M;
    const int64_t tl = (lanes + 127) / 128, tiles = tl * ((cols + TN - 1) / TN);
    if (tiles > 0x7fffffff / 8) return cudaErrorInvalidValue;
    p.tiles_l = (int)tl;
    p.tiles = (int)tiles;
    p.split = split;
    auto kern = fp8_matmul_tc_kernel<TOKENS, TN, TOut, MAP>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cfg.blockDim = dim3(C::THREADS, 1, 1);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = st;
    // Every tile its cluster, or as many CTAs as fit at once, walking the tiles (the small forms two
    // an SM: 1 x 65536 x 4096 44 us, 64 x 20000 x 4096 22; with one an SM 50 and 32).
    const int64_t most = (int64_t)C::PER_SM * sms;
    cfg.gridDim = dim3((unsigned)(split > 1 ? tiles * split : (tiles < most ? tiles : most)), 1, 1);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

// The form and split for a size.
template <typename TOut>
inline cudaError_t launch_fp8_matmul(const Args& g, int sms, cudaStream_t st) {
    const int64_t tok_tiles = (int64_t)((g.M + 127) / 128) * ((g.N + 255) / 256);
    if (g.M > 128 && tok_tiles >= sms / 2) {
        const bool map = (int64_t)g.N * sizeof(TOut) % 16 == 0 && (reinterpret_cast<uintptr_t>(g.out) & 15u) == 0;
        return map ? launch_tc<true, 256, TOut, true>(g, 1, sms, st) : launch_tc<true, 256, TOut, false>(g, 1, sms, st);
    }
    const int tn = g.M <= 16 ? 16 : (g.M <= 32 ? 32 : (g.M <= 64 ? 64 : 128));
    const int64_t tiles = (int64_t)((g.N + 127) / 128) * ((g.M + tn - 1) / tn);
    const int kb = (g.K + 127) / 128;
    // as many parts of K, of two blocks at least, as keep every CTA resident (two an SM); a
    // power of two, since odd clusters leave SMs of a GPC over
    int split = 1;
    while (split < 8 && tiles * split * 2 <= 2 * sms && kb / (split * 2) >= 2) split *= 2;
    if (tn == 16) return launch_tc<false, 16, TOut>(g, split, sms, st);
    if (tn == 32) return launch_tc<false, 32, TOut>(g, split, sms, st);
    if (tn == 64) return launch_tc<false, 64, TOut>(g, split, sms, st);
    return launch_tc<false, 128, TOut>(g, split, sms, st);
}

}  // namespace mm8
}  // namespace gdn
