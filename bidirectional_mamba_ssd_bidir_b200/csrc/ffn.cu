// ffn.cu -- the gated feed-forward block and its gradients on the tensor core.
//
// With g = u Wg^T and p = u Wu^T (Wg, Wu the two halves of W_in), h = act(g) * p, out = h Wd^T
// (Wd = W_out):
//
//   gh = gy Wd        gg = gh p act'(g)      gp = gh act(g)
//   gu = [gg gp] W_in          gW_in = [gg gp]^T u          gW_out = gy^T h
//
// act = SiLU: g sg, act' = sg (1 + g (1 - sg)); or GELU: g Phi(g), act' = Phi(g) + g phi(g).
//
// Two launches forward and two backward do all of it: the two projections, the activation and the
// product in one (h, and the projections when they are saved), then out; gh with the activation's
// gradient in its epilogue; and the three remaining products of the backward pass side by side (with few
// tokens gu in a launch of its own).
// Rounded to bf16 between them: h, gg, gp and the saved projections (the operands of the next
// product have to be bf16 for the tensor core; accumulation, activation and its derivative are
// float32).
//
// k_ffn, one kernel for all products D[M][N] = A B: persistent, warp-specialised, tiles of
// 128 CG x 256 over a group of CG CTAs (CG = 2: a CTA pair shares one tcgen05.mma of M = 256, each
// CTA holding half of A's rows and half of B's columns).  Warp 0 feeds the stage ring by TMA, warp 1
// of the group's first CTA issues the MMAs (N 256, K 16), warps 2-5 (2-9 with the activation's
// gradient) drain one 256-column TMEM accumulator while the other fills, each warp storing its own 32
// rows through its own staging boxes.
// Measured (8177 tokens, d_model 2048, d_ff 8192; bf16 cuBLAS rate 1663 TFLOP/s in a burst, 1390 sustained
// under the power cap): forward 670 to 759 us from card to card, 1.09 to 1.23 PFLOP/s; backward 1.60 to 1.72 ms,
// 0.96 to 1.03; the projections kernel alone 404 us, 1.36 PFLOP/s, the last launch of the backward pass 1.05.  In
// captures (1.57 to 1.65 GHz under the cap) the tensor pipe is active 75 % of the projections' time, 62 and 63 %
// of the two launches of plain products and 47 % of gh with the activation's gradient; L2 gives 44 % of its rate at
// most, the SM's memory pipes 72 %, so no unit is at its limit, and what the MN-major operands of the backward
// pass cost is not known.  Prefetching into L2 ahead of the loads made it 35 % slower, other orders of the tiles
// changed nothing.  Products with few tiles lose to the last wave (256 tiles on 74 pairs: 0.86).
// An operand may lie along K (K-major: rows of 64 k, the descriptor's usual form) or across it
// (MN-major: 64 x 64 boxes, 64 rows or columns wide), so nothing is transposed in memory.  Edges of
// any size come out of the tensor maps: loads outside a matrix read zero, stores there are dropped.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cstring>

#include "ffn.cuh"
#include "ragged.cuh"
#include "ssd_tc_common.cuh"

namespace ssd {
namespace {

enum Epi { EPI_PLAIN, EPI_GLU, EPI_GLU_BWD };

constexpr int kFK = 64;                          // K of a stage
constexpr uint32_t kFBox = 128 * 128;            // 128 rows of 64 bf16
constexpr uint32_t kFOutBox = 32 * 128;          // one warp's 32 rows of 64 columns
constexpr int kFThreads = 192, kFMaxProb = 3;
// The activation's gradient takes more work an element than one warp per SM sub-partition does in the
// time of a tile: eight epilogue warps there, each half of the columns.
template <int EPI> constexpr int kEpiWarps = EPI == EPI_GLU_BWD ? 8 : 4;
template <int EPI> constexpr int kFfnThreads = 64 + 32 * kEpiWarps<EPI>;
constexpr uint32_t kNarrowBox = 32 * 64;         // one warp's 32 rows of 32 columns

template <int EPI, int CG> struct FfnTile {
    static constexpr uint32_t kA = kFBox, kB = CG == 2 ? kFBox : 2 * kFBox, kStage = kA + kB;
    static constexpr int kBoxes = EPI == EPI_PLAIN ? 2 : 3;       // staging boxes of an epilogue warp
    static constexpr int kStages = CG == 2 ? (EPI == EPI_PLAIN ? 6 : 5) : (EPI == EPI_PLAIN ? 4 : 3);
    static constexpr uint32_t kOut = kStages * kStage;
    static constexpr uint32_t kBar = kOut + (EPI == EPI_GLU_BWD ? 8 * 3 * kNarrowBox : 4 * kBoxes * kFOutBox);
    static constexpr int kFull = 0, kEmpty = kStages, kAccFull = 2 * kStages, kAccEmpty = kAccFull + 2, kDone = kAccEmpty + 2,
                         kBars = kDone + 1;
    static constexpr uint32_t kMisc = (kBar + kBars * 8 + 15) & ~15u;
    static constexpr uint32_t kSmem = kMisc + 32 + 1024;
    static_assert(kSmem <= 232448, "shared memory budget");
};

// One product of a launch.  a, b: the operands' maps; d: the outputs' maps (D; or h, gate, up; or gg, gp, h).
struct FfnProb {
    CUtensorMap a, b, d[3];
    int M, N, K, a_mn, b_mn;
    int up_row;                    // EPI_GLU: first row of the up projection in W_in (the second half of B's columns)
    int tiles_m, tiles_n, tile0;   // its tiles, and the first one's number in the launch
};
struct FfnParams {
    FfnProb p[kFMaxProb];
    int nprob, ntiles, save, gelu, wait_prior;
    const __nv_bfloat16 *gu;       // EPI_GLU_BWD: [M][2N]
    int *status;
    long long wait_cycles;
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void arrive_in_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// The forms for a pair: M = 256 across two CTAs, barriers in the first one.
template <int CG> __device__ __forceinline__ void pair_load(uint32_t dst, const CUtensorMap *map, int c0, int c1, uint32_t bar) {
    if constexpr (CG == 1) tma_load_2d(dst, map, c0, c1, bar);
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
            : "memory");
}
template <int CG> __device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
    if constexpr (CG == 1) mma_ss(d, a, b, id, acc);
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(id), "r"(acc));
}
// arrives on the barrier at this offset of every CTA of the group once the MMAs issued so far are done
template <int CG> __device__ __forceinline__ void pair_commit(uint32_t bar) {
    if constexpr (CG == 1) mma_commit(bar);
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
            "h"((uint16_t)3)
            : "memory");
}

// The tile of number t: problem, first row and column.  Blocks of 8 row tiles walk along the columns,
// so the tiles in flight at one time share their rows of A and columns of B in L2.
struct FfnWhere {
    int p, m0, n0;
};
template <int CG> __device__ __forceinline__ FfnWhere tile_at(const FfnParams &prm, int t, int width) {
    int p = 0;
    while (p + 1 < prm.nprob && t >= prm.p[p + 1].tile0) ++p;
    const FfnProb &q = prm.p[p];
    const int i = t - q.tile0, band = 8 * q.tiles_n, b = i / band, r = i % band;
    const int rows = min(8, q.tiles_m - 8 * b);
    return {p, (8 * b + r % rows) * 128 * CG, (r / rows) * width};
}

// act(g), act'(g)
__device__ __forceinline__ void activation(const float (&g)[4], int gelu, float (&act)[4], float (&der)[4]) {
    if (gelu) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float cdf = 0.5f * (1.f + erff(g[i] * 0.7071067811865476f));
            act[i] = g[i] * cdf;
            der[i] = fmaf(g[i] * 0.3989422804014327f, ex2a(-0.7213475204444817f * g[i] * g[i]), cdf);
        }
    } else {
        float sg[4];
        sigmoids<4>(g, sg);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            act[i] = g[i] * sg[i];
            der[i] = sg[i] * fmaf(g[i], 1.f - sg[i], 1.f);
        }
    }
}

__device__ __forceinline__ uint4 pack8(const float *v) {
    return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

template <int EPI, int CG>
__global__ void __launch_bounds__(kFfnThreads<EPI>, 1) k_ffn(const __grid_constant__ FfnParams prm) {
    using L = FfnTile<EPI, CG>;
    constexpr int S = L::kStages;
    constexpr int kTileN = EPI == EPI_GLU ? 128 : 256;   // output columns of a tile
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(sm);
    auto bar = [&](int i) { return sbase + L::kBar + 8u * i; };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + L::kMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + L::kMisc + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_rank() : 0;
    const int first = blockIdx.x / CG, step = gridDim.x / CG;
    const uint32_t MASK = 0xffffffffu;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (threadIdx.x == 0) {
        *abort_flag = 0;
        *reinterpret_cast<volatile long long *>(abort_flag + 1) = prm.wait_cycles;
        for (int i = 0; i < L::kBars; ++i) mbar_init(bar(i), (i == L::kAccEmpty || i == L::kAccEmpty + 1) ? (uint32_t)(kEpiWarps<EPI> * CG) : 1u);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        if constexpr (CG == 2) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot)));
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot)));
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        }
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2) cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        // ------------------------------------------------------------ TMA loads (each CTA its own half)
        if (lane == 0) {
            long long g = 0;
            bool ok = true;
            if (prm.wait_prior) {                     // the launch before wrote the operands
                asm volatile("griddepcontrol.wait;" ::: "memory");
                asm volatile("fence.proxy.async;" ::: "memory");
            }
            for (int t = first; t < prm.ntiles && ok; t += step) {
                const FfnWhere w = tile_at<CG>(prm, t, kTileN);
                const FfnProb &q = prm.p[w.p];
                const int m = w.m0 + 128 * rank, nk = (q.K + kFK - 1) / kFK;
                for (int kt = 0; kt < nk; ++kt, ++g) {
                    const int st = (int)(g % S);
                    if (g >= S && !(ok = mbar_wait(bar(L::kEmpty + st), (uint32_t)((g / S) - 1) & 1, 1u, abort_flag,
                                                   prm.status, 141)))
                        break;
                    // the stage is complete when both CTAs' bytes have landed
                    const uint32_t full = CG == 2 ? in_cta(bar(L::kFull + st), 0) : bar(L::kFull + st);
                    if (rank == 0) mbar_expect_tx(bar(L::kFull + st), CG * L::kStage);
                    const uint32_t sa = sbase + st * L::kStage, sb = sa + L::kA;
                    const int k0 = kt * kFK;
                    if (q.a_mn) {
                        pair_load<CG>(sa, &q.a, m, k0, full);
                        pair_load<CG>(sa + kFBox / 2, &q.a, m + 64, k0, full);
                    } else {
                        pair_load<CG>(sa, &q.a, k0, m, full);
                    }
#pragma unroll
                    for (int h = 0; h < 2 / CG; ++h) {
                        const int half = CG == 2 ? (int)rank : h;   // which 128 columns of the tile's 256
                        const uint32_t dst = sb + h * kFBox;
                        if (EPI == EPI_GLU) {
                            pair_load<CG>(dst, &q.b, k0, w.n0 + half * q.up_row, full);
                        } else if (q.b_mn) {
                            pair_load<CG>(dst, &q.b, w.n0 + 128 * half, k0, full);
                            pair_load<CG>(dst + kFBox / 2, &q.b, w.n0 + 128 * half + 64, k0, full);
                        } else {
                            pair_load<CG>(dst, &q.b, k0, w.n0 + 128 * half, full);
                        }
                    }
                }
            }
            if (*abort_flag && rank == 0)
                for (long long x = g - 1; x >= 0 && x >= g - S; --x)
                    mbar_drain(bar(L::kFull + (int)(x % S)), (uint32_t)(x / S) & 1, prm.wait_cycles);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMAs
        if (rank == 0) {
            long long g = 0;
            int tc = 0;
            bool ok = true;
            for (int t = first; t < prm.ntiles && ok; t += step, ++tc) {
                const FfnProb &q = prm.p[tile_at<CG>(prm, t, kTileN).p];
                const int nk = (q.K + kFK - 1) / kFK, acc = tc & 1;
                // M 128 CG, N 256
                const uint32_t id = (idesc(256, q.a_mn, q.b_mn) & ~(31u << 24)) | ((uint32_t)(128 * CG >> 4) << 24);
                // K-major: rows of 128 bytes, 16 k = 32 bytes on; MN-major: boxes of 64 x 64 (8 KB
                // apart), 16 k = 16 rows of 128 bytes on
                const uint32_t la = q.a_mn ? kFBox / 2 : 16, lb = q.b_mn ? kFBox / 2 : 16;
                const uint32_t ka = q.a_mn ? 2048 : 32, kb = q.b_mn ? 2048 : 32;
                if (tc >= 2 && !(ok = mbar_wait(bar(L::kAccEmpty + acc), ((tc >> 1) - 1) & 1, MASK, abort_flag, prm.status, 142)))
                    break;
                tc_fence_after();
                for (int kt = 0; kt < nk; ++kt, ++g) {
                    const int st = (int)(g % S);
                    if (!(ok = mbar_wait(bar(L::kFull + st), (uint32_t)(g / S) & 1, MASK, abort_flag, prm.status, 143))) break;
                    tc_fence_after();
                    const uint32_t sa = sbase + st * L::kStage;
                    const SDesc da = make_sdesc(sa, la, 1024), db = make_sdesc(sa + L::kA, lb, 1024);
                    // (one branch for the stage's four: each electing its own lane took 4 % longer over the block)
                    if (elect_one()) {
#pragma unroll
                        for (int ks = 0; ks < kFK / 16; ++ks)
                            pair_mma<CG>(tmem + 256u * acc, da.at(ks * ka), db.at(ks * kb), id, (kt | ks) != 0);
                        pair_commit<CG>(bar(L::kEmpty + st));
                        if (kt == nk - 1) pair_commit<CG>(bar(L::kAccFull + acc));
                    }
                    __syncwarp();
                }
                if (!ok) break;
            }
            if (elect_one()) pair_commit<CG>(bar(L::kDone));
            __syncwarp();
        }
        // both CTAs leave only after every MMA issued has completed
        if (lane == 0) mbar_drain(bar(L::kDone), 0, prm.wait_cycles);
        __syncwarp();
    } else {
        // ------------------------------------------------------------ epilogue
        const int qd = warp & 3;
        const uint32_t tl = tmem + ((uint32_t)(32 * qd) << 16);
        const uint32_t boxes = L::kOut + (uint32_t)(warp - 2) * L::kBoxes * kFOutBox;
        int tc = 0, used = 0;                     // tiles; boxes handed to a store so far
        // box number `used` of the warp's ring, free again
        auto box = [&]() { return boxes + (uint32_t)(used % L::kBoxes) * kFOutBox; };
        auto put = [&](uint32_t b, int c8, const float *v) {   // 8 columns (chunk c8) of this thread's row
            *reinterpret_cast<uint4 *>(sm + b + swz(lane, c8)) = pack8(v);
        };
        auto send = [&](const CUtensorMap *map, uint32_t b, int n, int m) {
            if (lane == 0) tma_store_2d(map, sbase + b, n, m);
        };
        for (int t = first; t < prm.ntiles; t += step, ++tc) {
            const FfnWhere w = tile_at<CG>(prm, t, kTileN);
            const FfnProb &q = prm.p[w.p];
            const int acc = tc & 1, m0 = w.m0 + 128 * rank + 32 * qd;
            if constexpr (EPI == EPI_GLU_BWD) {
                // this warp's 128 columns in four steps of 32; a step's g and p are loaded a step ahead,
                // the first one's before the product is done
                const int half = (warp - 2) >> 2, m = m0 + lane, c0 = 128 * half;
                const __nv_bfloat16 *row = prm.gu + (long long)m * 2 * q.N + w.n0 + c0;
                const uint32_t b = L::kOut + (uint32_t)(warp - 2) * 3 * kNarrowBox;
                uint4 ng[4], np[4];
                auto load = [&](int c) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        ng[i] = np[i] = make_uint4(0u, 0u, 0u, 0u);
                        if (m < q.M && w.n0 + c0 + c + 8 * i < q.N) {   // N is a multiple of 8
                            ng[i] = *reinterpret_cast<const uint4 *>(row + c + 8 * i);
                            np[i] = *reinterpret_cast<const uint4 *>(row + q.N + c + 8 * i);
                        }
                    }
                };
                load(0);
                if (!mbar_wait(bar(L::kAccFull + acc), (tc >> 1) & 1, MASK, abort_flag, prm.status, 144)) break;
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < 128; c += 32) {
                    float gh[32];
                    tmem_ld32(tl + 256u * acc + c0 + c, gh);
                    uint4 cg_[4], cp[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        cg_[i] = ng[i];
                        cp[i] = np[i];
                    }
                    if (c + 32 < 128) load(c + 32);
                    if (lane == 0) bulk_wait_read0();
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t ga[4] = {cg_[i].x, cg_[i].y, cg_[i].z, cg_[i].w}, pa[4] = {cp[i].x, cp[i].y, cp[i].z, cp[i].w};
                        float gg[8], gp[8], hh[8];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float g4[4] = {bf16lo(ga[2 * e]), bf16hi(ga[2 * e]), bf16lo(ga[2 * e + 1]), bf16hi(ga[2 * e + 1])};
                            const float p4[4] = {bf16lo(pa[2 * e]), bf16hi(pa[2 * e]), bf16lo(pa[2 * e + 1]), bf16hi(pa[2 * e + 1])};
                            float act[4], der[4];
                            activation(g4, prm.gelu, act, der);
#pragma unroll
                            for (int z = 0; z < 4; ++z) {
                                const float d = gh[8 * i + 4 * e + z];
                                gg[4 * e + z] = d * p4[z] * der[z];
                                gp[4 * e + z] = d * act[z];
                                hh[4 * e + z] = act[z] * p4[z];
                            }
                        }
                        // rows of 64 bytes under the 64-byte swizzle
                        const uint32_t at = b + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4);
                        *reinterpret_cast<uint4 *>(sm + at) = pack8(gg);
                        *reinterpret_cast<uint4 *>(sm + at + kNarrowBox) = pack8(gp);
                        *reinterpret_cast<uint4 *>(sm + at + 2 * kNarrowBox) = pack8(hh);
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (w.n0 + c0 + c < q.N)
#pragma unroll
                        for (int x = 0; x < 3; ++x) send(&q.d[x], b + x * kNarrowBox, w.n0 + c0 + c, m0);
                    if (lane == 0) bulk_commit();
                }
            } else {
            if (!mbar_wait(bar(L::kAccFull + acc), (tc >> 1) & 1, MASK, abort_flag, prm.status, 144)) break;
            tc_fence_after();
            const uint32_t ta = tl + 256u * acc;
#pragma unroll 1
            for (int c = 0; c < kTileN; c += 64) {
                // boxes of this round are free once all but the rounds' stores in flight have been read
                const bool live = w.n0 + c < q.N;
                if (EPI == EPI_PLAIN) {
                    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                    __syncwarp();
                    const uint32_t b = box();
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float v[32];
                        tmem_ld32(ta + c + 32 * x, v);
#pragma unroll
                        for (int i = 0; i < 4; ++i) put(b, 4 * x + i, v + 8 * i);
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (live) send(&q.d[0], b, w.n0 + c, m0);
                    if (lane == 0) bulk_commit();
                    ++used;
                } else {
                    if (lane == 0) bulk_wait_read0();
                    __syncwarp();
                    const uint32_t b = boxes;
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float vg[32], vu[32];
                        tmem_ld32x2(ta + c + 32 * x, ta + 128 + c + 32 * x, vg, vu);
                        if (prm.save) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                put(b + kFOutBox, 4 * x + i, vg + 8 * i);
                                put(b + 2 * kFOutBox, 4 * x + i, vu + 8 * i);
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float g4[4] = {vg[4 * i], vg[4 * i + 1], vg[4 * i + 2], vg[4 * i + 3]};
                            float act[4], der[4];
                            activation(g4, prm.gelu, act, der);
#pragma unroll
                            for (int e = 0; e < 4; ++e) vu[4 * i + e] *= act[e];
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) put(b, 4 * x + i, vu + 8 * i);
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (live) {
                        send(&q.d[0], b, w.n0 + c, m0);
                        if (prm.save) {
                            send(&q.d[1], b + kFOutBox, w.n0 + c, m0);
                            send(&q.d[2], b + 2 * kFOutBox, w.n0 + c, m0);
                        }
                    }
                    if (lane == 0) bulk_commit();
                }
            }
            }
            // the accumulator has been read: the MMA warp may fill it again
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (CG == 2) arrive_in_cluster(in_cta(bar(L::kAccEmpty + acc), 0));
                else mbar_arrive(bar(L::kAccEmpty + acc));
            }
        }
        if (lane == 0) bulk_wait0();
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    // the pair ends together: a CTA's barriers are signalled by the other one until then
    if constexpr (CG == 2) cluster_sync_all();
    if (warp == 1) {
        tc_fence_after();
        if constexpr (CG == 2) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
        else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}

// ------------------------------------------------------------------ few tokens

// With few tokens (decoding) the weights are all there is to read, and the tile above would leave its
// rows empty and most SMs without a tile.  So the roles are exchanged: 128 rows of the weights are M,
// the tokens N (16 to 256, more in groups of 256), D^T[128][tokens] = W u^T.  EPI_GLU: 64 rows of the
// gate and the 64 rows beside them of the up projection make the 128.  Where the tiles are fewer than
// the SMs, a cluster of `split` CTAs shares one: each takes a part of K, leaves its float32 sums in its
// shared memory, and each adds up (in the order of the ranks, so the result does not depend on timing)
// and finishes its share of the tokens from all of them.  The second product's weights do not depend
// on the first: it is launched with programmatic dependent launch and has its first stages of them on
// the way before it waits for h.
//
// Both forms measured at d_model 2048, d_ff 8192 (us, this one / the other): 3 tokens 26 / 99, 128: 40 /
// 99, 256: 59 / 88, 512: 69 / 101, 1024: 120 / 126; at 768, 2048: 800 tokens 27 / 36.  Past 1024 tokens the
// persistent tiles fill the SMs there and hide their epilogues.  The rule goes by tokens alone, not by tiles: with
// cold caches 256 / 512 / 1024 tokens take 42 / 54 / 52 us at 1024, 4096 (the other form 63 / 54 / 60), 70 / 79 / 126
// at 2048, 8192 (91 / 101 / 124) and 136 / 227 / 392 at 4096, 16384 (196 / 233 / 331: there it should change
// over at 512).  Three tokens read the weights at 4.2 and 2.7 TB/s: 128 CTAs in each launch leave 20 SMs without one.
//
// gu = [gg gp] W_in of the backward pass has the longest K (2 d_ff) and, with few tokens, next to no tiles: beside
// the other two products it alone set the time.  Up to 2048 tokens it is a launch of this kernel, W_in
// taken as it lies (MN-major).  The whole backward pass at d_model 2048, d_ff 8192 (us, so / all three side by
// side): 16 tokens 81 / 172, 256: 119 / 181, 512: 124 / 196, 1024: 211 / 254, 1500: 310 / 324, 2048: 382 / 391; at
// 4096, 16384 with cold caches 256: 259 / 413, 1024: 734 / 788, 2048: 1492 / 1607, at 1024, 4096 2048: 136 / 157.
// What is left of few tokens or small widths is gh in its large tiles: 333 tokens at 488, 1160 put it on 20 SMs, 31
// of the three launches' 59 us with cold caches.
constexpr int kFewMax = 1024, kFewGrad = 2048;
template <int N> struct FewTile {
    static constexpr uint32_t kW = 128 * 128, kU = N * 128, kStage = kW + kU;
    // two CTAs to an SM, or one of 256 tokens
    static constexpr int kRoom = N == 256 ? 4 * kStage : 110592, kStages = kRoom / kStage > 6 ? 6 : kRoom / kStage;
    static constexpr uint32_t kBar = kStages * kStage;          // the sums [N][128] lie over the stages
    static constexpr uint32_t kMisc = (kBar + (2 * kStages + 1) * 8 + 15) & ~15u;
    static constexpr uint32_t kSmem = kMisc + 32 + 1024;
    static_assert(N * 128 * 4 <= kBar, "");
    static_assert((N == 256 ? 1 : 2) * (kSmem + 1024) <= 233472, "");
};
struct FewParams {
    CUtensorMap w, u;
    int rows, K, T, up_row;        // rows of the output (d_ff or d_model); tokens
    int split, save, gelu, wait_prior;
    int w_mn;                      // the weights lie [K][rows] (EPI_PLAIN)
    __nv_bfloat16 *out, *gu;       // out [T][rows]; gu [T][2 rows]
    int *status;
    long long wait_cycles;
};

template <int EPI, int N>
__global__ void __launch_bounds__(kFThreads) k_ffn_few(const __grid_constant__ FewParams prm) {
    using L = FewTile<N>;
    constexpr int S = L::kStages, kTmemCols = N < 32 ? 32 : N;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(sm);
    auto bar = [&](int i) { return sbase + L::kBar + 8u * i; };   // full 0 .., empty S .., 2 S: all products done
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + L::kMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + L::kMisc + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = blockIdx.x % prm.split, tile = blockIdx.x / prm.split, tok0 = N * blockIdx.y, ntok = min(N, prm.T - tok0);
    const int nk = (prm.K + kFK - 1) / kFK, k0 = nk * rank / prm.split, k1 = nk * (rank + 1) / prm.split;
    constexpr int kRows = EPI == EPI_GLU ? 64 : 128;              // output rows of a tile
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) {
        *abort_flag = 0;
        *reinterpret_cast<volatile long long *>(abort_flag + 1) = prm.wait_cycles;
        for (int i = 0; i < 2 * S + 1; ++i) mbar_init(bar(i), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "n"(kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (warp == 0) {
        if (lane == 0) {
            auto weights = [&](int kt, int st) {
                const uint32_t at = sbase + st * L::kStage;
                mbar_expect_tx(bar(st), L::kStage);
                if (EPI == EPI_GLU) {
                    tma_load_2d(at, &prm.w, kt * kFK, kRows * tile, bar(st));
                    tma_load_2d(at + L::kW / 2, &prm.w, kt * kFK, prm.up_row + kRows * tile, bar(st));
                } else if (prm.w_mn) {
                    tma_load_2d(at, &prm.w, kRows * tile, kt * kFK, bar(st));
                    tma_load_2d(at + L::kW / 2, &prm.w, kRows * tile + 64, kt * kFK, bar(st));
                } else {
                    tma_load_2d(at, &prm.w, kt * kFK, kRows * tile, bar(st));
                }
            };
            auto tokens = [&](int kt, int st) { tma_load_2d(sbase + st * L::kStage + L::kW, &prm.u, kt * kFK, tok0, bar(st)); };
            const int head = min(S, k1 - k0);
            for (int i = 0; i < head; ++i) weights(k0 + i, i);
            if (prm.wait_prior) {
                asm volatile("griddepcontrol.wait;" ::: "memory");
                asm volatile("fence.proxy.async;" ::: "memory");
            }
            for (int i = 0; i < head; ++i) tokens(k0 + i, i);
            int i = head;
            for (; i < k1 - k0; ++i) {
                const int st = i % S;
                if (!mbar_wait(bar(S + st), (uint32_t)(i / S - 1) & 1, 1u, abort_flag, prm.status, 181)) break;
                weights(k0 + i, st);
                tokens(k0 + i, st);
            }
            if (*abort_flag)
                for (int x = i - 1; x >= 0 && x >= i - S; --x) mbar_drain(bar(x % S), (uint32_t)(x / S) & 1, prm.wait_cycles);
        }
        __syncwarp();
    } else if (warp == 1) {
        const bool mn = EPI == EPI_PLAIN && prm.w_mn;              // (the layouts are k_ffn's)
        const uint32_t id = idesc(N, mn, 0), lw = mn ? L::kW / 2 : 16, kw = mn ? 2048 : 32;
        for (int i = 0; i < k1 - k0; ++i) {
            const int st = i % S;
            if (!mbar_wait(bar(st), (uint32_t)(i / S) & 1, 0xffffffffu, abort_flag, prm.status, 182)) break;
            tc_fence_after();
            const uint32_t at = sbase + st * L::kStage;
            const SDesc dw = make_sdesc(at, lw, 1024), du = make_sdesc(at + L::kW, 16, 1024);
#pragma unroll
            for (int ks = 0; ks < kFK / 16; ++ks) mma_ss_w(tmem, dw.at(ks * kw), du.at(ks * 32), id, (i | ks) != 0);
            mma_commit_w(bar(S + st));
        }
        mma_commit_w(bar(2 * S));
        __syncwarp();
    }
    // every product of this CTA is done (and with them the reads of the stages)
    const bool done = mbar_wait(bar(2 * S), 0, 0xffffffffu, abort_flag, prm.status, 183);
    __syncthreads();
    if (warp >= 2 && done) {
        tc_fence_after();
        const int qd = warp & 3;
        float *sum = reinterpret_cast<float *>(sm) + 32 * qd + lane;
        const uint32_t tl = tmem + ((uint32_t)(32 * qd) << 16);
#pragma unroll
        for (int c = 0; c < N; c += 16) {
            float v[16];
            tmem_ld16(tl + c, v);
#pragma unroll
            for (int e = 0; e < 16; ++e) sum[(c + e) * 128] = k1 > k0 ? v[e] : 0.f;   // a part without a k step adds nothing
        }
        tc_fence_before();
    }
    if (prm.split > 1) cluster_sync_all();
    else __syncthreads();
    if (!*abort_flag) {
        // tokens rank, rank + split, ..: 16 or 32 threads to one, four rows of the weights each (the row
        // counts are multiples of 8)
        constexpr int kPer = kRows / 4, kGroups = kFThreads / kPer;
        const int f = 4 * (threadIdx.x % kPer), grp = threadIdx.x / kPer, row = kRows * tile + f, step = prm.split * kGroups;
        if (row < prm.rows) {
            // the parts' sums of column c and weight rows l ..: all on the way at once, added in order
            auto total = [&](int c, int l, float (&t)[4]) {
                if (prm.split == 1) {
                    const float4 v = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(sm) + c * 128 + l);
                    t[0] = v.x; t[1] = v.y; t[2] = v.z; t[3] = v.w;
                    return;
                }
                const uint32_t at = sbase + 4u * (c * 128 + l);
                float4 v[8];
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    v[r] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (r < prm.split)
                        asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                                     : "=f"(v[r].x), "=f"(v[r].y), "=f"(v[r].z), "=f"(v[r].w) : "r"(in_cta(at, r)));
                }
                t[0] = t[1] = t[2] = t[3] = 0.f;
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    t[0] += v[r].x; t[1] += v[r].y; t[2] += v[r].z; t[3] += v[r].w;
                }
            };
            auto store = [&](__nv_bfloat16 *to, const float (&t)[4]) {
                *reinterpret_cast<uint2 *>(to) = make_uint2(pack_bf16(t[0], t[1]), pack_bf16(t[2], t[3]));
            };
            for (int c = rank + prm.split * grp; c < ntok; c += step) {
                const long long t = tok0 + c;
                if (EPI == EPI_GLU) {
                    float g[4], p[4], act[4], der[4];
                    total(c, f, g);
                    total(c, 64 + f, p);
                    activation(g, prm.gelu, act, der);
                    if (prm.save) {
                        store(prm.gu + t * 2 * prm.rows + row, g);
                        store(prm.gu + t * 2 * prm.rows + prm.rows + row, p);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) p[e] *= act[e];
                    store(prm.out + t * prm.rows + row, p);
                } else {
                    float d[4];
                    total(c, f, d);
                    store(prm.out + t * prm.rows + row, d);
                }
            }
        }
    }
    tc_fence_before();
    // the others' sums are read until all are through
    if (prm.split > 1) cluster_sync_all();
    else __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols));
    }
}

// ------------------------------------------------------------------ host side

// [rows][cols] bf16, rows `ld` elements apart; box [box_rows][64 or 32], swizzled over its row of 128 or 64 bytes
bool map_of(CUtensorMap *m, const void *base, uint64_t rows, uint64_t cols, uint64_t ld, uint32_t box_rows, uint32_t box_cols = 64) {
    EncodeTiled enc = get_encode();
    if (!enc) return false;
    const cuuint64_t dims[2] = {cols, rows}, strides[1] = {ld * 2};
    const cuuint32_t box[2] = {box_cols, box_rows}, estr[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Operand maps: X [M or N][K] K-major, or its transpose [K][M or N] (mn)
bool operand(CUtensorMap *m, const void *x, int n, int k, bool mn) {
    return mn ? map_of(m, x, k, n, n, 64) : map_of(m, x, n, k, k, 128);
}

template <int EPI, int CG> cudaError_t run_ffn(FfnParams &prm, cudaStream_t st) {
    const int width = EPI == EPI_GLU ? 128 : 256;
    prm.ntiles = 0;
    for (int i = 0; i < prm.nprob; ++i) {
        FfnProb &q = prm.p[i];
        q.tiles_m = (q.M + 128 * CG - 1) / (128 * CG);
        q.tiles_n = (q.N + width - 1) / width;
        q.tile0 = prm.ntiles;
        const long long n = (long long)q.tiles_m * q.tiles_n + prm.ntiles;
        if (n > 0x7fffffff) return cudaErrorInvalidValue;
        prm.ntiles = (int)n;
    }
    auto *kernel = k_ffn<EPI, CG>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)FfnTile<EPI, CG>::kSmem);
    if (e != cudaSuccess) return e;
    int dev = 0, sms = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    const int groups = prm.ntiles < sms / CG ? prm.ntiles : sms / CG;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = CG;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(groups * CG);
    cfg.blockDim = dim3(kFfnThreads<EPI>);
    cfg.dynamicSmemBytes = FfnTile<EPI, CG>::kSmem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = prm.wait_prior ? 2 : 1;            // set up while the launch before ends
    return cudaLaunchKernelEx(&cfg, kernel, prm);
}

// CTA pairs once there are two row tiles to pair.
template <int EPI> cudaError_t run_ffn_any(FfnParams &prm, cudaStream_t st) {
    int m = 0;
    for (int i = 0; i < prm.nprob; ++i) m = prm.p[i].M > m ? prm.p[i].M : m;
    return m > 128 ? run_ffn<EPI, 2>(prm, st) : run_ffn<EPI, 1>(prm, st);
}

FfnProb product(int M, int N, int K, bool a_mn, bool b_mn) {
    FfnProb q;
    memset(&q, 0, sizeof q);
    q.M = M; q.N = N; q.K = K; q.a_mn = a_mn; q.b_mn = b_mn;
    return q;
}

template <int EPI, int N> cudaError_t run_few(FewParams &prm, cudaStream_t st) {
    using L = FewTile<N>;
    const int tiles = (prm.rows + (EPI == EPI_GLU ? 63 : 127)) / (EPI == EPI_GLU ? 64 : 128), nk = (prm.K + kFK - 1) / kFK,
              groups = (prm.T + N - 1) / N;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    // as many parts of K as leave each CTA four steps and the tiles one wave
    prm.split = 1;
    while (prm.split < 8 && 2 * prm.split * tiles * groups <= sms && nk / (2 * prm.split) >= 4) prm.split *= 2;
    auto *kernel = k_ffn_few<EPI, N>;
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::kSmem)) != cudaSuccess) return e;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = prm.split;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(tiles * prm.split, groups);
    cfg.blockDim = dim3(kFThreads);
    cfg.dynamicSmemBytes = L::kSmem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = prm.wait_prior ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, prm);
}

template <int EPI> cudaError_t run_few_any(FewParams &prm, const void *w, int w_rows, const void *u, cudaStream_t st) {
    const int n = prm.T <= 16 ? 16 : prm.T <= 32 ? 32 : prm.T <= 64 ? 64 : prm.T <= 128 ? 128 : 256;
    if (!(prm.w_mn ? map_of(&prm.w, w, prm.K, w_rows, w_rows, 64) : map_of(&prm.w, w, w_rows, prm.K, prm.K, EPI == EPI_GLU ? 64 : 128)) ||
        !map_of(&prm.u, u, prm.T, prm.K, prm.K, n))
        return cudaErrorInvalidValue;
    switch (n) {
        case 16: return run_few<EPI, 16>(prm, st);
        case 32: return run_few<EPI, 32>(prm, st);
        case 64: return run_few<EPI, 64>(prm, st);
        case 128: return run_few<EPI, 128>(prm, st);
        default: return run_few<EPI, 256>(prm, st);
    }
}

cudaError_t launch_ffn_few(const FfnArgs &a, cudaStream_t st) {
    FewParams prm;
    memset(&prm, 0, sizeof prm);
    prm.rows = a.F; prm.K = a.D; prm.T = a.T; prm.up_row = a.F; prm.gelu = a.gelu; prm.save = a.gu != nullptr;
    prm.out = static_cast<__nv_bfloat16 *>(a.h); prm.gu = static_cast<__nv_bfloat16 *>(a.gu);
    prm.status = a.status; prm.wait_cycles = a.wait_cycles;
    cudaError_t e = run_few_any<EPI_GLU>(prm, a.W_in, 2 * a.F, a.u, st);
    if (e != cudaSuccess) return e;
    prm.rows = a.D; prm.K = a.F; prm.save = 0; prm.wait_prior = 1;
    prm.out = static_cast<__nv_bfloat16 *>(a.out);
    return run_few_any<EPI_PLAIN>(prm, a.W_out, a.D, a.h, st);
}

}  // namespace

bool ffn_supported() { return get_encode() != nullptr; }

cudaError_t launch_ffn(const FfnArgs &a, cudaStream_t st) {
    if (a.T <= kFewMax) return launch_ffn_few(a, st);
    FfnParams prm;
    memset(&prm, 0, sizeof prm);
    prm.nprob = 1; prm.gelu = a.gelu; prm.status = a.status; prm.wait_cycles = a.wait_cycles;
    prm.save = a.gu != nullptr;
    FfnProb &q = prm.p[0];
    q = product(a.T, a.F, a.D, false, false);
    q.up_row = a.F;
    bool ok = operand(&q.a, a.u, a.T, a.D, false) && operand(&q.b, a.W_in, 2 * a.F, a.D, false) &&
              map_of(&q.d[0], a.h, a.T, a.F, a.F, 32);
    if (a.gu)
        ok = ok && map_of(&q.d[1], a.gu, a.T, a.F, 2ull * a.F, 32) &&
             map_of(&q.d[2], static_cast<__nv_bfloat16 *>(a.gu) + a.F, a.T, a.F, 2ull * a.F, 32);
    if (!ok) return cudaErrorInvalidValue;
    static_assert(kFewMax >= 128, "more tokens than a single CTA's rows: pairs");
    cudaError_t e = run_ffn<EPI_GLU, 2>(prm, st);
    if (e != cudaSuccess) return e;
    prm.wait_prior = 1;
    q = product(a.T, a.D, a.F, false, false);
    if (!operand(&q.a, a.h, a.T, a.F, false) || !operand(&q.b, a.W_out, a.D, a.F, false) || !map_of(&q.d[0], a.out, a.T, a.D, a.D, 32))
        return cudaErrorInvalidValue;
    return run_ffn<EPI_PLAIN, 2>(prm, st);
}

cudaError_t launch_ffn_bwd(const FfnArgs &a, cudaStream_t st) {
    FfnParams prm;
    memset(&prm, 0, sizeof prm);
    prm.nprob = 1; prm.gelu = a.gelu; prm.status = a.status; prm.wait_cycles = a.wait_cycles;
    prm.gu = static_cast<const __nv_bfloat16 *>(a.gu);
    FfnProb &q = prm.p[0];
    // gh = gy Wd, then the activation's gradient
    q = product(a.T, a.F, a.D, false, true);
    __nv_bfloat16 *ggu = static_cast<__nv_bfloat16 *>(a.ggu);
    if (!operand(&q.a, a.gy, a.T, a.D, false) || !operand(&q.b, a.W_out, a.F, a.D, true) ||
        !map_of(&q.d[0], ggu, a.T, a.F, 2ull * a.F, 32, 32) || !map_of(&q.d[1], ggu + a.F, a.T, a.F, 2ull * a.F, 32, 32) ||
        !map_of(&q.d[2], a.h, a.T, a.F, a.F, 32, 32))
        return cudaErrorInvalidValue;
    cudaError_t e = run_ffn_any<EPI_GLU_BWD>(prm, st);
    if (e != cudaSuccess) return e;
    prm.wait_prior = 1;
    prm.nprob = 0;
    if (a.T <= kFewGrad) {
        // gu has few tiles and the longest K: the form for few tokens splits it over the SMs
        FewParams few;
        memset(&few, 0, sizeof few);
        few.rows = a.D; few.K = 2 * a.F; few.T = a.T; few.w_mn = 1; few.wait_prior = 1;
        few.out = static_cast<__nv_bfloat16 *>(a.gu_);
        few.status = a.status; few.wait_cycles = a.wait_cycles;
        if ((e = run_few_any<EPI_PLAIN>(few, a.W_in, a.D, ggu, st)) != cudaSuccess) return e;
    } else {
        // the longest products first: their tiles end last otherwise
        FfnProb &g = prm.p[prm.nprob++];
        g = product(a.T, a.D, 2 * a.F, false, true);
        if (!operand(&g.a, ggu, a.T, 2 * a.F, false) || !operand(&g.b, a.W_in, a.D, 2 * a.F, true) ||
            !map_of(&g.d[0], a.gu_, a.T, a.D, a.D, 32))
            return cudaErrorInvalidValue;
    }
    FfnProb &in = prm.p[prm.nprob++], &out = prm.p[prm.nprob++];
    in = product(2 * a.F, a.D, a.T, true, true);
    out = product(a.D, a.F, a.T, true, true);
    if (!operand(&in.a, ggu, 2 * a.F, a.T, true) || !operand(&in.b, a.u, a.D, a.T, true) ||
        !map_of(&in.d[0], a.gW_in, 2 * a.F, a.D, a.D, 32) ||
        !operand(&out.a, a.gy, a.D, a.T, true) || !operand(&out.b, a.h, a.F, a.T, true) ||
        !map_of(&out.d[0], a.gW_out, a.D, a.F, a.F, 32))
        return cudaErrorInvalidValue;
    return run_ffn_any<EPI_PLAIN>(prm, st);
}

}  // namespace ssd
