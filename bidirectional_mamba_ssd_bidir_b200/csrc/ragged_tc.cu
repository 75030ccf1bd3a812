// ragged_tc.cu -- the scan over packed ragged sequences on the tensor core: bf16, headdim 64,
// d_state 128, an even number of heads in a B/C group.
//
// A CTA walks one segment (ragged.cu) of one sequence for two heads of a group, in chunks of 128
// tokens.  In the chunk's scan order, with cs_i the inclusive sum of dt A and c = cs of the last token:
//
//   scores    = C B^T                                              both heads share them
//   P_ij      = scores_ij exp(cs_i - cs_j) dt_j,  j not after i     (one ex2 per element: cs_j and
//               dt_j are one number csd_j = cs_j - log2 dt_j, so the exponent never needs a rescue,
//               however steep the decay is)
//   y_i       = (P X)_i + exp(cs_i) C_i S^T + D x_i
//   S        <- exp(c) S + sum_j (w_j x_j) (outer) B_j,             w_j = dt_j exp(c - cs_j)
//
// Precision.  P and the copy of S that multiplies C are rounded to bf16 (operands of products whose
// result is a bf16 y).  S itself is a float32 output, so w x enters its product in two bf16 terms,
// high and rest: 2^-17 of w x instead of 2^-9.  S stays in registers in float32.
//
// Products (M = 128 each, float32 in TMEM), issued by warp 17 (one elected lane):
//   scores [0,128)     A = C, B = B tile, both K-major in smem
//   P X    [256,384)   A = P of a head (bf16, TMEM [0,64) and [64,128), written over the scores),
//                      B = X of the head (MN-major), N = 64 per head
//   C S^T  [384,512)   A = C, B = bf16 S of both heads (MN-major: row n, 128 columns (head, p))
//   new S  [128,256)   A = B^T (MN-major, M = n), B = w x high, then rest (MN-major), N = 128
//
// Warps: 0-15 the passes over tiles (TMEM lane quarter w & 3, column group w >> 2: head w >> 3, half
// of P), 16 the TMA loads, 17 the MMAs, 18 the y stores.  Per chunk j the passes are: P_j; the state
// (S <- ... and its bf16 copy for chunk j + 1); w x and the decay tables of chunk j + 1; y_j.  The
// products of j + 1 that need no state run while y_j is finished.
//
// Rows past the segment's end (another sequence's, or none) are zeroed in x and B before a product
// sees them, so nothing of theirs, NaN included, enters; their y rows are not written.
//
// STATES: the first of two launches when there are several segments: only w x and S, the state each
// segment adds and its decay.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cstring>

#include "ragged.cuh"
#include "ssd_tc_common.cuh"

namespace ssd {
namespace {

constexpr int kQ = 128;                                // tokens of a chunk
constexpr uint32_t kBox = 128 * 128;                   // 128 rows of 64 bf16: 16 KB
constexpr int kPassWarps = 16, kTcThreads = 32 * (kPassWarps + 3);
// shared memory: everything but the tables in 16 KB boxes; 227 KB in all
constexpr uint32_t kSX = 0;                            // x: two stages of two heads; becomes y
constexpr uint32_t kSW = 4 * kBox;                     // w x: high of two heads, rest of two heads
constexpr uint32_t kSB = 8 * kBox, kSC = 10 * kBox;    // B, C: two 64-column boxes each
constexpr uint32_t kSS = 12 * kBox;                    // bf16 S: rows n, a box per head
constexpr uint32_t kTab = 14 * kBox;                   // cs, csd: [2][128] float each
constexpr uint32_t kBars = kTab + 4 * kQ * 4;
enum TcBar {
    XF0 = 0, XF1, XE0, XE1, BF, BE, CF, CE,            // loads: full / empty
    PREP,                                              // chunk's w x and tables written
    SC, ST, YI, YF,                                    // products done: scores, new S, C S^T, P X
    RD0, RD1, RD2, RD3,                                // a lane quarter's scores are in registers
    PR, SB, YE,                                        // P written; bf16 S written; Y read
    SG0, SG1,                                          // y staged
    DONE,
    kNumBars
};
constexpr uint32_t kMisc = (kBars + kNumBars * 8 + 15) & ~15u;
constexpr uint32_t kTcSmem = kMisc + 32;
static_assert(kTcSmem <= 232448, "shared memory budget");
constexpr uint32_t kColS = 128, kColY = 256, kColYI = 384;   // TMEM columns (scores / P at 0)

struct TcMaps {
    CUtensorMap x, b, c, y;
};

template <bool STATES>
__global__ void __launch_bounds__(kTcThreads, 1) k_ragged_tc(const __grid_constant__ TcMaps maps,
                                                             const __grid_constant__ RaggedArgs a) {
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sbase = smem_u32(sm);
    auto bar = [&](int i) { return sbase + kBars + 8u * i; };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + kMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + kMisc + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t MASK = 0xffffffffu;
    const int pairs = a.H / 2, u = blockIdx.x / pairs, h0 = 2 * (blockIdx.x % pairs), grp = h0 / (a.H / a.G);
    const Segment sg = find_segment(a.seq, a.seg, u);
    if (blockIdx.x == 0 && !STATES) check_offsets(a.seq, a.status);
    if (sg.s < 0) return;                              // the same for the whole CTA, before any allocation
    const bool last = sg.k == sg.count - 1;
    if (STATES && last) return;
    if (sbase & 1023) {                                // the swizzled boxes need it (never seen)
        if (threadIdx.x == 0) atomicExch(a.status, 150);
        return;
    }
    const int t0 = sg.k * a.seg, len = min(a.seg, sg.len - t0), nc = (len + kQ - 1) / kQ;
    // row of packed token that is row 0 of chunk j's tiles; rows [v0(j), v1(j)) are the segment's
    auto base = [&](int j) { return a.dir > 0 ? sg.lo + t0 + j * kQ : sg.lo + sg.len - t0 - (j + 1) * kQ; };
    auto rows = [&](int j) { return min(kQ, len - j * kQ); };

    if (threadIdx.x == 0) {
        *abort_flag = 0;
        *reinterpret_cast<volatile long long *>(abort_flag + 1) = a.wait_cycles;
        for (int i = 0; i < kNumBars; ++i) {
            const bool w16 = i == PREP || i == PR || i == SB || i == YE || i == SG0 || i == SG1 || (STATES && (i == XE0 || i == XE1));
            mbar_init(bar(i), w16 ? kPassWarps : (i >= RD0 && i <= RD3) ? 4 : 1);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 17) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    auto wait = [&](int b, int phase, int code) { return mbar_wait(bar(b), (uint32_t)phase & 1, MASK, abort_flag, a.status, code); };

    if (warp == 16) {
        // ------------------------------------------------------------ loads
        if (lane == 0) {
            auto wait1 = [&](int b, int phase, int code) { return mbar_wait(bar(b), (uint32_t)phase & 1, 1u, abort_flag, a.status, code); };
            int nx = 0, nb = 0, ncc = 0;               // chunks asked for
            for (int j = 0; j < nc; ++j) {
                const int r = base(j), st = j & 1;
                if (j >= 2 && !wait1(XE0 + st, (j >> 1) - 1, 151)) break;
                mbar_expect_tx(bar(XF0 + st), 2 * kBox);
                for (int h = 0; h < 2; ++h) tma_load_2d(sbase + kSX + (2 * st + h) * kBox, &maps.x, 64 * (h0 + h), r, bar(XF0 + st));
                nx = j + 1;
                if (j >= 1 && !wait1(BE, j - 1, 152)) break;
                mbar_expect_tx(bar(BF), 2 * kBox);
                for (int h = 0; h < 2; ++h) tma_load_2d(sbase + kSB + h * kBox, &maps.b, 128 * grp + 64 * h, r, bar(BF));
                nb = j + 1;
                if (STATES) continue;
                if (j >= 1 && !wait1(CE, j - 1, 153)) break;
                mbar_expect_tx(bar(CF), 2 * kBox);
                for (int h = 0; h < 2; ++h) tma_load_2d(sbase + kSC + h * kBox, &maps.c, 128 * grp + 64 * h, r, bar(CF));
                ncc = j + 1;
            }
            if (*abort_flag) {                         // copies in flight land before the memory is given up
                for (int j = nx - 1; j >= 0 && j >= nx - 2; --j) mbar_drain(bar(XF0 + (j & 1)), (uint32_t)(j >> 1) & 1, a.wait_cycles);
                if (nb) mbar_drain(bar(BF), (uint32_t)(nb - 1) & 1, a.wait_cycles);
                if (ncc) mbar_drain(bar(CF), (uint32_t)(ncc - 1) & 1, a.wait_cycles);
            }
        }
        __syncwarp();
    } else if (warp == 17) {
        // ------------------------------------------------------------ products
        const uint32_t id_sc = idesc(128, 0, 0), id_px = idesc(64, 0, 1), id_yi = idesc(128, 0, 1), id_st = idesc(128, 1, 1);
        const SDesc dC = make_sdesc(sbase + kSC, 16, 1024), dBk = make_sdesc(sbase + kSB, 16, 1024);
        const SDesc dBm = make_sdesc(sbase + kSB, kBox, 1024), dW = make_sdesc(sbase + kSW, kBox, 1024),
                    dS = make_sdesc(sbase + kSS, kBox, 1024);
        for (int j = 0; j < nc; ++j) {
            if (!wait(PREP, j, 154) || !wait(BF, j, 155) || !wait(XF0 + (j & 1), j >> 1, 156)) break;
            if (!STATES) {
                if (!wait(CF, j, 157)) break;
                tc_fence_after();
                // K = n: 64 of them to a box, 16 to a step of 32 bytes
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {
                    const uint32_t off = (ks >> 2) * kBox + (ks & 3) * 32;
                    mma_ss_w(tmem, dC.at(off), dBk.at(off), id_sc, ks > 0);
                }
                mma_commit_w(bar(SC));
            }
            tc_fence_after();
            // K = tokens: 16 rows of 128 bytes to a step
#pragma unroll
            for (int ks = 0; ks < 16; ++ks)
                mma_ss_w(tmem + kColS, dBm.at((ks & 7) * 2048), dW.at((ks >> 3) * 2 * kBox + (ks & 7) * 2048), id_st, ks > 0);
            mma_commit_w(bar(ST));
            mma_commit_w(bar(BE));
            if (STATES) continue;
            if (!wait(SB, j, 158) || (j >= 1 && !wait(YE, j - 1, 159))) break;
            tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
                mma_ss_w(tmem + kColYI, dC.at((ks >> 2) * kBox + (ks & 3) * 32), dS.at(ks * 2048), id_yi, ks > 0);
            mma_commit_w(bar(YI));
            mma_commit_w(bar(CE));
            if (!wait(PR, j, 160)) break;
            tc_fence_after();
            const SDesc dX = make_sdesc(sbase + kSX + (j & 1) * 2 * kBox, kBox, 1024);
#pragma unroll
            for (int ks = 0; ks < 16; ++ks)
                mma_ts_w(tmem + kColY + 64 * (ks >> 3), tmem + 64 * (ks >> 3) + 8 * (ks & 7), dX.at((ks >> 3) * kBox + (ks & 7) * 2048),
                         id_px, (ks & 7) > 0);
            mma_commit_w(bar(YF));
        }
        mma_commit_w(bar(DONE));
        if (lane == 0) mbar_drain(bar(DONE), 0, a.wait_cycles);
        __syncwarp();
    } else if (warp == 18) {
        // ------------------------------------------------------------ y stores (whole chunks; a partial one is stored by the passes)
        if (!STATES && lane == 0) {
            for (int j = 0; j < nc; ++j) {
                const int st = j & 1;
                if (!mbar_wait(bar(SG0 + st), (uint32_t)(j >> 1) & 1, 1u, abort_flag, a.status, 161)) break;
                if (rows(j) == kQ) {
                    for (int h = 0; h < 2; ++h) tma_store_2d(&maps.y, sbase + kSX + (2 * st + h) * kBox, 64 * (h0 + h), base(j));
                    bulk_commit();
                    bulk_wait_read0();
                }
                mbar_arrive(bar(XE0 + st));
            }
            bulk_wait0();
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ passes
        const int q = warp & 3, cg = warp >> 2, hh = cg >> 1, half = cg & 1, h = h0 + hh;
        const int row = 32 * q + lane;                 // token row of a tile, or n of the state
        const uint32_t tl = tmem + ((uint32_t)(32 * q) << 16);
        float *cs_tab = reinterpret_cast<float *>(sm + kTab), *csd_tab = cs_tab + 2 * kQ;
        const float a2 = a.A[h] * 1.4426950408889634f, Dh = a.D ? a.D[h] : 0.f, bias = a.dt_bias ? a.dt_bias[h] : 0.f;
        const __nv_bfloat16 *dtp = static_cast<const __nv_bfloat16 *>(a.dt) + h;
        const size_t PN = 64 * 128;
        float S[32];                                   // S[h][32 half + i][row]
        // ---- start state
        {
            const size_t at = (size_t)h * PN + (size_t)(32 * half) * 128 + row;
            const float *in = nullptr;
            if (sg.k == 0) {
                if (STATES || last) {
                    const int si = slot_of_start(a.slots, sg.s, a.status);
                    if (si >= 0) in = static_cast<const float *>(a.slots.pool_in) + (size_t)si * a.H * PN;
                } else {
                    in = a.ws_state + (size_t)(u + sg.count - 1) * a.H * PN;
                }
            } else if (!STATES) {
                in = a.ws_state + (size_t)(u - sg.k) * a.H * PN;
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) S[i] = in ? in[at + i * 128] : 0.f;
            if (STATES && sg.k == 0) {
                // the sequence's start, kept where its last segment's own state would be (nothing reads that)
                float *keep = a.ws_state + (size_t)(u + sg.count - 1) * a.H * PN;
#pragma unroll
                for (int i = 0; i < 32; ++i) keep[at + i * 128] = S[i];
            }
            if (!STATES)
                for (int k = 1; k < sg.k; ++k) {
                    const size_t v = (size_t)(u - sg.k + k) * a.H;
                    const float d = ex2_ftz(a.ws_decay[v + h]);
                    const float *add = a.ws_state + v * PN + at;
#pragma unroll
                    for (int i = 0; i < 32; ++i) S[i] = fmaf(S[i], d, add[i * 128]);
                }
        }
        auto copy_state = [&]() {                      // bf16 S: row n, 32 columns of the head's box
            uint8_t *box = sm + kSS + hh * kBox;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<uint4 *>(box + swz(row, 4 * half + i)) =
                    make_uint4(pack_bf16(S[8 * i], S[8 * i + 1]), pack_bf16(S[8 * i + 2], S[8 * i + 3]),
                               pack_bf16(S[8 * i + 4], S[8 * i + 5]), pack_bf16(S[8 * i + 6], S[8 * i + 7]));
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(SB));
        };
        float dtr[4], kappa = 1.f, total = 0.f;        // dt of rows 4 lane ..; decay of the present chunk; of the segment (log2)
        auto load_dt = [&](int j) {
            const int b = base(j), n = rows(j);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = 4 * lane + e;
                const bool in = a.dir > 0 ? r < n : r >= kQ - n;
                dtr[e] = in ? __bfloat162float(dtp[(long long)(b + r) * a.lddt]) : -INFINITY;   // -inf: no token
            }
        };
        // tables and w x of chunk j, from dtr
        float next_kappa = 1.f;
        auto prepare = [&](int j) -> bool {
            const int st = j & 1, n = rows(j);
            float d[4], s[4], up[4], dn[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                d[e] = dtr[e] == -INFINITY ? 0.f : (a.dt_bias ? softplus(dtr[e] + bias) : dtr[e]);
                s[e] = d[e] * a2;
            }
            // inclusive sums from the first row on and from the last row back
            up[0] = s[0]; up[1] = up[0] + s[1]; up[2] = up[1] + s[2]; up[3] = up[2] + s[3];
            dn[3] = s[3]; dn[2] = dn[3] + s[2]; dn[1] = dn[2] + s[1]; dn[0] = dn[1] + s[0];
            float iu = up[3], id = dn[0];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float x = __shfl_up_sync(MASK, iu, o), y = __shfl_down_sync(MASK, id, o);
                if (lane >= o) iu += x;
                if (lane + o < 32) id += y;
            }
            const float tot = __shfl_sync(MASK, iu, 31);
            float eu = __shfl_up_sync(MASK, iu, 1), ed = __shfl_down_sync(MASK, id, 1);
            if (lane == 0) eu = 0.f;
            if (lane == 31) ed = 0.f;
            float cs[4], wv[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float tail = a.dir > 0 ? ed + (e < 3 ? dn[e < 3 ? e + 1 : 3] : 0.f) : eu + (e > 0 ? up[e > 0 ? e - 1 : 0] : 0.f);
                cs[e] = a.dir > 0 ? eu + up[e] : ed + dn[e];
                wv[e] = d[e] * ex2_ftz(tail);
            }
            next_kappa = ex2_ftz(tot);
            total += tot;
            if (!STATES && q == 0 && half == 0) {
                // the tables of the chunk before are read by the P pass: wait until all of it is over
                if (j >= 1 && !wait(PR, j - 1, 162)) return false;
                reinterpret_cast<float4 *>(cs_tab + hh * kQ)[lane] = make_float4(cs[0], cs[1], cs[2], cs[3]);
                reinterpret_cast<float4 *>(csd_tab + hh * kQ)[lane] =
                    make_float4(cs[0] - __log2f(d[0]), cs[1] - __log2f(d[1]), cs[2] - __log2f(d[2]), cs[3] - __log2f(d[3]));
            }
            // w of this thread's row: element lane & 3 of lane 8 q + lane / 4
            float wr = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float t = __shfl_sync(MASK, wv[e], 8 * q + (lane >> 2));
                if ((lane & 3) == e) wr = t;
            }
            if (!wait(XF0 + st, j >> 1, 163)) return false;
            const bool mine = a.dir > 0 ? row < n : row >= kQ - n;
            if (n < kQ) {                              // rows of no token: zero in x and B
                if (!wait(BF, j, 164)) return false;
                if (!mine)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        *reinterpret_cast<uint4 *>(sm + kSX + (2 * st + hh) * kBox + swz(row, 4 * half + i)) = make_uint4(0u, 0u, 0u, 0u);
                        *reinterpret_cast<uint4 *>(sm + kSB + hh * kBox + swz(row, 4 * half + i)) = make_uint4(0u, 0u, 0u, 0u);
                    }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t off = swz(row, 4 * half + i);
                const uint4 v = *reinterpret_cast<const uint4 *>(sm + kSX + (2 * st + hh) * kBox + off);
                const uint32_t in[4] = {v.x, v.y, v.z, v.w};
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = mul2(unpack2(in[e]), make_float2(wr, wr));
                    hi[e] = pack_bf16(f.x, f.y);
                    lo[e] = pack_bf16(f.x - bf16lo(hi[e]), f.y - bf16hi(hi[e]));
                }
                *reinterpret_cast<uint4 *>(sm + kSW + hh * kBox + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4 *>(sm + kSW + (2 + hh) * kBox + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(PREP));
                if (STATES) mbar_arrive(bar(XE0 + st));
            }
            return true;
        };

        bool ok = true;
        if (nc > 0) {
            load_dt(0);
            if (!STATES) copy_state();
            ok = prepare(0);
        }
        for (int j = 0; j < nc && ok; ++j) {
            const int st = j & 1;
            kappa = next_kappa;
            if (j + 1 < nc) load_dt(j + 1);
            float ecs = 0.f;
            if (!STATES) {
                // ---- P_j: this thread's row, columns [32 cg, 32 cg + 32)
                if (!(ok = wait(PREP, j, 165) && wait(SC, j, 166))) break;
                tc_fence_after();
                const bool diag = cg == q, live = a.dir > 0 ? cg <= q : cg >= q;
                float v[32];
                if (live) tmem_ld32(tl + 32 * cg, v);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(RD0 + q));
                // P goes over the scores once the quarter's four warps have them in registers
                if (!(ok = wait(RD0 + q, j, 167))) break;
                tc_fence_after();
                ecs = ex2_ftz(cs_tab[hh * kQ + row]);
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    uint32_t p[16];
                    const float c = cs_tab[z * kQ + row];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 e = *reinterpret_cast<const float4 *>(csd_tab + z * kQ + 32 * cg + 4 * i);
                        const float m0 = v[4 * i] * ex2_ftz(c - e.x), m1 = v[4 * i + 1] * ex2_ftz(c - e.y),
                                    m2 = v[4 * i + 2] * ex2_ftz(c - e.z), m3 = v[4 * i + 3] * ex2_ftz(c - e.w);
                        p[2 * i] = live ? pack_bf16(m0, m1) : 0u;
                        p[2 * i + 1] = live ? pack_bf16(m2, m3) : 0u;
                    }
                    if (diag)
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            // columns 2 i and 2 i + 1 of the quarter against row `lane` of it
                            const bool k0 = a.dir > 0 ? 2 * i <= lane : 2 * i >= lane, k1 = a.dir > 0 ? 2 * i + 1 <= lane : 2 * i + 1 >= lane;
                            p[i] &= (k0 ? 0x0000ffffu : 0u) | (k1 ? 0xffff0000u : 0u);
                        }
                    tmem_st16_nw(tl + 64 * z + 16 * cg, p);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(PR));
            }
            // ---- the state
            if (!(ok = wait(ST, j, 168))) break;
            tc_fence_after();
            {
                float ds[32];
                tmem_ld32(tl + kColS + 32 * cg, ds);
#pragma unroll
                for (int i = 0; i < 32; ++i) S[i] = fmaf(S[i], kappa, ds[i]);
            }
            if (!STATES && j + 1 < nc) {
                if (!(ok = wait(YI, j, 169))) break;   // C S^T has read the copy it is written over
                copy_state();
            }
            // ---- the next chunk's w x and tables
            tc_fence_before();
            if (j + 1 < nc && !(ok = prepare(j + 1))) break;
            if (!STATES) {
                // ---- y_j, in place over x_j
                if (!(ok = wait(YI, j, 170) && wait(YF, j, 171))) break;
                tc_fence_after();
                uint8_t *box = sm + kSX + (2 * st + hh) * kBox;
#pragma unroll
                for (int z = 0; z < 2; ++z) {          // 16 columns at a time: more do not fit beside S
                    float yp[16], yi[16];
                    tmem_ld16(tl + kColY + 32 * cg + 16 * z, yp);
                    tmem_ld16(tl + kColYI + 32 * cg + 16 * z, yi);
                    if (z == 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(YE));
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint4 *at = reinterpret_cast<uint4 *>(box + swz(row, 4 * half + 2 * z + i));
                        const uint4 x = *at;
                        const uint32_t in[4] = {x.x, x.y, x.z, x.w};
                        uint32_t o[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int c = 8 * i + 2 * e;
                            o[e] = pack_bf16(fmaf(Dh, bf16lo(in[e]), fmaf(ecs, yi[c], yp[c])),
                                             fmaf(Dh, bf16hi(in[e]), fmaf(ecs, yi[c + 1], yp[c + 1])));
                        }
                        *at = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                }
                const int n = rows(j);
                if (n == kQ) {
                    fence_async_smem();
                } else {
                    // the warp's 32 rows x 64 bytes, four lanes to a row, rows of the segment only
                    __syncwarp();
                    __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(a.y) + (long long)h * 64 + 32 * half;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = 32 * q + 8 * i + (lane >> 2), c = lane & 3;
                        if (a.dir > 0 ? r < n : r >= kQ - n)
                            *reinterpret_cast<uint4 *>(y + (long long)(base(j) + r) * a.ldy + 8 * c) =
                                *reinterpret_cast<const uint4 *>(box + swz(r, 4 * half + c));
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(SG0 + st));
            }
        }
        // ---- end state
        if (ok) {
            float *out = nullptr;
            if (STATES) {
                out = a.ws_state + (size_t)u * a.H * PN;
                if (q == 0 && half == 0 && lane == 0) a.ws_decay[(size_t)u * a.H + h] = total;
            } else if (last && a.slots.pool_out) {
                // (slot_of_end meets at a CTA barrier: its look for a second writer is done warp by warp here)
                const int v = a.slots.out ? a.slots.out[sg.s] : sg.s;
                bool good = v >= 0 && v < a.slots.n_out;
                if (v >= a.slots.n_out) report(a.status, kCodeSlotRange);
                if (good && a.slots.out) {
                    bool twice = false;
                    for (int i = lane; i < a.seq.nseq; i += 32) twice |= i != sg.s && a.slots.out[i] == v;
                    if (__any_sync(MASK, twice)) {
                        report(a.status, kCodeSlotTwice);
                        good = false;
                    }
                }
                if (good) out = static_cast<float *>(a.slots.pool_out) + (size_t)v * a.H * PN;
            }
            if (out) {
                out += (size_t)h * PN + (size_t)(32 * half) * 128 + row;
#pragma unroll
                for (int i = 0; i < 32; ++i) out[i * 128] = S[i];
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 17) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}

bool map_rows(CUtensorMap *m, const void *base, uint64_t rows, uint64_t cols, uint64_t ld) {
    EncodeTiled enc = get_encode();
    if (!enc) return false;
    const cuuint64_t dims[2] = {cols, rows}, strides[1] = {ld * 2};
    const cuuint32_t box[2] = {64, 128}, estr[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// Head shapes and layouts of the tensor-core form: what a tensor map takes (16-byte aligned rows).
bool ragged_tc_supported(const RaggedArgs &a, bool bf16) {
    auto ok = [](const void *p, long long ld) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 8 == 0; };
    return bf16 && a.P == 64 && a.N == 128 && (a.H / a.G) % 2 == 0 && a.seq.tokens > 0 && ok(a.x, a.ldx) && ok(a.B, a.ldB) &&
           ok(a.C, a.ldC) && ok(a.y, a.ldy) && (long long)a.units * (a.H / 2) <= 0x7fffffffLL && get_encode() != nullptr;
}

cudaError_t launch_ragged_tc(const RaggedArgs &a, cudaStream_t st) {
    TcMaps m;
    memset(&m, 0, sizeof m);
    const uint64_t T = a.seq.tokens, HP = 64ull * a.H, GN = 128ull * a.G;
    if (!map_rows(&m.x, a.x, T, HP, a.ldx) || !map_rows(&m.b, a.B, T, GN, a.ldB) || !map_rows(&m.c, a.C, T, GN, a.ldC) ||
        !map_rows(&m.y, a.y, T, HP, a.ldy))
        return cudaErrorInvalidValue;
    const unsigned grid = (unsigned)(a.units * (a.H / 2));
    cudaError_t e;
    if (a.seq.tokens > a.seg) {
        e = cudaFuncSetAttribute(k_ragged_tc<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kTcSmem);
        if (e != cudaSuccess) return e;
        k_ragged_tc<true><<<grid, kTcThreads, kTcSmem, st>>>(m, a);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    e = cudaFuncSetAttribute(k_ragged_tc<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kTcSmem);
    if (e != cudaSuccess) return e;
    k_ragged_tc<false><<<grid, kTcThreads, kTcSmem, st>>>(m, a);
    return cudaGetLastError();
}

}  // namespace ssd
