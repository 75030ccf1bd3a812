// ragged_tc.cu -- the scan over packed ragged sequences on the tensor core: bf16, headdim 64,
// d_state 128, an even number of heads in a B/C group.
//
// A CTA walks one segment (ragged.cu) of one sequence for two heads of a group, in chunks of 128
// tokens.  In the chunk's scan order, with cs_i the inclusive sum of dt A, c = cs of the last token and
// m a reference of the head and chunk:
//
//   scores    = C B^T, masked to j not after i                     both heads share them
//   w_j       = dt_j exp(m - cs_j),  rho_i = exp(cs_i - m)
//   y_i       = rho_i (scores (w x) + C (exp(m) S)^T)_i + D x_i
//   S        <- exp(c) S + exp(c - m) sum_j (w_j x_j) (outer) B_j
//
// With m about c / 2 the exponents of w and rho stay within half the chunk's decay: no factor of the decay
// touches an element of the scores, which are rounded to bf16 as they are and serve both heads.  A
// chunk that decays by more than 2^150 for one of the two heads takes the long form for both: m = c
// (no exponent of w is positive), P = scores times the decay, formed for each head, and x as it is in
// the place of w x.
//
// Precision.  The scores (or P), w x in their product and the copy of S that multiplies C are rounded
// to bf16 (operands of products whose result is a bf16 y).  S itself is a float32 output: w x enters its
// product in three bf16 terms, each the bf16 of what the ones before leave (2^-25 of w x in all; two
// terms, 2^-17, gave states 2e-6 off, twenty times float32's error), and S stays in registers in float32.
//
// Products (M = 128 each, float32 in TMEM):
//   scores    [0,128)    A = C, B = B tile, both K-major in smem
//   y         [256,512)  two buffers, chunk j in number j & 1: D x / rho, stored there before; then
//                        A = C, B = bf16 exp(m) S of both heads (MN-major: row n, 128 columns (head, p));
//                        then A = P (bf16, in TMEM over the scores: 32 columns of scores become 16 of P),
//                        B = high of w x (MN-major), N = 128.  y = rho (the sum).
//   new S     [128,256)  A = B^T (MN-major, M = n), B = the terms of w x one after the other (MN-major), N = 128
// In the long form C S^T, with S as it is, goes to the other buffer of y, 16 columns of each head's P
// take the place of 32 of scores, and P x is formed a head at a time, N = 64.
//
// The long form's P.  It is cut into 32 x 32 blocks; with b the last token before row block I,
// exp(cs_i - cs_j) dt_j = r_i q_j, r_i = exp(cs_i - cs_b), q_j = exp(cs_b - cs_j) dt_j.  P holds scores_ij q_j,
// and r_i takes the place of rho_i.  q grows past dt only in the diagonal block, by at most the decay
// of its 32 tokens: a row block that decays by more than 2^60 has r = 1 for its rows, its diagonal
// block's elements formed one by one, exp(cs_i - cs_j + log dt_j), and r_i q_j multiplied out elsewhere.
// k_ragged_tables forms the factors of every chunk and head beforehand, so the walk spends nothing on
// sums along tokens.
//
// Warps: 0-7 make P and y, 8-15 the state and w x (TMEM lane quarter w & 3; w >> 2 & 1: two of P's four
// column blocks, or the head), 16 the TMA loads, 17 to 19 the MMAs, by what they wait for.  The two
// groups run at their own pace.  Group one: P_j, then y of the chunk before, so that the products of
// chunk j run meanwhile.  Group two: S from the product of chunk j, its bf16 copy for chunk j + 1,
// D x / rho of chunk j + 1.  Each half of w x of chunk j + 1 once the products of chunk j have read theirs.
// Registers: a state warp holds 64 columns of S, so the groups are given 88 and 120 a thread and the last
// warpgroup 56 (128 (2 x 88 + 2 x 120 + 56) = 60416 of the 61440 launched with).
//
// What bounds it.  4.1 to 4.7 us a chunk and head pair (128 tokens; 32 KB of x and of y, 0.75 us at the
// HBM's share of an SM).  The products' operands alone take shared memory 2.8 K of the 8 K cycles (48
// products, 8 KB each; 16 in a row were seen to take 1096 cycles), the passes of the two groups about 4 K
// each, and what ties them is a chain: products read w x -> w x of the next chunk (0.9 K) -> its products
// (1.6 K) -> S (0.7 K).  Tried and not kept: one issuing warp for all products and one group of 16
// warps for all passes (12 K cycles a chunk), waits without the suspend hint (3 to 5 % slower), a second
// stage of B instead of the third term (no faster).
//
// Rows past the segment's end (another sequence's, or none) are zeroed in x and B before a product
// sees them, so nothing of theirs, NaN included, enters; their y rows are not written.
//
// With several segments k_ragged_states comes first: the state that each segment adds and its decay.
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
constexpr int kGroup = 8;                              // warps of a group

// shared memory: everything but the tables in 16 KB boxes; 227 KB in all
constexpr uint32_t kSX = 0;                            // x of two heads
constexpr uint32_t kSW = 2 * kBox;                     // w x: three terms of two heads each
constexpr uint32_t kSB = 8 * kBox, kSC = 10 * kBox;    // B, C: two 64-column boxes each
constexpr uint32_t kSS = 12 * kBox;                    // bf16 S: rows n, a box per head
// One chunk and head's table: the column factors, which every warp reads (copied to shared memory):
// q of the diagonal blocks, then of row blocks 1, 2, 3 (32, 64 and 96 columns); cs_b of the row blocks,
// the chunk's decay, the steep blocks' bits, m, and 0 in the long form or 1 + m - c.  Then per-row values.
// The short form reads rho, w and the scalars alone, and only they are written for it.
constexpr int kTabQd = 0, kTabQ = 128, kTabRef = 320, kTabTot = 324, kTabSteep = 325, kTabM = 326, kTabShort = 327, kTabShared = 328;
constexpr int kTabRho = 328, kTabW = 456, kTabCs = 584, kTabCsd = 712, kTabLen = 840;   // kTabRho: log2 rho
constexpr float kSteepBlock = 60.f, kSteepChunk = 150.f;
static_assert(kTabLen == kRaggedTable, "");
constexpr uint32_t kTab = 14 * kBox;                   // q of both heads
constexpr uint32_t kBars = kTab + 2 * kTabShared * 4;
enum TcBar {
    XF = 0, XE, BF, BF1, BE, BE1, CF, CE, TF,          // loads: full / empty; the tables
    PREP, PREP1,                                       // w x written (even and odd chunks)
    SC, ST, ST1, YI, YF0, YF1,                         // products done: scores, new S (even and odd), C S^T, y (by buffer)
    PR, PR1, SB, YB, YE0, YE1,                         // P written; S's copy; D x / rho; y read (by buffer)
    DONE,
    kNumBars
};
constexpr uint32_t kMisc = (kBars + kNumBars * 8 + 15) & ~15u;
constexpr uint32_t kTcSmem = kMisc + 32;
static_assert(kTcSmem <= 232448, "shared memory budget");
constexpr uint32_t kColS = 128, kColY = 256;           // TMEM columns (scores / P at 0; y: two buffers of 128)

// Chunk number of the j-th chunk of sequence s: as the segments are numbered (ragged.cu), with chunks
// for segments.
__device__ __forceinline__ int chunk_number(const Segment &sg, int seg, int j) { return sg.lo / kQ + sg.s + sg.k * (seg / kQ) + j; }

// The tables of one chunk for 8 heads, a warp to a head.  Sums along the tokens in float32 in log2
// units, from the first token on (cs) and from the last back (the exponent of w), so that w does not
// lose the digits of a difference of large sums.
constexpr int kTabThreads = 256, kTabHeads = kTabThreads / 32;
__global__ void __launch_bounds__(kTabThreads) k_ragged_tables(const __grid_constant__ RaggedArgs a) {
    __shared__ float d[kTabHeads][kQ + 1], tots[kTabHeads];
    const int c = blockIdx.x, g0 = blockIdx.y * kTabHeads, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Segment sg = find_segment(a.seq, kQ, c);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (sg.s < 0 || sg.len == 0) return;
    const int n = min(kQ, sg.len - sg.k * kQ);
    const int base = a.dir > 0 ? sg.lo + sg.k * kQ : sg.lo + sg.len - (sg.k + 1) * kQ;
    {
        const int h = g0 + (threadIdx.x & 7);
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 32 * i + (threadIdx.x >> 3);
            const bool in = h < a.H && (a.dir > 0 ? r < n : r >= kQ - n);
            v[i] = in ? __bfloat162float(static_cast<const __nv_bfloat16 *>(a.dt)[(long long)(base + r) * a.lddt + h]) : -INFINITY;
        }
        const float bias = a.dt_bias && h < a.H ? a.dt_bias[h] : 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)                    // -inf: no token
            d[threadIdx.x & 7][32 * i + (threadIdx.x >> 3)] = v[i] == -INFINITY ? 0.f : a.dt_bias ? softplus(v[i] + bias) : v[i];
    }
    __syncthreads();
    {
        const int i = warp;
        const float a2 = g0 + i < a.H ? a.A[g0 + i] * 1.4426950408889634f : 0.f;
        // lane: four tokens in scan order, 4 lane ..
        float dt[4], s[4], up[4], dn[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            dt[e] = d[i][a.dir > 0 ? 4 * lane + e : kQ - 1 - (4 * lane + e)];
            s[e] = dt[e] * a2;
        }
        up[0] = s[0]; up[1] = up[0] + s[1]; up[2] = up[1] + s[2]; up[3] = up[2] + s[3];
        dn[3] = 0.f; dn[2] = s[3]; dn[1] = dn[2] + s[2]; dn[0] = dn[1] + s[1];     // tokens behind
        float iu = up[3], id = dn[0] + s[0];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float x = __shfl_up_sync(0xffffffffu, iu, o), y = __shfl_down_sync(0xffffffffu, id, o);
            if (lane >= o) iu += x;
            if (lane + o < 32) id += y;
        }
        float eu = __shfl_up_sync(0xffffffffu, iu, 1), ed = __shfl_down_sync(0xffffffffu, id, 1);
        if (lane == 0) eu = 0.f;
        if (lane == 31) ed = 0.f;
        const float tot = __shfl_sync(0xffffffffu, iu, 31);
        if (lane == 0) tots[i] = tot;
        __syncthreads();
        if (g0 + i >= a.H) return;
        // (H is even, and the pairs begin at even heads)
        const bool small = -tots[i] <= kSteepChunk && -tots[i ^ 1] <= kSteepChunk;
        // m - c is a whole number of powers of two, so that exp(c - m) is exact and w keeps the accuracy of
        // the sum behind its token
        const float up2 = small ? rintf(-0.5f * tot) : 0.f, m = tot + up2;
        float *out = a.tables + ((size_t)c * a.H + g0 + i) * kTabLen;
        float cs[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) cs[e] = eu + up[e];
        // cs before and at the end of each scan block of 32 (its last lanes: 7, 15, 23, 31)
        float b[5];
        b[0] = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) b[k + 1] = __shfl_sync(0xffffffffu, cs[3], 8 * k + 7);
        const int blk = lane >> 3;
        const bool steep_own = (blk == 0 ? b[0] - b[1] : blk == 1 ? b[1] - b[2] : blk == 2 ? b[2] - b[3] : b[3] - b[4]) > kSteepBlock;
        const float own = blk == 0 ? b[0] : blk == 1 ? b[1] : blk == 2 ? b[2] : b[3];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int k = 4 * lane + e, row = a.dir > 0 ? k : kQ - 1 - k;      // row of the tile
            out[kTabRho + row] = small ? cs[e] - m : steep_own ? 0.f : cs[e] - own;
            out[kTabW + row] = dt[e] * ex2_ftz(ed + dn[e] + up2);
            if (small) continue;                       // the rest is the long form's
            out[kTabCs + row] = cs[e];
            out[kTabCsd + row] = cs[e] - __log2f(dt[e]);
            out[kTabQd + row] = dt[e] * ex2_ftz(own - cs[e]);
#pragma unroll
            for (int I = 1; I < 4; ++I)
                if (blk < I) out[kTabQ + 16 * I * (I - 1) + 32 * blk + (row & 31)] = dt[e] * ex2_ftz(b[I] - cs[e]);
        }
        if (lane == 0) {
            int steep = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                out[kTabRef + k] = b[k];
                if (b[k] - b[k + 1] > kSteepBlock) steep |= 1 << k;
            }
            out[kTabTot] = tot;
            out[kTabM] = m;
            out[kTabShort] = small ? up2 + 1.f : 0.f;
            out[kTabSteep] = __int_as_float(steep);
        }
    }
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
}

struct TcMaps {
    CUtensorMap x, b, c;
};

template <int R> __device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R> __device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

constexpr int kTcThreads = 640;

__global__ void __launch_bounds__(kTcThreads, 1) k_ragged_tc(const __grid_constant__ TcMaps maps,
                                                             const __grid_constant__ RaggedArgs a) {
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sbase = smem_u32(sm);
    auto bar = [&](int i) { return sbase + kBars + 8u * i; };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + kMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + kMisc + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t MASK = 0xffffffffu;
    // The launches of a call follow one another with programmatic dependent launch; what this one reads of
    // the ones before, it reads behind the wait.  (Every CTA waits, so that the next launch's wait covers all.)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    int job = blockIdx.x;
    if (a.order) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        job = a.order[job];
    }
    const int pairs = a.H / 2, u = job / pairs, h0 = 2 * (job % pairs), grp = h0 / (a.H / a.G);
    const Segment sg = find_segment(a.seq, a.seg, u);
    if (blockIdx.x == 0) check_offsets(a.seq, a.status);
    const bool last = sg.k == sg.count - 1;
    if (sg.s < 0) {                                    // the same for the whole CTA, before any allocation
        asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    if (sbase & 1023) {                                // the swizzled boxes need it (never seen)
        if (threadIdx.x == 0) atomicExch(a.status, 150);
        return;
    }
    const int t0 = sg.k * a.seg, len = min(a.seg, sg.len - t0), nc = (len + kQ - 1) / kQ;
    // row of packed token that is row 0 of chunk j's tiles; rows [v0(j), v1(j)) are the segment's
    auto base = [&](int j) { return a.dir > 0 ? sg.lo + t0 + j * kQ : sg.lo + sg.len - t0 - (j + 1) * kQ; };
    auto rows = [&](int j) { return min(kQ, len - j * kQ); };
    const int chunk0 = chunk_number(sg, a.seg, 0);

    if (threadIdx.x == 0) {
        *abort_flag = 0;
        *reinterpret_cast<volatile long long *>(abort_flag + 1) = a.wait_cycles;
        for (int i = 0; i < kNumBars; ++i) {
            const bool group = i == PR || i == PR1 || i == SB || i == YB || i == YE0 || i == YE1;
            mbar_init(bar(i), (i == PREP || i == PREP1 || i == XE) ? 2 * kGroup : group ? kGroup : i == DONE ? 3 : (i == BE || i == BE1) ? 2 : 1);
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
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const uint32_t tmem = *tmem_slot;
    auto wait = [&](int b, int phase, int code) { return mbar_wait(bar(b), (uint32_t)phase & 1, MASK, abort_flag, a.status, code); };

    // w x of chunk j in three bf16 terms: this thread's row, 32 of the head's columns; rows of no token zero
    auto weigh = [&](int j, int row, int hh, int side, float w) {
        const int n = rows(j);
        const bool mine = a.dir > 0 ? row < n : row >= kQ - n;
        const uint8_t *x = sm + kSX + hh * kBox;
        uint8_t *to = sm + kSW + hh * kBox;
        const float2 w2 = make_float2(w, w), m1 = make_float2(-1.f, -1.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t off = swz(row, 4 * side + i);
            uint4 v = *reinterpret_cast<const uint4 *>(x + off);
            if (!mine) v = make_uint4(0u, 0u, 0u, 0u);
            const uint32_t in[4] = {v.x, v.y, v.z, v.w};
            uint32_t t[3][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float2 f = mul2(unpack2(in[e]), w2);
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    t[k][e] = pack_bf16(f.x, f.y);
                    if (k < 2) f = fma2(unpack2(t[k][e]), m1, f);   // exact
                }
            }
#pragma unroll
            for (int k = 0; k < 3; ++k) *reinterpret_cast<uint4 *>(to + 2 * k * kBox + off) = make_uint4(t[k][0], t[k][1], t[k][2], t[k][3]);
        }
        fence_async_smem();
        __syncwarp();
    };
    if (warp >= 16) regs_down<56>();
    if (warp == 16) {
        // ------------------------------------------------------------ loads
        if (lane == 0) {
            auto wait1 = [&](int b, int phase, int code) { return mbar_wait(bar(b), (uint32_t)phase & 1, 1u, abort_flag, a.status, code); };
            int nx = 0, nb = 0, ncc = 0, nt = 0;       // chunks asked for (nt: tables, of long chunks alone)
            const float *tg = a.tables + ((size_t)chunk0 * a.H + h0) * kTabLen + kTabShort;
            float next = nc > 0 ? *tg : 0.f;
            for (int j = 0; j < nc; ++j) {
                const int r = base(j);
                if (j >= 1 && !wait1(XE, j - 1, 151)) break;
                mbar_expect_tx(bar(XF), 2 * kBox);
                for (int h = 0; h < 2; ++h) tma_load_2d(sbase + kSX + h * kBox, &maps.x, 64 * (h0 + h), r, bar(XF));
                nx = j + 1;
                if (j >= 1 && !wait1(BE + ((j - 1) & 1), (j - 1) >> 1, 152)) break;
                mbar_expect_tx(bar(BF + (j & 1)), 2 * kBox);
                for (int h = 0; h < 2; ++h)
                    tma_load_2d(sbase + kSB + h * kBox, &maps.b, 128 * grp + 64 * h, r, bar(BF + (j & 1)));
                nb = j + 1;
                if (j >= 1 && !wait1(CE, j - 1, 153)) break;
                mbar_expect_tx(bar(CF), 2 * kBox);
                for (int h = 0; h < 2; ++h) tma_load_2d(sbase + kSC + h * kBox, &maps.c, 128 * grp + 64 * h, r, bar(CF));
                ncc = j + 1;
                if (j + 2 < nc) {                      // its loads wait for buffers; from L2 they take half as long
                    for (int h = 0; h < 2; ++h) tma_prefetch_2d(&maps.x, 64 * (h0 + h), base(j + 2));
                    for (int h = 0; h < 2; ++h) tma_prefetch_2d(&maps.b, 128 * grp + 64 * h, base(j + 2));
                    for (int h = 0; h < 2; ++h) tma_prefetch_2d(&maps.c, 128 * grp + 64 * h, base(j + 2));
                }
                // the factors of the long form's P, once the P pass before has read its own
                if (j >= 1 && !wait1(PR + ((j - 1) & 1), (j - 1) >> 1, 162)) break;
                const bool small = next != 0.f;
                tg += (size_t)a.H * kTabLen;
                if (j + 1 < nc) next = *tg;
                if (small) continue;
                mbar_expect_tx(bar(TF), 2 * kTabShared * 4);
                for (int h = 0; h < 2; ++h)
                    bulk_load(sbase + kTab + h * kTabShared * 4, a.tables + ((size_t)(chunk0 + j) * a.H + h0 + h) * kTabLen,
                              kTabShared * 4, bar(TF));
                ++nt;
            }
            if (*abort_flag) {                         // copies in flight land before the memory is given up
                if (nx) mbar_drain(bar(XF), (uint32_t)(nx - 1) & 1, a.wait_cycles);
                if (nb) mbar_drain(bar(BF + ((nb - 1) & 1)), (uint32_t)((nb - 1) >> 1) & 1, a.wait_cycles);
                if (ncc) mbar_drain(bar(CF), (uint32_t)(ncc - 1) & 1, a.wait_cycles);
                if (nt) mbar_drain(bar(TF), (uint32_t)(nt - 1) & 1, a.wait_cycles);
            }
        }
        __syncwarp();
    } else if (warp == 17) {
        // ------------------------------------------------------------ products that read C: scores, C S^T
        {
            const uint32_t id_sc = idesc(128, 0, 0), id_yi = idesc(128, 0, 1);
            const SDesc dC = make_sdesc(sbase + kSC, 16, 1024), dBk = make_sdesc(sbase + kSB, 16, 1024), dS = make_sdesc(sbase + kSS, kBox, 1024);
            const float *tg = a.tables + ((size_t)chunk0 * a.H + h0) * kTabLen + kTabShort;
            float next = nc > 0 ? *tg : 0.f;
            for (int j = 0; j < nc; ++j) {
                const bool small = next != 0.f;
                tg += (size_t)a.H * kTabLen;
                if (j + 1 < nc) next = *tg;
                // P of the chunk before lies over the scores until its product has read it; a partial
                // chunk's B is zeroed in part first
                if (!wait(BF + (j & 1), j >> 1, 155) || !wait(CF, j, 157) || (j >= 1 && !wait(YF0 + ((j - 1) & 1), (j - 1) >> 1, 156)) ||
                    (rows(j) < kQ && !wait(PREP + (j & 1), j >> 1, 154)))
                    break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) {
                        const uint32_t off = (ks >> 2) * kBox + (ks & 3) * 32;
                        mma_ss(tmem, dC.at(off), dBk.at(off), id_sc, ks > 0);
                    }
                    mma_commit(bar(SC));
                    mma_commit(bar(BE + (j & 1)));
                }
                __syncwarp();
                // (the long form's goes into the other buffer, once the y before has been read there)
                if (!wait(SB, j, 158) || !wait(YB, j, 150) || (!small && j >= 1 && !wait(YE0 + ((j - 1) & 1), (j - 1) >> 1, 159))) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        mma_ss(tmem + kColY + 128 * (small ? j & 1 : (j & 1) ^ 1), dC.at((ks >> 2) * kBox + (ks & 3) * 32), dS.at(ks * 2048), id_yi,
                               small || ks > 0);
                    mma_commit(bar(YI));
                    mma_commit(bar(CE));
                }
                __syncwarp();
            }
        }
        if (elect_one()) mma_commit(bar(DONE));
        if (lane == 0) mbar_drain(bar(DONE), 0, a.wait_cycles);
        __syncwarp();
    } else if (warp == 18) {
        // ------------------------------------------------------------ the product of the state (K = tokens: 16 rows of 128 bytes to a step)
        const uint32_t id_st = idesc(128, 1, 1);
        const SDesc dBm = make_sdesc(sbase + kSB, kBox, 1024), dW = make_sdesc(sbase + kSW, kBox, 1024);
        for (int j = 0; j < nc; ++j) {
            if (!wait(PREP + (j & 1), j >> 1, 160) || !wait(BF + (j & 1), j >> 1, 172)) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int ks = 0; ks < 24; ++ks)
                    mma_ss(tmem + kColS, dBm.at((ks & 7) * 2048), dW.at((ks >> 3) * 2 * kBox + (ks & 7) * 2048), id_st, ks > 0);
                mma_commit(bar(ST + (j & 1)));
                mma_commit(bar(BE + (j & 1)));
            }
            __syncwarp();
        }
        if (elect_one()) mma_commit(bar(DONE));
        if (lane == 0) mbar_drain(bar(DONE), 0, a.wait_cycles);
        __syncwarp();
    } else if (warp == 19) {
        // ------------------------------------------------------------ P X
        {
            const uint32_t id_px = idesc(64, 0, 1), id_pw = idesc(128, 0, 1);
            const SDesc dX = make_sdesc(sbase + kSX, kBox, 1024), dW = make_sdesc(sbase + kSW, kBox, 1024);
            const float *tg = a.tables + ((size_t)chunk0 * a.H + h0) * kTabLen + kTabShort;
            float next = nc > 0 ? *tg : 0.f;
            for (int j = 0; j < nc; ++j) {
                const bool small = next != 0.f;
                tg += (size_t)a.H * kTabLen;
                if (j + 1 < nc) next = *tg;
                // in the short form C S^T lies under it: another thread's products, so they are waited for
                if (!wait(PREP + (j & 1), j >> 1, 174) || !wait(PR + (j & 1), j >> 1, 175) || !wait(YI, j, 177)) break;
                tc_fence_after();
                const uint32_t y = tmem + kColY + 128 * (j & 1);
                if (small) {
                    if (elect_one()) {
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks) mma_ts(y, tmem + 32 * (ks >> 1) + 8 * (ks & 1), dW.at(ks * 2048), id_pw, 1);
                        mma_commit(bar(YF0 + (j & 1)));
                    }
                } else if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < 16; ++ks)
                        mma_ts(y + 64 * (ks >> 3), tmem + 32 * (ks >> 1 & 3) + 16 * (ks >> 3) + 8 * (ks & 1),
                               dX.at((ks >> 3) * kBox + (ks & 7) * 2048), id_px, 1);
                    mma_commit(bar(YF0 + (j & 1)));
                }
                __syncwarp();
            }
        }
        if (elect_one()) mma_commit(bar(DONE));
        if (lane == 0) mbar_drain(bar(DONE), 0, a.wait_cycles);
        __syncwarp();
    } else if (warp < kGroup) {
        // ------------------------------------------------------------ P and y
        regs_down<88>();
        {
            const int q = warp & 3, hh = warp >> 2, h = h0 + hh, row = 32 * q + lane;
            const uint32_t tl = tmem + ((uint32_t)(32 * q) << 16);
            const float *tab = reinterpret_cast<const float *>(sm + kTab);
            const int rb = a.dir > 0 ? q : 3 - q;      // scan number of the row block
            const float *tg = a.tables + ((size_t)chunk0 * a.H + h0) * kTabLen;   // chunk 0's; a.H kTabLen on to the next
            const size_t step = (size_t)a.H * kTabLen;
            // ---- P_j: this thread's row, column blocks 2 hh and 2 hh + 1
            int longs = 0;                             // chunks of the long form so far
            auto make_p = [&](int j, bool small) -> bool {
                if (!small && !wait(TF, longs++, 165)) return false;
                const float *u0 = tab, *u1 = tab + kTabShared, *t0p = tg + j * step, *t1p = t0p + kTabLen;
                float cs0 = 0.f, cs1 = 0.f, rf0 = 1.f, rf1 = 1.f;
                bool steep0 = false, steep1 = false;
                if (!small) {
                    cs0 = t0p[kTabCs + row];
                    cs1 = t1p[kTabCs + row];
                    rf0 = ex2_ftz(cs0 - u0[kTabRef + rb]);
                    rf1 = ex2_ftz(cs1 - u1[kTabRef + rb]);
                    steep0 = __float_as_int(u0[kTabSteep]) >> rb & 1;
                    steep1 = __float_as_int(u1[kTabSteep]) >> rb & 1;
                }
                if (!wait(SC, j, 166)) return false;
                tc_fence_after();
#pragma unroll 1
                for (int x = 0; x < 2; ++x) {
                    const int cg = 2 * hh + x, cb = a.dir > 0 ? cg : 3 - cg;
                    if (cb > rb) {
                        const uint32_t zero[16] = {};
                        tmem_st16_nw(tl + 32 * cg, zero);
                        if (!small) tmem_st16_nw(tl + 32 * cg + 16, zero);
                        continue;
                    }
                    const bool diag = cb == rb;
                    float v[32];
                    tmem_ld32(tl + 32 * cg, v);
                    // columns of a diagonal block that are not after its row
                    if (diag) {
                        if (a.dir > 0)
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = i <= lane ? v[i] : 0.f;
                        else
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = i >= lane ? v[i] : 0.f;
                    }
                    if (small) {
                        uint32_t p[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) p[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
                        tmem_st16_nw(tl + 32 * cg, p);
                        continue;
                    }
#pragma unroll 1
                    for (int z = 0; z < 2; ++z) {
                        uint32_t p[16];
                        const bool steep = z ? steep1 : steep0;
                        if (!(diag && steep)) {
                            const float4 *qt = reinterpret_cast<const float4 *>(
                                tab + z * kTabShared + (diag ? kTabQd + 32 * cg : kTabQ + 16 * rb * (rb - 1) + 32 * cb));
                            if (steep) {
                                const float r = z ? rf1 : rf0;
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    const float4 e = qt[i];
                                    p[2 * i] = pack_bf16(v[4 * i] * r * e.x, v[4 * i + 1] * r * e.y);
                                    p[2 * i + 1] = pack_bf16(v[4 * i + 2] * r * e.z, v[4 * i + 3] * r * e.w);
                                }
                            } else {
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    const float4 e = qt[i];
                                    const float2 lo = mul2(make_float2(v[4 * i], v[4 * i + 1]), make_float2(e.x, e.y));
                                    const float2 hi = mul2(make_float2(v[4 * i + 2], v[4 * i + 3]), make_float2(e.z, e.w));
                                    p[2 * i] = pack_bf16(lo.x, lo.y);
                                    p[2 * i + 1] = pack_bf16(hi.x, hi.y);
                                }
                            }
                        } else {
                            // (a column past the row has a positive exponent, of any size: no product with it)
                            const float *ct = (z ? t1p : t0p) + kTabCsd + 32 * cg, c = z ? cs1 : cs0;
                            auto el = [&](int i) {
                                const bool in = a.dir > 0 ? i <= lane : i >= lane;
                                return in ? v[i] * ex2_ftz(c - ct[i]) : 0.f;
                            };
#pragma unroll
                            for (int i = 0; i < 16; ++i) p[i] = pack_bf16(el(2 * i), el(2 * i + 1));
                        }
                        // in place: the block's 32 score columns become 16 of each head
                        tmem_st16_nw(tl + 32 * cg + 16 * z, p);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(PR + (j & 1)));
                return true;
            };
            // ---- y_j: this thread's row of head h
            auto make_y = [&](int j, bool small, float lr, float cs) -> bool {
                const int buf = j & 1;
                if (!wait(YF0 + buf, j >> 1, 171) || (!small && !wait(YI, j, 170))) return false;
                tc_fence_after();
                const float rho = ex2_ftz(lr), ecs = ex2_ftz(cs);
                const float2 r2 = make_float2(rho, rho), e2 = make_float2(ecs, ecs);
                const int n = rows(j), r0 = row & ~1;
                const bool even_in = a.dir > 0 ? r0 < n : r0 >= kQ - n, odd_in = a.dir > 0 ? r0 + 1 < n : r0 + 1 >= kQ - n;
                __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(a.y) + (long long)(base(j) + r0) * a.ldy + h * 64;
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    float v[32];
                    tmem_ld32(tl + kColY + 128 * buf + 64 * hh + 32 * z, v);
                    if (small) {
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            const float2 t = mul2(make_float2(v[i], v[i + 1]), r2);
                            v[i] = t.x;
                            v[i + 1] = t.y;
                        }
                    } else {
                        float yi[32];
                        tmem_ld32(tl + kColY + 128 * (buf ^ 1) + 64 * hh + 32 * z, yi);
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            const float2 t = fma2(make_float2(yi[i], yi[i + 1]), e2, mul2(make_float2(v[i], v[i + 1]), r2));
                            v[i] = t.x;
                            v[i + 1] = t.y;
                        }
                    }
                    if (z == 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(YE0 + buf));
                    }
                    // 16 bytes of a row a lane, but whole sectors of 32 are stored: neighbouring lanes trade
                    // halves, so that each pair stores 32 bytes of the even row, then of the odd one
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t p[2][4];
#pragma unroll
                        for (int c = 0; c < 2; ++c)
#pragma unroll
                            for (int e = 0; e < 4; ++e) p[c][e] = pack_bf16(v[16 * i + 8 * c + 2 * e], v[16 * i + 8 * c + 2 * e + 1]);
                        const bool odd = lane & 1;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t got = __shfl_xor_sync(MASK, odd ? p[0][e] : p[1][e], 1);
                            if (odd) p[0][e] = got;
                            else p[1][e] = got;
                        }
                        // now p[0]: this lane's half of the even row's 32 bytes, p[1]: of the odd row's
                        __nv_bfloat16 *to = y + 32 * z + 16 * i + 8 * (lane & 1);
                        if (even_in) __stcs(reinterpret_cast<uint4 *>(to), make_uint4(p[0][0], p[0][1], p[0][2], p[0][3]));
                        if (odd_in) __stcs(reinterpret_cast<uint4 *>(to + a.ldy), make_uint4(p[1][0], p[1][1], p[1][2], p[1][3]));
                    }
                }
                return true;
            };
            // its half of w x of chunk j
            auto weigh_half = [&](int j, float w, bool small) -> bool {
                if (!wait(XF, j, 193)) return false;
                weigh(j, row, hh, 1, w);
                if (lane == 0) {
                    mbar_arrive(bar(PREP + (j & 1)));
                    if (small) mbar_arrive(bar(XE));   // the long form's product reads x itself
                }
                return true;
            };
            bool was_small = true, ok = true;
            float lr = 0.f, cs = 0.f;                  // log2 rho and cs of the row, of the chunk before
            const float *tw = tg + hh * kTabLen;       // own head's table of the chunk
            float nshort = nc > 0 ? tw[kTabShort] : 1.f;
            if (nc > 0) ok = weigh_half(0, tw[kTabW + row], nshort != 0.f);
            for (int j = 0; j <= nc && ok; ++j) {
                float nlr = 0.f, ncs = 0.f, nw = 0.f;
                const bool small = nshort != 0.f;
                if (j + 1 < nc) {
                    nw = tw[step + kTabW + row];
                    nshort = tw[step + kTabShort];
                }
                tw += step;
                if (j < nc) {
                    const float *t = tg + j * step + hh * kTabLen + row;
                    nlr = t[kTabRho];
                    ncs = t[kTabCs];                   // (not a number of ours in the short form, which has no use for it)
                }
                // after a chunk of the long form its y comes first: it frees both buffers of y, which
                // what P_j waits for may need
                if (j >= 1 && !was_small) ok = make_y(j - 1, false, lr, cs);
                if (ok && j < nc) ok = make_p(j, small);
                if (ok && j >= 1 && was_small) ok = make_y(j - 1, true, lr, cs);
                if (ok && j + 1 < nc) {
                    // both products have read the w x (P X of the long form: the x) of this chunk
                    if (!(ok = wait(YF0 + (j & 1), j >> 1, 194) && wait(ST + (j & 1), j >> 1, 195))) break;
                    if (!small && lane == 0) mbar_arrive(bar(XE));
                    ok = weigh_half(j + 1, nw, nshort != 0.f);
                }
                was_small = small;
                lr = nlr;
                cs = ncs;
            }
        }
    } else if (warp < 2 * kGroup) {
        // ------------------------------------------------------------ the state and w x
        regs_up<120>();
        const int q = warp & 3, hh = warp >> 2 & 1, h = h0 + hh, row = 32 * q + lane;   // n of the state, row of w x
        const uint32_t tl = tmem + ((uint32_t)(32 * q) << 16);
        const size_t PN = 64 * 128, at = (size_t)h * PN + row;
        float S[64];                                   // S[h][i][row]
        {
            const float *in = nullptr;
            const int v0 = first_state(sg, a.seg);
            if (sg.k == 0) {
                if (last) {
                    const int si = slot_of_start(a.slots, sg.s, a.status);
                    if (si >= 0) in = static_cast<const float *>(a.slots.pool_in) + (size_t)si * a.H * PN;
                } else {
                    in = a.ws_state + (size_t)(v0 + sg.count - 1) * a.H * PN;
                }
            } else {
                in = a.ws_state + (size_t)v0 * a.H * PN;
            }
#pragma unroll
            for (int i = 0; i < 64; ++i) S[i] = in ? in[at + i * 128] : 0.f;
            for (int k = 1; k < sg.k; ++k) {
                    const size_t v = (size_t)(v0 + k) * a.H;
                    const float d = ex2_ftz(a.ws_decay[v + h]);
                    const float *add = a.ws_state + v * PN + at;
#pragma unroll
                    for (int i = 0; i < 64; ++i) S[i] = fmaf(S[i], d, add[i * 128]);
                }
        }
        // Of the chunk that is next: w and log2 rho of this row, c and m (log2), its form
        float wr = 0.f, lr = 0.f, tot = 0.f, ref = 0.f;
        float shortness = 0.f;                         // kTabShort
        bool small = false;
        const float Dh = a.D ? a.D[h] : 0.f;
        auto load_w = [&](int j) {
            const float *t = a.tables + ((size_t)(chunk0 + j) * a.H + h) * kTabLen;
            wr = t[kTabW + row];
            lr = t[kTabRho + row];
            tot = t[kTabTot];
            ref = t[kTabM];
            shortness = t[kTabShort];
            small = shortness != 0.f;
        };
        auto copy_state = [&]() {                      // bf16 exp(m) S (long form: S): row n of the head's box
            const float f = small ? ex2_ftz(ref) : 1.f;
            const float2 f2 = make_float2(f, f);
            uint8_t *box = sm + kSS + hh * kBox;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 t = mul2(make_float2(S[8 * i + 2 * e], S[8 * i + 2 * e + 1]), f2);
                    o[e] = pack_bf16(t.x, t.y);
                }
                *reinterpret_cast<uint4 *>(box + swz(row, i)) = make_uint4(o[0], o[1], o[2], o[3]);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(SB));
        };
        uint8_t *xb = sm + kSX + hh * kBox;
        // chunk j has landed; rows of no token: zero in x (the long form's product reads it) and B
        auto land = [&](int j) -> bool {
            if (!wait(XF, j, 163)) return false;
            const int n = rows(j);
            if (n < kQ) {
                if (!wait(BF + (j & 1), j >> 1, 164)) return false;
                if (a.dir > 0 ? row >= n : row < kQ - n)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        *reinterpret_cast<uint4 *>(xb + swz(row, i)) = make_uint4(0u, 0u, 0u, 0u);
                        *reinterpret_cast<uint4 *>(sm + kSB + hh * kBox + swz(row, i)) = make_uint4(0u, 0u, 0u, 0u);
                    }
            }
            return true;
        };
        // D x / rho of chunk j into its buffer of y
        auto start_y = [&](int j) {
            const float f = Dh * ex2_ftz(-lr);
            const float2 f2 = make_float2(f, f);
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                float v[32];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(xb + swz(row, 4 * z + i));
                    const uint32_t in[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 t = mul2(unpack2(in[e]), f2);
                        v[8 * i + 2 * e] = t.x;
                        v[8 * i + 2 * e + 1] = t.y;
                    }
                }
                tmem_st32f_nw(tl + kColY + 128 * (j & 1) + 64 * hh + 32 * z, v);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(YB));
        };
        // its half of w x of chunk j
        auto prepare = [&](int j) {
            weigh(j, row, hh, 0, wr);
            if (lane == 0) {
                mbar_arrive(bar(PREP + (j & 1)));
                if (small) mbar_arrive(bar(XE));  // the long form's product reads x itself
            }
        };
        bool ok = true;
        if (nc > 0) {
            load_w(0);
            copy_state();
            if ((ok = land(0))) {
                start_y(0);
                prepare(0);
            }
        }

        for (int j = 0; j < nc && ok; ++j) {
            const float kappa = ex2_ftz(tot), add = small ? ex2_ftz(1.f - shortness) : 1.f;
            const bool was_small = small;
            if (j + 1 < nc) load_w(j + 1);
            if (!(ok = wait(ST + (j & 1), j >> 1, 168))) break;
            tc_fence_after();
            const float2 k2 = make_float2(kappa, kappa), a2 = make_float2(add, add);
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                float ds[32];
                tmem_ld32(tl + kColS + 64 * hh + 32 * z, ds);
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    const float2 n2 = fma2(make_float2(S[32 * z + i], S[32 * z + i + 1]), k2, mul2(make_float2(ds[i], ds[i + 1]), a2));
                    S[32 * z + i] = n2.x;
                    S[32 * z + i + 1] = n2.y;
                }
            }
            tc_fence_before();
            if (j + 1 == nc) break;
            if (!(ok = wait(YI, j, 169))) break;   // C S^T has read the copy it is written over
            copy_state();
            if (!was_small) {                      // P x of the long form has read x
                if (!(ok = wait(YF0 + (j & 1), j >> 1, 178))) break;
                if (lane == 0) mbar_arrive(bar(XE));
            }
            // the buffer of y is free: the y before last has been read (and the long form's C S^T there)
            if ((j >= 1 && !(ok = wait(YE0 + ((j - 1) & 1), (j - 1) >> 1, 179))) ||
                (!was_small && !(ok = wait(YE0 + (j & 1), j >> 1, 180))))
                break;
            tc_fence_after();
            if (!(ok = land(j + 1))) break;
            start_y(j + 1);
            if (was_small && !(ok = wait(YF0 + (j & 1), j >> 1, 176))) break;   // P X has read w x
            prepare(j + 1);
        }
        if (ok) {
            float *out = nullptr;
            if (last && a.slots.pool_out) {
                // (slot_of_end meets at a CTA barrier: its look for another user is done warp by warp here)
                const int v = a.slots.out ? a.slots.out[sg.s] : sg.s;
                bool good = v >= 0 && v < a.slots.n_out;
                if (v >= a.slots.n_out) report(a.status, kCodeSlotRange);
                if (good && __any_sync(MASK, slot_shared(a.slots, sg.s, a.seq.nseq, v, lane, 32))) {
                    report(a.status, kCodeSlotTwice);
                    good = false;
                }
                if (good) out = static_cast<float *>(a.slots.pool_out) + (size_t)v * a.H * PN;
            }
            if (out)
#pragma unroll
                for (int i = 0; i < 64; ++i) out[at + i * 128] = S[i];
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 17) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}

// ------------------------------------------------------------------ the segments' own states

// S of every segment but a sequence's last, from zero (the first segment: from the sequence's start
// state): the update above and nothing else.  Its products take half a chunk at a time (64 tokens), so
// that the next half is weighed while they run: 16 warps weigh, two buffers of w x, three stages of x and
// B, two accumulators; a chunk's sum is added to S while the next chunk's first half is multiplied.
// A segment of this kernel has whole chunks only.  One sequence of 32741 tokens, 64 heads: 135 us with cold
// caches (2.1 TB/s); on one card the whole call took 483 us with it, 501 when this was a walk of whole chunks.  x alone
// is 42 us at the HBM rate, the products' operand reads 50; a capture shows the tensor pipe 31 % active,
// shared memory 35 % and issue slots 45 %, so what is left is the chain load, weigh, multiply of a half.
constexpr int kHalf = 64, kStThreads = 576;
constexpr uint32_t kHBox = kHalf * 128;                // 64 rows of 64 bf16: 8 KB
constexpr uint32_t kTX = 0, kTB = 6 * kHBox, kTW = 12 * kHBox;   // x, B: three stages of two boxes; w x: two of six
constexpr uint32_t kTBars = 24 * kHBox;
enum StBar { HF = 0, HXE = 3, HBE = 6, HP = 9, HM = 11, HA = 13, HR = 15, HDONE = 17, kStBars };   // full; x, B empty; weighed; multiplied; sum full / read
constexpr uint32_t kTMisc = (kTBars + kStBars * 8 + 15) & ~15u, kStSmem = kTMisc + 32;
static_assert(kStSmem <= 232448, "shared memory budget");

struct StMaps {
    CUtensorMap x, b;
};

// The order in which k_ragged_tc takes its jobs (a segment and a pair of heads), longest first: CTAs start in
// the order of their numbers, and a long job that starts last is waited for by all other SMs.  A chunk
// counts 2, in the long form 5 (measured 4.4 and 10.5 us).  8 ragged prompts of 16384 tokens in all, 64 heads,
// 14 % of the chunks long: 291 us, 343 as they are numbered; one
// sequence of 32741 tokens, whose jobs are alike, the same either way (486 to 531 us from run to run).
// Sorted by 64 buckets; within one the order is open (results do not depend on it).  One CTA's work, while the
// others form the states.
constexpr int kBuckets = 64;
__device__ void order_jobs(const RaggedArgs &a, int *count) {
    const int pairs = a.H / 2, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, most = 5 * (a.seg / kQ);
    const size_t jobs = (size_t)a.units * pairs;
    int *bucket = a.order + jobs;
    if (threadIdx.x < kBuckets) count[threadIdx.x] = 0;
    __syncthreads();
    for (int u = warp; u < a.units; u += kStThreads / 32) {
        const Segment sg = find_segment(a.seq, a.seg, u);
        const int nc = sg.s < 0 ? 0 : (min(a.seg, sg.len - sg.k * a.seg) + kQ - 1) / kQ;
        const float *t = a.tables + (size_t)(sg.s < 0 ? 0 : chunk_number(sg, a.seg, 0)) * a.H * kTabLen + kTabShort;
        for (int p = lane; p < pairs; p += 32) {
            int cost = 0;
#pragma unroll 8
            for (int j = 0; j < nc; ++j) cost += t[((size_t)j * a.H + 2 * p) * kTabLen] != 0.f ? 2 : 5;
            const int b = kBuckets - 1 - (int)((long long)cost * (kBuckets - 1) / most);
            bucket[(size_t)u * pairs + p] = b;
            atomicAdd(&count[b], 1);
        }
    }
    __syncthreads();
    int before = 0;
    if (threadIdx.x < kBuckets)
        for (int b = 0; b < (int)threadIdx.x; ++b) before += count[b];
    __syncthreads();
    if (threadIdx.x < kBuckets) count[threadIdx.x] = before;
    __syncthreads();
    for (size_t i = threadIdx.x; i < jobs; i += kStThreads) a.order[atomicAdd(&count[bucket[i]], 1)] = (int)i;
}

__global__ void __launch_bounds__(kStThreads, 1) k_ragged_states(const __grid_constant__ StMaps maps,
                                                                 const __grid_constant__ RaggedArgs a) {
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sbase = smem_u32(sm);
    auto bar = [&](int i) { return sbase + kTBars + 8u * i; };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + kTMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + kTMisc + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t MASK = 0xffffffffu;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.x == 0) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        order_jobs(a, reinterpret_cast<int *>(sm));
        return;
    }
    const int job = blockIdx.x - 1, pairs = a.H / 2, v = job / pairs, h0 = 2 * (job % pairs), grp = h0 / (a.H / a.G);
    const Segment sg = find_state(a.seq, a.seg, v);
    if (sg.s < 0 || sg.k == sg.count - 1 || (sbase & 1023)) {   // (a misaligned base is reported by k_ragged_tc)
        asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    const int t0 = sg.k * a.seg, nc = a.seg / kQ, nh = 2 * nc;
    const int chunk0 = chunk_number(sg, a.seg, 0);
    // first row of half i: halves in the order of the rows, chunks in scan order
    auto base = [&](int i) {
        const int j = i >> 1;
        return (a.dir > 0 ? sg.lo + t0 + j * kQ : sg.lo + sg.len - t0 - (j + 1) * kQ) + kHalf * (i & 1);
    };
    if (threadIdx.x == 0) {
        *abort_flag = 0;
        *reinterpret_cast<volatile long long *>(abort_flag + 1) = a.wait_cycles;
        for (int i = 0; i < kStBars; ++i)
            mbar_init(bar(i), (i >= HXE && i < HBE) || (i >= HP && i < HM) || (i >= HR && i < HDONE) ? 16 : 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 17) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 256;" ::"r"(smem_u32(tmem_slot)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const uint32_t tmem = *tmem_slot;
    auto wait = [&](int b, int phase, int code) { return mbar_wait(bar(b), (uint32_t)phase & 1, MASK, abort_flag, a.status, code); };

    if (warp == 16) {
        if (lane == 0) {
            auto wait1 = [&](int b, int phase, int code) { return mbar_wait(bar(b), (uint32_t)phase & 1, 1u, abort_flag, a.status, code); };
            int n = 0;
            for (int i = 0; i < nh; ++i) {
                const int st = i % 3, r = base(i);
                if (i >= 3 && (!wait1(HXE + st, i / 3 - 1, 201) || !wait1(HBE + st, i / 3 - 1, 202))) break;
                mbar_expect_tx(bar(HF + st), 4 * kHBox);
                for (int h = 0; h < 2; ++h) {
                    tma_load_2d(sbase + kTX + (2 * st + h) * kHBox, &maps.x, 64 * (h0 + h), r, bar(HF + st));
                    tma_load_2d(sbase + kTB + (2 * st + h) * kHBox, &maps.b, 128 * grp + 64 * h, r, bar(HF + st));
                }
                n = i + 1;
            }
            if (*abort_flag)                           // copies in flight land before the memory is given up
                for (int i = n - 1; i >= 0 && i >= n - 3; --i) mbar_drain(bar(HF + i % 3), (uint32_t)(i / 3) & 1, a.wait_cycles);
        }
        __syncwarp();
    } else if (warp == 17) {
        const uint32_t id = idesc(128, 1, 1);
        for (int i = 0; i < nh; ++i) {
            const int st = i % 3, j = i >> 1;
            if (!wait(HP + (i & 1), i >> 1, 203) || !wait(HF + st, i / 3, 204) ||
                (!(i & 1) && j >= 2 && !wait(HR + (j & 1), (j >> 1) - 1, 205)))
                break;
            tc_fence_after();
            const SDesc db = make_sdesc(sbase + kTB + 2 * st * kHBox, kHBox, 1024), dw = make_sdesc(sbase + kTW + 6 * (i & 1) * kHBox, kHBox, 1024);
            if (elect_one()) {
#pragma unroll
                for (int ks = 0; ks < 12; ++ks)
                    mma_ss(tmem + 128 * (j & 1), db.at((ks & 3) * 2048), dw.at((ks >> 2) * 2 * kHBox + (ks & 3) * 2048), id, ks > 0 || (i & 1));
                mma_commit(bar(HM + (i & 1)));
                mma_commit(bar(HBE + st));
                if (i & 1) mma_commit(bar(HA + (j & 1)));
            }
            __syncwarp();
        }
        if (elect_one()) mma_commit(bar(HDONE));
        if (lane == 0) mbar_drain(bar(HDONE), 0, a.wait_cycles);
        __syncwarp();
    } else {
        // S: n = 32 q + its lane, 32 columns (head, p) from 32 cg on; w x: row and 16 columns of a head
        const int q = warp & 3, cg = warp >> 2, n = 32 * q + lane, hs = h0 + (cg >> 1);
        const int hw = warp >> 3, row = 32 * (warp & 1) + lane, c0 = 2 * (warp >> 1 & 3);
        const size_t PN = 64 * 128, at = (size_t)hs * PN + (size_t)(32 * (cg & 1)) * 128 + n;
        float S[32];
        const int si = sg.k == 0 ? slot_of_start(a.slots, sg.s, a.status) : -1;
        const float *in = si >= 0 ? static_cast<const float *>(a.slots.pool_in) + (size_t)si * a.H * PN + at : nullptr;
#pragma unroll
        for (int i = 0; i < 32; ++i) S[i] = in ? in[i * 128] : 0.f;
        if (sg.k == 0) {
            // the sequence's start, kept where its last segment's own state would be (nothing reads that):
            // by the time the scan starts from it the pool may hold the sequence's new state
            float *keep = a.ws_state + (size_t)(v - sg.k + sg.count - 1) * a.H * PN + at;
#pragma unroll
            for (int i = 0; i < 32; ++i) keep[i * 128] = S[i];
        }
        const size_t step = (size_t)a.H * kTabLen;
        const float *tw = a.tables + ((size_t)chunk0 * a.H + h0 + hw) * kTabLen + kTabW + row;
        const float *ts = a.tables + ((size_t)chunk0 * a.H + hs) * kTabLen;
        float w = *tw, total = 0.f;
        // S of chunk j
        auto add_chunk = [&](int j) -> bool {
            const float tot = ts[kTabTot], shortness = ts[kTabShort];
            ts += step;
            total += tot;
            if (!wait(HA + (j & 1), j >> 1, 206)) return false;
            tc_fence_after();
            float ds[32];
            tmem_ld32(tmem + ((uint32_t)(32 * q) << 16) + 128 * (j & 1) + 32 * cg, ds);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(HR + (j & 1)));
            const float kappa = ex2_ftz(tot), add = shortness != 0.f ? ex2_ftz(1.f - shortness) : 1.f;
            const float2 k2 = make_float2(kappa, kappa), a2 = make_float2(add, add);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                const float2 v = fma2(make_float2(S[i], S[i + 1]), k2, mul2(make_float2(ds[i], ds[i + 1]), a2));
                S[i] = v.x;
                S[i + 1] = v.y;
            }
            return true;
        };
        bool ok = true;
        for (int i = 0; i < nh && ok; ++i) {
            const int st = i % 3;
            const float2 w2 = make_float2(w, w), m1 = make_float2(-1.f, -1.f);
            if (i + 1 < nh) w = tw[((i + 1) >> 1) * step + kHalf * ((i + 1) & 1)];
            // (this buffer's products of two halves ago)
            if (!(ok = wait(HF + st, i / 3, 207) && (i < 2 || wait(HM + (i & 1), (i >> 1) - 1, 208)))) break;
            const uint8_t *x = sm + kTX + (2 * st + hw) * kHBox;
            uint8_t *to = sm + kTW + (6 * (i & 1) + hw) * kHBox;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const uint32_t off = swz(row, c0 + c);
                const uint4 v = *reinterpret_cast<const uint4 *>(x + off);
                const uint32_t xi[4] = {v.x, v.y, v.z, v.w};
                uint32_t t[3][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float2 f = mul2(unpack2(xi[e]), w2);
#pragma unroll
                    for (int k = 0; k < 3; ++k) {
                        t[k][e] = pack_bf16(f.x, f.y);
                        if (k < 2) f = fma2(unpack2(t[k][e]), m1, f);   // exact
                    }
                }
#pragma unroll
                for (int k = 0; k < 3; ++k) *reinterpret_cast<uint4 *>(to + 2 * k * kHBox + off) = make_uint4(t[k][0], t[k][1], t[k][2], t[k][3]);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(HP + (i & 1)));
                mbar_arrive(bar(HXE + st));
            }
            if ((i & 1) && i > 1) ok = add_chunk((i >> 1) - 1);
        }
        if (ok && add_chunk(nc - 1)) {
            float *out = a.ws_state + (size_t)v * a.H * PN + at;
#pragma unroll
            for (int i = 0; i < 32; ++i) out[i * 128] = S[i];
            if (q == 0 && (cg & 1) == 0 && lane == 0) a.ws_decay[(size_t)v * a.H + hs] = total;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 17) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 256;" ::"r"(tmem));
    }
}

bool map_rows(CUtensorMap *m, const void *base, uint64_t rows, uint64_t cols, uint64_t ld, uint32_t box_rows) {
    EncodeTiled enc = get_encode();
    if (!enc) return false;
    const cuuint64_t dims[2] = {cols, rows}, strides[1] = {ld * 2};
    const cuuint32_t box[2] = {64, box_rows}, estr[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// Head shapes and layouts of the tensor-core form: what a tensor map takes (16-byte aligned rows).
bool ragged_tc_supported(const RaggedArgs &a, bool bf16) {
    auto ok = [](const void *p, long long ld) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 8 == 0; };
    return bf16 && a.P == 64 && a.N == 128 && (a.H / a.G) % 2 == 0 && a.seq.tokens > 0 && ok(a.x, a.ldx) && ok(a.B, a.ldB) &&
           ok(a.C, a.ldC) && ok(a.y, a.ldy) && (long long)a.units * (a.H / 2) < 0x7fffffffLL && get_encode() != nullptr;
}

cudaError_t launch_ragged_tc(const RaggedArgs &a, cudaStream_t st) {
    TcMaps m;
    memset(&m, 0, sizeof m);
    const uint64_t T = a.seq.tokens, HP = 64ull * a.H, GN = 128ull * a.G;
    if (!map_rows(&m.x, a.x, T, HP, a.ldx, kQ) || !map_rows(&m.b, a.B, T, GN, a.ldB, kQ) || !map_rows(&m.c, a.C, T, GN, a.ldC, kQ))
        return cudaErrorInvalidValue;
    const unsigned grid = (unsigned)(a.units * (a.H / 2));
    k_ragged_tables<<<dim3(a.seq.tokens / kQ + a.seq.nseq, (a.H + kTabHeads - 1) / kTabHeads), kTabThreads, 0, st>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (a.states) {
        StMaps sm;
        memset(&sm, 0, sizeof sm);
        if (!map_rows(&sm.x, a.x, T, HP, a.ldx, kHalf) || !map_rows(&sm.b, a.B, T, GN, a.ldB, kHalf)) return cudaErrorInvalidValue;
        if ((e = cudaFuncSetAttribute(k_ragged_states, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kStSmem)) != cudaSuccess) return e;
        cfg.gridDim = dim3(a.states * (a.H / 2) + 1);  // and the CTA that sorts the jobs
        cfg.blockDim = dim3(kStThreads);
        cfg.dynamicSmemBytes = kStSmem;
        if ((e = cudaLaunchKernelEx(&cfg, k_ragged_states, sm, a)) != cudaSuccess) return e;
        cfg.gridDim = dim3(grid);
    }
    cfg.blockDim = dim3(kTcThreads);
    cfg.dynamicSmemBytes = kTcSmem;
    e = cudaFuncSetAttribute(k_ragged_tc, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kTcSmem);
    if (e != cudaSuccess) return e;
    return cudaLaunchKernelEx(&cfg, k_ragged_tc, m, a);
}

}  // namespace ssd
