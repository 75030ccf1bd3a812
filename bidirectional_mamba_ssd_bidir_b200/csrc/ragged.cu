// ragged.cu -- the selective scan over packed ragged sequences on the CUDA cores, in float32: every
// head size the library takes, both io types.  (bf16 with headdim 64 and d_state 128 runs on the
// tensor cores, ragged_tc.cu.)
//
//   S <- exp(dt A) S + dt x (outer) B,     y = C S + D x          per (sequence, head), in scan order
//
// The recurrence is evaluated as written, token by token, with the state in registers: thread
// (pg, nl) of a CTA holds P/16 rows x N/8 columns of it.  A step is about 3 P N / 128 fused
// multiply-adds a thread and a reduction of y over the 8 column lanes, so issue slots bound the
// kernel, not HBM (8 heads of 32 x 64, 7 sequences of 533 tokens in all, float32: 21 us, 33 with one token at
// a time and segments of 64).  Sequences are cut into segments of `seg` tokens when there are too few of them:
// a first launch forms each segment's end state from zero (the sequence's own start state for its
// first segment) and its decay; the second starts every segment from the states folded before it.
// (The recurrence is linear in its state.)
//
// Segment u = start / seg + i + k (k-th segment of sequence i): ceil(len / seg) consecutive numbers a
// sequence, disjoint between sequences whatever the lengths, and no pass over the lengths is needed:
// len <= (end / seg - start / seg + 1) seg - (start mod seg) leaves room for them.
#include "ragged.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 128, kTB = 16;   // threads of a CTA; tokens staged at a time

template <typename T, int P, int N, bool STATES>
__global__ void __launch_bounds__(kThreads) k_ragged(const __grid_constant__ RaggedArgs a) {
    constexpr int PPT = P / 16, NPT = N / 8, W = NPT < 4 ? NPT : 4, NQ = NPT / W;
    __shared__ float sx[kTB][P], sB[kTB][N], sC[kTB][N], sy[kTB][P], sdt[kTB], slog[kTB], sdec[kTB];
    const int u = blockIdx.x, h = blockIdx.y, g = h / (a.H / a.G);
    const Segment sg = STATES ? find_state(a.seq, a.seg, u) : find_segment(a.seq, a.seg, u);
    const int v0 = first_state(sg, a.seg);
    if (u == 0 && h == 0 && !STATES) check_offsets(a.seq, a.status);
    if (sg.s < 0) return;
    const bool last = sg.k == sg.count - 1;
    if (STATES && last) return;
    const int tid = threadIdx.x, nl = tid & 7, pg = tid >> 3;
    const int t0 = sg.k * a.seg, n = min(a.seg, sg.len - t0);
    // token of place i of the segment
    const int first = a.dir > 0 ? sg.lo + t0 : sg.lo + sg.len - 1 - t0;
    const size_t PN = (size_t)P * N;
    float S[PPT][NPT];
    // element (i, q, e) of a thread: row PPT pg + i, column W (nl + 8 q) + e
    auto at = [&](int i, int q) { return (size_t)(PPT * pg + i) * N + W * (nl + 8 * q); };
    auto each = [&](auto f) {
#pragma unroll
        for (int i = 0; i < PPT; ++i)
#pragma unroll
            for (int q = 0; q < NQ; ++q)
#pragma unroll
                for (int e = 0; e < W; ++e) f(S[i][q * W + e], at(i, q) + e);
    };
    each([&](float &s, size_t) { s = 0.f; });
    if (sg.k == 0) {
        if (STATES || last) {
            const int si = slot_of_start(a.slots, sg.s, a.status);
            if (si >= 0) {
                const float *in = static_cast<const float *>(a.slots.pool_in) + ((size_t)si * a.H + h) * PN;
                each([&](float &s, size_t o) { s = in[o]; });
            }
            if (STATES) {
                // kept for the scan in the place of the sequence's last segment, whose own end state
                // nothing reads: by then the pool may already hold the sequence's new state
                float *keep = a.ws_state + ((size_t)(v0 + sg.count - 1) * a.H + h) * PN;
                each([&](float &s, size_t o) { keep[o] = s; });
            }
        } else {
            const float *in = a.ws_state + ((size_t)(v0 + sg.count - 1) * a.H + h) * PN;
            each([&](float &s, size_t o) { s = in[o]; });
        }
    } else if (!STATES) {
        for (int k = 0; k < sg.k; ++k) {
            const size_t v = (size_t)(v0 + k) * a.H + h;
            const float d = expf(a.ws_decay[v]);
            const float *in = a.ws_state + v * PN;
            each([&](float &s, size_t o) { s = (k == 0 ? 0.f : s * d) + in[o]; });
        }
    }
    const float A = a.A[h], Dh = a.D ? a.D[h] : 0.f, bias = a.dt_bias ? a.dt_bias[h] : 0.f;
    const T *x = static_cast<const T *>(a.x) + (size_t)h * P, *B = static_cast<const T *>(a.B) + (size_t)g * N,
            *C = static_cast<const T *>(a.C) + (size_t)g * N, *dt = static_cast<const T *>(a.dt) + h;
    T *y = static_cast<T *>(a.y) + (size_t)h * P;
    float total = 0.f;
    for (int b0 = 0; b0 < n; b0 += kTB) {
        const int m = min(kTB, n - b0);
        __syncthreads();
        for (int i = tid; i < m * P; i += kThreads) sx[i / P][i % P] = to_f<T>(x[(first + a.dir * (long long)(b0 + i / P)) * a.ldx + i % P]);
        for (int i = tid; i < m * N; i += kThreads) {
            const long long t = first + a.dir * (long long)(b0 + i / N);
            sB[i / N][i % N] = to_f<T>(B[t * a.ldB + i % N]);
            if (!STATES) sC[i / N][i % N] = to_f<T>(C[t * a.ldC + i % N]);
        }
        if (tid < m) {
            float d = to_f<T>(dt[(first + a.dir * (long long)(b0 + tid)) * a.lddt]);
            if (a.dt_bias) d = softplus(d + bias);
            sdt[tid] = d;
            slog[tid] = d * A;
            sdec[tid] = expf(d * A);
        }
        __syncthreads();
        auto token = [&](int i) {
            const float d = sdt[i], dec = sdec[i];
            total += slog[i];
            float xd[PPT], acc[PPT];
#pragma unroll
            for (int p = 0; p < PPT; ++p) {
                xd[p] = sx[i][PPT * pg + p] * d;
                acc[p] = 0.f;
            }
#pragma unroll
            for (int q = 0; q < NQ; ++q)
#pragma unroll
                for (int e = 0; e < W; ++e) {
                    const int nn = W * (nl + 8 * q) + e;
                    const float b = sB[i][nn], c = STATES ? 0.f : sC[i][nn];
#pragma unroll
                    for (int p = 0; p < PPT; ++p) {
                        S[p][q * W + e] = fmaf(S[p][q * W + e], dec, xd[p] * b);
                        if (!STATES) acc[p] = fmaf(S[p][q * W + e], c, acc[p]);
                    }
                }
            if (!STATES) {
#pragma unroll
                for (int p = 0; p < PPT; ++p) {
#pragma unroll
                    for (int o = 4; o > 0; o >>= 1) acc[p] += __shfl_xor_sync(0xffffffffu, acc[p], o);
                    if (nl == 0) sy[i][PPT * pg + p] = fmaf(Dh, sx[i][PPT * pg + p], acc[p]);
                }
            }
        };
        // only S ties a token to the one before: four at a time hide the loads and the reductions
        if (m == kTB) {
#pragma unroll 4
            for (int i = 0; i < kTB; ++i) token(i);
        } else {
            for (int i = 0; i < m; ++i) token(i);
        }
        if (!STATES) {
            __syncthreads();
            for (int i = tid; i < m * P; i += kThreads)
                y[(first + a.dir * (long long)(b0 + i / P)) * a.ldy + i % P] = from_f<T>(sy[i / P][i % P]);
        }
    }
    if (STATES) {
        const size_t v = (size_t)u * a.H + h;
        float *out = a.ws_state + v * PN;
        each([&](float &s, size_t o) { out[o] = s; });
        if (tid == 0) a.ws_decay[v] = total;
    } else if (last) {
        const int so = slot_of_end(a.slots, sg.s, a.seq.nseq, a.status);
        if (so >= 0) {
            float *out = static_cast<float *>(a.slots.pool_out) + ((size_t)so * a.H + h) * PN;
            each([&](float &s, size_t o) { out[o] = s; });
        }
    }
}

template <typename T, int P, int N> cudaError_t run_ragged(const RaggedArgs &a, cudaStream_t st) {
    if (a.states) k_ragged<T, P, N, true><<<dim3(a.states, a.H), kThreads, 0, st>>>(a);
    k_ragged<T, P, N, false><<<dim3(a.units, a.H), kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

template <typename T> cudaError_t pick(const RaggedArgs &a, cudaStream_t st) {
#define SSD_PN(P_, N_) if (a.P == P_ && a.N == N_) return run_ragged<T, P_, N_>(a, st)
    SSD_PN(16, 16); SSD_PN(16, 32); SSD_PN(16, 64); SSD_PN(16, 128);
    SSD_PN(32, 16); SSD_PN(32, 32); SSD_PN(32, 64); SSD_PN(32, 128);
    SSD_PN(64, 16); SSD_PN(64, 32); SSD_PN(64, 64); SSD_PN(64, 128);
#undef SSD_PN
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_ragged_simt(const RaggedArgs &a, bool bf16, cudaStream_t st) {
    return bf16 ? pick<__nv_bfloat16>(a, st) : pick<float>(a, st);
}

}  // namespace ssd
