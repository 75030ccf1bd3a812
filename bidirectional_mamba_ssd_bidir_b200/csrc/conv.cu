// conv.cu -- the short depthwise causal convolution of the Mamba-2 layer as an operator of its own:
// packed ragged sequences, a carried state, both scan directions, and its gradients.
//
// In scan order (k = 0 first; token lo + k forward, hi - 1 - k in reverse), with width K and
// x_k for k < 0 the carried state (zero without one):
//
//   s_k  = b + sum_j w[K-1-j] x_{k-j}         j = 0 .. K-1
//   y_k  = silu(s_k)  (or s_k)
//
//   gs_k = gy_k silu'(s_k)                     silu' = sg (1 + s (1 - sg))
//   gx_k = sum_j w[K-1-j] gs_{k+j}             k + j inside the sequence
//   gw[K-1-j] = sum_k gs_k x_{k-j},  gb = sum_k gs_k
//
// Both passes move each element once.  Measured (bf16, 4352 channels, width 4): forward 16384 tokens 62 us,
// 4.6 TB/s, 0.71 of the copy rate; backward 16001 tokens 126 us, 3.3 TB/s, 0.51.  No unit is at its limit: a
// capture shows issue slots 53 and 49 % busy, ex2 and rcp's unit 56 and 29 %, and most stalls are for fixed
// latencies.  What is short is warps to hide them, 20 and 12 an SM (96 and 158 registers a thread), and whole
// waves: 3.2 and 2.6 of them.  Not faster: two channels a thread instead of four, more resident warps
// with 128 registers (backward 134 us), unpaired multiply-adds (66 and 131 us).
//
// A thread owns V = 4 neighbouring channels (1 where the channel count, a stride or an address does
// not allow 8- or 16-byte accesses) and walks a run of the packed rows with its taps and a sliding
// window of inputs in registers; the next rows are loaded before the present ones are computed.
// Runs are cut along the packed rows, not along the sequences: every CTA has the same work whatever
// the lengths are, and a sequence boundary inside a run only restarts the window.
#include "ragged.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 128;
constexpr int kRows = 8;          // rows loaded at a time
constexpr int kKMax = 8;

// Where a walk over packed rows is: the sequence of the present row and its bounds.
struct Walk {
    int s, lo, hi;                // sequence, its rows [lo, hi); s outside [0, nseq): no sequence
    __device__ __forceinline__ void set(const Packed &q, int i) {
        s = i;
        if (i >= 0 && i < q.nseq) {
            lo = seq_start(q, i);
            hi = max(lo, seq_start(q, i + 1));
        } else if (i < 0) {       // rows before the first sequence
            lo = 0;
            hi = seq_start(q, 0);
        } else {                  // rows behind the last
            lo = q.nseq > 0 ? seq_start(q, q.nseq) : 0;
            hi = q.tokens;
        }
    }
    // The same for a whole warp: one look at 32 starts at a time (the search above is a chain of loads,
    // and a run's first rows wait for it).
    __device__ __forceinline__ void find_warp(const Packed &q, int t) {
        if (!q.cu) {
            find(q, t);
            return;
        }
        const int lane = threadIdx.x & 31;
        int i = -1;
        for (int b = 0; b < q.nseq; b += 32) {
            const int n = __popc(__ballot_sync(0xffffffffu, b + lane < q.nseq && seq_start(q, b + lane) <= t));
            i += n;
            if (n < 32) break;
        }
        set(q, i);
        if (s >= 0 && t >= hi) set(q, q.nseq);
    }
    // the sequence of row t; rows in none get an index outside [0, nseq)
    __device__ __forceinline__ void find(const Packed &q, int t) {
        set(q, seq_find(q, t));
        if (s >= 0 && t >= hi) set(q, q.nseq);
    }
};

template <typename T, int V, int KM> __device__ __forceinline__ void load_taps(const ConvArgs &a, int K, int c0, float (&wr)[KM][V], float (&b)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
        b[v] = a.bias ? a.bias[c0 + v] : 0.f;
#pragma unroll
        for (int j = 0; j < KM; ++j) wr[j][v] = j < K ? a.w[(long long)(c0 + v) * K + (K - 1 - j)] : 0.f;
    }
}

// The per-sequence CTAs: everything that touches the state pools, so that reading a slot and
// writing it (in place, or another sequence's) stay inside one thread.  They compute the first
// K - 1 outputs of the sequence when it may start from a state, and store its last K - 1 inputs.
template <typename T, int V, int KT>
__device__ void conv_state(const ConvArgs &a, int s, int c0) {
    using R = typename Vec<T, V>::type;
    constexpr int KM = KT > 0 ? KT : kKMax;
    const int K = KT > 0 ? KT : a.K;
    const int si = slot_of_start(a.slots, s, a.status), so = slot_of_end(a.slots, s, a.seq.nseq, a.status);
    if (c0 >= a.C) return;
    const int lo = seq_start(a.seq, s), n = max(lo, seq_start(a.seq, s + 1)) - lo;
    const int first = a.dir > 0 ? lo : lo + n - 1;
    const T *x = static_cast<const T *>(a.x);
    auto row = [&](int k) { return *reinterpret_cast<const R *>(x + (long long)(first + a.dir * k) * a.ldx + c0); };
    R hist[KM > 1 ? KM - 1 : 1];          // the state's rows, oldest first
#pragma unroll
    for (int r = 0; r < KM - 1; ++r) {
        memset(&hist[r], 0, sizeof(R));
        if (r < K - 1 && si >= 0)
            hist[r] = *reinterpret_cast<const R *>(static_cast<const T *>(a.slots.pool_in) +
                                                   ((long long)si * (K - 1) + r) * a.C + c0);
    }
    // place p of the sequence with its history in front of it: row p of the state for p < K - 1
    auto at = [&](int p) {
        R v;
        memset(&v, 0, sizeof(R));
        if (p >= K - 1) return row(p - (K - 1));
#pragma unroll
        for (int r = 0; r < KM - 1; ++r)
            if (r == p) v = hist[r];
        return v;
    };
    if (a.slots.pool_in) {
        float wr[KM][V], b[V];
        load_taps<T, V, KM>(a, K, c0, wr, b);
        for (int k = 0; k < min(K - 1, n); ++k) {
            float acc[V];
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v] = b[v];
#pragma unroll
            for (int j = KM - 1; j >= 0; --j) {
                if (j >= K) continue;
                float f[V];
                unpack<T, V>(at(k - j + K - 1), f);
#pragma unroll
                for (int v = 0; v < V; ++v) acc[v] = fmaf(wr[j][v], f[v], acc[v]);
            }
            if (a.silu) {
                float sg[V];
                sigmoids<V>(acc, sg);
#pragma unroll
                for (int v = 0; v < V; ++v) acc[v] *= sg[v];
            }
            *reinterpret_cast<R *>(static_cast<T *>(a.y) + (long long)(first + a.dir * k) * a.ldy + c0) = pack<T, V>(acc);
        }
    }
    if (so >= 0) {
        R keep[KM > 1 ? KM - 1 : 1];
#pragma unroll
        for (int r = 0; r < KM - 1; ++r)
            if (r < K - 1) keep[r] = at(n + r);
#pragma unroll
        for (int r = 0; r < KM - 1; ++r)
            if (r < K - 1)
                *reinterpret_cast<R *>(static_cast<T *>(a.slots.pool_out) + ((long long)so * (K - 1) + r) * a.C + c0) =
                    keep[r];
    }
}

template <typename T, int V, int KT>
__global__ void __launch_bounds__(kThreads) k_conv(const __grid_constant__ ConvArgs a) {
    using R = typename Vec<T, V>::type;
    constexpr int KM = KT > 0 ? KT : kKMax;
    const int K = KT > 0 ? KT : a.K;
    const int unit = blockIdx.x / a.cblocks, c0 = ((blockIdx.x % a.cblocks) * kThreads + threadIdx.x) * V;
    if (blockIdx.x == 0) check_offsets(a.seq, a.status);
    if (unit >= a.units) {
        conv_state<T, V, KT>(a, unit - a.units, c0);
        return;
    }
    const bool live = c0 < a.C;                      // (a whole warp is needed to find the sequence)
    const int u0 = unit * a.run, n = min(a.run, a.seq.tokens - u0);
    const int first = a.dir > 0 ? u0 : u0 + n - 1;
    const T *xc = static_cast<const T *>(a.x) + (long long)first * a.ldx + c0;
    T *yc = static_cast<T *>(a.y) + (long long)first * a.ldy + c0;
    const long long sx = a.dir * a.ldx, sy = a.dir * a.ldy;
    // everything the first rows need is asked for at once: rows, the rows before them, taps, offsets
    R next[kRows], back[KM > 1 ? KM - 1 : 1];
    float wr[KM][V], b[V], win[KM][V];
    if (live) {
#pragma unroll
        for (int i = 0; i < kRows; ++i)
            if (i < n) next[i] = *reinterpret_cast<const R *>(xc + i * sx);
        const int behind = a.dir > 0 ? first : a.seq.tokens - 1 - first;
#pragma unroll
        for (int j = 0; j < KM - 1; ++j) back[j] = *reinterpret_cast<const R *>(xc - min(j + 1, behind) * sx);
        load_taps<T, V, KM>(a, K, c0, wr, b);
    }
    Walk w;
    w.find_warp(a.seq, first);
    if (!live) return;
    // k: the present row's place in its sequence, in scan order; left: rows of the sequence from it on
    int k = a.dir > 0 ? first - w.lo : w.hi - 1 - first, left = a.dir > 0 ? w.hi - first : first - w.lo + 1;
#pragma unroll
    for (int j = 0; j < KM; ++j) {
#pragma unroll
        for (int v = 0; v < V; ++v) win[j][v] = 0.f;
        // before its first shift the window holds the row j + 1 steps back
        if (j < KM - 1 && j < K - 1 && k > j) unpack<T, V>(back[j < KM - 1 ? j : 0], win[j]);
    }
    const int skip = a.slots.pool_in ? K - 1 : 0;   // those outputs belong to the per-sequence CTAs
    // the next row into the window, and its output
    auto step = [&](const R &in, R &out) {
#pragma unroll
        for (int j = KM - 1; j > 0; --j)
#pragma unroll
            for (int v = 0; v < V; ++v) win[j][v] = win[j - 1][v];
        unpack<T, V>(in, win[0]);
        float acc[V];
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = b[v];
#pragma unroll
        for (int j = KM - 1; j >= 0; --j) {
            if (KT == 0 && j >= K) continue;
            fma_v<V>(wr[j], win[j], acc);
        }
        if (a.silu) {
            float sg[V];
            sigmoids<V>(acc, sg);
            mul_v<V>(acc, sg, acc);
        }
        out = pack<T, V>(acc);
    };
    for (int i0 = 0; i0 < n; i0 += kRows) {
        R cur[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) cur[i] = next[i];
#pragma unroll
        for (int i = 0; i < kRows; ++i)
            if (i0 + kRows + i < n) next[i] = *reinterpret_cast<const R *>(xc + (i0 + kRows + i) * sx);
        // eight rows of one sequence, none of them the per-sequence CTAs' (the same for all threads)
        if (i0 + kRows <= n && left >= kRows && k >= skip && w.s >= 0 && w.s < a.seq.nseq) {
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                R out;
                step(cur[i], out);
                *reinterpret_cast<R *>(yc + (i0 + i) * sy) = out;
            }
            k += kRows;
            left -= kRows;
            continue;
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            if (i0 + i >= n) break;
            if (left == 0) {                        // a sequence starts here (the same for all threads)
                w.find(a.seq, first + a.dir * (i0 + i));
                k = 0;
                left = w.hi - w.lo;
#pragma unroll
                for (int j = 0; j < KM; ++j)
#pragma unroll
                    for (int v = 0; v < V; ++v) win[j][v] = 0.f;
            }
            R out;
            step(cur[i], out);
            if (k >= skip && w.s >= 0 && w.s < a.seq.nseq) *reinterpret_cast<R *>(yc + (i0 + i) * sy) = out;
            ++k;
            --left;
        }
    }
}

// ------------------------------------------------------------------ gradients

// One walk per run in scan order.  Step tau computes gs of its row and gx of the row K - 1 steps
// behind it, so a run of n rows takes n + K - 1 steps: the last ones only complete the gx of the
// run's own last rows.  A sequence's last K - 1 rows are completed with the zeros behind its end.
// gw and gb: sums over the run's own rows in registers, one partial row per run, added up by
// k_conv_sum in the order of the runs (no atomics, so the result does not depend on timing).
template <typename T, int V, int KT>
__global__ void __launch_bounds__(kThreads) k_conv_bwd(const __grid_constant__ ConvArgs a) {
    using R = typename Vec<T, V>::type;
    constexpr int KM = KT > 0 ? KT : kKMax;
    const int K = KT > 0 ? KT : a.K;
    const int unit = blockIdx.x / a.cblocks, c0 = ((blockIdx.x % a.cblocks) * kThreads + threadIdx.x) * V;
    if (blockIdx.x == 0) check_offsets(a.seq, a.status);
    const bool live = c0 < a.C;
    const int u0 = unit * a.run, n = min(a.run, a.seq.tokens - u0);
    const int first = a.dir > 0 ? u0 : u0 + n - 1;
    const int room = a.dir > 0 ? a.seq.tokens - first : first + 1;   // rows from `first` on, in scan order
    const int steps = min(n + K - 1, room);                          // steps that read a row
    const T *xc = static_cast<const T *>(a.x) + (long long)first * a.ldx + c0;
    const T *gc = static_cast<const T *>(a.gy) + (long long)first * a.ldg + c0;
    T *yc = static_cast<T *>(a.y) + (long long)first * a.ldy + c0;
    const long long sx = a.dir * a.ldx, sg_ = a.dir * a.ldg, sy = a.dir * a.ldy;
    constexpr int U = 4;
    R nx[U], ng[U], back[KM > 1 ? KM - 1 : 1];
    float wr[KM][V], b[V], win[KM][V], gs[KM][V], gw[KM][V], gb[V];
    if (live) {
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (i < steps) {
                nx[i] = *reinterpret_cast<const R *>(xc + i * sx);
                ng[i] = *reinterpret_cast<const R *>(gc + i * sg_);
            }
        const int behind = a.dir > 0 ? first : a.seq.tokens - 1 - first;
#pragma unroll
        for (int j = 0; j < KM - 1; ++j) back[j] = *reinterpret_cast<const R *>(xc - min(j + 1, behind) * sx);
        load_taps<T, V, KM>(a, K, c0, wr, b);
    }
    Walk w;
    w.find_warp(a.seq, first);
    if (!live) return;
    int k = a.dir > 0 ? first - w.lo : w.hi - 1 - first, left = a.dir > 0 ? w.hi - first : first - w.lo + 1;
#pragma unroll
    for (int j = 0; j < KM; ++j) {
#pragma unroll
        for (int v = 0; v < V; ++v) win[j][v] = gs[j][v] = gw[j][v] = 0.f;
        if (j < KM - 1 && j < K - 1 && k > j) unpack<T, V>(back[j < KM - 1 ? j : 0], win[j]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) gb[v] = 0.f;
    // place[j]: place in its sequence of the row j steps back (-1: in none)
    int place[KM];
#pragma unroll
    for (int j = 0; j < KM; ++j) place[j] = -1;
    bool inseq = w.s >= 0 && w.s < a.seq.nseq;
    // gs of the row in win[0]
    auto grad = [&](const R &gin, float (&g)[V]) {
        unpack<T, V>(gin, g);
        if (a.silu) {
            float s[V], sg[V];
#pragma unroll
            for (int v = 0; v < V; ++v) s[v] = b[v];
#pragma unroll
            for (int j = KM - 1; j >= 0; --j) {
                if (KT == 0 && j >= K) continue;
                fma_v<V>(wr[j], win[j], s);
            }
            sigmoids<V>(s, sg);
            // sg (1 + s (1 - sg)) = sg + t (1 - sg), t = s sg
            float t[V], d[V];
            mul_v<V>(s, sg, t);
#pragma unroll
            for (int v = 0; v < V; ++v) d[v] = 1.f - sg[v];
            fma_v<V>(t, d, sg, d);
            mul_v<V>(g, d, g);
        }
    };
    auto shift = [&]() {
#pragma unroll
        for (int j = KM - 1; j > 0; --j)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                win[j][v] = win[j - 1][v];
                gs[j][v] = gs[j - 1][v];
            }
    };
    auto sums = [&]() {                              // gw and gb of the row in win[0], gs[0]
        add_v<V>(gb, gs[0], gb);
#pragma unroll
        for (int j = 0; j < KM; ++j) {
            if (KT == 0 && j >= K) continue;
            fma_v<V>(gs[0], win[j], gw[j]);
        }
    };
    for (int i0 = 0; i0 < n + K - 1; i0 += U) {
        R cx[U], cg[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            cx[i] = nx[i];
            cg[i] = ng[i];
        }
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (i0 + U + i < steps) {
                nx[i] = *reinterpret_cast<const R *>(xc + (i0 + U + i) * sx);
                ng[i] = *reinterpret_cast<const R *>(gc + (i0 + U + i) * sg_);
            }
        // rows of one sequence, K - 1 rows into it and into the run (the same for all threads)
        if (KT > 0 && i0 >= K - 1 && i0 + U <= n && left >= U && k >= K - 1 && inseq) {
#pragma unroll
            for (int i = 0; i < U; ++i) {
                shift();
                unpack<T, V>(cx[i], win[0]);
                grad(cg[i], gs[0]);
                sums();
                float gx[V];
#pragma unroll
                for (int v = 0; v < V; ++v) gx[v] = 0.f;
                // entry j of gs is K - 1 - j rows ahead of the row K - 1 back
#pragma unroll
                for (int j = 0; j < KM; ++j) fma_v<V>(wr[KM - 1 - j], gs[j], gx);
                *reinterpret_cast<R *>(yc + (i0 + i - (K - 1)) * sy) = pack<T, V>(gx);
            }
            k += U;
            left -= U;
#pragma unroll
            for (int j = 0; j < KM; ++j) place[j] = k - 1 - j;
            continue;
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int tau = i0 + i;
            if (tau >= n + K - 1) break;
            shift();
#pragma unroll
            for (int j = KM - 1; j > 0; --j) place[j] = place[j - 1];
            if (tau < steps) {
                if (left == 0) {
                    w.find(a.seq, first + a.dir * tau);
                    inseq = w.s >= 0 && w.s < a.seq.nseq;
                    k = 0;
                    left = w.hi - w.lo;
#pragma unroll
                    for (int j = 0; j < KM; ++j)
#pragma unroll
                        for (int v = 0; v < V; ++v) win[j][v] = 0.f;
                }
                unpack<T, V>(cx[i], win[0]);
                grad(cg[i], gs[0]);
                place[0] = inseq ? k : -1;
                if (!inseq)
#pragma unroll
                    for (int v = 0; v < V; ++v) gs[0][v] = 0.f;
                if (inseq && tau < n) sums();
                ++k;
                --left;
            } else {
                place[0] = -1;
#pragma unroll
                for (int v = 0; v < V; ++v) gs[0][v] = 0.f;
            }
            // gx of the row K - 1 steps back: entry j of the window is its own sequence's row
            // (K - 1 - j) steps further on exactly when its place is larger by that much
            if (tau >= K - 1) {
                float gx[V];
#pragma unroll
                for (int v = 0; v < V; ++v) gx[v] = 0.f;
                int p0 = -1;
#pragma unroll
                for (int j = 0; j < KM; ++j)
                    if (j == K - 1) p0 = place[j];
#pragma unroll
                for (int j = 0; j < KM; ++j) {
                    if (j >= K || place[j] != p0 + (K - 1 - j)) continue;
#pragma unroll
                    for (int q = 0; q < KM; ++q)
                        if (q == K - 1 - j) fma_v<V>(wr[q], gs[j], gx);
                }
                // a row in no sequence has gradient zero
                if (p0 < 0)
#pragma unroll
                    for (int v = 0; v < V; ++v) gx[v] = 0.f;
                *reinterpret_cast<R *>(yc + (tau - (K - 1)) * sy) = pack<T, V>(gx);
            }
        }
    }
    float *part = a.part + (long long)unit * (K + 1) * a.C + c0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int j = 0; j < KM; ++j)
            if (j < K) part[(long long)(K - 1 - j) * a.C + v] = gw[j][v];
        part[(long long)K * a.C + v] = gb[v];
    }
}

// Adds the runs' partial sums: 32 columns (tap or bias, channel) a CTA, every eighth run a warp, the
// warps' sums joined in their order.
constexpr int kSumThreads = 256;
__global__ void __launch_bounds__(kSumThreads) k_conv_sum(const __grid_constant__ ConvArgs a) {
    __shared__ float part[kSumThreads / 32][32];
    const int K = a.K, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long i = (long long)blockIdx.x * 32 + lane, cols = (long long)(K + 1) * a.C;
    float s = 0.f;
    if (i < cols) {
#pragma unroll 4
        for (int u = warp; u < a.units; u += kSumThreads / 32) s += a.part[u * cols + i];
    }
    part[warp][lane] = s;
    __syncthreads();
    if (warp > 0 || i >= cols) return;
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < kSumThreads / 32; ++w) t += part[w][lane];
    const int k = (int)(i / a.C), c = (int)(i % a.C);
    if (k < K) a.gw[(long long)c * K + k] = t;
    else if (a.gb) a.gb[c] = t;
}

template <typename T, bool BWD> cudaError_t run_conv(ConvArgs a, bool vec, cudaStream_t st) {
    const int V = vec ? 4 : 1;
    const int rows = BWD ? a.units : a.units + (a.slots.pool_in || a.slots.pool_out ? a.seq.nseq : 0);
    if (rows == 0) return cudaSuccess;
    a.cblocks = (a.C + V * kThreads - 1) / (V * kThreads);
    if ((long long)a.cblocks * rows > 0x7fffffffLL) return cudaErrorInvalidValue;
    const unsigned grid = (unsigned)(a.cblocks * rows);
    auto go = [&](auto kernel) {
        kernel<<<grid, kThreads, 0, st>>>(a);
        return cudaGetLastError();
    };
#define SSD_CONV(KT)                                                                     \
    if constexpr (BWD) return vec ? go(k_conv_bwd<T, 4, KT>) : go(k_conv_bwd<T, 1, KT>); \
    else return vec ? go(k_conv<T, 4, KT>) : go(k_conv<T, 1, KT>)
    switch (a.K) {
        case 2: SSD_CONV(2);
        case 3: SSD_CONV(3);
        case 4: SSD_CONV(4);
        default: SSD_CONV(0);
    }
#undef SSD_CONV
}

bool vec_ok(const ConvArgs &a, int es) {
    const uintptr_t m = 4 * es - 1;
    auto ok = [&](const void *p, long long ld) { return (reinterpret_cast<uintptr_t>(p) & m) == 0 && ld % 4 == 0; };
    return a.C % 4 == 0 && ok(a.x, a.ldx) && ok(a.y, a.ldy) && ok(a.gy, a.ldg) && ok(a.slots.pool_in, a.C) &&
           ok(a.slots.pool_out, a.C);
}

// Rows of a run.  Long ones read fewer rows twice and set up less often; where that leaves SMs idle the
// run is halved until there are two CTAs an SM or 8 rows (143 rows x 320 channels: 64 rows 8.9 us, 8 rows
// 3.3 us).  The backward pass keeps one length: its workspace holds a row of sums per run.
constexpr int kRunFwd = 64, kRunMin = 8, kRunBwd = 128;

}  // namespace

cudaError_t launch_conv(ConvArgs a, bool bf16, cudaStream_t st) {
    a.gy = nullptr;
    a.ldg = 0;
    const long long blocks = (a.C + 4 * kThreads - 1) / (4 * kThreads);
    a.run = kRunFwd;
    while (a.run > kRunMin && (a.seq.tokens + a.run - 1) / a.run * blocks < 2 * 148) a.run /= 2;
    a.units = (a.seq.tokens + a.run - 1) / a.run;
    return bf16 ? run_conv<__nv_bfloat16, false>(a, vec_ok(a, 2), st) : run_conv<float, false>(a, vec_ok(a, 4), st);
}

size_t conv_bwd_partial_floats(long long tokens, int C, int K) {
    return (size_t)((tokens + kRunBwd - 1) / kRunBwd) * (K + 1) * C;
}

cudaError_t launch_conv_bwd(ConvArgs a, bool bf16, cudaStream_t st) {
    a.run = kRunBwd;
    a.units = (a.seq.tokens + a.run - 1) / a.run;
    cudaError_t e = bf16 ? run_conv<__nv_bfloat16, true>(a, vec_ok(a, 2), st) : run_conv<float, true>(a, vec_ok(a, 4), st);
    if (e != cudaSuccess) return e;
    const long long cols = (long long)(a.K + 1) * a.C;
    k_conv_sum<<<(unsigned)((cols + 31) / 32), kSumThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace ssd
