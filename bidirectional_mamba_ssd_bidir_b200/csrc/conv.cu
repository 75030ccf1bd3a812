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
// Both passes move each element once and do about ten operations on it, so HBM bounds them.  A
// thread owns V = 4 neighbouring channels (1 where the channel count, a stride or an address does
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
    if (c0 >= a.C) return;
    const int u0 = unit * a.run, n = min(a.run, a.seq.tokens - u0);
    const int first = a.dir > 0 ? u0 : u0 + n - 1;
    const T *xc = static_cast<const T *>(a.x) + (long long)first * a.ldx + c0;
    T *yc = static_cast<T *>(a.y) + (long long)first * a.ldy + c0;
    const long long sx = a.dir * a.ldx, sy = a.dir * a.ldy;
    R next[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
        if (i < n) next[i] = *reinterpret_cast<const R *>(xc + i * sx);
    Walk w;
    w.find(a.seq, first);
    float wr[KM][V], b[V], win[KM][V];
    load_taps<T, V, KM>(a, K, c0, wr, b);
    // k: the present row's place in its sequence, in scan order; left: rows of the sequence from it on
    int k = a.dir > 0 ? first - w.lo : w.hi - 1 - first, left = a.dir > 0 ? w.hi - first : first - w.lo + 1;
#pragma unroll
    for (int j = 0; j < KM; ++j) {
#pragma unroll
        for (int v = 0; v < V; ++v) win[j][v] = 0.f;
        // before its first shift the window holds the row j + 1 steps back
        if (j < K - 1 && k > j) unpack<T, V>(*reinterpret_cast<const R *>(xc - (j + 1) * sx), win[j]);
    }
    const int skip = a.slots.pool_in ? K - 1 : 0;   // those outputs belong to the per-sequence CTAs
    for (int i0 = 0; i0 < n; i0 += kRows) {
        R cur[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) cur[i] = next[i];
#pragma unroll
        for (int i = 0; i < kRows; ++i)
            if (i0 + kRows + i < n) next[i] = *reinterpret_cast<const R *>(xc + (i0 + kRows + i) * sx);
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
#pragma unroll
            for (int j = KM - 1; j > 0; --j)
#pragma unroll
                for (int v = 0; v < V; ++v) win[j][v] = win[j - 1][v];
            unpack<T, V>(cur[i], win[0]);
            float acc[V];
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v] = b[v];
#pragma unroll
            for (int j = KM - 1; j >= 0; --j) {
                if (KT == 0 && j >= K) continue;
#pragma unroll
                for (int v = 0; v < V; ++v) acc[v] = fmaf(wr[j][v], win[j][v], acc[v]);
            }
            if (a.silu) {
                float sg[V];
                sigmoids<V>(acc, sg);
#pragma unroll
                for (int v = 0; v < V; ++v) acc[v] *= sg[v];
            }
            if (k >= skip && w.s >= 0 && w.s < a.seq.nseq)
                *reinterpret_cast<R *>(yc + (i0 + i) * sy) = pack<T, V>(acc);
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
    if (c0 >= a.C) return;
    const int u0 = unit * a.run, n = min(a.run, a.seq.tokens - u0);
    const int first = a.dir > 0 ? u0 : u0 + n - 1;
    const int room = a.dir > 0 ? a.seq.tokens - first : first + 1;   // rows from `first` on, in scan order
    const int steps = min(n + K - 1, room);                          // steps that read a row
    const T *xc = static_cast<const T *>(a.x) + (long long)first * a.ldx + c0;
    const T *gc = static_cast<const T *>(a.gy) + (long long)first * a.ldg + c0;
    T *yc = static_cast<T *>(a.y) + (long long)first * a.ldy + c0;
    const long long sx = a.dir * a.ldx, sg_ = a.dir * a.ldg, sy = a.dir * a.ldy;
    constexpr int U = 4;
    R nx[U], ng[U];
#pragma unroll
    for (int i = 0; i < U; ++i)
        if (i < steps) {
            nx[i] = *reinterpret_cast<const R *>(xc + i * sx);
            ng[i] = *reinterpret_cast<const R *>(gc + i * sg_);
        }
    Walk w;
    w.find(a.seq, first);
    float wr[KM][V], b[V], win[KM][V], gs[KM][V], gw[KM][V], gb[V];
    load_taps<T, V, KM>(a, K, c0, wr, b);
    int k = a.dir > 0 ? first - w.lo : w.hi - 1 - first, left = a.dir > 0 ? w.hi - first : first - w.lo + 1;
#pragma unroll
    for (int j = 0; j < KM; ++j) {
#pragma unroll
        for (int v = 0; v < V; ++v) win[j][v] = gs[j][v] = gw[j][v] = 0.f;
        if (j < K - 1 && k > j) unpack<T, V>(*reinterpret_cast<const R *>(xc - (j + 1) * sx), win[j]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) gb[v] = 0.f;
    // place[j]: place in its sequence of the row j steps back (-1: in none)
    int place[KM];
#pragma unroll
    for (int j = 0; j < KM; ++j) place[j] = -1;
    bool inseq = w.s >= 0 && w.s < a.seq.nseq;
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
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int tau = i0 + i;
            if (tau >= n + K - 1) break;
#pragma unroll
            for (int j = KM - 1; j > 0; --j) {
                place[j] = place[j - 1];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    win[j][v] = win[j - 1][v];
                    gs[j][v] = gs[j - 1][v];
                }
            }
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
                float g[V];
                unpack<T, V>(cg[i], g);
                if (a.silu) {
                    float s[V], sg[V];
#pragma unroll
                    for (int v = 0; v < V; ++v) s[v] = b[v];
#pragma unroll
                    for (int j = KM - 1; j >= 0; --j) {
                        if (KT == 0 && j >= K) continue;
#pragma unroll
                        for (int v = 0; v < V; ++v) s[v] = fmaf(wr[j][v], win[j][v], s[v]);
                    }
                    sigmoids<V>(s, sg);
#pragma unroll
                    for (int v = 0; v < V; ++v) g[v] *= sg[v] * fmaf(s[v], 1.f - sg[v], 1.f);
                }
                place[0] = inseq ? k : -1;
                const bool sum = inseq && tau < n;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    gs[0][v] = inseq ? g[v] : 0.f;
                    if (sum) {
                        gb[v] += g[v];
#pragma unroll
                        for (int j = 0; j < KM; ++j) gw[j][v] = fmaf(g[v], win[j][v], gw[j][v]);
                    }
                }
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
                    if (j >= K) continue;
                    // (K - 1 - j) steps ahead of that row: tap wr[K - 1 - j]
                    const bool same = place[j] == p0 + (K - 1 - j);
                    if (same) {
#pragma unroll
                        for (int q = 0; q < KM; ++q)
                            if (q == K - 1 - j) {
#pragma unroll
                                for (int v = 0; v < V; ++v) gx[v] = fmaf(wr[q][v], gs[j][v], gx[v]);
                            }
                    }
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

// Adds the runs' partial sums: one thread per (tap or bias, channel), the runs in four interleaved
// sums that a fixed tree joins.
__global__ void __launch_bounds__(kThreads) k_conv_sum(const __grid_constant__ ConvArgs a) {
    const int K = a.K;
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x, cols = (long long)(K + 1) * a.C;
    if (i >= cols) return;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    int u = 0;
    for (; u + 4 <= a.units; u += 4)
#pragma unroll
        for (int q = 0; q < 4; ++q) s[q] += a.part[(u + q) * cols + i];
    for (; u < a.units; ++u) s[0] += a.part[u * cols + i];
    const float t = (s[0] + s[1]) + (s[2] + s[3]);
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

constexpr int kRunFwd = 64, kRunBwd = 128;

}  // namespace

cudaError_t launch_conv(ConvArgs a, bool bf16, cudaStream_t st) {
    a.run = kRunFwd;
    a.units = (a.seq.tokens + a.run - 1) / a.run;
    a.gy = nullptr;
    a.ldg = 0;
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
    k_conv_sum<<<(unsigned)((cols + kThreads - 1) / kThreads), kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace ssd
