// ragged.cuh -- what the kernels on packed ragged batches share: where a sequence lies in the
// packed rows, the state slots of a call, element types, and the launch interfaces of conv.cu,
// step.cu, ragged.cu and ragged_tc.cu.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cstring>

namespace ssd {

// Codes that the kernels on packed batches write into the status word when an index array does not
// hold what the call's contract says; the work concerned is skipped, nothing is read or written
// outside the buffers.  (Smaller codes are waits that gave up.)
constexpr int kCodeOffsets = 1001;    // cu_seqlens not ascending, or outside the packed rows
constexpr int kCodeSlotRange = 1002;  // a slot index past the pool
constexpr int kCodeSlotTwice = 1003;  // a slot that one sequence (or row) writes and another uses

// Sequences packed one after another: sequence i is rows [cu[i], cu[i+1]); cu == nullptr: each of
// the nseq sequences has `len` rows.
struct Packed {
    const int *cu;
    int nseq, tokens, len;
};

// The state slots of a call: sequence i starts from slot in[i] of pool_in (a negative index or no
// pool: from zero) and leaves its last state in slot out[i] of pool_out (negative: not stored).
// in/out == nullptr: slot i.
struct Slots {
    const void *pool_in;
    void *pool_out;
    const int *in, *out;
    int n_in, n_out;
};

struct ConvArgs {
    Packed seq;
    Slots slots;
    const void *x, *gy;
    void *y;                       // y, or gx in the backward pass
    long long ldx, ldy, ldg;       // row strides in elements
    const float *w, *bias;         // [C][K]; bias may be null
    int C, K, dir, silu;
    int run, units, cblocks;       // tokens a CTA walks, CTAs along the packed rows and along the channels
    int *status;                   // may be null
    float *part, *gw, *gb;         // backward: partial sums [units][K + 1][C]; gb may be null
};
cudaError_t launch_conv(ConvArgs a, bool bf16, cudaStream_t st);
cudaError_t launch_conv_bwd(ConvArgs a, bool bf16, cudaStream_t st);
size_t conv_bwd_partial_floats(long long tokens, int C, int K);

struct StepArgs {
    int rows, H, P, N, G, C, K;    // C = H P + 2 G N channels
    const void *xBC, *dt;
    long long ldx, lddt, ldy;
    const float *conv_w, *conv_b, *dt_bias, *A, *D;
    void *conv_state;              // [n_slots][K - 1][C]
    float *ssm_state;              // [n_slots][H][P][N]
    const int *slots;
    int n_slots;
    float *v;                      // [rows][C + 4]: the convolution's outputs, then the row's slot (or -1)
    void *y;
    int *status;
};
cudaError_t launch_step(const StepArgs &a, bool bf16, cudaStream_t st);

constexpr int kRaggedTable = 840;   // floats of a chunk and head's decay table (ragged_tc.cu)

struct RaggedArgs {
    Packed seq;
    Slots slots;                   // float32 pools [n][H][P][N]
    const void *x, *dt, *B, *C;
    long long ldx, lddt, ldB, ldC, ldy;
    const float *A, *D, *dt_bias;  // D, dt_bias may be null
    void *y;
    int H, P, N, G, dir;
    int seg, units;                // tokens of a segment (even), segments at most
    int states;                    // state numbers of the workspace (below); 0: no sequence has two segments
    float *ws_state, *ws_decay;    // [states][H][P][N] and [states][H]
    float *tables;                 // tensor-core form: [tokens / 128 + nseq][H][kRaggedTable]
    int *order;                    // its jobs, longest first, and scratch: 2 [units][H / 2] (null: as they are numbered)
    int *status;
    long long wait_cycles;
};
// Segment length for a call: whole tiles of `quant` tokens, as few as give about `ctas` CTAs.
inline int ragged_segment(long long tokens, long long ctas_per_segment, int quant, long long ctas) {
    long long s = (tokens * ctas_per_segment + ctas - 1) / ctas;
    s = (s + quant - 1) / quant * quant;
    return (int)(s < quant ? quant : s);
}
cudaError_t launch_ragged_simt(const RaggedArgs &a, bool bf16, cudaStream_t st);
// The tensor-core form (ragged_tc.cu); its segments are whole chunks of 128 tokens.
bool ragged_tc_supported(const RaggedArgs &a, bool bf16);
cudaError_t launch_ragged_tc(const RaggedArgs &a, cudaStream_t st);

#ifdef __CUDACC__
namespace {

__device__ __forceinline__ int seq_start(const Packed &s, int i) {
    if (!s.cu) return i * s.len;
    const int v = s.cu[i];
    return v < 0 ? 0 : (v > s.tokens ? s.tokens : v);
}

// The last sequence that starts at or before row t (-1: none).
__device__ __forceinline__ int seq_find(const Packed &s, int t) {
    if (!s.cu) return s.len > 0 ? min(t / s.len, s.nseq - 1) : -1;
    int lo = -1, hi = s.nseq;                 // start(lo) <= t < start(hi)
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (seq_start(s, m) <= t) lo = m;
        else hi = m;
    }
    return lo;
}

// Segment u of a call (ragged.cu): its sequence s (-1: none), which of the sequence's `count`
// segments it is, and the sequence's first row and length.  An empty sequence has one, empty, segment.
struct Segment {
    int s, k, count, lo, len;
};
// The last sequence i with before(start, i), which holds for a first part of them (-1: for none).
// Called by whole warps: 32 starts are looked at together, one step for up to 32 sequences and two for 1024
// (a search one by one is a chain of loads, and a kernel's first loads wait for it).
template <typename F> __device__ __forceinline__ int last_sequence(const Packed &q, F before) {
    const int lane = threadIdx.x & 31;
    int lo = 0;                               // those before `lo` have it, m more may
    for (int m = q.nseq; m > 0;) {
        const int st = (m + 31) / 32, at = lane * st;
        const int n = __popc(__ballot_sync(0xffffffffu, at < m && before(seq_start(q, lo + at), lo + at)));
        if (n == 0) break;
        const int skip = (n - 1) * st + 1;
        lo += skip;
        m = min(st - 1, m - skip);
    }
    return lo - 1;
}
__device__ __forceinline__ Segment segments_of(const Packed &q, int seg, int i) {
    Segment r{i, 0, 0, seq_start(q, i), 0};
    r.len = max(0, seq_start(q, i + 1) - r.lo);
    r.count = max(1, (r.len + seg - 1) / seg);
    return r;
}
__device__ __forceinline__ Segment find_segment(const Packed &q, int seg, int u) {
    const int i = last_sequence(q, [&](int start, int i) { return start / seg + i <= u; });
    if (i < 0) return Segment{-1, 0, 0, 0, 0};
    Segment r = segments_of(q, seg, i);
    r.k = u - (r.lo / seg + i);
    if (r.k < 0 || r.k >= r.count) r.s = -1;
    return r;
}

// States are kept between the launches for sequences of two or more segments alone: segment k of one that
// starts at row lo has state number lo / half + k, half = seg / 2.  The numbers of different sequences differ:
// with len > 2 half, ceil(len / seg) <= floor(len / half), and floor(lo / half) + floor(len / half) is at most the
// next sequence's first number.  So there are floor(tokens / half) numbers, however many sequences.
__device__ __forceinline__ int first_state(const Segment &s, int seg) { return s.lo / (seg / 2); }
// The segment of state number v (s = -1: none).  Row (v + 1) half - 1 is its sequence's: it is not before lo, as
// (lo / half + 1) half > lo, and at most lo + count half - 1 < lo + len.  Called by whole warps.
__device__ __forceinline__ Segment find_state(const Packed &q, int seg, int v) {
    const int half = seg / 2, t = (v + 1) * half - 1;
    const int i = last_sequence(q, [&](int start, int) { return start <= t; });
    if (i < 0) return Segment{-1, 0, 0, 0, 0};
    Segment r = segments_of(q, seg, i);
    r.k = v - r.lo / half;
    if (r.count < 2 || t >= r.lo + r.len || r.k < 0 || r.k >= r.count) r.s = -1;
    return r;
}

__device__ __forceinline__ void report(int *status, int code) {
    if (status) atomicCAS(status, 0, code);
}

// One CTA's look over cu_seqlens.
__device__ __forceinline__ void check_offsets(const Packed &s, int *status) {
    if (!s.cu || !status) return;
    bool bad = false;
    for (int i = threadIdx.x; i < s.nseq; i += blockDim.x)
        bad |= s.cu[i] < 0 || s.cu[i + 1] < s.cu[i] || s.cu[i + 1] > s.tokens;
    if (bad) report(status, kCodeOffsets);
}

// Slot that sequence i starts from (-1: zero state).
__device__ __forceinline__ int slot_of_start(const Slots &s, int i, int *status) {
    if (!s.pool_in) return -1;
    const int v = s.in ? s.in[i] : i;
    if (v >= s.n_in) {
        report(status, kCodeSlotRange);
        return -1;
    }
    return v < 0 ? -1 : v;
}
// Whether slot v, which sequence i is about to write, is another sequence's too: one that ends in it, or
// starts from it in the same pool (and might read it before or after).  Looked at by `step` threads.
__device__ __forceinline__ bool slot_shared(const Slots &s, int i, int nseq, int v, int first, int step) {
    const bool starts = s.in && s.pool_in == s.pool_out, from_own = !s.in && s.pool_in == s.pool_out;
    bool shared = from_own && v != i && v < nseq;
    if (!s.out && !starts) return shared;
    for (int j = first; j < nseq; j += step)
        shared |= j != i && ((s.out && s.out[j] == v) || (starts && s.in[j] == v));
    return shared;
}
// Slot that sequence i ends in (-1: not stored).  Called by every thread of the CTA: a slot that another
// sequence uses too is not stored.
__device__ __forceinline__ int slot_of_end(const Slots &s, int i, int nseq, int *status) {
    if (!s.pool_out) return -1;
    const int v = s.out ? s.out[i] : i;
    if (v < 0) return -1;
    if (v >= s.n_out) {
        report(status, kCodeSlotRange);
        return -1;
    }
    if (!s.out && (!s.in || s.pool_in != s.pool_out)) return v;
    if (__syncthreads_or(slot_shared(s, i, nseq, v, threadIdx.x, blockDim.x))) {
        report(status, kCodeSlotTwice);
        return -1;
    }
    return v;
}

// V consecutive elements as float32, and back (rounded to nearest even)
template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <typename T, int V> struct Vec;
template <> struct Vec<__nv_bfloat16, 4> { using type = uint2; };
template <> struct Vec<float, 4> { using type = uint4; };
template <> struct Vec<__nv_bfloat16, 1> { using type = __nv_bfloat16; };
template <> struct Vec<float, 1> { using type = float; };

template <typename T, int V>
__device__ __forceinline__ void unpack(const typename Vec<T, V>::type &r, float (&f)[V]) {
    T e[V];
    memcpy(e, &r, sizeof(r));
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = to_f<T>(e[i]);
}
template <typename T, int V>
__device__ __forceinline__ typename Vec<T, V>::type pack(const float (&f)[V]) {
    T e[V];
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = from_f<T>(f[i]);
    typename Vec<T, V>::type r;
    memcpy(&r, e, sizeof(r));
    return r;
}

__device__ __forceinline__ float softplus(float v) { return v > 20.f ? v : log1pf(expf(v)); }

__device__ __forceinline__ float ex2a(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcpa(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Pairs of float32 in one instruction (the packed forms of sm_100): a b + c, a b, a + b.
__device__ __forceinline__ void fma2_to(float &d0, float &d1, float a0, float a1, float b0, float b1, float c0, float c1) {
    asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
        "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
template <int V> __device__ __forceinline__ void fma_v(const float (&a)[V], const float (&b)[V], const float (&c)[V], float (&d)[V]) {
    if constexpr (V % 2 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 2) fma2_to(d[i], d[i + 1], a[i], a[i + 1], b[i], b[i + 1], c[i], c[i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] = fmaf(a[i], b[i], c[i]);
    }
}
// d += a b
template <int V> __device__ __forceinline__ void fma_v(const float (&a)[V], const float (&b)[V], float (&d)[V]) { fma_v<V>(a, b, d, d); }
template <int V> __device__ __forceinline__ void mul_v(const float (&a)[V], const float (&b)[V], float (&d)[V]) {
    if constexpr (V % 2 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 2)
            asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
                "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
                : "=f"(d[i]), "=f"(d[i + 1]) : "f"(a[i]), "f"(a[i + 1]), "f"(b[i]), "f"(b[i + 1]));
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] = a[i] * b[i];
    }
}
template <int V> __device__ __forceinline__ void add_v(const float (&a)[V], const float (&b)[V], float (&d)[V]) {
    if constexpr (V % 2 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 2)
            asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
                "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
                : "=f"(d[i]), "=f"(d[i + 1]) : "f"(a[i]), "f"(a[i + 1]), "f"(b[i]), "f"(b[i + 1]));
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] = a[i] + b[i];
    }
}

// sigma[i] = 1 / (1 + e^-v[i]), each from one ex2 and one rcp (approximations within 2 ulp, and the rounded
// argument of ex2 adds up to |v| ulp; results below 2^-126 flush to zero).  e^-v past the float range makes it 0, as it should be.
template <int V> __device__ __forceinline__ void sigmoids(const float (&v)[V], float (&sg)[V]) {
    float c[V], e[V];
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = -1.4426950408889634f;
    mul_v<V>(v, c, e);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        e[i] = ex2a(e[i]);
        c[i] = 1.f;
    }
    add_v<V>(e, c, e);
#pragma unroll
    for (int i = 0; i < V; ++i) sg[i] = rcpa(e[i]);
}

}  // namespace
#endif

}  // namespace ssd
