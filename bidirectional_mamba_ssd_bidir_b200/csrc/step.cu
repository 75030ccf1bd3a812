// step.cu -- one token of the Mamba-2 layer per row, for decoding: the causal convolution with its
// carried inputs, SiLU, the dt softplus and one step of the recurrence, both states updated in place.
//
//   v   = silu(conv_b + sum_k conv_w[:, k] [conv_state | xBC]_k)       x | B | C = v
//   d   = softplus(dt + dt_bias)
//   S  <- exp(d A) S + d x (outer) B,      y = C S + D x
//
// The float32 state is read once and written once (8 P N bytes a head), which is all but a percent of
// the bytes: HBM bounds a full batch, the two launches' latency a single row.  B and C belong to all
// heads of a group, and the convolution's own state may only be shifted after every head has read it,
// so the convolution is a kernel of its own (k_step_conv: each channel is owned by one thread).  The
// recurrence (k_step_state) is launched behind it with programmatic dependent launch: its CTAs start
// at once and have their states on the way into registers before they wait for the convolution.
// Measured (64 heads, headdim 64, d_state 128): 96 rows 75.7 us, 5.4 TB/s, 0.84 of the copy rate; one row
// 6.8 us on the device.
#include "ragged.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 128;

// The row's slot, or -1 where the row has nothing to do: a negative slot (padding), one past the
// pool, or one that another row names too (neither of them is updated).  Called by the whole CTA.
__device__ __forceinline__ int row_slot(const StepArgs &a, int r) {
    const int v = a.slots ? a.slots[r] : r;
    if (v < 0) return -1;
    if (v >= a.n_slots) {
        report(a.status, kCodeSlotRange);
        return -1;
    }
    if (!a.slots) return v;
    bool twice = false;
    for (int j = threadIdx.x; j < a.rows; j += blockDim.x) twice |= j != r && a.slots[j] == v;
    if (__syncthreads_or(twice)) {
        report(a.status, kCodeSlotTwice);
        return -1;
    }
    return v;
}

// One thread per channel; K - 1 rows of the state, all loads before the first store.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_step_conv(const __grid_constant__ StepArgs a) {
    const int r = blockIdx.x, c = blockIdx.y * kThreads + threadIdx.x, K = a.K;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int slot = row_slot(a, r);
    float *v = a.v + (long long)r * (a.C + 4);
    if (blockIdx.y == 0 && threadIdx.x == 0) v[a.C] = __int_as_float(slot);
    if (slot < 0 || c >= a.C) return;
    T *st = static_cast<T *>(a.conv_state) + (long long)slot * (K - 1) * a.C + c;
    const T now = static_cast<const T *>(a.xBC)[(long long)r * a.ldx + c];
    T old[7];
#pragma unroll
    for (int k = 0; k < 7; ++k)
        if (k < K - 1) old[k] = st[(long long)k * a.C];
    float s[1] = {a.conv_b ? a.conv_b[c] : 0.f}, sg[1];
    const float *w = a.conv_w + (long long)c * K;
#pragma unroll
    for (int k = 0; k < 7; ++k)
        if (k < K - 1) s[0] = fmaf(w[k], to_f<T>(old[k]), s[0]);
    s[0] = fmaf(w[K - 1], to_f<T>(now), s[0]);
    sigmoids<1>(s, sg);
    v[c] = s[0] * sg[0];
#pragma unroll
    for (int k = 1; k < 7; ++k)
        if (k < K - 1) st[(long long)(k - 1) * a.C] = old[k];
    if (K > 1) st[(long long)(K - 2) * a.C] = now;
}

// One CTA per (row, head, part of P): PB rows of the head's state, N / 4 lanes of four columns
// each.  Every thread has its PB N / 512 chunks of 16 bytes in flight before it waits.
template <int N, int PB> constexpr int step_threads() { return PB * N / 4 < kThreads ? PB * N / 4 : kThreads; }

template <typename T, int N, int PB>
__global__ void __launch_bounds__(kThreads) k_step_state(const __grid_constant__ StepArgs a) {
    constexpr int NL = N / 4, PG = step_threads<N, PB>() / NL, U = PB / PG;   // lanes of a state row, rows at a time, chunks
    static_assert(U >= 1 && PG * U == PB, "");
    const int r = blockIdx.y, parts = a.P / PB, h = blockIdx.x / parts, p0 = (blockIdx.x % parts) * PB;
    const int nl = threadIdx.x % NL, pg = threadIdx.x / NL;
    // the slot as the call gives it: a bounded address to load from; the convolution kernel decides
    // below whether the row counts
    int guess = a.slots ? a.slots[r] : r;
    guess = guess < 0 || guess >= a.n_slots ? 0 : guess;
    float4 *S = reinterpret_cast<float4 *>(a.ssm_state + (((long long)guess * a.H + h) * a.P + p0) * N) + nl;
    float4 s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) s[u] = __ldcs(S + (long long)(pg + PG * u) * NL);
    const float dtr = to_f<T>(static_cast<const T *>(a.dt)[(long long)r * a.lddt + h]) + (a.dt_bias ? a.dt_bias[h] : 0.f);
    const float d = softplus(dtr), dec = expf(d * a.A[h]), Dh = a.D ? a.D[h] : 0.f;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const float *v = a.v + (long long)r * (a.C + 4);
    if (__float_as_int(v[a.C]) < 0) return;
    const float *Bv = v + a.H * a.P + (h / (a.H / a.G)) * N, *Cv = Bv + a.G * N;
    const float4 B = *reinterpret_cast<const float4 *>(Bv + 4 * nl), C = *reinterpret_cast<const float4 *>(Cv + 4 * nl);
    T *y = static_cast<T *>(a.y) + (long long)r * a.ldy + h * a.P + p0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int p = pg + PG * u;
        const float x = v[h * a.P + p0 + p], xd = x * d;
        s[u].x = fmaf(s[u].x, dec, xd * B.x);
        s[u].y = fmaf(s[u].y, dec, xd * B.y);
        s[u].z = fmaf(s[u].z, dec, xd * B.z);
        s[u].w = fmaf(s[u].w, dec, xd * B.w);
        __stcs(S + (long long)p * NL, s[u]);
        float t = fmaf(s[u].x, C.x, s[u].y * C.y) + fmaf(s[u].z, C.z, s[u].w * C.w);
#pragma unroll
        for (int o = NL / 2; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o, NL);
        if (nl == 0) y[p] = from_f<T>(fmaf(Dh, x, t));
    }
}

template <typename T> cudaError_t run_step(const StepArgs &a, cudaStream_t st) {
    k_step_conv<T><<<dim3(a.rows, (a.C + kThreads - 1) / kThreads), kThreads, 0, st>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    auto go = [&](auto kernel, int pb, int threads) {
        cfg.blockDim = dim3(threads);
        cfg.gridDim = dim3(a.H * (a.P / pb), a.rows);
        return cudaLaunchKernelEx(&cfg, kernel, a);
    };
#define SSD_STEP(N_, P_) \
    if (a.N == N_ && a.P == P_) return go(k_step_state<T, N_, P_>, P_, step_threads<N_, P_>())
    SSD_STEP(16, 16); SSD_STEP(32, 16); SSD_STEP(64, 16); SSD_STEP(128, 16);
    SSD_STEP(16, 32); SSD_STEP(32, 32); SSD_STEP(64, 32); SSD_STEP(128, 32);
    SSD_STEP(16, 64); SSD_STEP(32, 64); SSD_STEP(64, 64); SSD_STEP(128, 64);
#undef SSD_STEP
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_step(const StepArgs &a, bool bf16, cudaStream_t st) {
    return bf16 ? run_step<__nv_bfloat16>(a, st) : run_step<float>(a, st);
}

}  // namespace ssd
