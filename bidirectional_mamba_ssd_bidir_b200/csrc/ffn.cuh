// ffn.cuh -- launch interface of the gated feed-forward block (ffn.cu).
#pragma once

#include <cuda_runtime.h>

namespace ssd {

// T tokens, d_model D, d_ff F, all bf16 row-major and contiguous:
//   u, out, gy, gu_ [T][D];  W_in, gW_in [2F][D] (gate rows, then up rows);  W_out, gW_out [D][F]
//   gu [T][2F] the saved projections;  h [T][F] and ggu [T][2F] scratch
struct FfnArgs {
    int T, D, F, gelu;
    const void *u, *W_in, *W_out;
    void *out, *h;
    void *gu;                      // forward: written when not null; backward: read
    const void *gy;
    void *ggu, *gu_, *gW_in, *gW_out;
    int *status;
    long long wait_cycles;
};
bool ffn_supported();
cudaError_t launch_ffn(const FfnArgs &a, cudaStream_t st);
cudaError_t launch_ffn_bwd(const FfnArgs &a, cudaStream_t st);

}  // namespace ssd
