// Layer norm and its RMS form over the rows of a readout (internal to libm2rnn.so).
#pragma once
#include <cuda_runtime.h>

#include <cstddef>

namespace m2rnn {

struct NormParams {
    int B, H, T, N;         // rows (b, h, t) of N values; plain rows: B = H = 1
    int x_fp32, y_fp32, dx_fp32;   // element types: fp32 or bf16 (dy has y's)
    int rms;                // no mean is subtracted
    float eps;
    const void* x;          // [B][H][T][N]
    const float* weight;    // [H][N], null = 1
    const float* bias;      // [H][N], null = 0
    void* y;                // [B][T][H][N]
    float* mean;            // [B][H][T]; forward output (may be null), backward input (null with rms)
    float* rstd;            // [B][H][T]
    // backward
    const void* dy;         // [B][T][H][N]
    void* dx;               // [B][H][T][N]
    float* dweight;         // [H][N], may be null
    float* dbias;           // [H][N], may be null
    float* part;            // [B*H][chunks][2][N] partial sums (workspace)
    int chunks;             // row blocks (CTAs) per (b, h)
};

cudaError_t launch_norm_fwd(const NormParams& p, cudaStream_t s);
cudaError_t launch_norm_bwd(const NormParams& p, cudaStream_t s);
// Column blocks of a head's [dweight | dbias]; those of all heads are at most 2^31 - 1.
__host__ __device__ inline unsigned norm_dw_blocks(int N) { return (2u * N + 31) / 32; }
// Row blocks per (b, h) of the backward: fixes the order of the weight gradient's sum.
int norm_bwd_chunks(int B, int H, int T, int N);

}  // namespace m2rnn
