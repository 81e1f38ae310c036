// Linear attention with a decay for each head: launch parameters and the
// launchers of its kernels (internal to libm2rnn.so).
//
//   S_t = f_t S_{t-1} + k_t v_tᵀ,   y_t = S_tᵀ q_t        (S_t is K x V)
//
// the M²RNN recurrence without the transition S·W, the tanh and the factor (1 - f_t)
// in front of the input, and therefore associative: a chunk of tokens can be
// evaluated with matrix products.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace m2rnn {

// Tokens between the checkpointed states (and per chunk of the tensor-core kernels).
constexpr int kLaChunk = 128;

// The limit of a kernel's waits, and the status word that one which runs out sets.
struct LaLimit {
    uint64_t ns;
    unsigned slot;
};
// Status words: 0 is shared by captured calls and by streams beyond the others,
// which have one each.
constexpr unsigned kLaSlots = 256;

struct LaParams {
    int B, H, G, T, K, V;   // G: head groups of k and q (divides H)
    int bf16;               // k, v, q, dy, y, dk, dv, dq are bf16 (else fp32)
    int f_is_logit;         // f holds gate logits
    int f_per_head;         // f and df are [H]: one constant for each head
    const void *k, *v, *q;
    const float* f;
    const float* S0;        // forward: initial state, may be null
    void* y;
    float* ST;              // may be null; may alias S0
    float* ckpt;            // [B*H][ceil(T/128)][V/4][K][4]: S before token 128c; forward: output, may be null; backward: input
    // backward
    const void* dy;
    const float* dST;       // may be null
    void *dk, *dq;          // what the kernels write: the outputs, or (grouped) fp32 per-head partials
    void* dv;
    float* df;              // [B*H][T]: the output, or (f_per_head) per-token values in the workspace
    float* dS0;             // may alias dST
    int out32;              // y, or dq, dk and dv, start on 32 bytes
    int dkq_fp32;           // dk and dq are fp32 whatever the inputs' type (per-head partials)
    // tensor-core kernels: time segments
    int segs;               // CTAs along T for each (b, h)
    int seg_chunks;         // chunks of 128 tokens per segment
    float* seg_state;       // [B*H][segs][K][V] (workspace)
    LaLimit limit;
    int fault;              // injected fault (m2rnn_debug_set_fault), 0 = none
};

// Time segments of the tensor-core kernels: CTAs along T for each (b, h), and
// their length in chunks.
struct LaPlan {
    int segs, seg_chunks;
};

// Row block of k and q that pair bh = b·H + h reads.
__host__ __device__ __forceinline__ int la_qk_pair(const LaParams& p, int bh) {
    return (bh / p.H) * p.G + (bh % p.H) / (p.H / p.G);
}

#ifdef __CUDACC__
// The f input of token t of pair bh, and the gate that it stands for.
__device__ __forceinline__ float la_f_input(const LaParams& p, int bh, int t) {
    return p.f_per_head ? p.f[bh % p.H] : p.f[(size_t)bh * p.T + t];
}
__device__ __forceinline__ float la_gate(const LaParams& p, float x) {
    return p.f_is_logit ? 1.f / (1.f + expf(-x)) : x;
}
__device__ __forceinline__ float la_to_f32(float x) { return x; }
__device__ __forceinline__ float la_to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <class T>
__device__ __forceinline__ T la_from_f32(float x);
template <>
__device__ __forceinline__ float la_from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 la_from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
#endif

// Token-by-token forward on the CUDA cores, any T and both types: the decode
// step, short prompts and the fp32 mode.
cudaError_t launch_la_rec(const LaParams& p, cudaStream_t s);
// Chunked tensor-core forward (bf16): y, ST and the checkpoints.
cudaError_t launch_la_fwd_tc(const LaParams& p, cudaStream_t s);
LaPlan la_plan(int B, int H, int T, bool backward);
// Workspace of a plan: segment states and decays.
size_t la_seg_bytes(const LaPlan& plan, int B, int H, int K, int V);
// Reads status word `slot` of the file's kernels, and clears it if it is set.
cudaError_t la_fwd_tc_status(unsigned slot, unsigned* word, cudaStream_t s);
// Chunked tensor-core backward (bf16).
cudaError_t launch_la_bwd_tc(const LaParams& p, cudaStream_t s);
// dL/dS at the segments' ends, into p.seg_state.
cudaError_t launch_la_seg_grads(const LaParams& p, cudaStream_t s);
cudaError_t la_bwd_tc_status(unsigned slot, unsigned* word, cudaStream_t s);
// fp32 backward on the CUDA cores.
cudaError_t launch_la_bwd_simt(const LaParams& p, cudaStream_t s);
// dk, dq [B, G, T, K] (bf16 or fp32) = sums of fp32 per-head partials over each group's heads, ascending.
cudaError_t launch_la_group_sum(const LaParams& p, const float* dk_part, const float* dq_part, void* dk, void* dq,
                                cudaStream_t s);
// df [H] = sums of per-token df over the batch and time, in a fixed order.
cudaError_t launch_la_df_sum(const LaParams& p, const float* df_tok, float* df, cudaStream_t s);

}  // namespace m2rnn
