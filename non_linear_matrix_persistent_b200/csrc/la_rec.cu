// Linear attention token by token on the CUDA cores: S = f S + k vᵀ, y = Sᵀ q.
//
// One CTA owns a slice of VS state columns of one (b, h) pair: columns are
// independent (the update and the readout never mix them), so the state is
// spread over as many CTAs as it has slices and no partial readout leaves a
// CTA.  A thread holds R rows of 4 adjacent columns in registers; y_t is the
// sum over rows, first inside the warp (shuffles over its row groups), then
// over the warps through shared memory, in a fixed order.
//
// For T = 1 the state is read and written once, 8·K·V bytes a pair against
// 2·(2K + V) bytes of inputs, so the kernel is bound by HBM; the threads of a
// CTA have their whole slice in flight before the first use.  Measured: 2048
// pairs of 128 x 128, 270 MB, 50.8 us, 82% of the copy rate; 16 pairs of 64 x
// 64 2.1 us, a launch and two trips to memory.
#include "kernels.h"
#include "linear_attention.h"

namespace m2rnn {
namespace {

template <class IO, int K, int VS>
struct RecCfg {
    static constexpr int kLanes = VS / 4;                       // threads along the columns
    static constexpr int kThreads = K * kLanes < 256 ? K * kLanes : 256;
    static constexpr int kGroups = kThreads / kLanes;           // row groups
    static constexpr int R = K / kGroups;                       // rows per thread
    static constexpr int kWarps = kThreads / 32;
};

template <class IO, int K, int VS>
__global__ void __launch_bounds__(RecCfg<IO, K, VS>::kThreads) m2rnn_la_rec_kernel(const LaParams p) {
    using C = RecCfg<IO, K, VS>;
    __shared__ float part[2][C::kWarps][VS];
    const int slices = p.V / VS;
    const int bh = blockIdx.x / slices, c0 = (blockIdx.x % slices) * VS;
    const int lane4 = threadIdx.x % C::kLanes, grp = threadIdx.x / C::kLanes;
    const int col = c0 + lane4 * 4;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const size_t qk = (size_t)la_qk_pair(p, bh) * p.T * K;
    const IO* k = static_cast<const IO*>(p.k) + qk;
    const IO* q = static_cast<const IO*>(p.q) + qk;
    const IO* v = static_cast<const IO*>(p.v) + (size_t)bh * p.T * p.V + col;
    IO* y = static_cast<IO*>(p.y) + (size_t)bh * p.T * p.V + c0;
    const size_t st = (size_t)bh * K * p.V + (size_t)grp * p.V + col;   // row grp + r·kGroups

    float4 S[C::R];
#pragma unroll
    for (int r = 0; r < C::R; ++r)
        S[r] = p.S0 ? *reinterpret_cast<const float4*>(p.S0 + st + (size_t)r * C::kGroups * p.V)
                    : make_float4(0.f, 0.f, 0.f, 0.f);

    const int nck = (p.T + kLaChunk - 1) / kLaChunk;
    for (int t = 0; t < p.T; ++t) {
        if (p.ckpt && t % kLaChunk == 0) {
            float* ck = p.ckpt + ((size_t)bh * nck + t / kLaChunk) * K * p.V + ((size_t)(col >> 2) * K + grp) * 4;
#pragma unroll
            for (int r = 0; r < C::R; ++r) *reinterpret_cast<float4*>(ck + r * C::kGroups * 4) = S[r];
        }
        const float f = la_gate(p, la_f_input(p, bh, t));
        float vv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) vv[i] = la_to_f32(v[(size_t)t * p.V + i]);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int r = 0; r < C::R; ++r) {
            const int row = grp + r * C::kGroups;
            const float kk = la_to_f32(k[(size_t)t * K + row]), qq = la_to_f32(q[(size_t)t * K + row]);
            S[r].x = fmaf(f, S[r].x, kk * vv[0]); S[r].y = fmaf(f, S[r].y, kk * vv[1]);
            S[r].z = fmaf(f, S[r].z, kk * vv[2]); S[r].w = fmaf(f, S[r].w, kk * vv[3]);
            o.x = fmaf(qq, S[r].x, o.x); o.y = fmaf(qq, S[r].y, o.y);
            o.z = fmaf(qq, S[r].z, o.z); o.w = fmaf(qq, S[r].w, o.w);
        }
#pragma unroll
        for (int d = C::kLanes; d < 32; d *= 2) {
            o.x += __shfl_xor_sync(~0u, o.x, d); o.y += __shfl_xor_sync(~0u, o.y, d);
            o.z += __shfl_xor_sync(~0u, o.z, d); o.w += __shfl_xor_sync(~0u, o.w, d);
        }
        float(&buf)[C::kWarps][VS] = part[t & 1];   // two buffers: one barrier a token
        if (lane < C::kLanes) *reinterpret_cast<float4*>(&buf[warp][lane * 4]) = o;
        __syncthreads();
        if (threadIdx.x < VS) {
            float s = buf[0][threadIdx.x];
#pragma unroll
            for (int w = 1; w < C::kWarps; ++w) s += buf[w][threadIdx.x];
            y[(size_t)t * p.V + threadIdx.x] = la_from_f32<IO>(s);
        }
    }
    if (p.ST) {
#pragma unroll
        for (int r = 0; r < C::R; ++r) *reinterpret_cast<float4*>(p.ST + st + (size_t)r * C::kGroups * p.V) = S[r];
    }
}

template <class IO, int K>
cudaError_t rec_v(const LaParams& p, cudaStream_t s) {
    const int pairs = p.B * p.H;
    if (p.V == 16)
        m2rnn_la_rec_kernel<IO, K, 16><<<pairs, RecCfg<IO, K, 16>::kThreads, 0, s>>>(p);
    else
        m2rnn_la_rec_kernel<IO, K, 32><<<pairs * (p.V / 32), RecCfg<IO, K, 32>::kThreads, 0, s>>>(p);
    return cudaGetLastError();
}
template <class IO>
cudaError_t rec_k(const LaParams& p, cudaStream_t s) {
    switch (p.K) {
        case 16: return rec_v<IO, 16>(p, s);
        case 32: return rec_v<IO, 32>(p, s);
        case 64: return rec_v<IO, 64>(p, s);
        case 128: return rec_v<IO, 128>(p, s);
    }
    return cudaErrorNotSupported;
}

// ------------------------------------------------------------------ backward
// fp32 on the CUDA cores (the debug mode), one CTA per (b, h) pair, walking blocks
// of kSub tokens from the last to the first with G = dL/dS at the block's end
// in shared memory.  Inside a block, with D_ts = f_{s+1}···f_t, a_t = f_1···f_t
// and b_s = D_{end,s} (all direct products, so a gate of exactly 0 is exact),
//   dq_t = a_t S dy_t + Σ_{s≤t} D_ts (dy_t·v_s) k_s
//   dk_s = b_s G v_s + Σ_{t≥s} D_ts (dy_t·v_s) q_t
//   dv_s = b_s Gᵀ k_s + Σ_{t≥s} D_ts (q_t·k_s) dy_t
//   df_u = Σ over sources s < u (S among them) and sinks t >= u (G among
//          them) of the path's product without f_u,
// where S is the state at the block's start, recomputed from the checkpoint.
constexpr int kSub = 16;
constexpr int kBwdThreads = 256;

__host__ __device__ inline size_t bwd_smem_floats(int K, int V) {
    return (size_t)2 * K * V + kSub * (4 * K + 2 * V) + 3 * kSub * (kSub + 1) + kSub + 64;
}

__global__ void __launch_bounds__(kBwdThreads) m2rnn_la_bwd_simt_kernel(const LaParams p) {
    extern __shared__ float sm[];
    const int K = p.K, V = p.V, tid = threadIdx.x, bh = blockIdx.x;
    float* S = sm;
    float* G = S + K * V;
    float* k = G + K * V;
    float* q = k + kSub * K;
    float* Sdy = q + kSub * K;      // [t][K]
    float* Gv = Sdy + kSub * K;     // [s][K]
    float* v = Gv + kSub * K;
    float* dy = v + kSub * V;
    float* QK = dy + kSub * V;      // [t][s]  q_t·k_s
    float* YV = QK + kSub * (kSub + 1);   // [t][s]  dy_t·v_s
    float* D = YV + kSub * (kSub + 1);    // [t][s]  s <= t
    float* f = D + kSub * (kSub + 1);
    float* red = f + kSub;
    const int ld = kSub + 1;
    const size_t qk0 = (size_t)la_qk_pair(p, bh) * p.T * K, vy0 = (size_t)bh * p.T * V, kq_out = (size_t)bh * p.T * K;
    const int nck = (p.T + kLaChunk - 1) / kLaChunk;
    for (int i = tid; i < K * V; i += kBwdThreads) G[i] = p.dST ? p.dST[(size_t)bh * K * V + i] : 0.f;

    for (int blk = (p.T + kSub - 1) / kSub - 1; blk >= 0; --blk) {
        const int t0 = blk * kSub, n = min(kSub, p.T - t0), c = t0 / kLaChunk;
        __syncthreads();
        // S at the block's start: the checkpoint advanced token by token
        for (int i = tid; i < K * V; i += kBwdThreads) {
            const int row = i / V, colv = i % V;
            float s = p.ckpt[((size_t)bh * nck + c) * K * V + ((colv >> 2) * K + row) * 4 + (colv & 3)];
            for (int t = c * kLaChunk; t < t0; ++t)
                s = fmaf(la_gate(p, la_f_input(p, bh, t)), s,
                         static_cast<const float*>(p.k)[qk0 + (size_t)t * K + row] *
                             static_cast<const float*>(p.v)[vy0 + (size_t)t * V + colv]);
            S[i] = s;
        }
        for (int i = tid; i < n * K; i += kBwdThreads) {
            k[i] = static_cast<const float*>(p.k)[qk0 + (size_t)t0 * K + i];
            q[i] = static_cast<const float*>(p.q)[qk0 + (size_t)t0 * K + i];
        }
        for (int i = tid; i < n * V; i += kBwdThreads) {
            v[i] = static_cast<const float*>(p.v)[vy0 + (size_t)t0 * V + i];
            dy[i] = static_cast<const float*>(p.dy)[vy0 + (size_t)t0 * V + i];
        }
        if (tid < n) f[tid] = la_gate(p, la_f_input(p, bh, t0 + tid));
        __syncthreads();
        {   // 16 x 16 products, one element a thread
            const int t = tid / kSub, s = tid % kSub;
            float a = 0.f, b = 0.f, d = 0.f;
            if (t < n && s <= t) {
                for (int i = 0; i < K; ++i) a = fmaf(q[t * K + i], k[s * K + i], a);
                for (int i = 0; i < V; ++i) b = fmaf(dy[t * V + i], v[s * V + i], b);
                d = 1.f;
                for (int u = s + 1; u <= t; ++u) d *= f[u];
            }
            QK[t * ld + s] = a; YV[t * ld + s] = b; D[t * ld + s] = d;
        }
        for (int e = tid; e < n * K; e += kBwdThreads) {
            const int t = e / K, i = e % K;
            float a = 0.f, b = 0.f;
            for (int j = 0; j < V; ++j) {
                a = fmaf(S[i * V + j], dy[t * V + j], a);
                b = fmaf(G[i * V + j], v[t * V + j], b);
            }
            Sdy[e] = a; Gv[e] = b;
        }
        // <S, G>, for the paths that cross the whole block
        float sg = 0.f;
        for (int i = tid; i < K * V; i += kBwdThreads) sg = fmaf(S[i], G[i], sg);
#pragma unroll
        for (int d = 16; d; d >>= 1) sg += __shfl_xor_sync(~0u, sg, d);
        if (tid % 32 == 0) red[tid / 32] = sg;
        __syncthreads();
        for (int e = tid; e < n * K; e += kBwdThreads) {
            const int t = e / K, i = e % K;
            float dq = Sdy[e] * (D[t * ld] * f[0]), dk = Gv[e] * D[(n - 1) * ld + t];
            for (int s = 0; s <= t; ++s) dq = fmaf(D[t * ld + s] * YV[t * ld + s], k[s * K + i], dq);
            for (int s = t; s < n; ++s) dk = fmaf(D[s * ld + t] * YV[s * ld + t], q[s * K + i], dk);
            static_cast<float*>(p.dq)[kq_out + (size_t)t0 * K + e] = dq;
            static_cast<float*>(p.dk)[kq_out + (size_t)t0 * K + e] = dk;
        }
        for (int e = tid; e < n * V; e += kBwdThreads) {
            const int s = e / V, j = e % V;
            float a = 0.f;
            for (int i = 0; i < K; ++i) a = fmaf(G[i * V + j], k[s * K + i], a);
            a *= D[(n - 1) * ld + s];
            for (int t = s; t < n; ++t) a = fmaf(D[t * ld + s] * QK[t * ld + s], dy[t * V + j], a);
            static_cast<float*>(p.dv)[vy0 + (size_t)t0 * V + e] = a;
        }
        if (tid < n) {
            const int u = tid;
            const float before = u > 0 ? D[(u - 1) * ld] * f[0] : 1.f;   // f_1···f_{u-1}, the block's start to u-1
            const float after = D[(n - 1) * ld + u];                      // u to the block's end
            float dot = 0.f;
            for (int w = 0; w < kBwdThreads / 32; ++w) dot += red[w];
            float d = before * after * dot;
            for (int t = u; t < n; ++t) {
                float sd = 0.f;
                for (int i = 0; i < K; ++i) sd = fmaf(q[t * K + i], Sdy[t * K + i], sd);
                float paths = before * sd;
                for (int s = 0; s < u; ++s) paths = fmaf(D[(u - 1) * ld + s] * QK[t * ld + s], YV[t * ld + s], paths);
                d = fmaf(D[t * ld + u], paths, d);
            }
            for (int s = 0; s < u; ++s) {
                float gd = 0.f;
                for (int i = 0; i < K; ++i) gd = fmaf(k[s * K + i], Gv[s * K + i], gd);
                d = fmaf(D[(u - 1) * ld + s] * after, gd, d);
            }
            // df/da = f (1 - f), with 1 - f = 1/(1 + e^a) free of cancellation for f near 1
            if (p.f_is_logit) d *= f[u] / (1.f + expf(la_f_input(p, bh, t0 + u)));
            p.df[(size_t)bh * p.T + t0 + u] = d;
        }
        __syncthreads();
        // G at the block's start
        const float A = D[(n - 1) * ld] * f[0];
        for (int i = tid; i < K * V; i += kBwdThreads) {
            const int row = i / V, colv = i % V;
            float g = A * G[i];
            for (int t = 0; t < n; ++t) g = fmaf(D[t * ld] * f[0] * q[t * K + row], dy[t * V + colv], g);
            G[i] = g;
        }
    }
    __syncthreads();
    for (int i = tid; i < K * V; i += kBwdThreads) p.dS0[(size_t)bh * K * V + i] = G[i];
}

// ------------------------------------------------------------------ sums
template <class O>
__global__ void m2rnn_la_group_sum_kernel(const float4* __restrict__ dk_part, const float4* __restrict__ dq_part, O* dk,
                                          O* dq, int B, int H, int G, size_t tk4) {
    const size_t per = (size_t)G * tk4, n = (size_t)B * per;
    const int hpg = H / G;
    for (size_t e = blockIdx.x * (size_t)blockDim.x + threadIdx.x; e < 2 * n; e += (size_t)gridDim.x * blockDim.x) {
        const bool second = e >= n;
        const size_t o = second ? e - n : e;
        const size_t b = o / per, rem = o % per, g = rem / tk4, r = rem % tk4;
        const float4* src = (second ? dq_part : dk_part) + (b * H + g * hpg) * tk4 + r;
        float4 s = src[0];
        for (int j = 1; j < hpg; ++j) {
            const float4 x = src[(size_t)j * tk4];
            s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
        }
        O* dst = (second ? dq : dk) + 4 * o;
        dst[0] = la_from_f32<O>(s.x); dst[1] = la_from_f32<O>(s.y);
        dst[2] = la_from_f32<O>(s.z); dst[3] = la_from_f32<O>(s.w);
    }
}

// One CTA per head; thread i sums tokens i, i + 1024, … of each batch row in
// ascending order, then a fixed tree over the threads.
__global__ void __launch_bounds__(1024) m2rnn_la_df_sum_kernel(const float* __restrict__ tok, float* df, int B, int H,
                                                               int T) {
    __shared__ float part[32];
    const int h = blockIdx.x;
    float s = 0.f;
    for (int b = 0; b < B; ++b)
        for (int t = threadIdx.x; t < T; t += 1024) s += tok[((size_t)b * H + h) * T + t];
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = s;
    __syncthreads();
    if (threadIdx.x < 32) {
        s = part[threadIdx.x];
#pragma unroll
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
        if (threadIdx.x == 0) df[h] = s;
    }
}

}  // namespace

cudaError_t launch_la_rec(const LaParams& p, cudaStream_t s) {
    return p.bf16 ? rec_k<__nv_bfloat16>(p, s) : rec_k<float>(p, s);
}

cudaError_t launch_la_bwd_simt(const LaParams& p, cudaStream_t s) {
    const size_t bytes = sizeof(float) * bwd_smem_floats(p.K, p.V);
    const cudaError_t e =
        cudaFuncSetAttribute(m2rnn_la_bwd_simt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    m2rnn_la_bwd_simt_kernel<<<p.B * p.H, kBwdThreads, bytes, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_la_group_sum(const LaParams& p, const float* dk_part, const float* dq_part, void* dk, void* dq,
                                cudaStream_t s) {
    const size_t tk4 = (size_t)p.T * p.K / 4, n = 2 * (size_t)p.B * p.G * tk4;
    if (n == 0) return cudaSuccess;
    const size_t want = (n + 255) / 256, cap = (size_t)kNumSMs * 8;
    const unsigned grid = (unsigned)(want < cap ? want : cap);
    const float4 *a = reinterpret_cast<const float4*>(dk_part), *b = reinterpret_cast<const float4*>(dq_part);
    if (p.bf16)
        m2rnn_la_group_sum_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(a, b, static_cast<__nv_bfloat16*>(dk),
                                                                     static_cast<__nv_bfloat16*>(dq), p.B, p.H, p.G, tk4);
    else
        m2rnn_la_group_sum_kernel<float><<<grid, 256, 0, s>>>(a, b, static_cast<float*>(dk), static_cast<float*>(dq),
                                                              p.B, p.H, p.G, tk4);
    return cudaGetLastError();
}

cudaError_t launch_la_df_sum(const LaParams& p, const float* df_tok, float* df, cudaStream_t s) {
    m2rnn_la_df_sum_kernel<<<p.H, 1024, 0, s>>>(df_tok, df, p.B, p.H, p.T);
    return cudaGetLastError();
}

}  // namespace m2rnn
