// Layer norm over rows of N values, forward and backward:
//   m = mean(x), r = 1/sqrt(mean((x - m)^2) + eps), n = (x - m) r, y = n w + b
//   g = dy w,  dx = r (g - mean(g) - n mean(g n)),  dw = Σ dy n,  db = Σ dy
// (the RMS form has m = 0 and no mean(g) term).  Everything is bound by HBM:
// x is read and y written once forward, x and dy read and dx written once
// backward.  A row's values stay in registers between the statistics and the
// output, so the variance is the two-pass one (exact for large means) at no
// extra traffic.
//
// Rows come as a head-first readout [B][H][T][N] and leave token-first
// [B][T][H][N], which is the transposition that the output projection needs;
// plain rows are the case B = H = 1.  A warp's rows are consecutive in x; in y
// each is a contiguous segment of N values, whole 32-byte sectors for N >= 16.
//
// The gradients of the weight and the bias are sums over rows: every thread
// keeps its columns' sums in registers over the rows of its CTA's block of one
// (b, h), the CTA's row groups are added through shared memory, and a second
// kernel adds the blocks in ascending order: no atomics, the same bits every
// time.
#include "kernels.h"
#include "layer_norm.h"

#include <cuda_bf16.h>

namespace m2rnn {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

template <int VEC>
__device__ __forceinline__ void load(const __nv_bfloat16* p, float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        const uint4 w = *reinterpret_cast<const uint4*>(p);
        v[0] = bf16lo_to_f32(w.x); v[1] = bf16hi_to_f32(w.x); v[2] = bf16lo_to_f32(w.y); v[3] = bf16hi_to_f32(w.y);
        v[4] = bf16lo_to_f32(w.z); v[5] = bf16hi_to_f32(w.z); v[6] = bf16lo_to_f32(w.w); v[7] = bf16hi_to_f32(w.w);
    } else {
        v[0] = __bfloat162float(*p);
    }
}
template <int VEC>
__device__ __forceinline__ void load(const float* p, float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        v[0] = *p;
    }
}
template <int VEC>
__device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        auto pack = [](float a, float b) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
            return *reinterpret_cast<const uint32_t*>(&h);
        };
        *reinterpret_cast<uint4*>(p) = make_uint4(pack(v[0], v[1]), pack(v[2], v[3]), pack(v[4], v[5]), pack(v[6], v[7]));
    } else {
        *p = __float2bfloat16_rn(v[0]);
    }
}
template <int VEC>
__device__ __forceinline__ void store(float* p, const float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *p = v[0];
    }
}

// Sum over the LPR threads of a row, the same value in each of them.  `buf`:
// a slot per warp, not the one of the previous call (for LPR > 32).
template <int LPR>
__device__ __forceinline__ float row_sum(float x, float* buf) {
#pragma unroll
    for (int d = (LPR < 32 ? LPR : 32) / 2; d; d >>= 1) x += __shfl_xor_sync(~0u, x, d);
    if constexpr (LPR > 32) {
        static_assert(LPR == kThreads, "a row takes part of a warp or the whole CTA");
        if (threadIdx.x % 32 == 0) buf[threadIdx.x / 32] = x;
        __syncthreads();
        x = buf[0];
#pragma unroll
        for (int w = 1; w < kThreads / 32; ++w) x += buf[w];
    }
    return x;
}

__device__ __forceinline__ size_t token_row(const NormParams& p, size_t r) {   // x's row (b, h, t) -> y's (b, t, h)
    if (p.H == 1) return r;
    const size_t bh = r / p.T, t = r % p.T;
    return ((bh / p.H) * p.T + t) * p.H + bh % p.H;
}

// LPR threads per row, CH groups of VEC values per thread: N <= LPR·VEC·CH.
template <class X, class Y, int VEC, int LPR, int CH>
__global__ void __launch_bounds__(kThreads) m2rnn_norm_fwd_kernel(const NormParams p) {
    __shared__ float buf[2][kThreads / 32];
    const int lane = threadIdx.x % LPR, N = p.N;
    const size_t rows = (size_t)p.B * p.H * p.T, step = (size_t)gridDim.x * (kThreads / LPR);
    const float inv = 1.f / (float)N;
    // every thread of a warp takes part in the shuffles: the loop bound is the CTA's
    for (size_t r0 = (size_t)blockIdx.x * (kThreads / LPR); r0 < rows; r0 += step) {
        const size_t r = r0 + threadIdx.x / LPR;
        const bool live = r < rows;
        const X* x = static_cast<const X*>(p.x) + (live ? r : 0) * N;
        float v[CH][VEC];
        float s = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int i = (c * LPR + lane) * VEC;
            if (live && i < N) {
                load<VEC>(x + i, v[c]);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[c][e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) s += v[c][e];
        }
        const float m = p.rms ? 0.f : row_sum<LPR>(s, buf[0]) * inv;
        s = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const bool in = (c * LPR + lane) * VEC < N;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                v[c][e] -= m;
                s = in ? fmaf(v[c][e], v[c][e], s) : s;
            }
        }
        const float rs = 1.f / sqrtf(row_sum<LPR>(s, buf[1]) * inv + p.eps);
        if constexpr (LPR > 32) __syncthreads();   // buf[] is free for the next row
        if (!live) continue;
        if (lane == 0) {
            if (p.mean && !p.rms) p.mean[r] = m;
            if (p.rstd) p.rstd[r] = rs;
        }
        const size_t wrow = (size_t)(p.H == 1 ? 0 : (r / p.T) % p.H) * N;
        Y* y = static_cast<Y*>(p.y) + token_row(p, r) * N;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int i = (c * LPR + lane) * VEC;
            if (i >= N) continue;
            float w[VEC], o[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) o[e] = v[c][e] * rs;
            if (p.weight) {
                load<VEC>(p.weight + wrow + i, w);
#pragma unroll
                for (int e = 0; e < VEC; ++e) o[e] *= w[e];
            }
            if (p.bias) {
                load<VEC>(p.bias + wrow + i, w);
#pragma unroll
                for (int e = 0; e < VEC; ++e) o[e] += w[e];
            }
            store<VEC>(y + i, o);
        }
    }
}

// One CTA per row block of one (b, h).
template <class X, class Y, class DX, int VEC, int LPR, int CH>
__global__ void __launch_bounds__(kThreads) m2rnn_norm_bwd_kernel(const NormParams p) {
    constexpr int kGroups = kThreads / LPR;                 // rows at a time
    __shared__ float buf[2][kThreads / 32];
    __shared__ float sums[LPR > 32 ? 1 : kThreads * VEC];   // row groups' partial sums, one chunk at a time
    const int lane = threadIdx.x % LPR, grp = threadIdx.x / LPR, N = p.N;
    const int bh = blockIdx.x / p.chunks, chunk = blockIdx.x % p.chunks;
    const int per = (p.T + p.chunks - 1) / p.chunks;
    const int t0 = chunk * per, t1 = min(p.T, t0 + per);
    const float inv = 1.f / (float)N;
    const size_t wrow = (size_t)(bh % p.H) * N;
    float w[CH][VEC], dw[CH][VEC], db[CH][VEC];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int i = (c * LPR + lane) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) { w[c][e] = 1.f; dw[c][e] = 0.f; db[c][e] = 0.f; }
        if (p.weight && i < N) load<VEC>(p.weight + wrow + i, w[c]);
    }
    for (int tb = t0; tb < t1; tb += kGroups) {
        const int t = tb + grp;
        const bool live = t < t1;
        const size_t r = (size_t)bh * p.T + (live ? t : t0);
        const X* x = static_cast<const X*>(p.x) + r * N;
        const Y* dy = static_cast<const Y*>(p.dy) + token_row(p, r) * N;
        const float m = p.rms ? 0.f : p.mean[r], rs = p.rstd[r];
        float n[CH][VEC], g[CH][VEC];
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int i = (c * LPR + lane) * VEC;
            if (live && i < N) {
                load<VEC>(x + i, n[c]);
                load<VEC>(dy + i, g[c]);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) { n[c][e] = m; g[c][e] = 0.f; }
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                n[c][e] = (n[c][e] - m) * rs;
                dw[c][e] = fmaf(g[c][e], n[c][e], dw[c][e]);
                db[c][e] += g[c][e];
                g[c][e] *= w[c][e];
                s1 += g[c][e];
                s2 = fmaf(g[c][e], n[c][e], s2);
            }
        }
        const float m1 = p.rms ? 0.f : row_sum<LPR>(s1, buf[0]) * inv;
        const float m2 = row_sum<LPR>(s2, buf[1]) * inv;
        if constexpr (LPR > 32) __syncthreads();
        if (!live) continue;
        DX* dx = static_cast<DX*>(p.dx) + r * N;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int i = (c * LPR + lane) * VEC;
            if (i >= N) continue;
            float o[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) o[e] = rs * (g[c][e] - m1 - n[c][e] * m2);
            store<VEC>(dx + i, o);
        }
    }
    if (!p.part) return;
    float* part = p.part + (size_t)blockIdx.x * 2 * N;
    if constexpr (LPR > 32) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int i = (c * LPR + lane) * VEC;
            if (i >= N) continue;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                part[i + e] = dw[c][e];
                part[N + i + e] = db[c][e];
            }
        }
    } else {
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int which = 0; which < 2; ++which) {
                __syncthreads();
#pragma unroll
                for (int e = 0; e < VEC; ++e) sums[(grp * LPR + lane) * VEC + e] = which ? db[c][e] : dw[c][e];
                __syncthreads();
                for (int i = threadIdx.x; i < LPR * VEC; i += kThreads) {
                    float s = sums[i];
#pragma unroll 8
                    for (int gg = 1; gg < kGroups; ++gg) s += sums[gg * LPR * VEC + i];
                    const int col = c * LPR * VEC + i;
                    if (col < N) part[which * N + col] = s;
                }
            }
    }
}

// dweight, dbias [H][N]: the row blocks' sums, added in ascending (b, block)
// order by eight groups of threads and then over the groups.
__global__ void __launch_bounds__(256) m2rnn_norm_dw_kernel(const NormParams p) {
    __shared__ float s[8][32];
    const int N = p.N, h = blockIdx.y, lane = threadIdx.x % 32, grp = threadIdx.x / 32;
    const int e = blockIdx.x * 32 + lane;                    // column of [dw | db]
    const int n = p.B * p.chunks;
    float a = 0.f;
    if (e < 2 * N)
        for (int j = grp; j < n; j += 8)
            a += p.part[((size_t)((j / p.chunks) * p.H + h) * p.chunks + j % p.chunks) * 2 * N + e];
    s[grp][lane] = a;
    __syncthreads();
    if (grp == 0 && e < 2 * N) {
#pragma unroll
        for (int g = 1; g < 8; ++g) a += s[g][lane];
        float* out = e < N ? p.dweight : p.dbias;
        if (out) out[(size_t)h * N + (e < N ? e : e - N)] = a;
    }
}

// Rows too long for registers: one CTA per row, the row read again (from L2)
// for each pass.
template <class X, class Y>
__global__ void __launch_bounds__(kThreads) m2rnn_norm_fwd_long_kernel(const NormParams p) {
    __shared__ float buf[2][kThreads / 32];
    const int N = p.N;
    const size_t rows = (size_t)p.B * p.H * p.T;
    const float inv = 1.f / (float)N;
    for (size_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const X* x = static_cast<const X*>(p.x) + r * N;
        float s = 0.f;
        if (!p.rms)
            for (int i = threadIdx.x; i < N; i += kThreads) s += to_f32(x[i]);
        const float m = p.rms ? 0.f : row_sum<kThreads>(s, buf[0]) * inv;
        s = 0.f;
        for (int i = threadIdx.x; i < N; i += kThreads) {
            const float d = to_f32(x[i]) - m;
            s = fmaf(d, d, s);
        }
        const float rs = 1.f / sqrtf(row_sum<kThreads>(s, buf[1]) * inv + p.eps);
        __syncthreads();
        if (threadIdx.x == 0) {
            if (p.mean && !p.rms) p.mean[r] = m;
            if (p.rstd) p.rstd[r] = rs;
        }
        const size_t wrow = (size_t)(p.H == 1 ? 0 : (r / p.T) % p.H) * N;
        Y* y = static_cast<Y*>(p.y) + token_row(p, r) * N;
        for (int i = threadIdx.x; i < N; i += kThreads) {
            float o[1] = {(to_f32(x[i]) - m) * rs};
            if (p.weight) o[0] *= p.weight[wrow + i];
            if (p.bias) o[0] += p.bias[wrow + i];
            store<1>(y + i, o);
        }
    }
}

// Backward of long rows: a CTA takes a row block; the weight's and bias's
// sums go through the block's own partial row in the workspace (each element
// is only ever touched by one thread).
template <class X, class Y, class DX>
__global__ void __launch_bounds__(kThreads) m2rnn_norm_bwd_long_kernel(const NormParams p) {
    __shared__ float buf[2][kThreads / 32];
    const int N = p.N, bh = blockIdx.x / p.chunks, chunk = blockIdx.x % p.chunks;
    const int per = (p.T + p.chunks - 1) / p.chunks;
    const int t0 = chunk * per, t1 = min(p.T, t0 + per);
    const float inv = 1.f / (float)N;
    const float* w = p.weight ? p.weight + (size_t)(bh % p.H) * N : nullptr;
    float* part = p.part ? p.part + (size_t)blockIdx.x * 2 * N : nullptr;
    if (part)
        for (int i = threadIdx.x; i < N; i += kThreads) part[i] = part[N + i] = 0.f;
    for (int t = t0; t < t1; ++t) {
        const size_t r = (size_t)bh * p.T + t;
        const X* x = static_cast<const X*>(p.x) + r * N;
        const Y* dy = static_cast<const Y*>(p.dy) + token_row(p, r) * N;
        DX* dx = static_cast<DX*>(p.dx) + r * N;
        const float m = p.rms ? 0.f : p.mean[r], rs = p.rstd[r];
        float s1 = 0.f, s2 = 0.f;
        for (int i = threadIdx.x; i < N; i += kThreads) {
            const float n = (to_f32(x[i]) - m) * rs, d = to_f32(dy[i]), g = w ? d * w[i] : d;
            s1 += g;
            s2 = fmaf(g, n, s2);
            if (part) {
                part[i] = fmaf(d, n, part[i]);
                part[N + i] += d;
            }
        }
        const float m1 = p.rms ? 0.f : row_sum<kThreads>(s1, buf[0]) * inv;
        const float m2 = row_sum<kThreads>(s2, buf[1]) * inv;
        __syncthreads();
        for (int i = threadIdx.x; i < N; i += kThreads) {
            const float n = (to_f32(x[i]) - m) * rs, d = to_f32(dy[i]), g = w ? d * w[i] : d;
            const float o[1] = {rs * (g - m1 - n * m2)};
            store<1>(dx + i, o);
        }
    }
}

unsigned capped(size_t want, int per_sm) {
    const size_t cap = (size_t)kNumSMs * per_sm;
    return (unsigned)(want < cap ? want : cap);
}

// Which layout a row length takes: f<VEC, LPR, CH>(), or false for rows too long for registers.
template <class F>
bool by_length(int N, F&& f) {
    if (N % 8 == 0) {   // rows start on 16 bytes in both types
        if (N <= 16) f.template operator()<8, 2, 1>();
        else if (N <= 32) f.template operator()<8, 4, 1>();
        else if (N <= 64) f.template operator()<8, 8, 1>();
        else if (N <= 128) f.template operator()<8, 16, 1>();
        else if (N <= 256) f.template operator()<8, 32, 1>();
        else if (N <= 1024) f.template operator()<8, 32, 4>();
        else if (N <= 2048) f.template operator()<8, 256, 1>();
        else if (N <= 4096) f.template operator()<8, 256, 2>();
        else if (N <= 8192) f.template operator()<8, 256, 4>();
        else return false;
    } else {
        if (N <= 256) f.template operator()<1, 32, 8>();
        else if (N <= 2048) f.template operator()<1, 256, 8>();
        else if (N <= 8192) f.template operator()<1, 256, 32>();
        else return false;
    }
    return true;
}

template <class X, class Y>
struct Fwd {
    const NormParams& p;
    cudaStream_t s;
    template <int VEC, int LPR, int CH>
    void operator()() {
        const size_t rows = (size_t)p.B * p.H * p.T, want = (rows + kThreads / LPR - 1) / (kThreads / LPR);
        m2rnn_norm_fwd_kernel<X, Y, VEC, LPR, CH><<<capped(want, 64), kThreads, 0, s>>>(p);
    }
};
template <class X, class Y, class DX>
struct Bwd {
    const NormParams& p;
    cudaStream_t s;
    template <int VEC, int LPR, int CH>
    void operator()() {
        m2rnn_norm_bwd_kernel<X, Y, DX, VEC, LPR, CH><<<p.B * p.H * p.chunks, kThreads, 0, s>>>(p);
    }
};

template <class X, class Y>
cudaError_t fwd(const NormParams& p, cudaStream_t s) {
    if (!by_length(p.N, Fwd<X, Y>{p, s}))
        m2rnn_norm_fwd_long_kernel<X, Y><<<capped((size_t)p.B * p.H * p.T, 8), kThreads, 0, s>>>(p);
    return cudaGetLastError();
}
template <class X, class Y, class DX>
cudaError_t bwd(const NormParams& p, cudaStream_t s) {
    if (!by_length(p.N, Bwd<X, Y, DX>{p, s}))
        m2rnn_norm_bwd_long_kernel<X, Y, DX><<<p.B * p.H * p.chunks, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}
template <class Y>
cudaError_t bwd_x(const NormParams& p, cudaStream_t s) {
    if (!p.x_fp32) return bwd<__nv_bfloat16, Y, __nv_bfloat16>(p, s);
    return p.dx_fp32 ? bwd<float, Y, float>(p, s) : bwd<float, Y, __nv_bfloat16>(p, s);
}

}  // namespace

cudaError_t launch_norm_fwd(const NormParams& p, cudaStream_t s) {
    if (p.x_fp32) return p.y_fp32 ? fwd<float, float>(p, s) : fwd<float, __nv_bfloat16>(p, s);
    return p.y_fp32 ? fwd<__nv_bfloat16, float>(p, s) : fwd<__nv_bfloat16, __nv_bfloat16>(p, s);
}

int norm_bwd_chunks(int B, int H, int T, int N) {
    // about four CTAs for each SM, and at least 8 of its row groups for a CTA
    const int lanes = N <= 256 ? (N + 7) / 8 : N <= 1024 ? 32 : 256;
    const int rows_at_once = kThreads / (lanes < 1 ? 1 : lanes);
    const long long pairs = (long long)B * H;
    long long chunks = (4LL * kNumSMs + pairs - 1) / pairs, most = T / (8LL * (rows_at_once < 1 ? 1 : rows_at_once));
    if (chunks > most) chunks = most;
    return (int)(chunks < 1 ? 1 : chunks);
}

cudaError_t launch_norm_bwd(const NormParams& p, cudaStream_t s) {
    cudaError_t e = p.y_fp32 ? bwd_x<float>(p, s) : bwd_x<__nv_bfloat16>(p, s);
    if (e != cudaSuccess || !p.part) return e;
    m2rnn_norm_dw_kernel<<<dim3((2 * p.N + 31) / 32, p.H), 256, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace m2rnn
