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
// kernel adds the blocks in a fixed order: no atomics, the same bits every
// time.
#include "kernels.h"
#include "launch.h"
#include "layer_norm.h"

#include <cuda_bf16.h>

namespace m2rnn {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

template <int VEC>
__device__ __forceinline__ void load(const float* p, float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        v[0] = *p;
    }
}
// VEC values as they lie in memory, to be unpacked when they are used: what a
// prefetch holds.
template <class T, int VEC>
struct Raw {
    static constexpr int kWords = VEC == 1 ? 1 : VEC * (int)sizeof(T) / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }
    __device__ __forceinline__ void get(const T* p) {
        if constexpr (VEC == 1) {
            if constexpr (sizeof(T) == 2) w[0] = *reinterpret_cast<const uint16_t*>(p);
            else w[0] = *reinterpret_cast<const uint32_t*>(p);
        } else {
#pragma unroll
            for (int i = 0; i < kWords; i += 4) {
                const uint4 x = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(p) + i);
                w[i] = x.x; w[i + 1] = x.y; w[i + 2] = x.z; w[i + 3] = x.w;
            }
        }
    }
    __device__ __forceinline__ float operator[](int e) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[e]);
        else return VEC == 1 || !(e & 1) ? bf16lo_to_f32(w[e / 2]) : bf16hi_to_f32(w[e / 2]);
    }
};

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

// Sums over the LPR threads of a row of U values, the same in each of them.
// `buf`: U slots per warp, not those of the previous call (for LPR > 32).
template <int LPR, int U>
__device__ __forceinline__ void row_sums(float (&x)[U], float (*buf)[U]) {
#pragma unroll
    for (int d = (LPR < 32 ? LPR : 32) / 2; d; d >>= 1)
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] += __shfl_xor_sync(~0u, x[u], d);
    if constexpr (LPR > 32) {
        static_assert(LPR == kThreads, "a row takes part of a warp or the whole CTA");
        if (threadIdx.x % 32 == 0)
#pragma unroll
            for (int u = 0; u < U; ++u) buf[threadIdx.x / 32][u] = x[u];
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            x[u] = buf[0][u];
#pragma unroll
            for (int w = 1; w < kThreads / 32; ++w) x[u] += buf[w][u];
        }
    }
}
template <int LPR>
__device__ __forceinline__ float row_sum(float x, float (*buf)[1]) {
    float v[1] = {x};
    row_sums<LPR, 1>(v, buf);
    return v[0];
}

// Row t of pair bh: x's row is bh·T + t, y's this.
__device__ __forceinline__ size_t token_row(const NormParams& p, int bh, int t) {
    return ((size_t)(bh / p.H) * p.T + t) * p.H + bh % p.H;
}

// Work items are pairs (row block of a (b, h)); `per` rows per block.
struct Block {
    int bh, t0, t1;
};
__device__ __forceinline__ Block block_of(const NormParams& p) {
    const int chunk = blockIdx.x % p.chunks, per = (p.T + p.chunks - 1) / p.chunks;
    return {(int)(blockIdx.x / p.chunks), chunk * per, min(p.T, (chunk + 1) * per)};
}

// Rows at a time and CTAs per SM: what hides the loads' latency within the
// registers, and for rows that take the whole CTA the barriers too.  Measured,
// us (see the kernels for the shapes):
//   forward, rows of 2048: 2 rows and 4 CTAs 14.8, 4 and 2 17.1, 1 and 6 20.4;
//            fp32 rows of 128: 4 rows and 2 CTAs 68, 2 and 4 82
//   backward, rows of 64: 3 rows 22.4, 2 25.7; rows of 2048: 2 rows 26.7, 3 32.2
constexpr int unroll_fwd(int values, bool cta) { return values >= 32 ? 1 : values >= 16 || cta ? 2 : 4; }
constexpr int ctas_fwd(int values, bool cta) { return cta && values < 16 ? 4 : 2; }
constexpr int unroll_bwd(int values, bool cta, bool bf16) { return values >= 16 ? 1 : cta || !bf16 ? 2 : 3; }

// 1/sqrt(x) to the last place or two: the approximation and one Newton step,
// which 0 and infinity do without.
__device__ __forceinline__ float inv_sqrt(float x) {
    const float r = rsqrtf(x), e = fmaf(-x * r, r, 1.f);
    return e == e ? fmaf(0.5f * r, e, r) : r;
}

// VEC values in pairs: additions, products and multiply-adds of two values take
// one instruction.  (One value at a time, issue slots and not HBM bounded rows
// of 64: forward 17.0 against 13.5 us, 67 MB moved.)
template <int VEC, class F>
__device__ __forceinline__ void by_pairs(F&& f) {   // f(i, i + 1)
#pragma unroll
    for (int e = 0; e < VEC; e += 2) f(e, VEC == 1 ? 0 : e + 1);
}

// LPR threads per row, CH groups of VEC values per thread (N <= LPR·VEC·CH), U
// rows at a time.  A CTA takes items of kGroups·U consecutive rows of one
// (b, h), a contiguous range of them, and has the next one's loads in flight
// while it works on one.  Measured against the copy rate of 6.45 TB/s: 2^18
// rows of 64 bf16 12.7 us (82%), 2^19 fp32 rows of 128 to bf16 68 us (92%),
// 8191 rows of 2048 bf16 14.9 us (70%: two barriers of the CTA a row group).
template <class X, class Y, int VEC, int LPR, int CH, int U>
__global__ void __launch_bounds__(kThreads, VEC == 8 && CH == 1 && LPR <= 32 ? 2 : 0)
    m2rnn_norm_fwd_kernel(const NormParams p) {
    constexpr int kGroups = kThreads / LPR, kRows = kGroups * U;
    constexpr bool kKeep = CH == 1 && VEC == 8;   // weight and bias stay in registers over the items of a head
    __shared__ float buf[2][kThreads / 32][U];
    const int lane = threadIdx.x % LPR, grp = threadIdx.x / LPR, N = p.N;
    const float inv = 1.f / (float)N;
    const unsigned per = (p.T + kRows - 1) / kRows, items = (unsigned)(p.B * p.H) * per;
    unsigned item = (unsigned)((unsigned long long)items * blockIdx.x / gridDim.x);
    const unsigned end = (unsigned)((unsigned long long)items * (blockIdx.x + 1) / gridDim.x);
    Raw<X, VEC> next[U][CH];
    int nbh = item / per, nblk = item % per;   // of the item to be fetched
    auto fetch = [&]() {
        const int t0 = nblk * kRows + grp;
        const X* x = static_cast<const X*>(p.x) + ((size_t)nbh * p.T + t0) * N;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int i = (c * LPR + lane) * VEC;
                if (t0 + u * kGroups < p.T && i < N) next[u][c].get(x + (size_t)u * kGroups * N + i);
                else next[u][c].zero();
            }
        if (++nblk == (int)per) { nblk = 0; ++nbh; }
    };
    int bh = nbh, blk = nblk, h = bh % p.H, b = bh / p.H;
    float w[kKeep ? VEC : 1], bias[kKeep ? VEC : 1];
    auto affine = [&](int i, float* wv, float* bv) {
        float x[VEC], z[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) { x[e] = 1.f; z[e] = 0.f; }
        if (i < N && p.weight) load<VEC>(p.weight + (size_t)h * N + i, x);
        if (i < N && p.bias) load<VEC>(p.bias + (size_t)h * N + i, z);
#pragma unroll
        for (int e = 0; e < VEC; ++e) { wv[e] = x[e]; bv[e] = z[e]; }
    };
    if (item < end) {
        fetch();
        if constexpr (kKeep) affine(lane * VEC, w, bias);
    }
    for (; item < end; ++item) {   // the same count for every thread
        const int t0 = blk * kRows + grp;
        float v[U][CH][VEC], s[U], m[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float2 a = make_float2(0.f, 0.f);
#pragma unroll
            for (int c = 0; c < CH; ++c) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[u][c][e] = next[u][c][e];
                if constexpr (VEC == 1) a.x += v[u][c][0];
                else by_pairs<VEC>([&](int i, int j) { a = __fadd2_rn(a, make_float2(v[u][c][i], v[u][c][j])); });
            }
            s[u] = a.x + a.y;
        }
        if (item + 1 < end) fetch();
        if (!p.rms) row_sums<LPR, U>(s, buf[0]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            m[u] = p.rms ? 0.f : s[u] * inv;
            float2 a = make_float2(0.f, 0.f);
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const float d = (c * LPR + lane) * VEC < N ? -m[u] : 0.f;   // nothing beside the row
                if constexpr (VEC == 1) {
                    v[u][c][0] += d;
                    a.x = fmaf(v[u][c][0], v[u][c][0], a.x);
                } else {
                    by_pairs<VEC>([&](int i, int j) {
                        const float2 x = __fadd2_rn(make_float2(v[u][c][i], v[u][c][j]), make_float2(d, d));
                        a = __ffma2_rn(x, x, a);
                        v[u][c][i] = x.x; v[u][c][j] = x.y;
                    });
                }
            }
            s[u] = a.x + a.y;
        }
        row_sums<LPR, U>(s, buf[1]);
        if constexpr (LPR > 32) __syncthreads();   // buf[] is free for the next rows
        float rs[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            rs[u] = inv_sqrt(s[u] * inv + p.eps);
            const int t = t0 + u * kGroups;
            if (lane == 0 && t < p.T) {
                const size_t r = (size_t)bh * p.T + t;
                if (p.mean && !p.rms) p.mean[r] = m[u];
                if (p.rstd) p.rstd[r] = rs[u];
            }
        }
        Y* y = static_cast<Y*>(p.y) + (((size_t)b * p.T + t0) * p.H + h) * N;
        const size_t ystep = (size_t)kGroups * p.H * N;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int i = (c * LPR + lane) * VEC;
            if (i >= N) continue;
            float wv[VEC], bv[VEC];
            if constexpr (!kKeep) affine(i, wv, bv);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (t0 + u * kGroups >= p.T) continue;
                float o[VEC];
                if constexpr (VEC == 1) {
                    o[0] = fmaf(v[u][c][0] * rs[u], wv[0], bv[0]);
                } else {
                    by_pairs<VEC>([&](int e, int f) {
                        const float2 x = __ffma2_rn(
                            __fmul2_rn(make_float2(v[u][c][e], v[u][c][f]), make_float2(rs[u], rs[u])),
                            kKeep ? make_float2(w[kKeep ? e : 0], w[kKeep ? f : 0]) : make_float2(wv[e], wv[f]),
                            kKeep ? make_float2(bias[kKeep ? e : 0], bias[kKeep ? f : 0]) : make_float2(bv[e], bv[f]));
                        o[e] = x.x; o[f] = x.y;
                    });
                }
                store<VEC>(y + u * ystep + i, o);
            }
        }
        if (++blk == (int)per) {   // the next (b, h)
            blk = 0;
            ++bh;
            if (++h == p.H) { h = 0; ++b; }
            if constexpr (kKeep) if (item + 1 < end) affine(lane * VEC, w, bias);
        }
    }
}

// A CTA takes a block of rows of one (b, h), U·kGroups at a time, the next ones
// in flight.  Measured with the sums' kernel: 2^18 rows of 64 bf16 22.6 us,
// 8191 rows of 2048 25.3 us, 101 MB each (15.6 us at the copy rate).  Bound by
// the loads that fit in flight beside the sums in 128 registers a thread, and
// by the second kernel (its early launch is worth 1 us).
template <class X, class Y, class DX, int VEC, int LPR, int CH, int U>
__global__ void __launch_bounds__(kThreads, VEC == 8 && CH == 1 ? 2 : 0) m2rnn_norm_bwd_kernel(const NormParams p) {
    constexpr int kGroups = kThreads / LPR, kRows = kGroups * U;
    __shared__ float buf[kThreads / 32][2 * U];
    __shared__ float sums[LPR > 32 ? 1 : kThreads * VEC];   // row groups' partial sums, one chunk at a time
    const int lane = threadIdx.x % LPR, grp = threadIdx.x / LPR, N = p.N;
    const Block b = block_of(p);
    const float inv = 1.f / (float)N;
    const size_t wrow = (size_t)(b.bh % p.H) * N, xrow = (size_t)b.bh * p.T;
    float w[CH][VEC], dw[CH][VEC], db[CH][VEC];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int i = (c * LPR + lane) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) { w[c][e] = 1.f; dw[c][e] = 0.f; db[c][e] = 0.f; }
        if (p.weight && i < N) load<VEC>(p.weight + wrow + i, w[c]);
    }
    Raw<X, VEC> nx[U][CH];
    Raw<Y, VEC> ny[U][CH];
    float nm[U], nr[U];
    auto fetch = [&](int t0) {
        const X* x = static_cast<const X*>(p.x) + (xrow + t0) * N;
        const Y* dy = static_cast<const Y*>(p.dy) + token_row(p, b.bh, t0) * N;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = t0 + u * kGroups;
            const bool live = t < b.t1;
            nm[u] = live && !p.rms ? p.mean[xrow + t] : 0.f;
            nr[u] = live ? p.rstd[xrow + t] : 0.f;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int i = (c * LPR + lane) * VEC;
                if (live && i < N) {
                    nx[u][c].get(x + (size_t)u * kGroups * N + i);
                    ny[u][c].get(dy + (size_t)u * kGroups * p.H * N + i);
                } else {
                    nx[u][c].zero();
                    ny[u][c].zero();
                }
            }
        }
    };
    fetch(b.t0 + grp);
    for (int tb = b.t0; tb < b.t1; tb += kRows) {
        float n[U][CH][VEC], g[U][CH][VEC], s[2 * U], rs[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            rs[u] = nr[u];
            float2 s1 = make_float2(0.f, 0.f), s2 = s1;
            const float2 r2 = make_float2(rs[u], rs[u]);
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                // beside the row, and behind the last (rs = 0), n is 0
                const float m = (c * LPR + lane) * VEC < N ? -nm[u] : 0.f;
                if constexpr (VEC == 1) {
                    const float a = (nx[u][c][0] + m) * rs[u], d = ny[u][c][0];
                    dw[c][0] = fmaf(d, a, dw[c][0]);
                    db[c][0] += d;
                    n[u][c][0] = a;
                    g[u][c][0] = d * w[c][0];
                    s1.x += g[u][c][0];
                    s2.x = fmaf(g[u][c][0], a, s2.x);
                } else {
                    by_pairs<VEC>([&](int e, int f) {
                        const float2 a = __fmul2_rn(__fadd2_rn(make_float2(nx[u][c][e], nx[u][c][f]), make_float2(m, m)), r2),
                                     d = make_float2(ny[u][c][e], ny[u][c][f]),
                                     wd = __ffma2_rn(d, a, make_float2(dw[c][e], dw[c][f])),
                                     bd = __fadd2_rn(make_float2(db[c][e], db[c][f]), d),
                                     gg = __fmul2_rn(d, make_float2(w[c][e], w[c][f]));
                        dw[c][e] = wd.x; dw[c][f] = wd.y;
                        db[c][e] = bd.x; db[c][f] = bd.y;
                        n[u][c][e] = a.x; n[u][c][f] = a.y;
                        g[u][c][e] = gg.x; g[u][c][f] = gg.y;
                        s1 = __fadd2_rn(s1, gg);
                        s2 = __ffma2_rn(gg, a, s2);
                    });
                }
            }
            s[2 * u] = s1.x + s1.y;
            s[2 * u + 1] = s2.x + s2.y;
        }
        fetch(tb + kRows + grp);
        row_sums<LPR, 2 * U>(s, buf);
        if constexpr (LPR > 32) __syncthreads();   // (two buffers in turn instead: no faster)
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = tb + u * kGroups + grp;
            if (t >= b.t1) continue;
            const float m1 = p.rms ? 0.f : s[2 * u] * inv, m2 = s[2 * u + 1] * inv;
            DX* dx = static_cast<DX*>(p.dx) + (xrow + t) * N;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int i = (c * LPR + lane) * VEC;
                if (i >= N) continue;
                float o[VEC];
                if constexpr (VEC == 1) {
                    o[0] = rs[u] * (g[u][c][0] - m1 - n[u][c][0] * m2);
                } else {
                    by_pairs<VEC>([&](int e, int f) {
                        const float2 x = __fmul2_rn(
                            make_float2(rs[u], rs[u]),
                            __ffma2_rn(make_float2(n[u][c][e], n[u][c][f]), make_float2(-m2, -m2),
                                       __fadd2_rn(make_float2(g[u][c][e], g[u][c][f]), make_float2(-m1, -m1))));
                        o[e] = x.x; o[f] = x.y;
                    });
                }
                store<VEC>(dx + i, o);
            }
        }
    }
    if (!p.part) return;
    cudaTriggerProgrammaticLaunchCompletion();   // the sums' kernel may be set up; it waits for this one's end
    float* part = p.part + (size_t)blockIdx.x * 2 * N;
    if constexpr (LPR > 32) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int i = (c * LPR + lane) * VEC;
            if (i >= N) continue;
            store<VEC>(part + i, dw[c]);   // both 32-byte aligned where VEC is 8: N is a multiple of 8
            store<VEC>(part + N + i, db[c]);
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
                    float a = sums[i];
#pragma unroll 8
                    for (int gg = 1; gg < kGroups; ++gg) a += sums[gg * LPR * VEC + i];
                    const int col = c * LPR * VEC + i;
                    if (col < N) part[which * N + col] = a;
                }
            }
    }
}

// dweight, dbias [H][N]: the row blocks' sums, added in ascending (b, block)
// order by 32 groups of threads and then over the groups.  Launched while the
// backward kernel runs out, whose end it waits for.  A CTA takes 32 columns of a
// head; heads and column blocks share the grid's first dimension, since the others
// end at 65535.  Backward with 32, 16 and 8 groups: 8192 rows of 2048 25.8, 28.0 and
// 32.0 us; 2^18 rows of 64 23.2, 25.1 and 28.3.
__global__ void __launch_bounds__(1024) m2rnn_norm_dw_kernel(const NormParams p) {
    __shared__ float s[32][32];
    const int N = p.N, lane = threadIdx.x % 32, grp = threadIdx.x / 32;
    const unsigned blocks = norm_dw_blocks(N), h = blockIdx.x / blocks;
    const int e = (int)(blockIdx.x % blocks) * 32 + lane;    // column of [dw | db]
    const int n = p.B * p.chunks;
    float a = 0.f;
    cudaGridDependencySynchronize();
    if (e < 2 * N)
#pragma unroll 8
        for (int j = grp; j < n; j += 32)
            a += p.part[((size_t)((j / p.chunks) * p.H + h) * p.chunks + j % p.chunks) * 2 * N + e];
    s[grp][lane] = a;
    __syncthreads();
    if (grp == 0 && e < 2 * N) {
#pragma unroll
        for (int g = 1; g < 32; ++g) a += s[g][lane];
        float* out = e < N ? p.dweight : p.dbias;
        if (out) out[(size_t)h * N + (e < N ? e : e - N)] = a;
    }
}

// Rows too long for registers: one CTA per row, the row read again (from L2)
// for each pass.
template <class X, class Y>
__global__ void __launch_bounds__(kThreads) m2rnn_norm_fwd_long_kernel(const NormParams p) {
    __shared__ float buf[2][kThreads / 32][1];
    const int N = p.N;
    const float inv = 1.f / (float)N;
    const Block b = block_of(p);
    for (int t = b.t0; t < b.t1; ++t) {
        const size_t r = (size_t)b.bh * p.T + t;
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
        const size_t wrow = (size_t)(b.bh % p.H) * N;
        Y* y = static_cast<Y*>(p.y) + token_row(p, b.bh, t) * N;
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
    __shared__ float buf[2][kThreads / 32][1];
    const int N = p.N;
    const Block b = block_of(p);
    const float inv = 1.f / (float)N;
    const float* w = p.weight ? p.weight + (size_t)(b.bh % p.H) * N : nullptr;
    float* part = p.part ? p.part + (size_t)blockIdx.x * 2 * N : nullptr;
    if (part)
        for (int i = threadIdx.x; i < N; i += kThreads) part[i] = part[N + i] = 0.f;
    for (int t = b.t0; t < b.t1; ++t) {
        const size_t r = (size_t)b.bh * p.T + t;
        const X* x = static_cast<const X*>(p.x) + r * N;
        const Y* dy = static_cast<const Y*>(p.dy) + token_row(p, b.bh, t) * N;
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

// Which layout a row length takes, f<VEC, LPR, CH>(), or false for rows too
// long for registers.  Measured, us, 2^24 bf16 values, forward / backward:
//   a warp for a row, or the CTA: rows of 264 32 / 55, or 79 / 105; of 1024 17 / 29,
//     or 24 / 35; one value at a time, rows of 100 40 / 102, or 333 / 383; of 255
//     24 / 56, or 139 / 157
//   one group of 8 a thread, or two: rows of 2048 15 / 26, or 22 / 33
//   in registers, or read again: rows of 8192 19 / 39, or 51 / 209; of 8191 45 / 53,
//     or 53 / 233; of 4097 52 / 61, or 40 / 197
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
unsigned capped(size_t want, int per_sm) {
    const size_t cap = (size_t)kNumSMs * per_sm;
    return (unsigned)(want < cap ? want : cap);
}

template <class X, class Y>
struct Fwd {
    const NormParams& p;
    cudaStream_t s;
    template <int VEC, int LPR, int CH>
    void operator()() {
        constexpr int U = unroll_fwd(VEC * CH, LPR > 32), kRows = kThreads / LPR * U;
        const size_t items = (size_t)p.B * p.H * ((p.T + kRows - 1) / kRows);
        m2rnn_norm_fwd_kernel<X, Y, VEC, LPR, CH, U><<<capped(items, ctas_fwd(VEC * CH, LPR > 32)), kThreads, 0, s>>>(p);
    }
};
template <class X, class Y, class DX>
struct Bwd {
    const NormParams& p;
    cudaStream_t s;
    template <int VEC, int LPR, int CH>
    void operator()() {
        constexpr int U = unroll_bwd(VEC * CH, LPR > 32, sizeof(X) + sizeof(Y) == 4);
        m2rnn_norm_bwd_kernel<X, Y, DX, VEC, LPR, CH, U><<<p.B * p.H * p.chunks, kThreads, 0, s>>>(p);
    }
};

template <class X, class Y>
cudaError_t fwd(const NormParams& p, cudaStream_t s) {
    if (!by_length(p.N, Fwd<X, Y>{p, s}))
        m2rnn_norm_fwd_long_kernel<X, Y><<<p.B * p.H * p.chunks, kThreads, 0, s>>>(p);
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

// Row blocks of each (b, h): at most `ctas` CTAs in all where there are fewer
// pairs (one wave), each with at least `least` times the rows that it takes at a
// time.  Measured, us, backward with least = 1, 4 and 16: 512 rows of 2048 8.3, 7.1,
// 10.1; 16 heads of 2048 rows of 64 7.3, 7.3, 9.3; 1024 rows of 64 5.1, 5.7, 9.1.
int chunks_for(int B, int H, int T, int N, int ctas, int least) {
    const int lanes = N % 8 ? (N <= 256 ? 32 : 256) : N <= 256 ? (N + 7) / 8 : N <= 1024 ? 32 : 256;
    const int at_once = kThreads / lanes;
    const long long pairs = (long long)B * H;
    long long chunks = ctas / pairs, most = T / ((long long)least * at_once);
    if (chunks > most) chunks = most;
    return (int)(chunks < 1 ? 1 : chunks);
}

}  // namespace

cudaError_t launch_norm_fwd(const NormParams& q, cudaStream_t s) {
    NormParams p = q;
    p.chunks = chunks_for(p.B, p.H, p.T, p.N, 8 * kNumSMs, 1);   // rows too long for registers
    if (p.x_fp32) return p.y_fp32 ? fwd<float, float>(p, s) : fwd<float, __nv_bfloat16>(p, s);
    return p.y_fp32 ? fwd<__nv_bfloat16, float>(p, s) : fwd<__nv_bfloat16, __nv_bfloat16>(p, s);
}

int norm_bwd_chunks(int B, int H, int T, int N) { return chunks_for(B, H, T, N, 2 * kNumSMs, 4); }

cudaError_t launch_norm_bwd(const NormParams& p, cudaStream_t s) {
    cudaError_t e = p.y_fp32 ? bwd_x<float>(p, s) : bwd_x<__nv_bfloat16>(p, s);
    if (e != cudaSuccess || !p.part) return e;
    return launch_dependent(m2rnn_norm_dw_kernel, dim3(norm_dw_blocks(p.N) * p.H), 1024, 0, s, p);
}

}  // namespace m2rnn
