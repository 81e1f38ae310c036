// Backward of linear attention in chunks of 128 tokens on the tensor cores
// (bf16), walking from the last chunk to the first.
//
// With S the state at the chunk's start (a checkpoint), G = dL/dS at its end,
// and a, b, D the decays of the forward,
//   dq_t = a_t (dY Sᵀ)_t + (dP' K)_t          P'  = (Q Kᵀ) ∘ D
//   dk_s = b_s (V Gᵀ)_s  + (dP'ᵀ Q)_s         dP' = (dY Vᵀ) ∘ D
//   dv_s = b_s (K G)_s   + (P'ᵀ dY)_s
//   G'   = a_end G + Σ_t (a_t q_t) dy_tᵀ
// The scores are computed transposed (lane = source s, column = sink t): P'ᵀ
// then stays in tensor memory as the A operand of dv, and dP'ᵀ goes to shared
// memory, for dq and dk (for K = 64 dk's copy stays in tensor memory too).
//
// The gate's gradient.  f_u df_u is the sum over all paths from a source
// s < u (a token, or S) to a sink t >= u (a token, or G):
//   Σ_{t>=u, s<u} D_ts (q_t·k_s)(dy_t·v_s) + Σ_{t>=u} q_t·(a_t S dy_t)
//   + Σ_{s<u} k_s·(b_s G v_s) + a_end <S, G>
// It is summed as it stands (suffix sums over t in registers, sums over s
// across lanes), never as a difference of running totals: those cancel, and
// for a gate near 0 the division by f_u would amplify what is left.  Gates
// below 2^-100 act as 2^-100 there, which keeps that quotient; every other
// gradient has the gate itself.
//
// Rounding: P', dP' and the copy of G that gives dv enter in two bf16 terms each
// (2^-16 of them is left out), so what rounds dq, dk and dv is their own bf16:
// relative error 1.7e-3, against 2.4e-3 with one term each.  S and G enter the
// products that df also reads, and a_t q_t enters G, as three terms (fp32
// accuracy).
//
// One CTA per (b, h) or time segment of it.  16 warps compute (thread = token
// or state row = tensor-memory lane, the four warpgroups sharing the columns),
// one issues the products, one moves tiles, one computes decays and df.
//
// Measured: 128 pairs of 64 x 64 over 2048 tokens 139 us (the reads of k, v, q,
// dy and the checkpoints and the writes of dk, dv, dq take 42.6 us at the copy
// rate of 6.45 TB/s), of 128 x 128 over 4096 tokens 530 us (191 us); the second
// terms are 16 and 62 us of these.  As in the forward a chunk's chain of waits
// bounds it, 8.7 and 16.5 us a chunk, and 96 registers a thread, of which
// 128 x 128 spills 63: one CTA an SM, 19 warps.
#include "kernels.h"
#include "la_tc.cuh"

namespace m2rnn {
namespace {

struct BwdMaps {
    CUtensorMap q, k, v, dy, dq, dk, dv;
};

// What the threads leave for df.
struct DfScratch {
    float alpha[4][128], beta[4][128];   // parts of the dot products, by warpgroup
    float total[4][128];                 // by source: its paths to each block of 32 sinks
    float cut[4][128];                   // by gate u: paths from each block of sources to sinks u.. of u's block
};
static_assert(sizeof(DfScratch) <= kTileBytes / 2, "half a tile");

// Two schedules.  Up to 64 x 128 and 128 x 64 (kRoomy) the terms of S, of G
// and of a q have shared memory of their own: both states' products run while
// the scores are worked on, and the sum for G while the outputs' products do.
// For 128 x 128 the terms of S, then those of G, then those of a q share two
// buffers and the place of dP'; dq, dk and dv go to global memory from
// registers, so that the next tiles are fetched as soon as a q has been formed
// and nothing waits for staged outputs to leave.
//
// dP'ᵀ [s][t] takes two tiles a term.  Sinks before their source have none, so of
// the low term's first tile (t < 64) the rows s >= 64 are neither written nor
// used: the products that would read them leave those lanes of the result alone.
template <int KP, int VP>
struct BCfg {
    static constexpr int NW = 16, kThreads = (NW + 3) * 32;
    static constexpr int kQ = KP / 64 * kTileBytes, kV = VP / 64 * kTileBytes, kStage = 2 * kQ + 2 * kV;
    static constexpr int kStages = KP == 64 && VP == 64 ? 2 : 1;
    static constexpr bool kRoomy = KP * VP < 128 * 128;
    static constexpr int kOp = KP * VP * 2;                     // one bf16 term of a state
    // 64 x 64: the low term of dP'ᵀ waits in tensor memory until the states' products
    // are done and then goes to 8 KB of its own (t < 64) and the v tile
    static constexpr bool kLateLo = KP == 64 && VP == 64;
    static constexpr int kOffStage = kLateLo ? kTileBytes / 2 : 0;
    static constexpr int kOffX = kOffStage + kStages * kStage;  // the states' terms
    static constexpr int kX = (kRoomy ? 6 : 2) * kOp;
    static constexpr int kOffP = kOffX + kX;                    // dP'ᵀ [s][t], 32 KB
    // df's scratch: its own place, or the v tile once V Gᵀ is done (for 128 x 128
    // the quarter of it that the low term of dP' does not use)
    static constexpr bool kOwnScratch = KP == 64 && VP == 64;
    static constexpr int kAtScratch = kRoomy ? 0 : kTileBytes / 2;
    static constexpr int kOffScratch = kOffP + 2 * kTileBytes;
    static constexpr int kOffTab = kOffScratch + (kOwnScratch ? (int)sizeof(DfScratch) : 0);
    static constexpr int kOffBar = kOffTab + (int)sizeof(LaTablesZ);
    static constexpr int kBars = 19;
    static constexpr int kOffGamma = kOffBar + kBars * 8 + 8;   // parts of a_end <S, G>, by warp
    static constexpr int kSmem = kOffGamma + NW * 4;
    static_assert(kSmem <= 227 * 1024, "shared memory");
    static_assert(kX >= (kRoomy ? 3 : 2) * kQ && kOp <= 2 * kTileBytes, "terms of a q; third terms");
    // where the terms of G go, from kOffX; without room the third terms are at kOffP
    static constexpr int kG0 = kRoomy ? 3 * kOp : 0;
    // the low term of dP'ᵀ of the other shapes: over state terms that are no longer
    // read (those of S, or where G's are done too and those of a q come early, of G),
    // or the v tile.  Where it shares its place with a q, a q waits for the outputs'
    // products (64 x 64 so: 152 us where it takes 139, see above).
    static constexpr bool kEarlyAq = KP == 64;
    static constexpr int kOffLo = kRoomy ? kOffX + (kEarlyAq ? kG0 : 0) : 2 * kQ;
    static_assert(!kEarlyAq || kLateLo || (kG0 >= 3 * kQ && kX - kG0 >= 2 * kTileBytes), "a q beside the low term of dP'");
    static_assert(kRoomy ? kLateLo || kX >= 2 * kTileBytes : kV >= 2 * kTileBytes && kStages == 1, "room for the low term of dP'");
    static_assert(!kRoomy || KP == 64 || kG0 >= 2 * kTileBytes, "G's terms are still read");
    // Tensor memory: the two score matrices, dq, dk, dv and the sum for G.
    // Where the last two do not fit beside the others they go over dY·Vᵀ once
    // the scores have been read (for 128 x 128 the sum for G over dq instead).
    static constexpr bool kOwnDv = KP == 64;
    static constexpr int kP = 0, kDP = 128, kDQ = 256, kDK = kDQ + KP, kDV = kOwnDv ? kDK + KP : kDP,
                         kDG = KP == 128 ? (VP == 64 ? kDP + 64 : kDQ) : VP == 64 ? kDV + VP : kDP;
    // the scores' columns are free for the next chunk once the products that read them are done
    static constexpr bool kEarly = KP == 64 && VP == 64;
    static constexpr int NS = KP * VP / 512;                    // state elements per thread
    static constexpr int NL = NS < 16 ? NS : 16;
    static constexpr int NQ = KP / 4, NV = VP / 4;              // columns of dq, dk and of dv per thread
};

// Column sums over the 32 lanes of N = 8 or 16 values a lane: lane l gets
// column l·N/32's.
template <int N>
__device__ __forceinline__ float column_sums(float (&r)[N]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int w = N / 2; w; w >>= 1) {
        const int d = w * 32 / N;
        const bool up = lane & d;
#pragma unroll
        for (int e = 0; e < w; ++e) {
            const float send = up ? r[e] : r[e + w], keep = up ? r[e + w] : r[e];
            r[e] = keep + __shfl_xor_sync(~0u, send, d);
        }
    }
#pragma unroll
    for (int d = 16 / N; d; d >>= 1) r[0] += __shfl_xor_sync(~0u, r[0], d);
    return r[0];
}

// One source's block of 32 sinks: from the raw scores (lane = source s, 32
// columns of sinks t0..t0+31) P'ᵀ and dP'ᵀ in two bf16 terms, back over the scores
// in tensor memory (8 columns of high terms, 8 of low ones for every 16 sinks;
// dP'ᵀ where TS) and, dP'ᵀ, to `dp(column)` and, where LO, `dp_lo(column)` in shared memory; returns
// the source's sum of paths into the block, and leaves in cut[] by gate u the
// sums over the warp's sources before u of the paths to sinks u.. of the block.
// The decay is r·c[t].  `first`: the lane in the source's own block (sinks t >=
// s), else -1.  ZERO: the chunk has gates beneath the floor, paths through which
// are smaller in everything but df, or blocks too steep for the product: the diagonal takes
// an exponential each.  (One body for diagonal and other blocks: the two would
// not fit the instruction cache together.)
// PW: columns at a time, 16 or, where registers are short, 8.
template <bool ZERO, int PW, bool TS, bool LO, class Place, class PlaceLo>
__device__ __forceinline__ float score_block(uint32_t tp, uint32_t tdp, const LaTablesZ* tab, int t0, float Fs, float Is,
                                             float Zs, float r, int first, float* cut, Place dp, PlaceLo dp_lo) {
    const int lane = threadIdx.x & 31;
    float run = 0.f;
#pragma unroll
    for (int h = 16; h >= 0; h -= 16) {
        uint32_t pp[8], ppl[8], pd[8], pdl[8];
#pragma unroll
        for (int g = 16 - PW; g >= 0; g -= PW) {
            uint32_t x[PW], y[PW];
            tmem_ld<PW>(tp + h + g, x);
            tmem_ld<PW>(tdp + h + g, y);
            float d[PW], z[ZERO ? PW : 1];
#pragma unroll
            for (int e = 0; e < PW; e += 4) {
                const int at = h + g + e;
                const float4 c = *reinterpret_cast<const float4*>(&tab->c[t0 + at]);
                d[e] = r * c.x; d[e + 1] = r * c.y; d[e + 2] = r * c.z; d[e + 3] = r * c.w;
                if (ZERO && first >= 0) {
                    const float4 f = *reinterpret_cast<const float4*>(&tab->F[t0 + at]);
                    const float4 w = la_whole(tab, t0 + at);
                    d[e] = ex2_approx((f.x - Fs) + (w.x - Is)); d[e + 1] = ex2_approx((f.y - Fs) + (w.y - Is));
                    d[e + 2] = ex2_approx((f.z - Fs) + (w.z - Is)); d[e + 3] = ex2_approx((f.w - Fs) + (w.w - Is));
                }
#pragma unroll
                for (int o = 0; o < 4; ++o) d[e + o] = at + o >= first ? d[e + o] : 0.f;
                if constexpr (ZERO) {
                    const float4 zs = *reinterpret_cast<const float4*>(&tab->Z[t0 + at]);
                    // (Z falls with t: before the source, where d is 0, the difference is positive)
                    z[e] = d[e] * ex2_approx(fminf(zs.x - Zs, 0.f));
                    z[e + 1] = d[e + 1] * ex2_approx(fminf(zs.y - Zs, 0.f));
                    z[e + 2] = d[e + 2] * ex2_approx(fminf(zs.z - Zs, 0.f));
                    z[e + 3] = d[e + 3] * ex2_approx(fminf(zs.w - Zs, 0.f));
                }
            }
            tc_wait_ld();
            reg_fence(x);
            reg_fence(y);
            float R[PW];
#pragma unroll
            for (int e = PW - 2; e >= 0; e -= 2) {
                const float2 P = make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])),
                             Q = make_float2(__uint_as_float(y[e]), __uint_as_float(y[e + 1])),
                             D = make_float2(d[e], d[e + 1]);
                float2 PD = __fmul2_rn(P, D);
                const float2 W = __fmul2_rn(PD, Q);
                float2 QD = __fmul2_rn(Q, D);
                if constexpr (ZERO) {
                    const float2 Zd = make_float2(z[e], z[e + 1]);
                    PD = __fmul2_rn(P, Zd);
                    QD = __fmul2_rn(Q, Zd);
                }
                split2(PD.x, PD.y, pp[(g + e) / 2], ppl[(g + e) / 2]);
                split2(QD.x, QD.y, pd[(g + e) / 2], pdl[(g + e) / 2]);
                run += W.y;
                R[e + 1] = h + g + e + 1 > first ? run : 0.f;   // sources strictly before the gate
                run += W.x;
                R[e] = h + g + e > first ? run : 0.f;
            }
#pragma unroll
            for (int e = 0; e < PW; e += 8) {
                const int w = (g + e) / 2;
                *reinterpret_cast<uint4*>(dp(t0 + h + g + e)) = make_uint4(pd[w], pd[w + 1], pd[w + 2], pd[w + 3]);
                if (LO) *reinterpret_cast<uint4*>(dp_lo(t0 + h + g + e)) = make_uint4(pdl[w], pdl[w + 1], pdl[w + 2], pdl[w + 3]);
            }
            const float c = column_sums(R);
            if (!(lane & (32 / PW - 1))) cut[t0 + h + g + lane / (32 / PW)] = c;
        }
        tmem_st_32x32b<8>(tp + h, pp);       // inside the half that has been read
        tmem_st_32x32b<8>(tp + h + 8, ppl);
        if constexpr (TS) {
            tmem_st_32x32b<8>(tdp + h, pd);
            tmem_st_32x32b<8>(tdp + h + 8, pdl);
        }
    }
    return run;
}

template <int KP, int VP>
__global__ void __launch_bounds__(BCfg<KP, VP>::kThreads, 1)
    m2rnn_la_bwd_tc_kernel(const LaParams p, const __grid_constant__ BwdMaps maps) {
    using C = BCfg<KP, VP>;
    constexpr int NW = C::NW;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int bh = blockIdx.x / p.segs, seg = blockIdx.x % p.segs;
    const int nchunks = (p.T + kLaChunk - 1) / kLaChunk;
    const int c0 = seg * p.seg_chunks, n = min(nchunks - c0, p.seg_chunks);
    auto chunk_of = [&](int i) { return c0 + n - 1 - i; };
    auto stage_of = [&](int i) { return i % C::kStages; };
    auto stage_phase = [&](int i) { return (uint32_t)(i / C::kStages) & 1u; };

    LaTablesZ* tab = reinterpret_cast<LaTablesZ*>(smem + C::kOffTab);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    const uint32_t b_full = bar(0), r_s = bar(2), b_in = bar(3), r_g = bar(4), b_g = bar(5), r_p = bar(6),
                   b_dv = bar(7), r_dv = bar(8), b_out = bar(9), r_aq = bar(10), b_dg = bar(11), r_out = bar(12),
                   b_free = bar(13), b_tab = bar(14), b_drain = bar(15), b_sc = bar(16),
                   r_df = bar(17);   // two, for chunks in turn: the copies may be a chunk behind df
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kBars);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    float* gammas = reinterpret_cast<float*>(smem + C::kOffGamma);
    const LaLimit limit = p.limit;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 19; ++i) mbar_init(bar(i), 1);
        for (uint32_t b : {r_s, r_g, r_p, r_dv, r_aq, r_out}) mbar_init(b, NW);   // one arrival a warp
        if (!C::kRoomy) mbar_init(b_full, 2);   // dy comes later than the other tiles
        *abort_flag = 0;
        fence_mbarrier_init();
    }
    if (warp == NW) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    constexpr uint32_t tmem = 0;   // the CTA has all 512 columns
    const uint32_t sbase = smem_u32(smem);

    if (warp == NW) {
        // ------------------------------------------------------ products
        constexpr uint32_t id_sc = idesc_bf16_f32(128, 128, 0, 0),     // scores
            id_ki = idesc_bf16_f32(128, KP, 0, 0),                     // dY Sᵀ, V Gᵀ
            id_vi = idesc_bf16_f32(128, VP, 0, 1),                     // K G; P'ᵀ dY
            id_dq = idesc_bf16_f32(128, KP, 1, 1),                     // dP' K
            id_dk = idesc_bf16_f32(128, KP, 0, 1),                     // dP'ᵀ Q
            id_dg = idesc_bf16_f32(KP, VP, 1, 1);                      // (a Q)ᵀ dY
        const Desc d_tile = sw128_desc(sbase, 16), d_mn = sw128_desc(sbase, kTileBytes),
                       d_op = sw128_desc(sbase, KP * 128);
        const uint32_t one = lane == 0;
        constexpr uint32_t X = C::kOffX >> 4, OP = C::kOp >> 4, XP = C::kOffP >> 4;
        auto kmajor = [](int ks, int rows) { return (uint32_t)((ks >> 2) * (rows * 128 >> 4) + (ks & 3) * 2); };
        // rows (128 tokens) times a state in three terms, the first two at x; the
        // smallest first: an accumulation rounds at the size that the sum has by then
        auto times_state = [&](uint32_t d, uint32_t rows, uint32_t x) {
#pragma unroll
            for (int e = 2; e >= 0; --e) {
                const uint32_t op = e < 2 || C::kRoomy ? x + e * OP : XP;
#pragma unroll
                for (int ks = 0; ks < VP / 16; ++ks)
                    mma_ss(d, d_tile + rows + kmajor(ks, 128), d_op + op + kmajor(ks, KP), id_ki,
                                  e < 2 || ks > 0, one);
            }
        };
        auto tiles = [&](int i, uint32_t& q, uint32_t& k, uint32_t& v, uint32_t& dy) {
            q = (C::kOffStage + stage_of(i) * C::kStage) >> 4;
            k = q + (C::kQ >> 4);
            v = k + (C::kQ >> 4);
            dy = v + (C::kV >> 4);
        };
        auto scores = [&](int i) {
            uint32_t q, k, v, dy;
            tiles(i, q, k, v, dy);
#pragma unroll
            for (int ks = 0; ks < KP / 16; ++ks)
                mma_ss(C::kP, d_tile + k + kmajor(ks, 128), d_tile + q + kmajor(ks, 128), id_sc, ks > 0, one);
#pragma unroll
            for (int ks = 0; ks < VP / 16; ++ks)
                mma_ss(C::kDP, d_tile + v + kmajor(ks, 128), d_tile + dy + kmajor(ks, 128), id_sc, ks > 0, one);
            mma_commit(b_sc, one);
        };
        bool ok = true;
        for (int i = 0; i < n; ++i) {
            const int ph = i & 1;
            uint32_t q, k, v, dy;
            tiles(i, q, k, v, dy);
            auto inter_dv = [&]() {   // K G with G's first two terms
#pragma unroll
                for (int e = 1; e >= 0; --e)
#pragma unroll
                    for (int ks = 0; ks < KP / 16; ++ks)
                        mma_ss(C::kDV, d_tile + k + kmajor(ks, 128), d_op + X + (C::kG0 >> 4) + e * OP + ks * 128, id_vi,
                               e < 1 || ks > 0, one);
            };
            if (!(ok = la_wait(b_full + stage_of(i) * 8, stage_phase(i), abort_flag, limit))) break;
            if (C::kEarly) {
                if (i > 0 && !(ok = la_wait(b_out, ph ^ 1, abort_flag, limit))) break;
                scores(i);
            }
            if (!(ok = la_wait(r_s, ph, abort_flag, limit))) break;
            tc_fence_after();
            if (!C::kEarly && C::kRoomy) scores(i);
            times_state(C::kDQ, dy, X);                     // dY Sᵀ
            if (C::kRoomy) {
                times_state(C::kDK, v, X + (C::kG0 >> 4));  // V Gᵀ
                if (C::kOwnDv) inter_dv();
            }
            mma_commit(b_in, one);
            if (!C::kRoomy) scores(i);
            if (!C::kRoomy) {
                if (!(ok = la_wait(r_g, ph, abort_flag, limit))) break;
                tc_fence_after();
                times_state(C::kDK, v, X);
                mma_commit(b_g, one);
            }
            auto sum_for_G = [&]() -> bool {
                if (!la_wait(r_aq, ph, abort_flag, limit)) return false;
                // 64 x 128: its columns hold dk's operand until the products with that are done
                if (C::kDG == C::kDP && KP == 64 && !la_wait(b_out, ph, abort_flag, limit)) return false;
                tc_fence_after();
#pragma unroll
                for (int x = 2; x >= 0; --x) {      // the terms of a q
                    const uint32_t op = x < 2 || C::kRoomy ? X + x * (C::kQ >> 4) : XP;
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        mma_ss(C::kDG, d_mn + op + ks * 128, d_mn + dy + ks * 128, id_dg,
                                      x < 2 || ks > 0, one);
                }
                mma_commit(b_dg, one);
                return true;
            };
            if (!(ok = la_wait(r_p, ph, abort_flag, limit))) break;
            tc_fence_after();
            if (!C::kOwnDv) {
                inter_dv();
                mma_commit(b_dv, one);
            }
            // the low terms first.  dq: contraction over s, the rows of the dP'ᵀ and k tiles
            const uint32_t lo = C::kOffLo >> 4;   // (the v tile has one stage where it takes the low term)
            const Desc d_lo = C::kLateLo ? sw128_desc(sbase, C::kOffStage + stage_of(i) * C::kStage + 2 * C::kQ) : d_mn + lo;
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                if (ks < 4) mma_ss(C::kDQ, d_lo + ks * 128, d_mn + k + ks * 128, id_dq, 1, one);
                else mma_ss_half<true>(C::kDQ, d_lo + ks * 128, d_mn + k + ks * 128, id_dq, one);   // sinks t >= 64
            }
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) mma_ss(C::kDQ, d_mn + XP + ks * 128, d_mn + k + ks * 128, id_dq, 1, one);
            // dk and dv: over t, 16 sinks at a time, A from tensor memory (8 columns each term) or the dP'ᵀ tiles
#pragma unroll
            for (int x = 1; x >= 0; --x)
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {
                    const Desc b = d_mn + q + ks * 128;
                    if (KP == 64) mma_ts(C::kDK, C::kDP + ks * 16 + x * 8, b, id_dk, 1, one);
                    else if (x == 0) mma_ss(C::kDK, d_tile + XP + kmajor(ks, 128), b, id_dk, 1, one);
                    else if (ks >= 4) mma_ss(C::kDK, d_tile + lo + kmajor(ks, 128), b, id_dk, 1, one);
                    else mma_ss_half<false>(C::kDK, d_tile + lo + kmajor(ks, 128), b, id_dk, one);   // sources s < 64
                }
            if (!C::kOwnDv) {
                if (!(ok = la_wait(r_dv, ph, abort_flag, limit))) break;
                tc_fence_after();
            }
#pragma unroll
            for (int x = 1; x >= 0; --x)
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) mma_ts(C::kDV, C::kP + ks * 16 + x * 8, d_mn + dy + ks * 128, id_vi, 1, one);
            mma_commit(b_out, one);
            if (!(ok = sum_for_G())) break;
        }
        mma_commit(b_drain, one);   // nothing is in flight when the CTA ends
        if (lane == 0) la_drain(b_drain, 0, limit);
        __syncwarp();
    } else if (warp == NW + 1) {
        // ------------------------------------------------------ copies
        if (lane == 0) {
            const int qk = la_qk_pair(p, bh);
            int loaded = 0, started = 0;   // chunks whose every load, whose first load has been issued
            auto load = [&](int i, bool rest, bool dys) {   // the q, k and v tiles, the dy tile
                if (p.fault == 1 && i > 0) return;   // injected: the copies stop after the first chunk
                if (rest) started = i + 1;
                if (dys) loaded = i + 1;
                const int t = chunk_of(i) * kLaChunk;
                const uint32_t base = sbase + C::kOffStage + stage_of(i) * C::kStage, full = b_full + stage_of(i) * 8;
                if (C::kRoomy) {
                    mbar_arrive_expect_tx(full, C::kStage);
                } else {
                    if (rest) mbar_arrive_expect_tx(full, C::kStage - C::kV);
                    if (dys) mbar_arrive_expect_tx(full, C::kV);
                }
                if (dys)
#pragma unroll
                    for (int x = 0; x < VP / 64; ++x)
                        tma_tile(base + 2 * C::kQ + C::kV + x * kTileBytes, &maps.dy, x * 64, t, bh, full);
                if (!rest) return;
#pragma unroll
                for (int x = 0; x < KP / 64; ++x) {
                    tma_tile(base + x * kTileBytes, &maps.q, x * 64, t, qk, full);
                    tma_tile(base + C::kQ + x * kTileBytes, &maps.k, x * 64, t, qk, full);
                }
#pragma unroll
                for (int x = 0; x < VP / 64; ++x)
                    tma_tile(base + 2 * C::kQ + x * kTileBytes, &maps.v, x * 64, t, bh, full);
            };
            // the next chunk's checkpoint into L2 (its tiles too, or two chunks
            // ahead, was 8% slower for 128 pairs of 128 x 128 over 4096 tokens)
            auto prefetch = [&](int i) {
                if (i < n && !p.fault)
                    bulk_prefetch(p.ckpt + ((size_t)bh * nchunks + chunk_of(i)) * p.K * p.V, p.K * p.V * 4);
            };
            for (int i = 0; i < C::kStages && i < n; ++i) load(i, true, true);
            bool ok = true;
            int i = 0;
            for (; i < n; ++i) {
                prefetch(i + 1);
                if (!C::kRoomy) {
                    if (!(ok = la_wait_lane(r_aq, i & 1, abort_flag, limit) &&
                          la_wait_lane(r_df + (i & 1) * 8, (i >> 1) & 1, abort_flag, limit))) break;
                    if (i + 1 < n) load(i + 1, true, false);
                    if (!(ok = la_wait_lane(b_dg, i & 1, abort_flag, limit))) break;
                    if (i + 1 < n) load(i + 1, false, true);
                    continue;
                }
                const int ph = i & 1, t = chunk_of(i) * kLaChunk;
                const uint32_t base = sbase + C::kOffStage + stage_of(i) * C::kStage;
                if (!(ok = la_wait_lane(r_out, ph, abort_flag, limit))) break;
                if (!p.dkq_fp32)
                    for (int x = 0; x < KP / 64; ++x)
                        if (x * 64 < p.K) {
                            tma_store_tile(&maps.dq, (C::kOwnScratch ? base + 2 * C::kQ : sbase + C::kOffP) + x * kTileBytes,
                                           x * 64, t, bh);
                            tma_store_tile(&maps.dk, base + x * kTileBytes, x * 64, t, bh);
                        }
                for (int x = 0; x < VP / 64; ++x)
                    if (x * 64 < p.V)
                        tma_store_tile(&maps.dv, base + 2 * C::kQ + C::kV + x * kTileBytes, x * 64, t, bh);
                tma_store_commit();
                tma_store_wait_read();
                mbar_arrive(b_free);
                if (!(ok = la_wait_lane(r_df + ph * 8, (i >> 1) & 1, abort_flag, limit))) break;
                if (i + C::kStages < n) load(i + C::kStages, true, true);
            }
            if (!ok) {   // leave no copy in flight
                if (!C::kRoomy && loaded < started) load(started - 1, false, true);
                for (int j = i; j < loaded; ++j) la_drain(b_full + stage_of(j) * 8, stage_phase(j), limit);
            }
        }
        __syncwarp();
    } else if (warp == NW + 2) {
        // ------------------------------------------------------ decays and df: four tokens a lane
        float fx[4], fnext[4];
        la_load_f(p, bh, chunk_of(0), fx);
        if (n > 1) la_load_f(p, bh, chunk_of(1), fnext);
        la_tables<true>(tab, p, fx, p.T - chunk_of(0) * kLaChunk, kLogFloorBwd);
        __syncwarp();
        if (lane == 0) mbar_arrive(b_tab);
        for (int i = 0; i < n; ++i) {
            const int ph = i & 1, c = chunk_of(i);
            if (!la_wait(r_p, ph, abort_flag, limit)) break;
            const DfScratch* sc = reinterpret_cast<const DfScratch*>(
                smem + (C::kOwnScratch ? C::kOffScratch : C::kOffStage + stage_of(i) * C::kStage + 2 * C::kQ + C::kAtScratch));
            const int block = lane >> 3, t0 = lane * 4;
            float x[4] = {0.f, 0.f, 0.f, 0.f}, al[4], be[4], past[3][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                al[e] = be[e] = 0.f;
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    al[e] += sc->alpha[g][t0 + e];
                    be[e] += sc->beta[g][t0 + e];
                    x[e] += g <= block ? sc->cut[g][t0 + e] : 0.f;
                }
                // this source's paths to sinks beyond block J
                past[2][e] = sc->total[3][t0 + e];
                past[1][e] = past[2][e] + sc->total[2][t0 + e];
                past[0][e] = past[1][e] + sc->total[1][t0 + e];
            }
            float gamma = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) gamma += gammas[w];
            __syncwarp();
            if (lane == 0) mbar_arrive(r_df + ph * 8);
            // sums over sources before each token of this lane (exclusive)
            auto before = [&](const float (&v)[4], float (&o)[4]) {
                float s[4] = {v[0], v[0] + v[1], v[0] + v[1] + v[2], v[0] + v[1] + v[2] + v[3]};
                float run = s[3];
#pragma unroll
                for (int d = 1; d < 32; d *= 2) {
                    const float y = __shfl_up_sync(~0u, run, d);
                    if (lane >= d) run += y;
                }
                const float pre = __shfl_up_sync(~0u, run, 1);
                o[0] = lane ? pre : 0.f;
#pragma unroll
                for (int e = 1; e < 4; ++e) o[e] = o[0] + s[e - 1];
            };
            float o[4];
            before(be, o);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] += o[e] + gamma;
#pragma unroll
            for (int J = 0; J < 3; ++J) {
                before(past[J], o);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] += block == J ? o[e] : 0.f;
            }
            // sums over sinks from each token on (inclusive)
            float s[4] = {al[0] + al[1] + al[2] + al[3], al[1] + al[2] + al[3], al[2] + al[3], al[3]}, run = s[0];
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const float y = __shfl_down_sync(~0u, run, d);
                if (lane + d < 32) run += y;
            }
            float post = __shfl_down_sync(~0u, run, 1);
            post = lane < 31 ? post : 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[e] += s[e] + post;
                const int t = c * kLaChunk + t0 + e;
                if (t < p.T) {
                    // x = f df: the gate's gradient, or the logit's, df f (1 - f) with 1 - f = 1/(1 + e^a)
                    // (a gate at the floor: df times the gate itself)
                    const float f = la_gate(p, fx[e]), g = f < kGateFloorBwd ? kGateFloorBwd : f;
                    p.df[(size_t)bh * p.T + t] =
                        !p.f_is_logit ? x[e] / g : x[e] * (f < kGateFloorBwd ? f / g : 1.f) / (1.f + expf(fx[e]));
                }
            }
            if (i + 1 < n) {
#pragma unroll
                for (int e = 0; e < 4; ++e) fx[e] = fnext[e];
                if (i + 2 < n) la_load_f(p, bh, chunk_of(i + 2), fnext);
                la_tables<true>(tab, p, fx, p.T - chunk_of(i + 1) * kLaChunk, kLogFloorBwd);
                __syncwarp();
                if (lane == 0) mbar_arrive(b_tab);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------ elementwise work
        const int wg = warp >> 2, quarter = warp & 3;
        const int row = quarter * 32 + lane;                     // token of the chunk
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;   // tensor-memory lane base
        const uint32_t mylane = tmem + lanes;
        // this thread's part of S and G: row kap, columns [v0, v0 + NS)
        const int kap = KP == 128 ? row : quarter * 16 + (lane & 15);
        const int v0 = KP == 128 ? wg * C::NS : (wg * 2 + (lane >> 4)) * C::NS;
        const bool mine = kap < p.K;
        float G[C::NS];
        {
            const float* src = p.segs > 1 ? p.seg_state + ((size_t)bh * p.segs + seg) * p.K * p.V
                               : p.dST    ? p.dST + (size_t)bh * p.K * p.V
                                          : nullptr;
#pragma unroll
            for (int j = 0; j < C::NS; j += 4) {
                const float4 x = src && mine && v0 + j < p.V
                                     ? *reinterpret_cast<const float4*>(src + (size_t)kap * p.V + v0 + j)
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
                G[j] = x.x; G[j + 1] = x.y; G[j + 2] = x.z; G[j + 3] = x.w;
            }
        }
        auto arrive = [&](uint32_t b) {   // this warp's writes are done: shared memory for the products, tensor memory
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(b);
        };
        // three bf16 terms of a state's elements j..j+7, the first two from x on
        auto put_terms = [&](const float (&v)[8], int j, int x) {
            uint4 hi, mid, lo;
            split3(v[0], v[1], hi.x, mid.x, lo.x);
            split3(v[2], v[3], hi.y, mid.y, lo.y);
            split3(v[4], v[5], hi.z, mid.z, lo.z);
            split3(v[6], v[7], hi.w, mid.w, lo.w);
            const uint32_t at = (v0 >> 6) * (KP * 128) + sw128(kap, ((v0 & 63) + j) >> 3);
            *reinterpret_cast<uint4*>(smem + x + at) = hi;
            *reinterpret_cast<uint4*>(smem + x + C::kOp + at) = mid;
            *reinterpret_cast<uint4*>(smem + (C::kRoomy ? x + 2 * C::kOp : C::kOffP) + at) = lo;
        };
        auto put_G = [&]() {
#pragma unroll
            for (int j = 0; j < C::NS; j += 8) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = G[j + e];
                put_terms(x, j, C::kOffX + C::kG0);
            }
        };
        float Sn[C::NS];   // the next chunk's S
        auto load_S = [&](int c) {
            const float* ck = p.ckpt + ((size_t)bh * nchunks + c) * p.K * p.V;
#pragma unroll
            for (int j = 0; j < C::NS; j += 4) {
                const float4 s4 = mine && v0 + j < p.V
                                      ? *reinterpret_cast<const float4*>(ck + ((size_t)((v0 + j) >> 2) * p.K + kap) * 4)
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
                Sn[j] = s4.x; Sn[j + 1] = s4.y; Sn[j + 2] = s4.z; Sn[j + 3] = s4.w;
            }
        };
        // the terms of S (and of G) for the chunk to come, and this thread's part of <S, G>
        float gamma_next = 0.f;
        auto put_S = [&]() {
            gamma_next = 0.f;
#pragma unroll
            for (int j = 0; j < C::NS; j += 8) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[e] = Sn[j + e];
                    gamma_next = fmaf(x[e], G[j + e], gamma_next);
                }
                put_terms(x, j, C::kOffX);
            }
            if (C::kRoomy) put_G();
            arrive(r_s);
        };
        load_S(chunk_of(0));
        put_S();
        constexpr bool kLoadEarly = C::NS <= 16;   // registers
        auto tile_at = [&](int col) { return (col >> 6) * kTileBytes + sw128(row, (col & 63) >> 3); };

        for (int i = 0; i < n; ++i) {
            const int ph = i & 1, c = chunk_of(i);
            uint8_t* stage = smem + C::kOffStage + stage_of(i) * C::kStage;
            float gamma = gamma_next;
            if (kLoadEarly && i + 1 < n) load_S(chunk_of(i + 1));
            if (!la_wait(b_tab, ph, abort_flag, limit)) break;
            const float Ft = tab->F[row], It = tab->I[row], Fe = tab->F[127], Ie = tab->I[127];
            const float Zt = tab->Z[row], Ze = tab->Z[127];
            // decays for df, and for everything else
            const float at0 = ex2_approx(Ft + It), bt0 = ex2_approx((Fe - Ft) + (Ie - It)), A0 = ex2_approx(Fe + Ie);
            const float at = at0 * ex2_approx(Zt), bt = bt0 * ex2_approx(Ze - Zt), A = A0 * ex2_approx(Ze);
            gamma *= A0;
#pragma unroll
            for (int d = 16; d; d >>= 1) gamma += __shfl_xor_sync(~0u, gamma, d);
            if (!la_wait(b_full + stage_of(i) * 8, stage_phase(i), abort_flag, limit)) break;
            if (!C::kRoomy) {
                if (!la_wait(b_in, ph, abort_flag, limit)) break;
                tc_fence_after();
                put_G();             // over the terms of S
                arrive(r_g);
            }
            // ---- a_t (S dy_t) and b_s (G v_s) in place, and their dot products with q and k
            auto scale_rows = [&](uint32_t col0, float w0, float w, const uint8_t* tile) {
                float dot = 0.f;
#pragma unroll
                for (int j = 0; j < C::NQ; j += 16) {
                    const int col = wg * C::NQ + j;
                    uint32_t x[16];
                    tmem_ld<16>(mylane + col0 + col, x);
                    const uint4 y0 = *reinterpret_cast<const uint4*>(tile + tile_at(col)),
                                y1 = *reinterpret_cast<const uint4*>(tile + tile_at(col + 8));
                    const uint32_t y[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
                    tc_wait_ld();
                    reg_fence(x);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float s = __uint_as_float(x[e]);
                        dot = fmaf(s, e & 1 ? bf16hi_to_f32(y[e / 2]) : bf16lo_to_f32(y[e / 2]), dot);
                        x[e] = __float_as_uint(w * s);
                    }
                    tmem_st16(mylane + col0 + col, x);
                }
                return w0 * dot;
            };
            auto scale_dv = [&]() {
#pragma unroll
                for (int j = 0; j < C::NV; j += 16) {
                    const int col = wg * C::NV + j;
                    uint32_t x[16];
                    tmem_ld<16>(mylane + C::kDV + col, x);
                    tc_wait_ld();
                    reg_fence(x);
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(bt * __uint_as_float(x[e]));
                    tmem_st16(mylane + C::kDV + col, x);
                }
            };
            DfScratch* sc = reinterpret_cast<DfScratch*>(C::kOwnScratch ? smem + C::kOffScratch
                                                                        : stage + 2 * C::kQ + C::kAtScratch);
            auto scale_all = [&]() -> bool {
                if (!la_wait(b_in, ph, abort_flag, limit)) return false;
                tc_fence_after();
                const float alpha = scale_rows(C::kDQ, at0, at, stage);
                if (!C::kRoomy && !la_wait(b_g, ph, abort_flag, limit)) return false;
                tc_fence_after();
                const float beta = scale_rows(C::kDK, bt0, bt, stage + C::kQ);
                if (C::kOwnDv) scale_dv();
                sc->alpha[wg][row] = alpha;
                sc->beta[wg][row] = beta;
                if (lane == 0) gammas[warp] = gamma;
                return true;
            };
            if (!C::kRoomy) {
                if (!scale_all()) break;
            } else {
                // the scratch and dP' may be written: df has been read, the states' products are done, dq has left
                if (!C::kOwnScratch && !la_wait(b_in, ph, abort_flag, limit)) break;
                if (C::kOwnScratch && i > 0 && !la_wait(r_df + (ph ^ 1) * 8, ((i - 1) >> 1) & 1, abort_flag, limit)) break;
                if (!C::kOwnScratch && i > 0 && !la_wait(b_free, ph ^ 1, abort_flag, limit)) break;
            }
            if (!la_wait(b_sc, ph, abort_flag, limit)) break;
            tc_fence_after();
            uint8_t* dp = smem + C::kOffP;
            // ---- a_t q_t in three terms
            auto put_aq = [&]() {
#pragma unroll
                for (int j = 0; j < C::NQ; j += 8) {
                    const uint32_t pos = tile_at(wg * C::NQ + j);
                    const uint4 x = *reinterpret_cast<const uint4*>(stage + pos);
                    uint4 hi, mid, lo;
                    split3(at * bf16lo_to_f32(x.x), at * bf16hi_to_f32(x.x), hi.x, mid.x, lo.x);
                    split3(at * bf16lo_to_f32(x.y), at * bf16hi_to_f32(x.y), hi.y, mid.y, lo.y);
                    split3(at * bf16lo_to_f32(x.z), at * bf16hi_to_f32(x.z), hi.z, mid.z, lo.z);
                    split3(at * bf16lo_to_f32(x.w), at * bf16hi_to_f32(x.w), hi.w, mid.w, lo.w);
                    uint8_t* X = smem + C::kOffX + pos;
                    *reinterpret_cast<uint4*>(X) = hi;
                    *reinterpret_cast<uint4*>(X + C::kQ) = mid;
                    *reinterpret_cast<uint4*>(C::kRoomy ? X + 2 * C::kQ : dp + pos) = lo;
                }
                arrive(r_aq);
            };
            // ---- P'ᵀ, dP'ᵀ and df's sums: source s = row, sinks of block wg
            float run = 0.f;
            auto place_lo = [&](int col) -> uint8_t* {
                if constexpr (C::kLateLo) return (col < 64 ? smem : stage + 2 * C::kQ) + sw128(row, (col & 63) >> 3);
                else return (C::kRoomy ? smem : stage) + C::kOffLo + tile_at(col);
            };
            const bool low = wg >= 2 || quarter < 2;   // the low term's rows s >= 64 of sinks t < 64 are not read
            if (wg < quarter) {   // sinks before the source
                const uint32_t z[16] = {};
#pragma unroll
                for (int e = 0; e < 32; e += 16) {
                    tmem_st16(mylane + C::kP + wg * 32 + e, z);
                    if (KP == 64) tmem_st16(mylane + C::kDP + wg * 32 + e, z);
                }
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    *reinterpret_cast<uint4*>(dp + tile_at(wg * 32 + e)) = make_uint4(0, 0, 0, 0);
                    if (!C::kLateLo && low) *reinterpret_cast<uint4*>(place_lo(wg * 32 + e)) = make_uint4(0, 0, 0, 0);
                }
            } else {
                const uint32_t tp = mylane + C::kP + wg * 32, tdp = mylane + C::kDP + wg * 32;
                float* cut = sc->cut[quarter];
                auto place = [&](int col) { return dp + tile_at(col); };
                const int first = wg == quarter ? lane : -1;
                // the decay from the source to the block before the sinks' (for its own block, a reciprocal)
                const float Fp = wg ? tab->F[wg * 32 - 1] : 0.f, Ip = wg ? tab->I[wg * 32 - 1] : 0.f;
                const float r = ex2_approx((Fp - Ft) + (Ip - It));
                constexpr int N = C::NS <= 16 ? 16 : 8;
                if (Ze != 0.f || tab->steep != 0.f)
                    run = score_block<true, N, KP == 64, !C::kLateLo>(tp, tdp, tab, wg * 32, Ft, It, Zt, r, first, cut, place, place_lo);
                else
                    run = score_block<false, N, KP == 64, !C::kLateLo>(tp, tdp, tab, wg * 32, Ft, It, Zt, r, first, cut, place, place_lo);
            }
            sc->total[wg][row] = run;
            if (C::kRoomy && !scale_all()) break;
            tc_wait_st();
            if (C::kLateLo && low) {
#pragma unroll
                for (int h = 0; h < 32; h += 16) {
                    uint32_t x[8];
                    tmem_ld<8>(mylane + C::kDP + wg * 32 + h + 8, x);
                    tc_wait_ld();
                    reg_fence(x);
                    *reinterpret_cast<uint4*>(place_lo(wg * 32 + h)) = make_uint4(x[0], x[1], x[2], x[3]);
                    *reinterpret_cast<uint4*>(place_lo(wg * 32 + h + 8)) = make_uint4(x[4], x[5], x[6], x[7]);
                }
            }
            arrive(r_p);
            if (!kLoadEarly && i + 1 < n) load_S(chunk_of(i + 1));
            if (!C::kOwnDv) {
                if (!la_wait(b_dv, ph, abort_flag, limit)) break;
                tc_fence_after();
                scale_dv();
                tc_wait_st();
                arrive(r_dv);
            }
            if (C::kEarlyAq) put_aq();   // over the terms of S, whose products are done
            if (!la_wait(b_out, ph, abort_flag, limit)) break;
            tc_fence_after();
            if (C::kRoomy && !C::kEarlyAq) put_aq();   // over the states' terms and the low term of dP'
            const int t = c * kLaChunk + row;
            // 16 columns of dq, dk or dv: the per-head parts of a shared q's or k's gradient, or packed
            auto take = [&](uint32_t col, uint32_t (&x)[16]) {
                tmem_ld<16>(mylane + col, x);
                tc_wait_ld();
                reg_fence(x);
            };
            auto part_out = [&](void* out, int col, const uint32_t (&x)[16]) {
                if (t >= p.T || col >= p.K) return;
                uint4* g = reinterpret_cast<uint4*>(static_cast<float*>(out) + ((size_t)bh * p.T + t) * p.K + col);
#pragma unroll
                for (int e = 0; e < 4; ++e) g[e] = make_uint4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
            };
            auto pack16 = [&](const uint32_t (&x)[16], uint32_t* o) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    o[e] = pack_bf16(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
            };
            auto stage_out = [&](uint8_t* tile, int col, const uint32_t* o) {
                *reinterpret_cast<uint4*>(tile + tile_at(col)) = make_uint4(o[0], o[1], o[2], o[3]);
                *reinterpret_cast<uint4*>(tile + tile_at(col + 8)) = make_uint4(o[4], o[5], o[6], o[7]);
            };
            // straight to the output, [pair][T][width] bf16
            auto rows_out = [&](void* out, int width, int col, const uint32_t* o) {
                if (t >= p.T || col >= width) return;
                __nv_bfloat16* g = static_cast<__nv_bfloat16*>(out) + ((size_t)bh * p.T + t) * width + col;
                if (p.out32) {
                    st_global_v8(g, o);
                } else {
                    *reinterpret_cast<uint4*>(g) = make_uint4(o[0], o[1], o[2], o[3]);
                    *reinterpret_cast<uint4*>(g + 8) = make_uint4(o[4], o[5], o[6], o[7]);
                }
            };
            uint32_t okk[C::kRoomy ? C::NQ / 2 : 8], ov[C::kRoomy ? C::NV / 2 : 8];
            // ---- dq, by way of dP' or the v tile
#pragma unroll
            for (int j = 0; j < C::NQ; j += 16) {
                const int col = wg * C::NQ + j;
                uint32_t x[16], o[8];
                take(C::kDQ + col, x);
                if (p.dkq_fp32) part_out(p.dq, col, x);
                pack16(x, o);
                if (C::kRoomy) stage_out(C::kOwnScratch ? stage + 2 * C::kQ : dp, col, o);
                else if (!p.dkq_fp32) rows_out(p.dq, p.K, col, o);
            }
            if (!C::kRoomy) put_aq();
            // ---- dk and dv, kept until their tiles are free
#pragma unroll
            for (int j = 0; j < C::NQ; j += 16) {
                const int col = wg * C::NQ + j;
                uint32_t x[16];
                take(C::kDK + col, x);
                if (p.dkq_fp32) part_out(p.dk, col, x);
                pack16(x, okk + (C::kRoomy ? j / 2 : 0));
                if (!C::kRoomy && !p.dkq_fp32) rows_out(p.dk, p.K, col, okk);
            }
#pragma unroll
            for (int j = 0; j < C::NV; j += 16) {
                const int col = wg * C::NV + j;
                uint32_t x[16];
                take(C::kDV + col, x);
                pack16(x, ov + (C::kRoomy ? j / 2 : 0));
                if (!C::kRoomy) rows_out(p.dv, p.V, col, ov);
            }
            // ---- G = A G + the chunk's sum
            if (!la_wait(b_dg, ph, abort_flag, limit)) break;
            tc_fence_after();
#pragma unroll
            for (int j = 0; j < C::NS; j += C::NL) {
                uint32_t d[C::NL];
                if constexpr (KP == 128)
                    tmem_ld<C::NL>(mylane + C::kDG + wg * C::NS + j, d);
                else   // threads 16..31: the same lanes, NS columns on
                    tmem_ld_16x32bx2<C::NL, C::NS>(mylane + C::kDG + wg * 2 * C::NS + j, d);
                tc_wait_ld();
                reg_fence(d);
#pragma unroll
                for (int e = 0; e < C::NL; ++e) G[j + e] = fmaf(A, G[j + e], __uint_as_float(d[e]));
            }
            if (i + 1 < n) put_S();   // every read of this chunk's sums is done, and every product of terms
            if (C::kRoomy) {
#pragma unroll
                for (int j = 0; j < C::NQ; j += 16) stage_out(stage, wg * C::NQ + j, okk + j / 2);
#pragma unroll
                for (int j = 0; j < C::NV; j += 16) stage_out(stage + 2 * C::kQ + C::kV, wg * C::NV + j, ov + j / 2);
                arrive(r_out);
            }
        }
        if (c0 == 0 && mine) {
#pragma unroll
            for (int j = 0; j < C::NS; j += 4)
                if (v0 + j < p.V)
                    *reinterpret_cast<float4*>(p.dS0 + (size_t)bh * p.K * p.V + (size_t)kap * p.V + v0 + j) =
                        make_float4(G[j], G[j + 1], G[j + 2], G[j + 3]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == NW) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int KP, int VP>
cudaError_t launch(const LaParams& p, const BwdMaps& m, cudaStream_t s) {
    using C = BCfg<KP, VP>;
    auto kern = m2rnn_la_bwd_tc_kernel<KP, VP>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    kern<<<p.B * p.H * p.segs, C::kThreads, C::kSmem, s>>>(p, m);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_la_bwd_tc(const LaParams& q, cudaStream_t s) {
    LaParams p = q;
    p.out32 = !((reinterpret_cast<uintptr_t>(p.dq) | reinterpret_cast<uintptr_t>(p.dk) |
                 reinterpret_cast<uintptr_t>(p.dv)) & 31u);
    const size_t qk = (size_t)p.B * p.G, vy = (size_t)p.B * p.H;
    BwdMaps m;
    if (!la_tensor_map(&m.q, p.q, p.K, p.T, qk) || !la_tensor_map(&m.k, p.k, p.K, p.T, qk) ||
        !la_tensor_map(&m.v, p.v, p.V, p.T, vy) || !la_tensor_map(&m.dy, p.dy, p.V, p.T, vy) ||
        !la_tensor_map(&m.dv, p.dv, p.V, p.T, vy))
        return cudaErrorNotSupported;
    m.dq = m.dk = m.dv;   // not used for per-head parts
    if (!p.dkq_fp32 && (!la_tensor_map(&m.dq, p.dq, p.K, p.T, vy) || !la_tensor_map(&m.dk, p.dk, p.K, p.T, vy)))
        return cudaErrorNotSupported;
    if (p.segs > 1) {
        const cudaError_t e = launch_la_seg_grads(p, s);
        if (e != cudaSuccess) return e;
    }
    if (p.K <= 64) return p.V <= 64 ? launch<64, 64>(p, m, s) : launch<64, 128>(p, m, s);
    return p.V <= 64 ? launch<128, 64>(p, m, s) : launch<128, 128>(p, m, s);
}

cudaError_t la_bwd_tc_status(unsigned slot, unsigned* word, cudaStream_t s) { return la_read_status(slot, word, s); }

}  // namespace m2rnn
