// Linear attention in chunks of 128 tokens on the tensor cores (bf16).
//
// With L_t the cumulative log-decay inside a chunk, D_ts = 2^(L_t - L_s),
// a_t = 2^(L_t), b_s = 2^(L_end - L_s) and S the state at its start,
//   y_t  = a_t (Q S)_t + ((Q Kᵀ ∘ D) V)_t          (s <= t)
//   S'   = a_end S + Σ_s (b_s k_s) v_sᵀ
// Four matrix products, every accumulator in tensor memory; the state's fp32
// master stays in registers over the whole walk.
//
// A CTA walks the chunks of one (b, h), or of one of its time segments.  16
// warps compute: thread = token row (or state row) = tensor-memory lane, the
// four warpgroups sharing the columns.  One more warp issues the products, one
// moves tiles, one computes decays a chunk ahead.  Only S -> Q S -> y and the
// state's sum -> S form a chain over the chunks; P of the next chunk is formed
// while the sum of this one is computed.
//
// Rounding: the masked scores and the copy of S that multiplies Q enter in two
// bf16 terms each (2^-16 of them is left out; each term of y passes through
// exactly one of them), so what rounds y is its own bf16: relative error 1.7e-3
// of the whole, against 2.3e-3 with one term each.  b_s k_s enters as three
// terms, so the state keeps fp32 accuracy over any number of chunks.
//
// Decays without an exponential per score: for a row t and a block of 32
// columns, D_ts = 2^(L_t - L_e)·2^(L_e - L_s) with e the block's last token.
// The second factor is shared by all rows.  Left of the diagonal both are at
// most 1; in the diagonal block the first is the reciprocal of a decay, within
// fp32's range unless the block decays by more than 2^-90: such chunks take one
// exponential per score there.
//
// Measured: 128 pairs of 64 x 64 over 2048 tokens 56 us (137 MB: 21.3 us at the
// copy rate of 6.45 TB/s), of 128 x 128 over 4096 tokens 177 us (547 MB: 84.9
// us); the second terms are 8 and 30 us of these.  Neither HBM nor the tensor pipe
// nor issue is full: a chunk's waits from product to elementwise work and back
// (2.9 and 5.1 us a chunk) bound it, with one CTA an SM (shared and tensor memory)
// and 128 of the 148 SMs.
#include <mutex>

#include "kernels.h"
#include "la_tc.cuh"

namespace m2rnn {

bool la_tensor_map(CUtensorMap* map, const void* x, int width, int T, size_t rows) {
    using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static Encode encode = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) ==
                cudaSuccess &&
            found == cudaDriverEntryPointSuccess)
            encode = reinterpret_cast<Encode>(fn);
    });
    if (!encode) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)T, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)width * 2, (cuuint64_t)width * 2 * T};
    const cuuint32_t box[3] = {64, 128, 1}, step[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(x), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

struct Maps {
    CUtensorMap q, k, v, y;
};

constexpr int kNW = 16, kFwdThreads = (kNW + 3) * 32;   // compute warps; one each for products, copies, decays

// Three bf16 terms of eight scaled values: two to their places, the third
// returned, or all three to their places.
__device__ __forceinline__ uint4 put_scaled(uint4 x, uint8_t* d0, uint8_t* d1, float w) {
    uint4 hi, mid, lo;
    split3(w * bf16lo_to_f32(x.x), w * bf16hi_to_f32(x.x), hi.x, mid.x, lo.x);
    split3(w * bf16lo_to_f32(x.y), w * bf16hi_to_f32(x.y), hi.y, mid.y, lo.y);
    split3(w * bf16lo_to_f32(x.z), w * bf16hi_to_f32(x.z), hi.z, mid.z, lo.z);
    split3(w * bf16lo_to_f32(x.w), w * bf16hi_to_f32(x.w), hi.w, mid.w, lo.w);
    *reinterpret_cast<uint4*>(d0) = hi;
    *reinterpret_cast<uint4*>(d1) = mid;
    return lo;
}
__device__ __forceinline__ void put_scaled(uint4 x, uint8_t* d0, uint8_t* d1, uint8_t* d2, float w) {
    *reinterpret_cast<uint4*>(d2) = put_scaled(x, d0, d1, w);
}

// A warp's writes are done (shared memory for the products, tensor memory):
// one arrival a warp.
__device__ __forceinline__ void warp_arrive(uint32_t b) {
    fence_proxy_async_smem();
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(b);
}

// Σ_s k_s ⊗ v_s over a chunk with one side in three scaled terms, into
// D[KP][VP].  a, b: the sides' first tiles (units of 16 bytes from the
// descriptor's start); astep, bstep: from one term to the next, 0 for the side
// that is not scaled.  The smallest terms come first: an accumulation rounds at
// the size that the sum has by then.
template <int KP, int VP>
__device__ __forceinline__ void outer_sum(uint32_t d, Desc mn, uint32_t a, uint32_t astep, uint32_t b, uint32_t bstep,
                                          uint32_t one) {
    constexpr uint32_t id = idesc_bf16_f32(KP, VP, 1, 1);
#pragma unroll
    for (int x = 2; x >= 0; --x)
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
            mma_ss(d, mn + a + x * astep + ks * 128, mn + b + x * bstep + ks * 128, id, x < 2 || ks > 0, one);
}

// The thread's part of a [KP][VP] accumulator or state: row kap, NS columns
// from v0.  128 rows have a tensor-memory lane each; 64 rows have 16 lanes in
// every quarter, which two half warps read.
template <int KP, int VP>
struct Part {
    static constexpr int NS = KP * VP / (kNW * 32), NL = NS < 16 ? NS : 16;
    int kap, v0;
    uint32_t col;   // tensor-memory column of the warp's load
    __device__ __forceinline__ Part() {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wg = warp >> 2, quarter = warp & 3;
        kap = KP == 128 ? quarter * 32 + lane : quarter * 16 + (lane & 15);
        v0 = KP == 128 ? wg * NS : (wg * 2 + (lane >> 4)) * NS;
        col = KP == 128 ? wg * NS : wg * 2 * NS;
    }
    // S = A S + the accumulator
    __device__ __forceinline__ void add(uint32_t acc, float A, float (&S)[NS]) const {
#pragma unroll
        for (int j = 0; j < NS; j += NL) {
            uint32_t d[NL];
            if constexpr (KP == 128) tmem_ld<NL>(acc + col + j, d);
            else tmem_ld_16x32bx2<NL, NS>(acc + col + j, d);   // threads 16..31: the same lanes, NS columns on
            tc_wait_ld();
            reg_fence(d);
#pragma unroll
            for (int e = 0; e < NL; ++e) S[j + e] = fmaf(A, S[j + e], __uint_as_float(d[e]));
        }
    }
    __device__ __forceinline__ void load(const float* src, int K, int V, float (&S)[NS]) const {
#pragma unroll
        for (int j = 0; j < NS; j += 4) {
            const float4 x = src && kap < K && v0 + j < V ? *reinterpret_cast<const float4*>(src + (size_t)kap * V + v0 + j)
                                                          : make_float4(0.f, 0.f, 0.f, 0.f);
            S[j] = x.x; S[j + 1] = x.y; S[j + 2] = x.z; S[j + 3] = x.w;
        }
    }
    __device__ __forceinline__ void store(float* dst, int K, int V, const float (&S)[NS]) const {
#pragma unroll
        for (int j = 0; j < NS; j += 4)
            if (kap < K && v0 + j < V)
                *reinterpret_cast<float4*>(dst + (size_t)kap * V + v0 + j) = make_float4(S[j], S[j + 1], S[j + 2], S[j + 3]);
    }
};

// The decay warp: tables of the walk's chunks into two buffers in turn, a chunk
// ahead of their use.  b_tab, t_free: two barriers each, one per buffer.
template <class ChunkOf>
__device__ __forceinline__ void decay_warp(const LaParams& p, int bh, int n, ChunkOf chunk_of, LaTables* tab, uint32_t b_tab,
                                           uint32_t t_free, volatile int* abort_flag) {
    float fx[4], fnext[4];
    la_load_f(p, bh, chunk_of(0), fx);
    for (int i = 0; i < n; ++i) {
        if (i + 1 < n) la_load_f(p, bh, chunk_of(i + 1), fnext);
        if (i >= 2 && !la_wait(t_free + (i & 1) * 8, ((i - 2) >> 1) & 1, abort_flag, p.limit)) break;
        la_tables(tab + (i & 1), p, fx, p.T - chunk_of(i) * kLaChunk, kLogFloorFwd);
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(b_tab + (i & 1) * 8);
#pragma unroll
        for (int e = 0; e < 4; ++e) fx[e] = fnext[e];
    }
    __syncwarp();
}

// ------------------------------------------------------------------ forward

template <int KP, int VP>
struct Cfg {
    static constexpr int kQ = KP / 64 * kTileBytes, kV = VP / 64 * kTileBytes, kStage = 2 * kQ + kV;
    static constexpr int kStages = KP == 64 && VP == 64 ? 3 : 2;
    static constexpr bool kScaleV = VP < KP;                    // the narrower side carries the decays
    static constexpr int kTerm = kScaleV ? kV : kQ;
    // 128 x 128 has no room for the scaled side's three terms: they go over the
    // k tile, the q tile and the state operand, once Q S is done.  The state's low
    // term goes over the k tile before that, whose values wait in registers.
    static constexpr bool kInPlace = KP * VP == 128 * 128;
    // 128 x 64 has room for all but the state's low term: it shares its place
    // with the scaled side's third
    static constexpr bool kShareLo = KP == 128 && VP == 64;
    static constexpr bool kStageY = !kInPlace && VP <= KP;      // y by TMA, over the q tile; else from registers
    static constexpr int kOffS = kStages * kStage;              // bf16 state operand [KP][VP]
    static constexpr int kOffX = kOffS + KP * VP * 2;           // the terms
    static constexpr int kOffLo = kOffX + (kShareLo ? 2 : 3) * kTerm;   // the state operand's low term
    static constexpr int kOffTab = kInPlace ? kOffX : kOffLo + KP * VP * 2;
    static constexpr int kOffBar = kOffTab + 2 * (int)sizeof(LaTables);
    static constexpr int kBars = 22;
    static constexpr int kSmem = kOffBar + kBars * 8 + 16;
    static_assert(kSmem <= 227 * 1024, "shared memory");
    static_assert(!kInPlace || KP * VP * 2 <= kQ, "the state's low term over the k tile");
    static_assert(!kShareLo || KP * VP * 2 <= kTerm, "the state's low term over the third of the scaled side");
    // tensor memory: scores (two of them where they fit: the next chunk's are
    // computed early), P·V, Q·S, the state's sum
    static constexpr int kScores = VP == 64 ? 2 : 1;
    static constexpr int kPV = kScores * 128, kQS = kPV + VP, kDS = kQS + VP;
    static_assert(kDS + VP <= 512, "tensor memory");
    static constexpr int NY = VP / 4;                           // columns of y per thread
};

template <int KP, int VP>
__global__ void __launch_bounds__(kFwdThreads, 1)
    m2rnn_la_fwd_tc_kernel(const LaParams p, const __grid_constant__ Maps maps) {
    using C = Cfg<KP, VP>;
    using Pt = Part<KP, VP>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int bh = blockIdx.x / p.segs, seg = blockIdx.x % p.segs;
    const int nchunks = (p.T + kLaChunk - 1) / kLaChunk;
    const int c0 = seg * p.seg_chunks, n = min(nchunks - c0, p.seg_chunks);
    auto chunk_of = [&](int i) { return c0 + i; };
    auto stage_of = [&](int i) { return i % C::kStages; };
    auto stage_phase = [&](int i) { return (uint32_t)(i / C::kStages) & 1u; };

    LaTables* tab = reinterpret_cast<LaTables*>(smem + C::kOffTab);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    // b_qk, b_v: one per stage; pairs of barriers serve chunks in turn, where one side may be a chunk ahead
    const uint32_t b_qk = bar(0), b_v = bar(3), b_sc = bar(6), b_tab = bar(8), t_free = bar(10), r_y = bar(12),
                   r_p = bar(14), r_s = bar(15), r_k = bar(16), b_pv = bar(17), b_ds = bar(18), b_drain = bar(19),
                   r_raw = bar(20);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kBars);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const LaLimit limit = p.limit;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 21; ++i) mbar_init(bar(i), 1);
        for (uint32_t b : {t_free, t_free + 8, r_y, r_y + 8, r_p, r_s, r_k, r_raw}) mbar_init(b, kNW);
        *abort_flag = 0;
        fence_mbarrier_init();
    }
    if (warp == kNW) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    constexpr uint32_t tmem = 0;   // the CTA has all 512 columns
    const uint32_t sbase = smem_u32(smem);

    if (warp == kNW) {
        // ------------------------------------------------------ products
        constexpr uint32_t id_sc = idesc_bf16_f32(128, 128, 0, 0), id_v = idesc_bf16_f32(128, VP, 0, 1);
        const Desc d_tile = sw128_desc(sbase, 16), d_mn = sw128_desc(sbase, kTileBytes),
                       d_op = sw128_desc(sbase, KP * 128);   // the state operand's terms
        constexpr uint32_t X = C::kOffX >> 4, XS = C::kTerm >> 4;
        auto tile = [](int ks) { return (uint32_t)((ks >> 2) * (kTileBytes >> 4) + (ks & 3) * 2); };
        const uint32_t one = lane == 0;
        auto scores = [&](int i) {   // Q Kᵀ
            const uint32_t q = stage_of(i) * (C::kStage >> 4), k = q + (C::kQ >> 4);
            tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < KP / 16; ++ks)
                mma_ss((i % C::kScores) * 128, d_tile + q + tile(ks), d_tile + k + tile(ks), id_sc, ks > 0, one);
            mma_commit(b_sc + (i & 1) * 8, one);
        };
        // P V, Q S (which waits for S) and the state's sum of a chunk in this order,
        // the next chunk's scores as soon as its tiles are there and their place is free
        if (la_wait(b_qk, 0, abort_flag, limit)) {
            scores(0);
            for (int i = 0; i < n; ++i) {
                const int ph = i & 1, s = stage_of(i), s1 = stage_of(i + 1);
                const uint32_t q = s * (C::kStage >> 4), k = q + (C::kQ >> 4), v = k + (C::kQ >> 4);
                bool next = i + 1 == n;
                auto next_scores = [&](bool wait) -> bool {
                    if (next) return true;
                    if (wait) {
                        if (C::kScores == 1 && !la_wait(b_pv, ph, abort_flag, limit)) return false;
                        if (!la_wait(b_qk + s1 * 8, stage_phase(i + 1), abort_flag, limit)) return false;
                    } else if (!__all_sync(~0u, (C::kScores == 2 || mbar_test_wait(b_pv, ph)) &&
                                                    mbar_test_wait(b_qk + s1 * 8, stage_phase(i + 1)))) {
                        return true;
                    }
                    scores(i + 1);
                    next = true;
                    return true;
                };
                if (!la_wait(b_v + s * 8, stage_phase(i), abort_flag, limit)) break;
                if (!la_wait(r_p, ph, abort_flag, limit)) break;
                tc_fence_after();
#pragma unroll
                for (int x = 1; x >= 0; --x)         // the low terms first
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)   // P: of each block's 32 columns 16 of high terms (bf16 pairs), 16 of low ones
                        mma_ts(C::kPV, (i % C::kScores) * 128 + (ks >> 1) * 32 + x * 16 + (ks & 1) * 8, d_mn + v + ks * 128,
                               id_v, x < 1 || ks > 0, one);
                if (!la_wait(r_s, ph, abort_flag, limit)) break;
                tc_fence_after();
#pragma unroll
                for (int x = 1; x >= 0; --x) {
                    const uint32_t op = x == 0 ? C::kOffS >> 4 : C::kInPlace ? k : C::kOffLo >> 4;
#pragma unroll
                    for (int ks = 0; ks < KP / 16; ++ks)
                        mma_ss(C::kQS, d_tile + q + tile(ks), d_op + op + ks * 128, id_v, x < 1 || ks > 0, one);
                }
                mma_commit(b_pv, one);
                // (of two score matrices the other is free since r_s: y of the chunk before had been read)
                if (C::kScores == 2) next_scores(false);
                if (!la_wait(r_k, ph, abort_flag, limit)) break;
                tc_fence_after();
                if (C::kScores == 1) next_scores(false);
                if (C::kInPlace) {
                    constexpr uint32_t id = idesc_bf16_f32(KP, VP, 1, 1);
#pragma unroll
                    for (int x = 2; x >= 0; --x) {   // the smallest terms first
                        const uint32_t a = x == 0 ? k : x == 1 ? q : C::kOffS >> 4;
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks)
                            mma_ss(C::kDS, d_mn + a + ks * 128, d_mn + v + ks * 128, id, x < 2 || ks > 0, one);
                    }
                } else if (C::kScaleV) {
                    outer_sum<KP, VP>(C::kDS, d_mn, k, 0, X, XS, one);
                } else {
                    outer_sum<KP, VP>(C::kDS, d_mn, X, XS, v, 0, one);
                }
                mma_commit(b_ds, one);
                if (!next_scores(true)) break;
            }
        }
        mma_commit(b_drain, one);   // nothing is in flight when the CTA ends
        if (lane == 0) la_drain(b_drain, 0, limit);
        __syncwarp();
    } else if (warp == kNW + 1) {
        // ------------------------------------------------------ copies
        if (lane == 0) {
            const int qk = la_qk_pair(p, bh);
            int nqk = 0, nv = 0;   // chunks whose tiles have been asked for
            auto load_qk = [&](int i) {
                if (p.fault == 1 && i > 0) return;   // injected: the copies stop after the first chunk
                nqk = i + 1;
                const int s = stage_of(i), t = chunk_of(i) * kLaChunk;
                const uint32_t base = sbase + s * C::kStage, full = b_qk + s * 8;
                mbar_arrive_expect_tx(full, 2 * C::kQ);
#pragma unroll
                for (int x = 0; x < KP / 64; ++x) {
                    tma_tile(base + x * kTileBytes, &maps.q, x * 64, t, qk, full);
                    tma_tile(base + C::kQ + x * kTileBytes, &maps.k, x * 64, t, qk, full);
                }
            };
            auto load_v = [&](int i) {
                if (p.fault == 1 && i > 0) return;
                nv = i + 1;
                const int s = stage_of(i), t = chunk_of(i) * kLaChunk;
                const uint32_t base = sbase + s * C::kStage + 2 * C::kQ, full = b_v + s * 8;
                mbar_arrive_expect_tx(full, C::kV);
#pragma unroll
                for (int x = 0; x < VP / 64; ++x) tma_tile(base + x * kTileBytes, &maps.v, x * 64, t, bh, full);
            };
            for (int i = 0; i < C::kStages && i < n; ++i) {
                load_qk(i);
                load_v(i);
            }
            bool ok = true;
            for (int i = 0; i < n; ++i) {
                // the stage is free: its products are done, y has been staged
                if (!(ok = la_wait_lane(r_y + (i & 1) * 8, (i >> 1) & 1, abort_flag, limit))) break;
                if (C::kStageY) {
#pragma unroll
                    for (int x = 0; x < VP / 64; ++x)
                        if (x * 64 < p.V)
                            tma_store_tile(&maps.y, sbase + stage_of(i) * C::kStage + x * kTileBytes, x * 64,
                                           chunk_of(i) * kLaChunk, bh);
                    tma_store_commit();
                    tma_store_wait_read();
                }
                if (i + C::kStages < n) {
                    load_qk(i + C::kStages);
                    load_v(i + C::kStages);
                }
            }
            if (!ok) {   // leave no copy in flight
                for (int j = max(0, nqk - C::kStages); j < nqk; ++j) la_drain(b_qk + stage_of(j) * 8, stage_phase(j), limit);
                for (int j = max(0, nv - C::kStages); j < nv; ++j) la_drain(b_v + stage_of(j) * 8, stage_phase(j), limit);
            }
        }
        __syncwarp();
    } else if (warp == kNW + 2) {
        decay_warp(p, bh, n, chunk_of, tab, b_tab, t_free, abort_flag);
    } else {
        // ------------------------------------------------------ elementwise work
        const int wg = warp >> 2, quarter = warp & 3;
        const int row = quarter * 32 + lane;                          // token of the chunk
        const uint32_t mine = tmem + ((uint32_t)(quarter * 32) << 16);   // tensor-memory lane base
        const Pt part;
        float S[Pt::NS];
        part.load(p.segs > 1 ? p.seg_state + ((size_t)bh * p.segs + seg) * p.K * p.V
                  : p.S0     ? p.S0 + (size_t)bh * p.K * p.V
                             : nullptr,
                  p.K, p.V, S);
        // S before chunk i of the walk: its two bf16 terms for Q·S, the checkpoint
        auto put_operand = [&](int i) -> bool {
            if (C::kInPlace && !la_wait(r_raw, i & 1, abort_flag, limit)) return false;   // every k is in registers
            uint8_t* op = smem + C::kOffS + (part.v0 >> 6) * (KP * 128);
            uint8_t* lo = smem + (C::kInPlace ? stage_of(i) * C::kStage + C::kQ : C::kOffLo) + (part.v0 >> 6) * (KP * 128);
#pragma unroll
            for (int j = 0; j < Pt::NS; j += 8) {
                uint4 hi, rest;
                split2(S[j], S[j + 1], hi.x, rest.x);
                split2(S[j + 2], S[j + 3], hi.y, rest.y);
                split2(S[j + 4], S[j + 5], hi.z, rest.z);
                split2(S[j + 6], S[j + 7], hi.w, rest.w);
                const uint32_t at = sw128(part.kap, ((part.v0 & 63) + j) >> 3);
                *reinterpret_cast<uint4*>(op + at) = hi;
                *reinterpret_cast<uint4*>(lo + at) = rest;
            }
            warp_arrive(r_s);
            if (p.ckpt && part.kap < p.K) {   // [V/4][K][4]: a warp's rows are adjacent
                float* ck = p.ckpt + ((size_t)bh * nchunks + chunk_of(i)) * p.K * p.V;
#pragma unroll
                for (int j = 0; j < Pt::NS; j += 4)
                    if (part.v0 + j < p.V)
                        *reinterpret_cast<float4*>(ck + ((size_t)((part.v0 + j) >> 2) * p.K + part.kap) * 4) =
                            make_float4(S[j], S[j + 1], S[j + 2], S[j + 3]);
            }
            return true;
        };
        // the scaled side: its tile's place in a stage, 16-byte chunks of the row for this thread
        constexpr int kOffTerm = C::kScaleV ? 2 * C::kQ : C::kQ, kCh = C::kTerm / 128 / 16 / 4;
        auto pos_of = [&](int j) {
            const int ch = wg * kCh + j;
            return (uint32_t)((ch >> 3) * kTileBytes + sw128(row, ch & 7));
        };
        uint4 raw[C::kInPlace ? kCh : 1];        // of k, kept while the state's low term is in its tile
        float at = 0.f, w = 0.f, A = 0.f;        // of the chunk whose P has been formed last
        // P = masked, decayed scores in bf16, over the scores: row `row`, block wg of 32 columns
        auto put_P = [&](int i) -> bool {
            if (!la_wait(b_tab + (i & 1) * 8, (i >> 1) & 1, abort_flag, limit)) return false;
            const LaTables* tb = tab + (i & 1);
            const float Ft = tb->F[row], It = tb->I[row], Fe = tb->F[127], Ie = tb->I[127];
            at = ex2_approx(Ft + It);
            A = ex2_approx(Fe + Ie);
            w = ex2_approx((Fe - Ft) + (Ie - It));
            if (!la_wait(b_sc + (i & 1) * 8, (i >> 1) & 1, abort_flag, limit)) return false;
            tc_fence_after();
            const uint32_t at_ = mine + (i % C::kScores) * 128 + wg * 32;
            uint32_t pk[16], lo[16];
            if (wg > quarter) {
#pragma unroll
                for (int e = 0; e < 16; ++e) pk[e] = lo[e] = 0;
            } else {
                uint32_t sc[32];
                tmem_ld<32>(at_, sc);
                const float r = ex2_approx((Ft - tb->F[wg * 32 + 31]) + (It - tb->I[wg * 32 + 31]));
                const int last = wg < quarter ? 31 : lane;   // the row's last column of the block
                tc_wait_ld();
                reg_fence(sc);
                if (wg < quarter || tb->steep == 0.f) {
                    const float2 r2 = make_float2(r, r);
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const float4 cs = *reinterpret_cast<const float4*>(&tb->c[wg * 32 + e]);
                        const float2 x = __fmul2_rn(__fmul2_rn(r2, make_float2(cs.x, cs.y)),
                                                    make_float2(__uint_as_float(sc[e]), __uint_as_float(sc[e + 1]))),
                                     y = __fmul2_rn(__fmul2_rn(r2, make_float2(cs.z, cs.w)),
                                                    make_float2(__uint_as_float(sc[e + 2]), __uint_as_float(sc[e + 3])));
                        split2(e <= last ? x.x : 0.f, e + 1 <= last ? x.y : 0.f, pk[e / 2], lo[e / 2]);
                        split2(e + 2 <= last ? y.x : 0.f, e + 3 <= last ? y.y : 0.f, pk[e / 2 + 1], lo[e / 2 + 1]);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const float4 fs = *reinterpret_cast<const float4*>(&tb->F[wg * 32 + e]);
                        const float4 is = la_whole(tb, wg * 32 + e);
                        auto d = [&](int o, float f, float w_) {
                            return e + o <= lane ? __uint_as_float(sc[e + o]) * ex2_approx((Ft - f) + (It - w_)) : 0.f;
                        };
                        split2(d(0, fs.x, is.x), d(1, fs.y, is.y), pk[e / 2], lo[e / 2]);
                        split2(d(2, fs.z, is.z), d(3, fs.w, is.w), pk[e / 2 + 1], lo[e / 2 + 1]);
                    }
                }
            }
            tmem_st16(at_, pk);
            tmem_st16(at_ + 16, lo);
            tc_wait_st();
            warp_arrive(r_p);
            if constexpr (C::kInPlace) {   // (the scores, which read the k tile too, are done)
                if (!la_wait(b_qk + stage_of(i) * 8, stage_phase(i), abort_flag, limit)) return false;
#pragma unroll
                for (int j = 0; j < kCh; ++j)
                    raw[j] = *reinterpret_cast<const uint4*>(smem + stage_of(i) * C::kStage + kOffTerm + pos_of(j));
                __syncwarp();
                if (lane == 0) mbar_arrive(r_raw);
            }
            return true;
        };
        // the scaled side's terms of chunk i (their buffer is free: the last sum is done)
        auto put_terms = [&](int i) -> bool {
            uint8_t* stage = smem + stage_of(i) * C::kStage;
            if constexpr (C::kInPlace) {
                if (!la_wait(b_pv, i & 1, abort_flag, limit)) return false;   // Q S has read q and S
#pragma unroll
                for (int j = 0; j < kCh; ++j) {
                    const uint32_t pos = pos_of(j);
                    put_scaled(raw[j], stage + kOffTerm + pos, stage + pos, smem + C::kOffS + pos, w);
                }
            } else {
                if (!la_wait((C::kScaleV ? b_v : b_qk) + stage_of(i) * 8, stage_phase(i), abort_flag, limit)) return false;
                uint8_t* X = smem + C::kOffX;
                uint4 third[kCh];
#pragma unroll
                for (int j = 0; j < kCh; ++j) {
                    const uint32_t pos = pos_of(j);
                    third[j] = put_scaled(*reinterpret_cast<const uint4*>(stage + kOffTerm + pos), X + pos, X + C::kTerm + pos, w);
                }
                if (C::kShareLo && !la_wait(b_pv, i & 1, abort_flag, limit)) return false;   // Q S has read the low term
#pragma unroll
                for (int j = 0; j < kCh; ++j) *reinterpret_cast<uint4*>(X + 2 * C::kTerm + pos_of(j)) = third[j];
            }
            warp_arrive(r_k);
            if (lane == 0) mbar_arrive(t_free + (i & 1) * 8);    // this chunk's tables are no longer read
            return true;
        };
        bool ok = true;
        ok = (C::kInPlace || put_operand(0)) && put_P(0) && (!C::kInPlace || put_operand(0)) && put_terms(0);
        for (int i = 0; ok && i < n; ++i) {
            const int ph = i & 1;
            const float at_i = at, A_i = A;
            // ---- y = a (Q S) + P V
            if (!la_wait(b_pv, ph, abort_flag, limit)) break;
            tc_fence_after();
            const int t = chunk_of(i) * kLaChunk + row;
#pragma unroll
            for (int j = 0; j < C::NY; j += 16) {
                const int col = wg * C::NY + j;
                uint32_t pv[16], qs[16], o[8];
                tmem_ld<16>(mine + C::kPV + col, pv);
                tmem_ld<16>(mine + C::kQS + col, qs);
                tc_wait_ld();
                reg_fence(pv);
                reg_fence(qs);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    o[e] = pack_bf16(fmaf(at_i, __uint_as_float(qs[2 * e]), __uint_as_float(pv[2 * e])),
                                     fmaf(at_i, __uint_as_float(qs[2 * e + 1]), __uint_as_float(pv[2 * e + 1])));
                if (C::kStageY) {
                    uint8_t* dst = smem + stage_of(i) * C::kStage + (col >> 6) * kTileBytes;
                    *reinterpret_cast<uint4*>(dst + sw128(row, (col & 63) >> 3)) = make_uint4(o[0], o[1], o[2], o[3]);
                    *reinterpret_cast<uint4*>(dst + sw128(row, ((col & 63) >> 3) + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
                } else if (t < p.T && col < p.V) {
                    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y) + ((size_t)bh * p.T + t) * p.V + col;
                    if (p.out32) {
                        st_global_v8(y, o);
                    } else {
                        *reinterpret_cast<uint4*>(y) = make_uint4(o[0], o[1], o[2], o[3]);
                        *reinterpret_cast<uint4*>(y + 8) = make_uint4(o[4], o[5], o[6], o[7]);
                    }
                }
            }
            // ---- the next chunk's P while the state's sum is computed
            if (i + 1 < n && !(ok = put_P(i + 1))) break;
            // ---- S = A S + the chunk's sum
            if (!la_wait(b_ds, ph, abort_flag, limit)) break;
            tc_fence_after();
            part.add(mine + C::kDS, A_i, S);
            warp_arrive(r_y + (i & 1) * 8);
            if (i + 1 < n) {
                ok = put_operand(i + 1) && put_terms(i + 1);
            }
        }
        if (p.ST && c0 + n == nchunks) part.store(p.ST + (size_t)bh * p.K * p.V, p.K, p.V, S);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kNW) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------ segment sums

// What a segment's tokens add to the state at its end, from a zero start
// (REV: to the state's gradient at its start): Σ w_s k_s v_sᵀ (Σ w_t q_t dy_tᵀ)
// with w the decay to the segment's end (from its start through t).  The walk
// starts at that end, so w is a running product times the chunk's decay and no
// chunk's sum is scaled again: a chunk's terms are written while the last
// one's products run.  The chunks' sums are added in registers, which round to
// nearest: one accumulation in tensor memory over the segment lost up to 1e-6
// of the state where gates are close to 1.
template <int KP, int VP>
struct SumCfg {
    static constexpr int kQ = KP / 64 * kTileBytes, kV = VP / 64 * kTileBytes, kStage = kQ + kV;
    static constexpr bool kScaleV = VP < KP;
    static constexpr int kTerm = kScaleV ? kV : kQ;
    static constexpr int kSets = KP * VP < 128 * 128 ? 2 : 1;   // sets of terms
    static constexpr int kOffX = 2 * kStage;
    static constexpr int kOffTab = kOffX + kSets * 3 * kTerm;
    static constexpr int kOffBar = kOffTab + 2 * (int)sizeof(LaTables);
    static constexpr int kBars = 11;
    static constexpr int kSmem = kOffBar + kBars * 8 + 16;
    static_assert(kSmem <= 227 * 1024, "shared memory");
};

template <int KP, int VP, bool REV>
__global__ void __launch_bounds__(kFwdThreads, 1)
    m2rnn_la_sum_tc_kernel(const LaParams p, const __grid_constant__ Maps maps, float* seg_decay) {
    using C = SumCfg<KP, VP>;
    using Pt = Part<KP, VP>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int bh = blockIdx.x / p.segs, seg = blockIdx.x % p.segs;
    if (REV ? seg == 0 : seg == p.segs - 1) return;   // no segment starts from this sum
    const int nchunks = (p.T + kLaChunk - 1) / kLaChunk;
    const int c0 = seg * p.seg_chunks, n = min(nchunks - c0, p.seg_chunks);
    auto chunk_of = [&](int i) { return REV ? c0 + i : c0 + n - 1 - i; };

    LaTables* tab = reinterpret_cast<LaTables*>(smem + C::kOffTab);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    const uint32_t b_full = bar(0), b_tab = bar(2), t_free = bar(4), b_ds = bar(6), r_k = bar(8), b_drain = bar(10);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kBars);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const LaLimit limit = p.limit;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 11; ++i) mbar_init(bar(i), 1);
        for (uint32_t b : {t_free, t_free + 8, r_k, r_k + 8}) mbar_init(b, kNW);
        *abort_flag = 0;
        fence_mbarrier_init();
    }
    if (warp == kNW) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    constexpr uint32_t tmem = 0;   // the CTA has all 512 columns
    const uint32_t sbase = smem_u32(smem);

    if (warp == kNW) {
        const Desc d_mn = sw128_desc(sbase, kTileBytes);
        const uint32_t one = lane == 0;
        for (int i = 0; i < n; ++i) {
            if (!la_wait(b_full + (i & 1) * 8, (i >> 1) & 1, abort_flag, limit)) break;
            if (!la_wait(r_k + (i & 1) * 8, (i >> 1) & 1, abort_flag, limit)) break;
            tc_fence_after();
            const uint32_t k = (i & 1) * (C::kStage >> 4), v = k + (C::kQ >> 4),
                           x = (C::kOffX + (i % C::kSets) * 3 * C::kTerm) >> 4, xs = C::kTerm >> 4;
            if (C::kScaleV) outer_sum<KP, VP>((i & 1) * VP, d_mn, k, 0, x, xs, one);
            else outer_sum<KP, VP>((i & 1) * VP, d_mn, x, xs, v, 0, one);
            mma_commit(b_ds + (i & 1) * 8, one);
        }
        mma_commit(b_drain, one);
        if (lane == 0) la_drain(b_drain, 0, limit);
        __syncwarp();
    } else if (warp == kNW + 1) {
        if (lane == 0) {
            const int qk = la_qk_pair(p, bh);
            int loaded = 0;
            auto load = [&](int i) {
                if (p.fault == 1 && i > 0) return;
                loaded = i + 1;
                const int t = chunk_of(i) * kLaChunk;
                const uint32_t base = sbase + (i & 1) * C::kStage, full = b_full + (i & 1) * 8;
                mbar_arrive_expect_tx(full, C::kStage);
#pragma unroll
                for (int x = 0; x < KP / 64; ++x) tma_tile(base + x * kTileBytes, &maps.k, x * 64, t, qk, full);
#pragma unroll
                for (int x = 0; x < VP / 64; ++x) tma_tile(base + C::kQ + x * kTileBytes, &maps.v, x * 64, t, bh, full);
            };
            load(0);
            if (n > 1) load(1);
            bool ok = true;
            for (int i = 0; i + 2 < n; ++i) {
                if (!(ok = la_wait_lane(b_ds + (i & 1) * 8, (i >> 1) & 1, abort_flag, limit))) break;
                load(i + 2);
            }
            if (!ok)
                for (int j = max(0, loaded - 2); j < loaded; ++j) la_drain(b_full + (j & 1) * 8, (j >> 1) & 1, limit);
        }
        __syncwarp();
    } else if (warp == kNW + 2) {
        decay_warp(p, bh, n, chunk_of, tab, b_tab, t_free, abort_flag);
    } else {
        const int wg = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane;
        const Part<KP, VP> part;
        float carry = 1.f, S[Pt::NS];
#pragma unroll
        for (int e = 0; e < Pt::NS; ++e) S[e] = 0.f;
        auto add = [&](int j) -> bool {   // chunk j's sum
            if (!la_wait(b_ds + (j & 1) * 8, (j >> 1) & 1, abort_flag, limit)) return false;
            tc_fence_after();
            part.add(((uint32_t)(quarter * 32) << 16) + (j & 1) * VP, 1.f, S);
            return true;
        };
        bool ok = true;
        for (int i = 0; i < n; ++i) {
            if (!(ok = la_wait(b_tab + (i & 1) * 8, (i >> 1) & 1, abort_flag, limit))) break;
            const LaTables* tb = tab + (i & 1);
            const float Ft = tb->F[row], It = tb->I[row], Fe = tb->F[127], Ie = tb->I[127];
            const float w = carry * ex2_approx(REV ? Ft + It : (Fe - Ft) + (Ie - It));
            carry *= ex2_approx(Fe + Ie);
            __syncwarp();
            if (lane == 0) mbar_arrive(t_free + (i & 1) * 8);
            if (!(ok = la_wait(b_full + (i & 1) * 8, (i >> 1) & 1, abort_flag, limit))) break;
            if (i >= C::kSets && !(ok = add(i - C::kSets))) break;   // whose terms these replace
            const uint8_t* src = smem + (i & 1) * C::kStage + (C::kScaleV ? C::kQ : 0);
            uint8_t* dst = smem + C::kOffX + (i % C::kSets) * 3 * C::kTerm;
            constexpr int kCh = C::kTerm / 128 / 16 / 4;
#pragma unroll
            for (int e = 0; e < kCh; ++e) {
                const int ch = wg * kCh + e;
                const uint32_t pos = (ch >> 3) * kTileBytes + sw128(row, ch & 7);
                put_scaled(*reinterpret_cast<const uint4*>(src + pos), dst + pos, dst + pos + C::kTerm, dst + pos + 2 * C::kTerm, w);
            }
            warp_arrive(r_k + (i & 1) * 8);
        }
        for (int j = max(0, n - C::kSets); ok && j < n; ++j) ok = add(j);
        if (ok) {
            part.store(p.seg_state + ((size_t)bh * p.segs + seg) * p.K * p.V, p.K, p.V, S);
            if (threadIdx.x == 0) seg_decay[(size_t)bh * p.segs + seg] = carry;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kNW) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Segment sums -> segment start states, in place: start_0 = init,
// start_{i+1} = decay_i start_i + sum_i (reverse: from the last segment, for
// the gradient at segment ends).  A thread takes four adjacent elements, eight
// segments' sums in flight (one at a time: 39 us more for 16 pairs of 128 x
// 128 over 4096 tokens, forward and backward).
__global__ void m2rnn_la_seg_scan_kernel(const LaParams p, const float* seg_decay, const float* init,
                                         int reverse) {
    const int kv4 = p.K * p.V / 4;
    const size_t e = blockIdx.x * (size_t)blockDim.x + threadIdx.x;
    if (e >= (size_t)p.B * p.H * kv4) return;
    const size_t bh = e / kv4, o = e % kv4;
    float4* st = reinterpret_cast<float4*>(p.seg_state) + bh * p.segs * kv4 + o;
    float4 s = init ? reinterpret_cast<const float4*>(init)[bh * kv4 + o] : make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int N = 8;
    for (int i0 = 0; i0 < p.segs; i0 += N) {
        float4 d[N];
        float a[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int g = reverse ? p.segs - 1 - i0 - j : i0 + j;
            if (i0 + j < p.segs) { d[j] = st[(size_t)g * kv4]; a[j] = seg_decay[bh * p.segs + g]; }
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int g = reverse ? p.segs - 1 - i0 - j : i0 + j;
            if (i0 + j >= p.segs) break;
            st[(size_t)g * kv4] = s;
            s.x = fmaf(a[j], s.x, d[j].x); s.y = fmaf(a[j], s.y, d[j].y);
            s.z = fmaf(a[j], s.z, d[j].z); s.w = fmaf(a[j], s.w, d[j].w);
        }
    }
}

float* decays_of(const LaParams& p) {   // behind the segment states in the workspace
    return p.seg_state + (size_t)p.B * p.H * p.segs * p.K * p.V;
}

template <int KP, int VP>
struct FwdKernel {
    static cudaError_t launch(const LaParams& p, const Maps& m, cudaStream_t s) {
        auto kern = m2rnn_la_fwd_tc_kernel<KP, VP>;
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<KP, VP>::kSmem);
        if (e != cudaSuccess) return e;
        kern<<<p.B * p.H * p.segs, kFwdThreads, Cfg<KP, VP>::kSmem, s>>>(p, m);
        return cudaGetLastError();
    }
};
template <bool REV>
struct Sum {
    template <int KP, int VP>
    struct Kernel {
        static cudaError_t launch(const LaParams& p, const Maps& m, cudaStream_t s) {
            auto kern = m2rnn_la_sum_tc_kernel<KP, VP, REV>;
            const cudaError_t e =
                cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SumCfg<KP, VP>::kSmem);
            if (e != cudaSuccess) return e;
            kern<<<p.B * p.H * p.segs, kFwdThreads, SumCfg<KP, VP>::kSmem, s>>>(p, m, decays_of(p));
            return cudaGetLastError();
        }
    };
};
template <template <int, int> class Kernel>
cudaError_t launch_shape(const LaParams& p, const Maps& m, cudaStream_t s) {
    if (p.K <= 64)
        return p.V <= 64 ? Kernel<64, 64>::launch(p, m, s) : Kernel<64, 128>::launch(p, m, s);
    return p.V <= 64 ? Kernel<128, 64>::launch(p, m, s) : Kernel<128, 128>::launch(p, m, s);
}

cudaError_t launch_scan(const LaParams& p, const float* init, int reverse, cudaStream_t s) {
    const size_t n = (size_t)p.B * p.H * p.K * p.V / 4;
    m2rnn_la_seg_scan_kernel<<<(unsigned)((n + 127) / 128), 128, 0, s>>>(p, decays_of(p), init, reverse);
    return cudaGetLastError();
}

}  // namespace

// Segments while there are SMs for them, if the chunks that a walk is spared
// pay for the sums that run before it, a launch and a pass over k and v (q and
// dy).  Those cost more the more CTAs share the memory.  Measured, us, one
// walk against segments of T/128 chunks (64 x 128 and 128 x 64 lie between the
// two shapes and turn at the same lengths):
//   forward            64 x 64                                128 x 128
//    1 pair    4 chunks 15.3 / 15.2,  5  17.9 / 15.3     4  26.8 / 26.1,   5  31.6 / 25.9
//   24 pairs   5        17.9 / 17.2,  6  20.5 / 18.0     5  31.9 / 29.8,   6  36.8 / 30.8
//   37 pairs   6        20.8 / 20.6,  8  26.3 / 22.1     6  37.5 / 37.5,   8  48.4 / 41.2
//   48 pairs  10        32.1 / 32.2, 12  37.5 / 32.5    10  58.5 / 57.5,  12  68.6 / 60.1
//   74 pairs  24        70.7 / 77.1                     16  90.0 / 96.4,  24   130 / 125
//   backward
//    1 pair    2 chunks 19.5 / 19.8,  3  26.8 / 19.9     2  37.6 / 35.6,   3  52.9 / 35.6
//   48 pairs   3        26.9 / 24.7,  6  51.2 / 35.9     2  38.4 / 40.3,   3  55.2 / 44.8
//   74 pairs   4        36.1 / 36.4,  6  52.4 / 48.7     4  73.9 / 75.4,   6   107 / 97
LaPlan la_plan(int B, int H, int T, bool backward) {
    const int chunks = (T + kLaChunk - 1) / kLaChunk;
    const long long pairs = (long long)B * H;
    if (pairs * 2 > kNumSMs) return {1, chunks};
    const int most = kNumSMs / (int)pairs, want = most < chunks ? most : chunks, per = (chunks + want - 1) / want;
    const int need = backward ? 2 + (int)pairs / 64 : 4 + (int)(pairs * pairs) / 512;
    if (chunks - per < need) return {1, chunks};
    return {(chunks + per - 1) / per, per};
}

size_t la_seg_bytes(const LaPlan& plan, int B, int H, int K, int V) {
    return plan.segs <= 1 ? 0 : sizeof(float) * (size_t)B * H * plan.segs * ((size_t)K * V + 1);
}

cudaError_t launch_la_fwd_tc(const LaParams& q, cudaStream_t s) {
    LaParams p = q;
    p.out32 = !(reinterpret_cast<uintptr_t>(p.y) & 31u);
    Maps m;
    if (!la_tensor_map(&m.q, p.q, p.K, p.T, (size_t)p.B * p.G) || !la_tensor_map(&m.k, p.k, p.K, p.T, (size_t)p.B * p.G) ||
        !la_tensor_map(&m.v, p.v, p.V, p.T, (size_t)p.B * p.H) || !la_tensor_map(&m.y, p.y, p.V, p.T, (size_t)p.B * p.H))
        return cudaErrorNotSupported;
    if (p.segs > 1) {
        cudaError_t e = launch_shape<Sum<false>::Kernel>(p, m, s);
        if (e != cudaSuccess) return e;
        if ((e = launch_scan(p, p.S0, 0, s)) != cudaSuccess) return e;
    }
    return launch_shape<FwdKernel>(p, m, s);
}

// The same sums for the gradient: what a segment's tokens add to dL/dS at its
// start, then dL/dS at every segment's end.
cudaError_t launch_la_seg_grads(const LaParams& p, cudaStream_t s) {
    Maps m;
    if (!la_tensor_map(&m.k, p.q, p.K, p.T, (size_t)p.B * p.G) || !la_tensor_map(&m.v, p.dy, p.V, p.T, (size_t)p.B * p.H))
        return cudaErrorNotSupported;
    m.q = m.k;
    m.y = m.v;
    const cudaError_t e = launch_shape<Sum<true>::Kernel>(p, m, s);
    return e != cudaSuccess ? e : launch_scan(p, p.dST, 1, s);
}

cudaError_t la_fwd_tc_status(unsigned slot, unsigned* word, cudaStream_t s) { return la_read_status(slot, word, s); }

}  // namespace m2rnn
