// Linear attention in chunks of 128 tokens on the tensor cores (bf16).
//
// With L_t the cumulative log-decay inside a chunk, D_ts = 2^(L_t - L_s),
// a_t = 2^(L_t), b_s = 2^(L_end - L_s) and S the state at its start,
//   y_t  = a_t (Q S)_t + ((Q Kᵀ ∘ D) V)_t          (s <= t)
//   S'   = a_end S + Σ_s (b_s k_s) v_sᵀ
// Four matrix products, every accumulator in tensor memory; the state's fp32
// master stays in registers over the whole walk.
//
// A CTA walks the chunks of one (b, h), or of one of its time segments.  8 or
// 16 warps compute: thread = token row (or state row) = tensor-memory lane, the
// warpgroups sharing the columns.  One more warp issues the products, another
// fetches tiles two chunks ahead, stores y and computes the next chunk's
// decays.  A chunk is a chain of waits (product -> elementwise -> product):
// two CTAs of 8 warps share an SM where they fit, else a CTA has 16.
//
// Rounding: the masked scores and the copy of S that multiplies Q are bf16
// operands (each term of y passes through exactly one of them, and y is
// rounded to bf16 itself); b_s k_s enters as three bf16 terms, so the state
// keeps fp32 accuracy over any number of chunks.
//
// Decays without an exponential per score: for a row t and a block of 32
// columns, D_ts = 2^(L_t - L_e)·2^(L_e - L_s) with e the block's last token.
// The second factor is shared by all rows.  Left of the diagonal both are at
// most 1; in the diagonal block the first is the reciprocal of a decay, within
// fp32's range unless the block decays by more than 2^-90: such chunks take one
// exponential per score there.
#include <cstdlib>
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

// FWD: the forward.  SUM: only the segment's own contribution to its final
// state (from a zero start).  RSUM: the same backwards in time, with decays
// from the segment's start: Σ_t a_t k_t v_tᵀ.
enum Kind { FWD, SUM, RSUM };

// NW compute warps: 8 (two CTAs share an SM where they fit) or 16 (one CTA
// that has an SM to itself).
template <int KP, int VP, int NW>
struct Cfg {
    static constexpr int kThreads = (NW + 2) * 32, WG = NW / 4;
    static constexpr int kQ = KP / 64 * kTileBytes, kV = VP / 64 * kTileBytes, kStage = 2 * kQ + kV;
    static constexpr int kOffS = 2 * kStage;                    // bf16 state operand [KP][VP]
    static constexpr int kOffTab = kOffS + KP * VP * 2;
    static constexpr int kOffBar = kOffTab + (int)sizeof(LaTables);
    static constexpr int kBars = 13;
    static constexpr int kSmem = kOffBar + kBars * 8 + 16;
    static constexpr int kCtas = NW == 8 && kSmem <= 113 * 1024 ? 2 : 1;
    // tensor memory: scores (P in bf16 over them), P·V, Q·S, the state's sum.
    // With two CTAs an SM, P·V takes the second half of the scores, which P leaves free.
    static constexpr bool kPacked = kCtas == 2;
    static constexpr int kTmem = kPacked ? 256 : 512;
    static constexpr int kPV = kPacked ? 64 : 128, kQS = kPV + VP, kDS = kQS + VP;
    static_assert(kDS + VP <= kTmem, "tensor memory");
    static constexpr int NS = VP / WG / (KP == 128 ? 1 : 2);    // state columns per thread
    static constexpr int NL = NS < 16 ? NS : 16;                // per tensor-memory load
    static constexpr int NY = VP / WG;                          // columns of y per thread
    // Tensor-memory column of the 16 columns of P that hold score block j (of
    // 32 columns; warpgroup j % WG computes it): inside that warpgroup's own
    // score columns, so that no warp writes over scores that another reads.
    static constexpr __device__ int p_col(int j) { return kPacked ? (j & 1) * 32 + (j >> 1) * 16 : j * 32; }
};

template <int KP, int VP, int NW, Kind KIND>
__global__ void __launch_bounds__(Cfg<KP, VP, NW>::kThreads, Cfg<KP, VP, NW>::kCtas)
    m2rnn_la_fwd_tc_kernel(const LaParams p, const __grid_constant__ Maps maps, float* seg_decay) {
    using C = Cfg<KP, VP, NW>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int bh = blockIdx.x / p.segs, seg = blockIdx.x % p.segs;
    const int nchunks = (p.T + kLaChunk - 1) / kLaChunk;
    const int c0 = seg * p.seg_chunks, n = min(nchunks - c0, p.seg_chunks);
    if ((KIND == SUM && seg == p.segs - 1) || (KIND == RSUM && seg == 0)) return;   // no segment starts from this sum
    auto chunk_of = [&](int i) { return KIND == RSUM ? c0 + n - 1 - i : c0 + i; };

    LaTables* tab = reinterpret_cast<LaTables*>(smem + C::kOffTab);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    const uint32_t b_full = bar(0), b_sc = bar(2), r_k = bar(3), b_ds1 = bar(4), r_p = bar(5), b_pv = bar(6),
                   r_lo = bar(7), b_ds2 = bar(8), r_s = bar(9), b_tab = bar(10), b_drain = bar(11), r_y = bar(12);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kBars);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const uint64_t limit = p.wait_limit_ns;

    if (threadIdx.x == 0) {
        mbar_init(bar(0), 1);
        mbar_init(bar(1), 1);
        for (uint32_t b : {b_sc, b_ds1, b_pv, b_ds2, b_tab, b_drain}) mbar_init(b, 1);
        for (uint32_t b : {r_k, r_p, r_lo, r_s, r_y}) mbar_init(b, NW);   // one arrival a warp
        *abort_flag = 0;
        fence_mbarrier_init();
    }
    if (warp == NW) {
        tmem_alloc(smem_u32(tmem_slot), C::kTmem);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t sbase = smem_u32(smem);

    if (warp == NW) {
        // ------------------------------------------------------ products
        constexpr uint32_t id_sc = idesc_bf16_f32(128, 128, 0, 0), id_qs = idesc_bf16_f32(128, VP, 0, 1),
                           id_pv = idesc_bf16_f32(128, VP, 0, 1), id_ds = idesc_bf16_f32(KP, VP, 1, 1);
        const uint64_t d_tile = sw128_desc(sbase, 16), d_mn = sw128_desc(sbase, kTileBytes),
                       d_s = sw128_desc(sbase + C::kOffS, KP * 128);
        bool ok = true;
        for (int i = 0; i < n; ++i) {
            const int s = i & 1, ph = i & 1;
            // operand positions in units of 16 bytes
            const uint32_t q = s * (C::kStage >> 4), k = q + (C::kQ >> 4), v = k + (C::kQ >> 4);
            // the state's product: A = a scaled k tile, its rows (tokens) along the contraction
            auto state_product = [&](uint32_t a, bool first) {
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                    tc_mma_f16_ss(tmem + C::kDS, d_mn + a + ks * 128, d_mn + v + ks * 128, id_ds, !(first && ks == 0));
            };
            if (!(ok = la_wait(b_full + s * 8, (i >> 1) & 1, abort_flag, limit))) break;
            if (KIND == FWD) {
                if (!(ok = la_wait(r_s, ph, abort_flag, limit))) break;
                tc_fence_after();
                if (lane == 0) {
#pragma unroll
                    for (int ks = 0; ks < KP / 16; ++ks) {
                        const uint32_t off = (ks >> 2) * (kTileBytes >> 4) + (ks & 3) * 2;
                        tc_mma_f16_ss(tmem, d_tile + q + off, d_tile + k + off, id_sc, ks > 0);
                    }
#pragma unroll
                    for (int ks = 0; ks < KP / 16; ++ks) {
                        const uint32_t off = (ks >> 2) * (kTileBytes >> 4) + (ks & 3) * 2;
                        tc_mma_f16_ss(tmem + C::kQS, d_tile + q + off, d_s + ks * 128, id_qs, ks > 0);
                    }
                    tc_commit(b_sc);
                }
            }
            if (!(ok = la_wait(r_k, ph, abort_flag, limit))) break;
            tc_fence_after();
            if (lane == 0) {
                state_product(k, true);
                state_product(q, false);
                tc_commit(b_ds1);
            }
            if (KIND == FWD) {
                if (!(ok = la_wait(r_p, ph, abort_flag, limit))) break;
                tc_fence_after();
                if (lane == 0) {
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        tc_mma_f16_ts(tmem + C::kPV, tmem + C::p_col(ks >> 1) + (ks & 1) * 8, d_mn + v + ks * 128, id_pv,
                                      ks > 0);
                    tc_commit(b_pv);
                }
            }
            if (!(ok = la_wait(r_lo, ph, abort_flag, limit))) break;
            tc_fence_after();
            if (lane == 0) {
                state_product(k, false);
                tc_commit(b_ds2);
            }
        }
        if (lane == 0) {   // nothing is in flight when the CTA ends
            tc_commit(b_drain);
            la_drain(b_drain, 0, limit);
        }
        __syncwarp();
    } else if (warp == NW + 1) {
        // ------------------------------------------------------ copies and decays
        const int qk = la_qk_pair(p, bh);
        int loaded = 0;
        auto load = [&](int i) {   // lane 0: the tiles of the walk's i-th chunk
            if (p.fault == 1 && i > 0) return;   // injected: the copies stop after the first chunk
            loaded = i + 1;
            const int s = i & 1, t = chunk_of(i) * kLaChunk;
            const uint32_t base = sbase + s * C::kStage, full = b_full + s * 8;
            mbar_arrive_expect_tx(full, KIND == FWD ? C::kStage : C::kQ + C::kV);
#pragma unroll
            for (int x = 0; x < KP / 64; ++x) {
                if (KIND == FWD) tma_tile(base + x * kTileBytes, &maps.q, x * 64, t, qk, full);
                tma_tile(base + C::kQ + x * kTileBytes, &maps.k, x * 64, t, qk, full);
            }
#pragma unroll
            for (int x = 0; x < VP / 64; ++x) tma_tile(base + 2 * C::kQ + x * kTileBytes, &maps.v, x * 64, t, bh, full);
        };
        if (lane == 0) {
            load(0);
            if (n > 1) load(1);
        }
        float fx[4], fnext[4];
        la_load_f(p, bh, chunk_of(0), fx);
        la_load_f(p, bh, n > 1 ? chunk_of(1) : chunk_of(0), fnext);
        la_tables(tab, p, fx, p.T - chunk_of(0) * kLaChunk, kLogFloorFwd);
        __syncwarp();
        if (lane == 0) mbar_arrive(b_tab);
        bool ok = true;
        int i = 0;
        for (; i < n; ++i) {
            const int ph = i & 1;
            if (i + 1 < n) {   // the next chunk's decays, once this one's are no longer read
#pragma unroll
                for (int e = 0; e < 4; ++e) fx[e] = fnext[e];
                if (i + 2 < n) la_load_f(p, bh, chunk_of(i + 2), fnext);
                if (!(ok = la_wait(KIND == FWD ? r_p : r_k, ph, abort_flag, limit))) break;
                la_tables(tab, p, fx, p.T - chunk_of(i + 1) * kLaChunk, kLogFloorFwd);
                __syncwarp();
                if (lane == 0) mbar_arrive(b_tab);
            }
            // the stage is free when its products are done and y, staged over its q (and k) tile, has left
            if (!(ok = la_wait(KIND == FWD ? r_y : b_ds2, ph, abort_flag, limit))) break;
            if (lane == 0) {
                if (KIND == FWD) {
#pragma unroll
                    for (int x = 0; x < VP / 64; ++x)
                        if (x * 64 < p.V)
                            tma_store_tile(&maps.y, sbase + (i & 1) * C::kStage + x * kTileBytes, x * 64,
                                           chunk_of(i) * kLaChunk, bh);
                    tma_store_commit();
                    tma_store_wait_read();
                }
                if (i + 2 < n) load(i + 2);
            }
        }
        if (!ok && lane == 0)   // leave no copy in flight
            for (int j = i; j < loaded; ++j) la_drain(b_full + (j & 1) * 8, (j >> 1) & 1, limit);
        __syncwarp();
    } else {
        // ------------------------------------------------------ elementwise work
        const int wg = warp >> 2, quarter = warp & 3;
        const int row = quarter * 32 + lane;                     // token of the chunk
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;   // tensor-memory lane base
        // This thread's part of the state: row kap, columns [v0, v0 + NS).  The
        // sum of 128 state rows has a lane for each; that of 64 rows has 16
        // lanes in every quarter, which two half warps read.
        const int kap = KP == 128 ? row : quarter * 16 + (lane & 15);
        const int v0 = KP == 128 ? wg * C::NS : (wg * 2 + (lane >> 4)) * C::NS;
        const bool mine = kap < p.K;
        float S[C::NS];
        {
            const float* src = KIND != FWD ? nullptr
                               : p.segs > 1 ? p.seg_state + ((size_t)bh * p.segs + seg) * p.K * p.V
                               : p.S0       ? p.S0 + (size_t)bh * p.K * p.V
                                            : nullptr;
#pragma unroll
            for (int j = 0; j < C::NS; j += 4) {
                const float4 x = src && mine && v0 + j < p.V
                                     ? *reinterpret_cast<const float4*>(src + (size_t)kap * p.V + v0 + j)
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
                S[j] = x.x; S[j + 1] = x.y; S[j + 2] = x.z; S[j + 3] = x.w;
            }
        }
        auto arrive = [&](uint32_t b) {   // this warp's writes are done: shared memory for the products, tensor memory
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(b);
        };
        auto store_state = [&](float* dst) {
            if (!mine) return;
#pragma unroll
            for (int j = 0; j < C::NS; j += 4)
                if (v0 + j < p.V)
                    *reinterpret_cast<float4*>(dst + (size_t)kap * p.V + v0 + j) =
                        make_float4(S[j], S[j + 1], S[j + 2], S[j + 3]);
        };
        auto write_operand = [&]() {   // bf16 copy of S for Q·S
            uint8_t* op = smem + C::kOffS + (v0 >> 6) * (KP * 128);
#pragma unroll
            for (int j = 0; j < C::NS; j += 8)
                *reinterpret_cast<uint4*>(op + sw128(kap, ((v0 & 63) + j) >> 3)) =
                    make_uint4(pack_bf16(S[j], S[j + 1]), pack_bf16(S[j + 2], S[j + 3]), pack_bf16(S[j + 4], S[j + 5]),
                               pack_bf16(S[j + 6], S[j + 7]));
        };
        if (KIND == FWD) {
            write_operand();
            arrive(r_s);
        }
        float decay = 1.f;

        for (int i = 0; i < n; ++i) {
            const int s = i & 1, ph = i & 1, c = chunk_of(i);
            uint8_t* stage = smem + s * C::kStage;
            if (KIND == FWD && p.ckpt && mine) {   // [V/4][K][4]: a warp's rows are adjacent
                float* ck = p.ckpt + ((size_t)bh * nchunks + c) * p.K * p.V;
#pragma unroll
                for (int j = 0; j < C::NS; j += 4)
                    if (v0 + j < p.V)
                        *reinterpret_cast<float4*>(ck + ((size_t)((v0 + j) >> 2) * p.K + kap) * 4) =
                            make_float4(S[j], S[j + 1], S[j + 2], S[j + 3]);
            }
            if (!la_wait(b_tab, ph, abort_flag, limit)) break;
            const float Ft = tab->F[row], It = tab->I[row], Fe = tab->F[127], Ie = tab->I[127];
            const float at = ex2_approx(Ft + It), A = ex2_approx(Fe + Ie);
            const float w = KIND == RSUM ? at : ex2_approx((Fe - Ft) + (Ie - It));
            if (!la_wait(b_full + s * 8, (i >> 1) & 1, abort_flag, limit)) break;
            if (KIND == FWD && !la_wait(b_sc, ph, abort_flag, limit)) break;
            tc_fence_after();
            // ---- w k in three bf16 terms: over the k tile, over the q tile, and kept
            constexpr int kCh = KP / 8 / C::WG;                 // 16-byte chunks of the row for this thread
            uint32_t lo[kCh][4];
#pragma unroll
            for (int j = 0; j < kCh; ++j) {
                const int ch = wg * kCh + j;
                const uint32_t at_ = (ch >> 3) * kTileBytes + sw128(row, ch & 7);
                uint4* kp = reinterpret_cast<uint4*>(stage + C::kQ + at_);
                const uint4 x = *kp;
                uint4 hi, mid;
                split3(w * bf16lo_to_f32(x.x), w * bf16hi_to_f32(x.x), hi.x, mid.x, lo[j][0]);
                split3(w * bf16lo_to_f32(x.y), w * bf16hi_to_f32(x.y), hi.y, mid.y, lo[j][1]);
                split3(w * bf16lo_to_f32(x.z), w * bf16hi_to_f32(x.z), hi.z, mid.z, lo[j][2]);
                split3(w * bf16lo_to_f32(x.w), w * bf16hi_to_f32(x.w), hi.w, mid.w, lo[j][3]);
                *kp = hi;
                *reinterpret_cast<uint4*>(stage + at_) = mid;
            }
            arrive(r_k);
            if (KIND == FWD) {
                // ---- P = masked, decayed scores in bf16, back to tensor memory
#pragma unroll
                for (int j = wg; j < 4; j += C::WG) {          // block of 32 columns
                    uint32_t pk[16];
                    if (j > quarter) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) pk[e] = 0;
                    } else {
                        uint32_t sc[32];
                        tmem_ld_32x32b<32>(tmem + lanes + j * 32, sc);
                        tc_wait_ld();
                        reg_fence(sc);
                        if (j < quarter || tab->steep == 0.f) {
                            const float r = ex2_approx((Ft - tab->F[j * 32 + 31]) + (It - tab->I[j * 32 + 31]));
                            const int last = j < quarter ? 31 : lane;   // the row's last column of the block
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                const float4 cs = *reinterpret_cast<const float4*>(&tab->c[j * 32 + e]);
                                const float2 lo2 = __fmul2_rn(__fmul2_rn(make_float2(r, r), make_float2(cs.x, cs.y)),
                                                              make_float2(__uint_as_float(sc[e]), __uint_as_float(sc[e + 1]))),
                                             hi2 = __fmul2_rn(__fmul2_rn(make_float2(r, r), make_float2(cs.z, cs.w)),
                                                              make_float2(__uint_as_float(sc[e + 2]), __uint_as_float(sc[e + 3])));
                                pk[e / 2] = pack_bf16(e <= last ? lo2.x : 0.f, e + 1 <= last ? lo2.y : 0.f);
                                pk[e / 2 + 1] = pack_bf16(e + 2 <= last ? hi2.x : 0.f, e + 3 <= last ? hi2.y : 0.f);
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                const float4 fs = *reinterpret_cast<const float4*>(&tab->F[j * 32 + e]);
                                const float4 is = *reinterpret_cast<const float4*>(&tab->I[j * 32 + e]);
                                auto d = [&](int o, float f, float w_) {
                                    return e + o <= lane ? __uint_as_float(sc[e + o]) * ex2_approx((Ft - f) + (It - w_))
                                                         : 0.f;
                                };
                                pk[e / 2] = pack_bf16(d(0, fs.x, is.x), d(1, fs.y, is.y));
                                pk[e / 2 + 1] = pack_bf16(d(2, fs.z, is.z), d(3, fs.w, is.w));
                            }
                        }
                    }
                    tmem_st16(tmem + lanes + C::p_col(j), pk);
                }
                tc_wait_st();
                arrive(r_p);
            }
            // ---- the state's third term, once the first two are multiplied
            if (!la_wait(b_ds1, ph, abort_flag, limit)) break;
#pragma unroll
            for (int j = 0; j < kCh; ++j) {
                const int ch = wg * kCh + j;
                *reinterpret_cast<uint4*>(stage + C::kQ + (ch >> 3) * kTileBytes + sw128(row, ch & 7)) =
                    make_uint4(lo[j][0], lo[j][1], lo[j][2], lo[j][3]);
            }
            arrive(r_lo);
            // ---- y = a (Q S) + P V, kept until the stage is free
            uint32_t o[C::NY / 2];
            if (KIND == FWD) {
                if (!la_wait(b_pv, ph, abort_flag, limit)) break;
                tc_fence_after();
#pragma unroll
                for (int j = 0; j < C::NY; j += 16) {
                    uint32_t pv[16], qs[16];
                    tmem_ld<16>(tmem + lanes + C::kPV + wg * C::NY + j, pv);
                    tmem_ld<16>(tmem + lanes + C::kQS + wg * C::NY + j, qs);
                    tc_wait_ld();
                    reg_fence(pv);
                    reg_fence(qs);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        o[j / 2 + e] = pack_bf16(fmaf(at, __uint_as_float(qs[2 * e]), __uint_as_float(pv[2 * e])),
                                                 fmaf(at, __uint_as_float(qs[2 * e + 1]), __uint_as_float(pv[2 * e + 1])));
                }
            }
            // ---- S = A S + the chunk's sum
            if (!la_wait(b_ds2, ph, abort_flag, limit)) break;
            tc_fence_after();
#pragma unroll
            for (int j = 0; j < C::NS; j += C::NL) {
                uint32_t d[C::NL];
                if constexpr (KP == 128)
                    tmem_ld<C::NL>(tmem + lanes + C::kDS + wg * C::NS + j, d);
                else   // threads 16..31: the same lanes, NS columns on
                    tmem_ld_16x32bx2<C::NL, C::NS>(tmem + lanes + C::kDS + wg * 2 * C::NS + j, d);
                tc_wait_ld();
                reg_fence(d);
#pragma unroll
                for (int e = 0; e < C::NL; ++e) S[j + e] = fmaf(A, S[j + e], __uint_as_float(d[e]));
            }
            decay *= A;
            if (KIND == FWD) {
                if (i + 1 < n) {
                    write_operand();
                    arrive(r_s);
                }
#pragma unroll
                for (int j = 0; j < C::NY; j += 8) {
                    const int col = wg * C::NY + j;
                    *reinterpret_cast<uint4*>(stage + (col >> 6) * kTileBytes + sw128(row, (col & 63) >> 3)) =
                        make_uint4(o[j / 2], o[j / 2 + 1], o[j / 2 + 2], o[j / 2 + 3]);
                }
                arrive(r_y);
            } else {
                tc_fence_before();   // ordered before the next chunk's r_k arrival
            }
        }
        if (KIND != FWD) {
            store_state(p.seg_state + ((size_t)bh * p.segs + seg) * p.K * p.V);
            if (threadIdx.x == 0) seg_decay[(size_t)bh * p.segs + seg] = decay;
        } else if (p.ST && c0 + n == nchunks) {
            store_state(p.ST + (size_t)bh * p.K * p.V);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == NW) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmem);
    }
}

// Segment sums -> segment start states, in place: start_0 = init,
// start_{i+1} = decay_i start_i + sum_i (reverse: from the last segment, for
// the gradient at segment ends).  A thread takes four adjacent elements.
__global__ void m2rnn_la_seg_scan_kernel(const LaParams p, const float* __restrict__ seg_decay, const float* init,
                                         int reverse) {
    const int kv4 = p.K * p.V / 4;
    const size_t e = blockIdx.x * (size_t)blockDim.x + threadIdx.x;
    if (e >= (size_t)p.B * p.H * kv4) return;
    const size_t bh = e / kv4, o = e % kv4;
    float4* st = reinterpret_cast<float4*>(p.seg_state) + bh * p.segs * kv4 + o;
    float4 s = init ? reinterpret_cast<const float4*>(init)[bh * kv4 + o] : make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < p.segs; ++i) {
        const int g = reverse ? p.segs - 1 - i : i;
        const float4 d = st[(size_t)g * kv4];
        st[(size_t)g * kv4] = s;
        const float a = seg_decay[bh * p.segs + g];
        s.x = fmaf(a, s.x, d.x); s.y = fmaf(a, s.y, d.y); s.z = fmaf(a, s.z, d.z); s.w = fmaf(a, s.w, d.w);
    }
}

template <int KP, int VP, int NW, Kind KIND>
cudaError_t launch_nw(const LaParams& p, const Maps& m, float* seg_decay, cudaStream_t s) {
    using C = Cfg<KP, VP, NW>;
    auto kern = m2rnn_la_fwd_tc_kernel<KP, VP, NW, KIND>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    kern<<<p.B * p.H * p.segs, C::kThreads, C::kSmem, s>>>(p, m, seg_decay);
    return cudaGetLastError();
}
template <int KP, int VP, Kind KIND>
cudaError_t launch(const LaParams& p, const Maps& m, float* seg_decay, cudaStream_t s) {
    if constexpr (Cfg<KP, VP, 8>::kCtas == 2) {
        if ((long long)p.B * p.H * p.segs > kNumSMs) return launch_nw<KP, VP, 8, KIND>(p, m, seg_decay, s);
    }
    return launch_nw<KP, VP, 16, KIND>(p, m, seg_decay, s);
}
template <Kind KIND>
cudaError_t launch_shape(const LaParams& p, const Maps& m, float* seg_decay, cudaStream_t s) {
    if (p.K <= 64)
        return p.V <= 64 ? launch<64, 64, KIND>(p, m, seg_decay, s) : launch<64, 128, KIND>(p, m, seg_decay, s);
    return p.V <= 64 ? launch<128, 64, KIND>(p, m, seg_decay, s) : launch<128, 128, KIND>(p, m, seg_decay, s);
}

float* decays_of(const LaParams& p) {   // behind the segment states in the workspace
    return p.seg_state + (size_t)p.B * p.H * p.segs * p.K * p.V;
}

}  // namespace

LaPlan la_fwd_plan(int B, int H, int T, int K, int V) {
    const int chunks = (T + kLaChunk - 1) / kLaChunk, per_sm = K <= 64 && V <= 64 ? 2 : 1;
    const long long pairs = (long long)B * H, slots = (long long)kNumSMs * per_sm;
    long long segs = 1;
    if (pairs * 2 <= kNumSMs && chunks >= 4) segs = slots / pairs;
#ifdef LA_TUNE
    if (const char* e = getenv("LA_SEGS")) segs = atoi(e);
#endif
    if (segs > chunks / 2) segs = chunks / 2;
    if (segs < 1) segs = 1;
    const int per = (int)((chunks + segs - 1) / segs);
    return {(chunks + per - 1) / per, per};
}

size_t la_seg_bytes(const LaPlan& plan, int B, int H, int K, int V) {
    return plan.segs <= 1 ? 0 : sizeof(float) * (size_t)B * H * plan.segs * ((size_t)K * V + 1);
}

cudaError_t launch_la_fwd_tc(const LaParams& p, cudaStream_t s) {
    Maps m;
    if (!la_tensor_map(&m.q, p.q, p.K, p.T, (size_t)p.B * p.G) || !la_tensor_map(&m.k, p.k, p.K, p.T, (size_t)p.B * p.G) ||
        !la_tensor_map(&m.v, p.v, p.V, p.T, (size_t)p.B * p.H) || !la_tensor_map(&m.y, p.y, p.V, p.T, (size_t)p.B * p.H))
        return cudaErrorNotSupported;
    if (p.segs > 1) {
        cudaError_t e = launch_shape<SUM>(p, m, decays_of(p), s);
        if (e != cudaSuccess) return e;
        const size_t n = (size_t)p.B * p.H * p.K * p.V / 4;
        m2rnn_la_seg_scan_kernel<<<(unsigned)((n + 127) / 128), 128, 0, s>>>(p, decays_of(p), p.S0, 0);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return launch_shape<FWD>(p, m, nullptr, s);
}

// The same sums for the gradient: what a segment's tokens add to dL/dS at its
// start, then dL/dS at every segment's end.
cudaError_t launch_la_seg_grads(const LaParams& p, cudaStream_t s) {
    Maps m;
    if (!la_tensor_map(&m.k, p.q, p.K, p.T, (size_t)p.B * p.G) || !la_tensor_map(&m.v, p.dy, p.V, p.T, (size_t)p.B * p.H))
        return cudaErrorNotSupported;
    m.q = m.k;
    m.y = m.v;
    cudaError_t e = launch_shape<RSUM>(p, m, decays_of(p), s);
    if (e != cudaSuccess) return e;
    const size_t n = (size_t)p.B * p.H * p.K * p.V / 4;
    m2rnn_la_seg_scan_kernel<<<(unsigned)((n + 127) / 128), 128, 0, s>>>(p, decays_of(p), p.dST, 1);
    return cudaGetLastError();
}

// Reads and clears the status word of this file's kernels.
cudaError_t la_fwd_tc_status(unsigned* word, cudaStream_t s) { return la_read_status(word, s); }

}  // namespace m2rnn
