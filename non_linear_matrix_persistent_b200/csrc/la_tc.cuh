// Pieces shared by the tensor-core kernels of linear attention: tiles of 128
// tokens fetched by TMA into 128-byte-swizzled shared memory, their matrix
// descriptors, decays, operand splitting and bounded waits.
//
// A tile [128 rows][64 columns] of bf16 takes 16 KB: row r at r·128 bytes, its
// 16-byte chunk c at position c ^ (r & 7) (the 128-byte swizzle).  A width of
// 128 is two such tiles; widths of 16 and 32 run as 64, with the columns and
// the rows behind the last token filled with zeros by the copy.  The same tile
// serves as a K-major operand (contraction along the columns) and as an
// MN-major one (contraction along the rows), so no transposed copy exists.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>

#include "linear_attention.h"
#include "ptx.cuh"

namespace m2rnn {

constexpr int kTileBytes = 128 * 128;   // 128 tokens x 64 bf16

// The kernels' device status: words for each source file, read and cleared by
// m2rnn_linear_attention_status.  A wait that runs out sets its call's.
static __device__ unsigned g_la_status[kLaSlots];

// Floor of a gate's base-2 logarithm.  Forward: 2^-256, which every product of
// decays flushes to 0, so a gate of 0 (or below 2^-126) discards the state.
// Backward: 2^-100, so that the sums over paths through a gate of 0, divided
// by the gate again, still give its gradient; in the other gradients the rest
// of such a gate's exponent is made up for (LaTablesZ::Z).
constexpr float kLogFloorFwd = -256.f, kLogFloorBwd = -100.f, kGateFloorBwd = 7.888609052210118e-31f;

// log2 of a gate split into an integer and a fraction in [-1/2, 1/2]: sums of
// the integers are exact, so differences of cumulative sums keep their
// precision behind a gate close to 0.  A NaN stays a NaN.
// `rest`: what the floor took away (a gate of 0 has a logarithm of -300 here).
__device__ __forceinline__ void la_log2(const LaParams& p, float x, float floor_, float& whole, float& frac,
                                        float& rest) {
    float l = p.f_is_logit ? -1.4426950408889634f * log1pf(expf(-x)) : log2f(x);
    rest = l < floor_ ? fmaxf(l, -300.f) - floor_ : 0.f;
    l = l < floor_ ? floor_ : l;
    whole = rintf(l);
    frac = l - whole;
}

// Cumulative log-decays of a chunk's 128 tokens, from the chunk's start
// through the token, by one warp (4 tokens a lane): F + I in shared memory
// (128 whole parts of -256 at most: 16 bits),
// and c[t] = the decay from t to the last token of its block of 32 or, with
// FROM_PREV, from the last token of the block before through t.
// steep: some block of 32 decays by more than 2^-90.  Elsewhere the decay
// between two tokens of one block is the product of a decay to the block's end
// and the reciprocal of another, both far inside fp32's range: c[] serves the
// diagonal blocks too.
struct LaTables {
    float F[128], c[128];
    short I[128];
    float steep, pad[3];
};
__device__ __forceinline__ float4 la_whole(const LaTables* tab, int t) {   // I[t..t+3]
    const short4 w = *reinterpret_cast<const short4*>(&tab->I[t]);
    return make_float4(w.x, w.y, w.z, w.w);
}
struct LaTablesZ : LaTables {
    float Z[128];   // exponents beneath the floor, from the chunk's start through the token: 0 or negative
};
// The fraction back into [-1/2, 1/2]: a cumulative sum keeps the precision of
// its small part, which the decays between neighbours are made of.
__device__ __forceinline__ void la_carry(float& frac, float& whole) {
    const float r = rintf(frac);
    frac -= r;
    whole += r;
}
template <bool FROM_PREV = false, class Tab = LaTables>
__device__ __forceinline__ void la_tables(Tab* tab, const LaParams& p, const float (&x)[4], int valid, float floor_) {
    const int lane = threadIdx.x & 31;
    float F[4], I[4], Z[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float rest;
        la_log2(p, x[i], floor_, I[i], F[i], rest);
        if (lane * 4 + i >= valid) { F[i] = 0.f; I[i] = 0.f; rest = 0.f; }   // behind the last token: a gate of 1
        Z[i] = rest + (i > 0 ? Z[i > 0 ? i - 1 : 0] : 0.f);
        if (i > 0) {
            F[i] += F[i - 1];
            I[i] += I[i - 1];
            la_carry(F[i], I[i]);
        }
    }
    float f = F[3], w = I[3];
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const float a = __shfl_up_sync(~0u, f, d), b = __shfl_up_sync(~0u, w, d);
        if (lane >= d) { f += a; w += b; }
        la_carry(f, w);
    }
    const float f0 = __shfl_up_sync(~0u, f, 1), w0 = __shfl_up_sync(~0u, w, 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        F[i] += lane ? f0 : 0.f;
        I[i] += lane ? w0 : 0.f;
        la_carry(F[i], I[i]);
    }
    if constexpr (FROM_PREV) {
        float z = Z[3];
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const float a = __shfl_up_sync(~0u, z, d);
            if (lane >= d) z += a;
        }
        z -= Z[3];
        *reinterpret_cast<float4*>(&tab->Z[lane * 4]) = make_float4(z + Z[0], z + Z[1], z + Z[2], z + Z[3]);
    }
    // the block's last token, or the one before the block
    float fe = __shfl_sync(~0u, F[3], FROM_PREV ? (lane & ~7) - 1 : lane | 7),
          we = __shfl_sync(~0u, I[3], FROM_PREV ? (lane & ~7) - 1 : lane | 7);
    {
        const float pe = __shfl_sync(~0u, F[3] + I[3], lane < 8 ? 0 : (lane & ~7) - 1),
                    ee = __shfl_sync(~0u, F[3] + I[3], lane | 7);
        const bool any = __any_sync(~0u, !(ee - (lane < 8 ? 0.f : pe) > -90.f));
        if (lane == 0) tab->steep = any ? 1.f : 0.f;
    }
    float sign = 1.f;
    if (FROM_PREV) {
        if (lane < 8) { fe = 0.f; we = 0.f; }
        sign = -1.f;
    }
    *reinterpret_cast<float4*>(&tab->F[lane * 4]) = make_float4(F[0], F[1], F[2], F[3]);
    *reinterpret_cast<short4*>(&tab->I[lane * 4]) = make_short4((short)I[0], (short)I[1], (short)I[2], (short)I[3]);
    *reinterpret_cast<float4*>(&tab->c[lane * 4]) =
        make_float4(ex2_approx(sign * ((fe - F[0]) + (we - I[0]))), ex2_approx(sign * ((fe - F[1]) + (we - I[1]))),
                    ex2_approx(sign * ((fe - F[2]) + (we - I[2]))), ex2_approx(sign * ((fe - F[3]) + (we - I[3]))));
}
// The f inputs of chunk c for la_tables; 0 behind the last token.
__device__ __forceinline__ void la_load_f(const LaParams& p, int bh, int c, float (&x)[4]) {
    const int t = c * kLaChunk + (threadIdx.x & 31) * 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = t + i < p.T ? la_f_input(p, bh, t + i) : 0.f;
}

// ---------------------------------------------------------------- operands
// Byte position of the 16-byte chunk `ch` (of 8) of row `row` in a swizzled tile.
__device__ __forceinline__ uint32_t sw128(int row, int ch) { return row * 128 + ((ch ^ (row & 7)) << 4); }

// A descriptor as its two words: positions are added to the lower one alone.
struct Desc {
    uint32_t lo, hi;
};
__device__ __forceinline__ Desc operator+(Desc d, uint32_t at) { return {d.lo + at, d.hi}; }
// Descriptor of a 128-byte-swizzled operand.  K-major: lbo unused, sbo = 1024
// (8 rows).  MN-major: lbo = bytes from one 64-column tile to the next, sbo =
// 1024 (8 contraction rows).
__device__ __forceinline__ Desc sw128_desc(uint32_t saddr, uint32_t lbo) {
    const uint64_t d = smem_desc(saddr, lbo, 1024) | (2ull << 61);
    return {(uint32_t)d, (uint32_t)(d >> 32)};
}

// Products issued by a whole warp, of which the lane with `one` != 0 issues: the
// operands are the same in every lane, so that they are computed and kept in
// uniform registers.
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, Desc a, Desc b, uint32_t idesc, uint32_t accumulate, uint32_t one) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %2};\n\t"
        "mov.b64 b, {%3, %4};\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "setp.ne.b32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d_tmem),
        "r"(a.lo), "r"(a.hi), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"(accumulate), "r"(one)
        : "memory");
}
// The same, leaving 64 lanes of D as they are: the lower half, or the upper one.
template <bool LOWER>
__device__ __forceinline__ void mma_ss_half(uint32_t d_tmem, Desc a, Desc b, uint32_t idesc, uint32_t one) {
    constexpr uint32_t lo = LOWER ? 0xFFFFFFFFu : 0u, hi = ~lo;   // lanes 0-63, lanes 64-127 not written
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %2};\n\t"
        "mov.b64 b, {%3, %4};\n\t"
        "setp.eq.b32 p, 0, 0;\n\t"
        "setp.ne.b32 q, %6, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, {%7, %7, %8, %8}, p;\n\t}" ::"r"(d_tmem),
        "r"(a.lo), "r"(a.hi), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"(one), "r"(lo), "r"(hi)
        : "memory");
}
// The same with A in tensor memory: 128 lanes, two bf16 per 32-bit column.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, Desc b, uint32_t idesc, uint32_t accumulate,
                                       uint32_t one) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "setp.ne.b32 q, %6, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"(accumulate), "r"(one)
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar, uint32_t one) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(one)
        : "memory");
}

// Tensor-memory store of 16 columns (32x32b).
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// Tensor-memory load of N (8, 16 or 32) adjacent columns of this thread's lane.
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[N]) {
    tmem_ld_32x32b<N>(taddr, r);
}

// 32 bytes to a 32-byte aligned address: one whole sector.
__device__ __forceinline__ void st_global_v8(void* dst, const uint32_t* v) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// x = hi + lo to 2^-16 of x: lo is what hi left over (exact in fp32), rounded to
// nearest.
__device__ __forceinline__ void split2(float x0, float x1, uint32_t& hi, uint32_t& lo) {
    hi = pack_bf16(x0, x1);
    lo = pack_bf16(x0 - bf16lo_to_f32(hi), x1 - bf16hi_to_f32(hi));
}
// x = hi + mid + lo to about 2^-26 of x: each term is what the bf16 before it
// left over (exact in fp32), rounded to nearest.
__device__ __forceinline__ void split3(float x0, float x1, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
    hi = pack_bf16(x0, x1);
    x0 -= bf16lo_to_f32(hi);
    x1 -= bf16hi_to_f32(hi);
    mid = pack_bf16(x0, x1);
    lo = pack_bf16(x0 - bf16lo_to_f32(mid), x1 - bf16hi_to_f32(mid));
}

// ---------------------------------------------------------------- TMA
// Box of 128 tokens x 64 columns at column x, token t of row block z.
__device__ __forceinline__ void tma_tile(uint32_t dst, const CUtensorMap* map, int x, int t, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(t), "r"(z), "r"(bar)
        : "memory");
}

// `bytes` (a multiple of 16) from a 16-byte aligned address into L2.
__device__ __forceinline__ void bulk_prefetch(const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}
// The same box from shared memory; columns and rows outside the tensor are left out.
__device__ __forceinline__ void tma_store_tile(const CUtensorMap* map, uint32_t src, int x, int t, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map),
                 "r"(x), "r"(t), "r"(z), "r"(src)
                 : "memory");
}
__device__ __forceinline__ void tma_store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// The stores committed by this thread have read their shared memory.
__device__ __forceinline__ void tma_store_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

// ---------------------------------------------------------------- waits
// Bounded mbarrier wait of a whole warp: false when it runs longer than the
// limit or another thread of the CTA has given up.  The outcome is the warp's:
// what follows it (tensor-memory accesses, shuffles, the way out) takes all 32
// lanes, and lanes that answered for themselves could part between a phase that
// completes and a limit that runs out.  Nor does a barrier move on by two phases
// while some lanes see the first: the next one waits for this warp.  The vote
// also tells the compiler that the outcome is uniform, so that what the issuing
// warp computes stays in uniform registers, where the products take their
// operands from.  (64 attempts in an asm loop and a vote behind them: 128 pairs
// of 128 x 128 forward 6% slower.)
__device__ __forceinline__ bool la_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, LaLimit limit) {
    uint64_t t0 = 0;
    for (int k = 1;; ++k) {
        if (__all_sync(~0u, mbar_try_wait(bar, parity))) return true;
        if ((k & 63) == 0) {
            const uint64_t t = globaltimer_ns();
            if (t0 == 0) t0 = t;
            const bool late = t - t0 > limit.ns;
            if (__any_sync(~0u, late || *abort_flag)) {
                if (late) {
                    *abort_flag = 1;
                    atomicOr(&g_la_status[limit.slot], 1u);
                }
                __syncwarp();
                return false;
            }
        }
    }
}
// The same for a single lane, which the rest of its warp awaits at a __syncwarp.
__device__ __forceinline__ bool la_wait_lane(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                             LaLimit limit) {
    uint64_t t0 = 0;
    for (int k = 1;; ++k) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((k & 63) == 0) {
            if (*abort_flag) return false;
            const uint64_t t = globaltimer_ns();
            if (t0 == 0) t0 = t;
            if (t - t0 > limit.ns) {
                *abort_flag = 1;
                atomicOr(&g_la_status[limit.slot], 1u);
                return false;
            }
        }
    }
}
// The same without the abort flag: for copies and products in flight before the CTA exits.
__device__ __forceinline__ void la_drain(uint32_t bar, uint32_t parity, LaLimit limit) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity))
        if (globaltimer_ns() - t0 > limit.ns) {
            atomicOr(&g_la_status[limit.slot], 1u);
            return;
        }
}

// ---------------------------------------------------------------- host
// Reads and clears a status word of this source file.
static inline cudaError_t la_read_status(unsigned slot, unsigned* word, cudaStream_t s) {
    const unsigned zero = 0;
    const size_t at = slot * sizeof zero;
    cudaError_t e = cudaMemcpyFromSymbolAsync(word, g_la_status, sizeof *word, at, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e == cudaSuccess && *word) {
        e = cudaMemcpyToSymbolAsync(g_la_status, &zero, sizeof zero, at, cudaMemcpyHostToDevice, s);
        if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    }
    return e;
}
// Tensor map of x [rows][T][width] bf16: boxes of 128 tokens x 64 columns.
bool la_tensor_map(CUtensorMap* map, const void* x, int width, int T, size_t rows);

}  // namespace m2rnn
