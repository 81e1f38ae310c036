// C ABI of linear attention and of the layer norm: argument validation,
// workspace carving and dispatch (declared in include/m2rnn.h).
#include "linear_attention.h"

#include <cstring>
#include <initializer_list>
#include <mutex>

#include "../../include/m2rnn.h"
#include "kernels.h"
#include "layer_norm.h"

namespace {

constexpr size_t kRefused = ~(size_t)0;

bool state_dim_ok(int n) { return n == 16 || n == 32 || n == 64 || n == 128; }

bool any_misaligned(std::initializer_list<const void*> ptrs) {
    for (const void* p : ptrs)
        if (reinterpret_cast<uintptr_t>(p) & 15u) return true;
    return false;
}

m2rnn_status check(const m2rnn_la_dims* d) {
    if (d == nullptr || d->B < 0 || d->H < 0 || d->T < 0) return M2RNN_ERR_INVALID_ARG;
    if (d->mode != M2RNN_MODE_BF16_TC && d->mode != M2RNN_MODE_FP32_DEBUG) return M2RNN_ERR_INVALID_ARG;
    if (d->qk_heads < 0 || (d->qk_heads > 0 && (d->qk_heads > d->H || d->H % d->qk_heads != 0)))
        return M2RNN_ERR_INVALID_ARG;
    if ((d->f_is_logit & ~1) || (d->f_per_head & ~1)) return M2RNN_ERR_INVALID_ARG;
    if (!state_dim_ok(d->K) || !state_dim_ok(d->V)) return M2RNN_ERR_UNSUPPORTED_SHAPE;
    // pairs, and tokens over all pairs, index 32-bit grids and coordinates
    if ((long long)d->B * d->H > (1 << 24) || d->T > (1 << 30)) return M2RNN_ERR_UNSUPPORTED_SHAPE;
    return M2RNN_OK;
}

int groups(const m2rnn_la_dims* d) { return d->qk_heads > 0 ? d->qk_heads : d->H; }
size_t pairs(const m2rnn_la_dims* d) { return (size_t)d->B * d->H; }
size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// Per-head fp32 dk and dq before the sum over each group's heads.
size_t group_bytes(const m2rnn_la_dims* d) {
    return groups(d) == d->H ? 0 : round256(2 * sizeof(float) * pairs(d) * d->T * d->K);
}
// Per-token df before the sum over batch and time.
size_t df_bytes(const m2rnn_la_dims* d) { return d->f_per_head ? round256(sizeof(float) * pairs(d) * d->T) : 0; }

// Prompts run on the tensor cores, whose chunk costs the same at any fill;
// short ones run token by token, which costs a step each.  Measured, us, tokens
// against chunks at T = 8, 11, 12 and 16:
//    16 pairs of 16 x 16      5.3 / 6.8,  6.8 / 6.8,  7.3 / 6.8,  9.2 / 6.8
//    16 pairs of 64 x 64      5.2 / 7.0,  6.5 / 7.0,  6.8 / 7.0,  8.6 / 6.9
//   128 pairs of 64 x 64      6.2 / 8.1,  7.8 / 8.0,  8.2 / 8.0, 10.3 / 8.1
//   128 pairs of 128 x 128   10.4 / 12.5, 13.1 / 12.6, 13.8 / 12.6, 17.2 / 12.4
// (More pairs than SMs would turn later, up to T = 20: 512 pairs of 64 x 64 22.0
// against 26.5 at 16.)
bool fwd_on_tensor_cores(const m2rnn_la_dims* d) { return d->mode == M2RNN_MODE_BF16_TC && d->T > 11; }

bool bwd_on_tensor_cores(const m2rnn_la_dims* d) { return d->mode == M2RNN_MODE_BF16_TC; }
m2rnn::LaPlan plan_of(const m2rnn_la_dims* d, bool backward) { return m2rnn::la_plan(d->B, d->H, d->T, backward); }
size_t seg_bytes(const m2rnn_la_dims* d, bool backward) {
    if (!(backward ? bwd_on_tensor_cores(d) : fwd_on_tensor_cores(d))) return 0;
    return m2rnn::la_seg_bytes(plan_of(d, backward), d->B, d->H, d->K, d->V);
}

m2rnn::LaParams params(const m2rnn_la_dims* d) {
    m2rnn::LaParams p;
    std::memset(&p, 0, sizeof p);
    p.B = d->B; p.H = d->H; p.T = d->T; p.K = d->K; p.V = d->V;
    p.G = groups(d);
    p.bf16 = d->mode == M2RNN_MODE_BF16_TC;
    p.f_is_logit = d->f_is_logit;
    p.f_per_head = d->f_per_head;
    p.segs = 1;
    p.seg_chunks = (d->T + m2rnn::kLaChunk - 1) / m2rnn::kLaChunk;
    p.limit = {m2rnn::wait_limit_ns(), 0};
    p.fault = m2rnn::injected_fault();
    return p;
}

// What a failed CUDA call leaves behind for cudaGetLastError(), which the
// launches ask: taken away where a call fails, and before one begins, so that an
// error is reported by the call that it belongs to alone.
void drop_last_error() { (void)cudaGetLastError(); }
m2rnn_status status_of(cudaError_t e) {
    if (e == cudaSuccess) return M2RNN_OK;
    drop_last_error();
    return M2RNN_ERR_CUDA;
}

// The status words in use: a stream's is found by its device and its id, which no
// other stream is given in the life of the process.
struct StatusWords {
    std::mutex lock;
    unsigned count = 1;         // word 0 is the shared one
    bool shared = false;        // it has been given to a call
    int device[m2rnn::kLaSlots];
    unsigned long long id[m2rnn::kLaSlots];
};
StatusWords g_words;

// A stream by its device and id.  One that is being captured is not told apart:
// its calls are those of the stream that will replay them.
struct StreamKey {
    int device = 0;
    unsigned long long id = 0;
    bool known = false, capturing = false;
};
StreamKey key_of(cudaStream_t s) {
    StreamKey k;
    cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
    if (cudaGetDevice(&k.device) == cudaSuccess && cudaStreamIsCapturing(s, &capture) == cudaSuccess) {
        k.capturing = capture != cudaStreamCaptureStatusNone;
        k.known = !k.capturing && cudaStreamGetId(s, &k.id) == cudaSuccess;
    }
    if (!k.known) drop_last_error();
    return k;
}
unsigned find_word(const StreamKey& k) {   // (with the lock held) 0: none
    for (unsigned i = 1; k.known && i < g_words.count; ++i)
        if (g_words.id[i] == k.id && g_words.device[i] == k.device) return i;
    return 0;
}
// The word of a call that is about to be launched.
unsigned word_for_call(cudaStream_t s) {
    const StreamKey k = key_of(s);
    const std::lock_guard<std::mutex> hold(g_words.lock);
    if (const unsigned i = find_word(k)) return i;
    if (k.known && g_words.count < m2rnn::kLaSlots) {
        g_words.device[g_words.count] = k.device;
        g_words.id[g_words.count] = k.id;
        return g_words.count++;
    }
    g_words.shared = true;
    return 0;
}

// No tokens: the state (or its gradient) passes through.
m2rnn_status pass_through(float* out, const float* in, size_t n, cudaStream_t s) {
    if (!out || out == in || n == 0) return M2RNN_OK;
    return status_of(in ? cudaMemcpyAsync(out, in, n * sizeof(float), cudaMemcpyDeviceToDevice, s)
                        : cudaMemsetAsync(out, 0, n * sizeof(float), s));
}

}  // namespace

extern "C" {

size_t m2rnn_linear_attention_workspace(const m2rnn_la_dims* d, int backward) {
    if (check(d) != M2RNN_OK) return kRefused;
    if (pairs(d) * d->T == 0) return 0;
    if (!backward) return seg_bytes(d, false);
    return group_bytes(d) + df_bytes(d) + seg_bytes(d, true);
}

m2rnn_status m2rnn_linear_attention_forward(const m2rnn_la_dims* d, const void* k, const void* v, const void* q,
                                            const float* f, const float* S0, void* y, float* ST, float* ckpt,
                                            void* workspace, size_t ws_bytes, m2rnn_stream_t stream) {
    const m2rnn_status st = check(d);
    if (st != M2RNN_OK) return st;
    if (pairs(d) * d->T > 0 && (!k || !v || !q || !f || !y)) return M2RNN_ERR_INVALID_ARG;
    if (any_misaligned({k, v, q, f, S0, y, ST, ckpt, workspace})) return M2RNN_ERR_MISALIGNED;
    const size_t need = m2rnn_linear_attention_workspace(d, 0);
    if (need > 0 && (!workspace || ws_bytes < need)) return M2RNN_ERR_WORKSPACE;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    drop_last_error();
    if (pairs(d) * d->T == 0) return pass_through(ST, S0, pairs(d) * d->K * d->V, s);
    m2rnn::LaParams p = params(d);
    p.k = k; p.v = v; p.q = q; p.f = f; p.S0 = S0; p.y = y; p.ST = ST; p.ckpt = ckpt;
    if (!fwd_on_tensor_cores(d)) return status_of(m2rnn::launch_la_rec(p, s));
    p.limit.slot = word_for_call(s);
    const m2rnn::LaPlan plan = plan_of(d, false);
    p.segs = plan.segs; p.seg_chunks = plan.seg_chunks;
    p.seg_state = static_cast<float*>(workspace);
    return status_of(m2rnn::launch_la_fwd_tc(p, s));
}

m2rnn_status m2rnn_linear_attention_backward(const m2rnn_la_dims* d, const void* k, const void* v, const void* q,
                                             const float* f, const float* ckpt, const void* dy, const float* dST,
                                             void* dk, void* dv, void* dq, float* df, float* dS0, void* workspace,
                                             size_t ws_bytes, m2rnn_stream_t stream) {
    const m2rnn_status st = check(d);
    if (st != M2RNN_OK) return st;
    if (pairs(d) * d->T > 0 && (!k || !v || !q || !f || !ckpt || !dy || !dk || !dv || !dq || !df))
        return M2RNN_ERR_INVALID_ARG;
    if ((pairs(d) > 0 && !dS0) || (d->f_per_head && d->H > 0 && !df)) return M2RNN_ERR_INVALID_ARG;
    if (any_misaligned({k, v, q, f, ckpt, dy, dST, dk, dv, dq, df, dS0, workspace})) return M2RNN_ERR_MISALIGNED;
    const size_t need = m2rnn_linear_attention_workspace(d, 1);
    if (need > 0 && (!workspace || ws_bytes < need)) return M2RNN_ERR_WORKSPACE;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    drop_last_error();
    if (pairs(d) * d->T == 0) {
        if (d->f_per_head && d->H > 0) {
            const m2rnn_status z = status_of(cudaMemsetAsync(df, 0, sizeof(float) * d->H, s));
            if (z != M2RNN_OK) return z;
        }
        return pass_through(dS0, dST, pairs(d) * d->K * d->V, s);
    }
    m2rnn::LaParams p = params(d);
    p.k = k; p.v = v; p.q = q; p.f = f; p.ckpt = const_cast<float*>(ckpt); p.dy = dy; p.dST = dST;
    p.dk = dk; p.dq = dq; p.dv = dv; p.df = df; p.dS0 = dS0;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    if (group_bytes(d)) {
        p.dkq_fp32 = 1;
        p.dk = ws;
        p.dq = reinterpret_cast<float*>(ws) + pairs(d) * d->T * d->K;
    }
    if (d->f_per_head) p.df = reinterpret_cast<float*>(ws + group_bytes(d));
    cudaError_t e;
    if (bwd_on_tensor_cores(d)) {
        p.limit.slot = word_for_call(s);
        const m2rnn::LaPlan plan = plan_of(d, true);
        p.segs = plan.segs; p.seg_chunks = plan.seg_chunks;
        p.seg_state = reinterpret_cast<float*>(ws + group_bytes(d) + df_bytes(d));
        e = m2rnn::launch_la_bwd_tc(p, s);
    } else {
        e = m2rnn::launch_la_bwd_simt(p, s);
    }
    if (e == cudaSuccess && group_bytes(d))
        e = m2rnn::launch_la_group_sum(p, static_cast<const float*>(p.dk), static_cast<const float*>(p.dq), dk, dq, s);
    if (e == cudaSuccess && d->f_per_head) e = m2rnn::launch_la_df_sum(p, p.df, df, s);
    return status_of(e);
}

m2rnn_status m2rnn_linear_attention_status(m2rnn_stream_t stream) {
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const StreamKey k = key_of(s);
    unsigned slots[2], n = 0, any = 0;
    {
        const std::lock_guard<std::mutex> hold(g_words.lock);
        if (const unsigned i = find_word(k)) slots[n++] = i;
        if (g_words.shared || k.capturing) slots[n++] = 0;   // (a stream that is being captured cannot be synchronised: an error)
    }
    for (unsigned i = 0; i < n; ++i) {
        unsigned word[2] = {0, 0};
        for (cudaError_t e : {m2rnn::la_fwd_tc_status(slots[i], &word[0], s), m2rnn::la_bwd_tc_status(slots[i], &word[1], s)})
            if (e != cudaSuccess) return status_of(e);
        any |= word[0] | word[1];
    }
    return any ? M2RNN_ERR_DEVICE_TIMEOUT : M2RNN_OK;
}

// ------------------------------------------------------------------ layer norm

static m2rnn_status check_norm(const m2rnn_norm_dims* d) {
    if (d == nullptr || d->B < 0 || d->H < 0 || d->T < 0 || d->N < 1) return M2RNN_ERR_INVALID_ARG;
    if ((d->x_fp32 & ~1) || (d->y_fp32 & ~1) || (d->dx_fp32 & ~1) || (d->rms & ~1)) return M2RNN_ERR_INVALID_ARG;
    if (d->dx_fp32 && !d->x_fp32) return M2RNN_ERR_INVALID_ARG;
    if (!(d->eps >= 0.f)) return M2RNN_ERR_INVALID_ARG;
    // pairs index 32-bit grids, rows and blocks of rows 32-bit counters
    if ((long long)d->B * d->H > (1 << 24) || d->T > (1 << 30) || d->N > (1 << 28)) return M2RNN_ERR_UNSUPPORTED_SHAPE;
    if ((long long)d->B * d->H * d->T > (1LL << 35)) return M2RNN_ERR_UNSUPPORTED_SHAPE;
    return M2RNN_OK;
}
// The weight's and bias's gradients are summed by one CTA for 32 of their columns.
static m2rnn_status check_norm_sums(const m2rnn_norm_dims* d) {
    const m2rnn_status st = check_norm(d);
    if (st != M2RNN_OK) return st;
    return (long long)m2rnn::norm_dw_blocks(d->N) * d->H > 0x7FFFFFFFLL ? M2RNN_ERR_UNSUPPORTED_SHAPE : M2RNN_OK;
}

static m2rnn::NormParams norm_params(const m2rnn_norm_dims* d) {
    m2rnn::NormParams p;
    std::memset(&p, 0, sizeof p);
    p.B = d->B; p.H = d->H; p.T = d->T; p.N = d->N;
    p.x_fp32 = d->x_fp32; p.y_fp32 = d->y_fp32; p.dx_fp32 = d->dx_fp32; p.rms = d->rms; p.eps = d->eps;
    return p;
}

m2rnn_status m2rnn_layer_norm_forward(const m2rnn_norm_dims* d, const void* x, const float* weight, const float* bias,
                                      void* y, float* mean, float* rstd, m2rnn_stream_t stream) {
    const m2rnn_status st = check_norm(d);
    if (st != M2RNN_OK) return st;
    if ((size_t)d->B * d->H * d->T == 0) return M2RNN_OK;
    if (!x || !y) return M2RNN_ERR_INVALID_ARG;
    if (any_misaligned({x, weight, bias, y, mean, rstd})) return M2RNN_ERR_MISALIGNED;
    drop_last_error();
    m2rnn::NormParams p = norm_params(d);
    p.x = x; p.weight = weight; p.bias = bias; p.y = y; p.mean = mean; p.rstd = rstd;
    return status_of(m2rnn::launch_norm_fwd(p, reinterpret_cast<cudaStream_t>(stream)));
}

size_t m2rnn_layer_norm_workspace(const m2rnn_norm_dims* d) {
    if (check_norm_sums(d) != M2RNN_OK) return kRefused;
    if ((size_t)d->B * d->H * d->T == 0) return 0;
    return sizeof(float) * 2 * d->N * ((size_t)d->B * d->H * m2rnn::norm_bwd_chunks(d->B, d->H, d->T, d->N));
}

m2rnn_status m2rnn_layer_norm_backward(const m2rnn_norm_dims* d, const void* dy, const void* x, const float* weight,
                                       const float* mean, const float* rstd, void* dx, float* dweight, float* dbias,
                                       void* workspace, size_t ws_bytes, m2rnn_stream_t stream) {
    const bool sums = dweight || dbias;
    const m2rnn_status st = sums ? check_norm_sums(d) : check_norm(d);
    if (st != M2RNN_OK) return st;
    if (any_misaligned({dy, x, weight, mean, rstd, dx, dweight, dbias, workspace})) return M2RNN_ERR_MISALIGNED;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    drop_last_error();
    if ((size_t)d->B * d->H * d->T == 0) {
        for (float* g : {dweight, dbias})
            if (g && d->H > 0) {
                const m2rnn_status z = status_of(cudaMemsetAsync(g, 0, sizeof(float) * d->H * d->N, s));
                if (z != M2RNN_OK) return z;
            }
        return M2RNN_OK;
    }
    if (!dy || !x || !rstd || !dx || (!d->rms && !mean)) return M2RNN_ERR_INVALID_ARG;
    if (sums && (!workspace || ws_bytes < m2rnn_layer_norm_workspace(d))) return M2RNN_ERR_WORKSPACE;
    m2rnn::NormParams p = norm_params(d);
    p.dy = dy; p.x = x; p.weight = weight; p.mean = const_cast<float*>(mean); p.rstd = const_cast<float*>(rstd);
    p.dx = dx; p.dweight = dweight; p.dbias = dbias;
    p.part = sums ? static_cast<float*>(workspace) : nullptr;
    p.chunks = m2rnn::norm_bwd_chunks(d->B, d->H, d->T, d->N);
    return status_of(m2rnn::launch_norm_bwd(p, s));
}

}  // extern "C"
