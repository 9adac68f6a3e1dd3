// api_tokens.cpp -- C ABI of the adapters and of the log probabilities: argument
// checks and dispatch.  Everything is checked before anything is enqueued.
#include <hip/hip_runtime.h>

#include <cmath>

#include "api_checks.h"
#include "qmm.h"
#include "token_internal.h"

using namespace qmm;

namespace {

bool is_float(qmm_dtype t) { return t == QMM_T_F32 || t == QMM_T_F16 || t == QMM_T_BF16; }

constexpr float kLog2e = 1.4426950408889634f;
constexpr int64_t kMaxWorkgroups = (int64_t)1 << 24;  // of 256 threads in one grid

bool lora_fits(int64_t T, int64_t K, int64_t N, int64_t rank) {
    return T <= kMaxSize && K <= kMaxSize && N <= kMaxSize && rank <= kLoraMaxRank && T * ceil_div(N, 64) < kMaxWorkgroups;
}

bool logprobs_fit(int64_t T, int64_t V) { return V <= kMaxVocab && T <= kMaxWorkgroups && T * ceil_div(V, 2048) < kMaxWorkgroups; }

}  // namespace

extern "C" {

// ------------------------------------------------------------------ adapters ---

size_t qmm_lora_matmul_workspace_bytes(int64_t T, int64_t K, int64_t rank) {
    if (T <= 0 || K <= 0 || rank <= 0 || !lora_fits(T, K, 1, rank)) return 0;
    return (size_t)lora_shape(T, K, rank).total;
}

qmm_status lora_matmul(const void *X, qmm_dtype xt, int64_t T, int64_t K, int64_t ldx, const void *A, int64_t a_stride,
                       int64_t lda, const void *B, int64_t b_stride, int64_t ldb, qmm_dtype wt, int64_t n_adapters,
                       int64_t rank, int64_t N, const int32_t *adapters, const float *scales, const void *base,
                       int64_t ld_base, void *out, int64_t ld_out, void *workspace, size_t workspace_bytes,
                       void *stream) {
    if (T < 0 || K <= 0 || N < 0 || rank <= 0 || n_adapters < 0 || ldx < K || lda < K || ldb < rank || ld_out < N ||
        (base && ld_base < N))
        return QMM_ERR_INVALID;
    if (!is_float(xt) || !is_float(wt)) return QMM_ERR_INVALID;
    if (!span_ok({{n_adapters, a_stride}, {rank, lda}}) || !span_ok({{n_adapters, b_stride}, {N, ldb}}) ||
        !span_ok({{T, ldx}}) || !span_ok({{T, ld_out}}) || (base && !span_ok({{T, ld_base}})))
        return QMM_ERR_INVALID;
    if (wt != (xt == QMM_T_F32 ? QMM_T_BF16 : xt) || n_adapters > kMaxSize || !lora_fits(T, K, N, rank))
        return QMM_ERR_UNSUPPORTED;
    if (T == 0 || N == 0) return QMM_OK;
    const int64_t es = size_of(xt);
    if (!X || !adapters || !out || (n_adapters > 0 && (!A || !B)) || !aligned_to(X, es) || !aligned_to(out, es) ||
        !aligned_to(base, es) || !aligned_to(A, 2) || !aligned_to(B, 2) || !aligned_to(adapters, 4) || !aligned_to(scales, 4))
        return QMM_ERR_INVALID;
    LoraParams p{};
    const LoraShape z = lora_shape(T, K, rank);
    if (!workspace || !aligned_to(workspace, 256)) return QMM_ERR_WORKSPACE;
    // lanes read their own columns of base before they write them, and no others'
    if (base && !(base == out && (ld_base == ld_out || T == 1)) &&
        may_overlap({base, {T, 1}, {es * ld_base, 0}, es * N}, {out, {T, 1}, {es * ld_out, 0}, es * N}))
        return QMM_ERR_INVALID;
    if (may_overlap({X, {T, 1}, {es * ldx, 0}, es * K}, {out, {T, 1}, {es * ld_out, 0}, es * N})) return QMM_ERR_INVALID;
    if (workspace_bytes < (size_t)z.total) return QMM_ERR_WORKSPACE;
    p.X = X;
    p.A = A;
    p.B = B;
    p.base = base;
    p.out = out;
    p.ldx = ldx;
    p.a_stride = a_stride;
    p.lda = lda;
    p.b_stride = b_stride;
    p.ldb = ldb;
    p.ld_base = ld_base;
    p.ld_out = ld_out;
    p.adapters = adapters;
    p.scales = scales;
    p.T = (int)T;
    p.K = (int)K;
    p.N = (int)N;
    p.rank = (int)rank;
    p.n_adapters = (int)n_adapters;
    p.rp = z.rp;
    p.splits = z.splits;
    p.per = z.per;
    p.z = (float *)workspace;
    return record_status(launch_lora(p, z, xt, (hipStream_t)stream), z.rows == 64 ? "lora_rows64" : "lora_rows16");
}

// --------------------------------------------------------- log probabilities ---

size_t qmm_token_logprobs_workspace_bytes(int64_t T, int64_t V) {
    if (T <= 0 || V <= 0 || !logprobs_fit(T, V)) return 0;
    int64_t most = 0;
    for (int64_t es : {2, 4}) {
        const int64_t n = logprob_shape(T, V, es, true).total;
        if (n > most) most = n;
    }
    return (size_t)most;
}

qmm_status token_logprobs(const void *logits, qmm_dtype xt, int64_t T, int64_t V, int64_t ld, const int64_t *tokens,
                          int64_t ld_tokens, int64_t n, int64_t top, float scale, float *logprobs, float *entropy,
                          int64_t *top_ids, float *top_logprobs, void *workspace, size_t workspace_bytes, void *stream) {
    if (T < 0 || V <= 0 || ld < V || n < 0 || top < 0 || !(scale > 0.0f) || !std::isfinite(scale * kLog2e)) return QMM_ERR_INVALID;
    if (n > 0 && ld_tokens < n) return QMM_ERR_INVALID;
    if (!is_float(xt)) return QMM_ERR_INVALID;
    if (!span_ok({{T, ld}}) || !span_ok({{T, ld_tokens}})) return QMM_ERR_INVALID;
    if (top > QMM_MAX_TOP || n > kMaxSize || !logprobs_fit(T, V)) return QMM_ERR_UNSUPPORTED;
    if (T == 0) return QMM_OK;
    const int64_t es = size_of(xt);
    if (!logits || !aligned_to(logits, es) || !aligned_to(entropy, 4)) return QMM_ERR_INVALID;
    if (n > 0 && (!tokens || !logprobs || !aligned_to(tokens, 8) || !aligned_to(logprobs, 4))) return QMM_ERR_INVALID;
    if (top > 0 && (!top_ids || !top_logprobs || !aligned_to(top_ids, 8) || !aligned_to(top_logprobs, 4)))
        return QMM_ERR_INVALID;
    const LogprobShape z = logprob_shape(T, V, es, top > 0);
    if (!workspace || !aligned_to(workspace, 256) || workspace_bytes < (size_t)z.total) return QMM_ERR_WORKSPACE;
    LogprobParams p{};
    p.logits = logits;
    p.ld = ld;
    p.tokens = tokens;
    p.ld_tokens = ld_tokens;
    p.logprobs = logprobs;
    p.entropy = entropy;
    p.top_lp = top_logprobs;
    p.top_ids = top_ids;
    p.scale = scale * kLog2e;
    p.scale_e = scale;
    p.T = (int)T;
    p.V = (int)V;
    p.n = (int)n;
    p.top = (int)top;
    p.chunks = (int)z.chunks;
    p.groups = (int)z.groups;
    p.part = (float *)workspace;
    p.gmax = (float *)((char *)workspace + z.gmax_off);
    return record_status(launch_logprobs(p, z, xt, (hipStream_t)stream), z.loads == 8 ? "logprobs_wide" : "logprobs_narrow");
}

}  // extern "C"
