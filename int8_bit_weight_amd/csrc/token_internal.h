// token_internal.h -- internal declarations of the adapters (k_lora.hip) and the
// log probabilities of tokens (k_logprobs.hip).
#pragma once

#include "qmm_internal.h"

namespace qmm {

// ------------------------------------------------------- log probabilities ---

constexpr int kTopGroup = 32;      // tokens of which the first launch keeps the largest logit
constexpr int64_t kMaxVocab = (int64_t)1 << 28;

struct LogprobParams {
    const void *logits;
    int64_t ld;
    const int64_t *tokens;
    int64_t ld_tokens;
    float *logprobs, *entropy, *top_lp;
    int64_t *top_ids;
    float scale, scale_e; // log2(e) times the caller's; the caller's
    int T, V, n, top;
    int chunks, groups;   // of a row
    float *part;          // [T][chunks][3]: largest logit m, sum of e = exp(z - z(m)), sum of e log2(e)
    float *gmax;          // [T][groups]
};

// A wavefront of the first launch takes `loads` 16-byte loads a lane.
struct LogprobShape {
    int loads;
    int64_t chunks, groups, gmax_off, total;
};

inline LogprobShape logprob_shape(int64_t T, int64_t V, int64_t es, bool top) {
    LogprobShape z{};
    const int64_t vec = 16 / es;
    const int64_t span = V + vec - 1;  // from the 16 bytes that hold a row's first element
    z.loads = T * ceil_div(span, 64 * vec * 8) >= 2048 ? 8 : 2;
    z.chunks = ceil_div(span, 64 * vec * z.loads);
    z.groups = z.chunks * (64 * vec * z.loads / kTopGroup);
    z.gmax_off = round_up(T * z.chunks * 12, 256);
    z.total = z.gmax_off + (top ? T * z.groups * 4 : 0);
    return z;
}

hipError_t launch_logprobs(const LogprobParams &p, const LogprobShape &z, qmm_dtype xt, hipStream_t s);

// ----------------------------------------------------------------- adapters ---

struct LoraParams {
    const void *X, *A, *B, *base;
    void *out;
    int64_t ldx, a_stride, lda, b_stride, ldb, ld_base, ld_out;
    const int32_t *adapters;
    const float *scales;
    int T, K, N, rank, n_adapters;
    int rp, splits, per;             // rank in whole 16s; ranges of k, of `per` 32s each
    float *z;                        // [splits][T][rp]
};

constexpr int kLoraMaxRank = 128;

// How a call is cut: rows of a workgroup, 16 or (of many rows) 64; ranges of k.
struct LoraShape {
    int rows, rp, splits, per;
    int64_t total;
};

inline LoraShape lora_shape(int64_t T, int64_t K, int64_t rank) {
    LoraShape z{};
    // us a call with 64 and with 16 rows a workgroup, K = 4096, 8 adapters in runs / in turn:
    //   T                  96                    160                   256                   400
    //   N 4096, rank 16    16, 37 / 10, 12       17, 37 / 12, 17       17, 37 / 16, 23       17, 37 / 23, 35
    //   N 14336, rank 64   29, 71 / 28, 44       30, 73 / 44, 66       30, 74 / 68, 96       31, 74 / 99, 146
    z.rows = T > (rank > 32 ? 128 : 256) ? 64 : 16;
    z.rp = (int)round_up(rank, 16);
    const int64_t steps = ceil_div(K, 32), tiles = ceil_div(T, z.rows);
    int64_t splits = ceil_div(512, tiles);  // two workgroups to a CU
    if (splits > ceil_div(steps, z.rows == 64 ? 8 : 4)) splits = ceil_div(steps, z.rows == 64 ? 8 : 4);
    if (splits > 16) splits = 16;
    z.per = (int)round_up(ceil_div(steps, splits), z.rows == 64 ? 2 : 1);
    z.splits = (int)ceil_div(steps, z.per);
    z.total = (int64_t)z.splits * T * z.rp * 4;
    return z;
}

hipError_t launch_lora(const LoraParams &p, const LoraShape &z, qmm_dtype xt, hipStream_t s);

}  // namespace qmm
