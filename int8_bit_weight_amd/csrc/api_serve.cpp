// api_serve.cpp -- C ABI of the drafted-token verification operators: argument
// checks and dispatch.  Everything is checked before anything is enqueued.
#include <hip/hip_runtime.h>

#include <cmath>

#include "api_checks.h"
#include "qmm.h"
#include "serve_internal.h"

using namespace qmm;

namespace {

bool group_ok(int64_t g) { return g == 32 || g == 64 || (g > 0 && g % 128 == 0); }

bool has_scales(const qmm_kv_cache *c) { return c->type == QMM_T_S8 || c->type == QMM_T_Q4; }

// The checks of a cache that every call on it makes.
qmm_status check_cache(const qmm_kv_cache *c) {
    if (!c || c->num_pages < 1 || c->page_size < 1 || c->n_heads < 1 || c->head_dim < 1) return QMM_ERR_INVALID;
    if (c->type != QMM_T_F16 && c->type != QMM_T_BF16 && c->type != QMM_T_S8 && c->type != QMM_T_Q4) return QMM_ERR_INVALID;
    if (!c->k || !c->v) return QMM_ERR_INVALID;
    if (!span_ok({{c->num_pages, c->page_stride}, {c->page_size, c->token_stride}, {c->n_heads, c->head_stride}}))
        return QMM_ERR_INVALID;
    if (has_scales(c)) {
        if (!c->k_scale || !c->v_scale || !aligned_to(c->k_scale, 4) || !aligned_to(c->v_scale, 4))
            return QMM_ERR_INVALID;
        if (!span_ok({{c->num_pages, c->scale_page_stride},
                      {c->page_size, c->scale_token_stride},
                      {c->n_heads, c->scale_head_stride}}))
            return QMM_ERR_INVALID;
    }
    if (c->head_dim > 256 || c->head_dim % (c->type == QMM_T_Q4 ? 16 : 8) != 0 || c->page_size >= (1 << 20) || c->num_pages > kMaxSize ||
        c->n_heads > kMaxSize)
        return QMM_ERR_UNSUPPORTED;
    // rows of 8 elements: 16 bytes, int8 8 bytes; 4-bit rows of 16 elements: 8 bytes, which their strides count
    const size_t a = has_scales(c) ? 8 : 16;
    if (!aligned_to(c->k, a) || !aligned_to(c->v, a) || (c->num_pages > 1 && c->page_stride % 8) ||
        (c->page_size > 1 && c->token_stride % 8) || (c->n_heads > 1 && c->head_stride % 8))
        return QMM_ERR_UNSUPPORTED;
    return QMM_OK;
}

// The checks of rows beside a cache and its slots, and the kernels' arguments.
qmm_status kv_rows(const void *K, int64_t k_token_stride, int64_t k_head_stride, const void *V, int64_t v_token_stride,
                   int64_t v_head_stride, qmm_dtype xt, int64_t T, const int64_t *slots, const qmm_kv_cache *c,
                   KvAppendParams &p, bool &vec) {
    if (T < 0 || (xt != QMM_T_F32 && xt != QMM_T_F16 && xt != QMM_T_BF16)) return QMM_ERR_INVALID;
    const qmm_status st = check_cache(c);
    if (st != QMM_OK) return st;
    if (!span_ok({{T, k_token_stride}, {c->n_heads, k_head_stride}}) ||
        !span_ok({{T, v_token_stride}, {c->n_heads, v_head_stride}}))
        return QMM_ERR_INVALID;
    if (T > kMaxSize || T * c->n_heads > kGridThreads >> kv_append_lanes_log2(c->head_dim))
        return QMM_ERR_UNSUPPORTED;
    if (T == 0) return QMM_OK;
    const size_t es = (size_t)size_of(xt);
    if (!K || !V || !slots || !aligned_to(slots, 8) || !aligned_to(K, es) || !aligned_to(V, es)) return QMM_ERR_INVALID;
    p.src[0] = K;
    p.src[1] = V;
    p.tok[0] = k_token_stride;
    p.tok[1] = v_token_stride;
    p.head[0] = k_head_stride;
    p.head[1] = v_head_stride;
    p.dst[0] = c->k;
    p.dst[1] = c->v;
    p.scale[0] = c->k_scale;
    p.scale[1] = c->v_scale;
    p.slots = slots;
    p.n_slots = c->num_pages * c->page_size;
    p.page_stride = c->page_stride;
    p.token_stride = c->token_stride;
    p.head_stride = c->head_stride;
    p.sp_stride = c->scale_page_stride;
    p.st_stride = c->scale_token_stride;
    p.sh_stride = c->scale_head_stride;
    p.rows = T * c->n_heads;
    p.H = (int)c->n_heads;
    p.D = (int)c->head_dim;
    p.page = (int)c->page_size;
    const int64_t a = (int64_t)(16 / es);
    vec = aligned_to(K, 16) && aligned_to(V, 16) && k_token_stride % a == 0 && k_head_stride % a == 0 &&
          v_token_stride % a == 0 && v_head_stride % a == 0;
    return QMM_OK;
}

// The checks of an attention call and its kernels' arguments, but for what a row sees, of which
// most_keys is a bound.
qmm_status attention(const void *Q, int64_t q_token_stride, int64_t q_head_stride, qmm_dtype xt, int64_t T, int64_t Hq,
                     const qmm_kv_cache *c, const int32_t *block_table, int64_t ld_table, int64_t table_width,
                     const int32_t *ctx_lens, const int32_t *cu_new, int64_t R, int64_t mask_cols, float scale, void *O,
                     int64_t o_token_stride, int64_t o_head_stride, void *workspace, size_t workspace_bytes,
                     int64_t most_keys, TreeParams &p, TreeShape &z) {
    if (T < 0 || Hq < 1 || R < 0 || table_width < 0 || ld_table < table_width) return QMM_ERR_INVALID;
    if (xt != QMM_T_F16 && xt != QMM_T_BF16 && xt != QMM_T_F32) return QMM_ERR_INVALID;
    if (!std::isfinite(scale)) return QMM_ERR_INVALID;
    const qmm_status st = check_cache(c);
    if (st != QMM_OK) return st;
    if (Hq % c->n_heads != 0) return QMM_ERR_INVALID;
    if (!span_ok({{T, q_token_stride}, {Hq, q_head_stride}}) || !span_ok({{T, o_token_stride}, {Hq, o_head_stride}}))
        return QMM_ERR_INVALID;
    if (xt == QMM_T_F32 || (has_scales(c) ? xt != QMM_T_BF16 : xt != c->type)) return QMM_ERR_UNSUPPORTED;
    if (T > kMaxSize || Hq > 65535 || T * (Hq / c->n_heads) > kMaxSize || R > kMaxSize || table_width > INT32_MAX || mask_cols > INT32_MAX ||
        table_width * c->page_size > kTreeMaxKeys)
        return QMM_ERR_UNSUPPORTED;
    if (T == 0 || R == 0) return QMM_OK;
    if (!Q || !O || !ctx_lens || !cu_new || !aligned_to(ctx_lens, 4) || !aligned_to(cu_new, 4) || !aligned_to(Q, 2) ||
        !aligned_to(O, 2) || (table_width > 0 && (!block_table || !aligned_to(block_table, 4))))
        return QMM_ERR_INVALID;
    p.Q = Q;
    p.O = O;
    p.q_tok = q_token_stride;
    p.q_head = q_head_stride;
    p.o_tok = o_token_stride;
    p.o_head = o_head_stride;
    p.k = c->k;
    p.v = c->v;
    p.k_scale = c->k_scale;
    p.v_scale = c->v_scale;
    p.page_stride = c->page_stride;
    p.token_stride = c->token_stride;
    p.head_stride = c->head_stride;
    p.sp_stride = c->scale_page_stride;
    p.st_stride = c->scale_token_stride;
    p.sh_stride = c->scale_head_stride;
    p.table = block_table;
    p.ctx_lens = ctx_lens;
    p.cu_new = cu_new;
    p.ld_table = ld_table;
    p.T = (int)T;
    p.Hq = (int)Hq;
    p.Hkv = (int)c->n_heads;
    p.G = (int)(Hq / c->n_heads);
    p.D = (int)c->head_dim;
    p.R = (int)R;
    p.width = (int)table_width;
    p.page = (int)c->page_size;
    // with 2^(l-1) < page <= 2^l the multiplier is below 2^32, and above 2^(31+l) / page by less than one part in 2^31 of it
    while ((1 << (p.page_shift)) < p.page) ++p.page_shift;
    p.page_shift += 31;
    p.page_mul = (uint32_t)((((uint64_t)1 << p.page_shift) + p.page - 1) / p.page);
    p.num_pages = (int)c->num_pages;
    p.scale = std::fabs(scale) * 1.4426950408889634f;
    p.q_flip = scale < 0 ? (int)0x80008000 : 0;
    p.q_vec = aligned_to(Q, 16) && q_token_stride % 8 == 0 && q_head_stride % 8 == 0;
    p.o_vec = aligned_to(O, 8) && o_token_stride % 4 == 0 && o_head_stride % 4 == 0;
    const int64_t keys = table_width * c->page_size;
    z = tree_shape(T, p.G, R, p.Hkv, p.D, keys < most_keys ? keys : most_keys, c->type == QMM_T_Q4);
    if (!workspace || !aligned_to(workspace, 256)) return QMM_ERR_WORKSPACE;
    // rows whose sums are not finite are computed again from Q once O has been written
    if (may_overlap({Q, {T, Hq}, {2 * q_token_stride, 2 * q_head_stride}, 2 * c->head_dim},
                    {O, {T, Hq}, {2 * o_token_stride, 2 * o_head_stride}, 2 * c->head_dim}))
        return QMM_ERR_INVALID;
    if (workspace_bytes < (size_t)z.total) return QMM_ERR_WORKSPACE;
    p.hdr = (TreeHeader *)workspace;
    p.part = (float *)((char *)workspace + z.hdr_bytes);
    p.slot_rows = z.slot_rows;
    p.wgs = (int)z.wgs;
    return QMM_OK;
}

}  // namespace

extern "C" {

// --------------------------------------------------- group-scaled product ---

size_t qmm_q4_group_packed_bytes(int64_t K, int64_t N, int64_t group) {
    if (K <= 0 || N <= 0 || !group_ok(group) || K > kMaxSize || N > kMaxSize) return 0;
    const Q4gLayout L = q4g_layout(K, N, group);
    return q4g_fits(L) ? (size_t)L.total : 0;
}

qmm_status q4_group_repack(const uint8_t *codes, int64_t ldc, const void *scales, qmm_dtype st, int64_t lds,
                           const uint8_t *zeros, int64_t ldz, int64_t K, int64_t N, int64_t group,
                           void *packed, size_t packed_bytes, void *stream) {
    if (K <= 0 || N <= 0 || group <= 0 || !codes || !scales || !packed || !aligned_to(packed, 256) ||
        !aligned_to(scales, 2))
        return QMM_ERR_INVALID;
    if (st != QMM_T_F16 && st != QMM_T_BF16) return QMM_ERR_INVALID;
    if (ldc < ceil_div(K, 2) || lds < ceil_div(K, group) || (zeros && ldz < ceil_div(K, group))) return QMM_ERR_INVALID;
    if (!group_ok(group) || K > kMaxSize || N > kMaxSize) return QMM_ERR_UNSUPPORTED;
    const Q4gLayout L = q4g_layout(K, N, group);
    if (!q4g_fits(L)) return QMM_ERR_UNSUPPORTED;
    if (packed_bytes < (size_t)L.total) return QMM_ERR_WORKSPACE;
    return record_status(launch_q4g_repack(codes, ldc, scales, st == QMM_T_BF16, lds, zeros, ldz, group, L,
                                           (uint8_t *)packed, (hipStream_t)stream),
                         "q4g_repack");
}

// The most a call of these sizes needs, whatever the alignment of its rows.
size_t qmm_q4_group_matmul_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t group, qmm_dtype xt) {
    if (M <= 0 || K <= 0 || N <= 0 || !group_ok(group) || M > kQ4gMaxRows || K > kMaxSize || N > kMaxSize) return 0;
    const Q4gLayout L = q4g_layout(K, N, group);
    return q4g_fits(L) ? (size_t)q4g_shape(M, N, xt == QMM_T_F32 ? 3 : 1, false, L).total : 0;
}

qmm_status q4_group_matmul(const void *X, qmm_dtype xt, int64_t M, int64_t K, int64_t ldx, const void *Wpacked,
                           int64_t N, int64_t group, void *Y, int64_t ldy, void *workspace, size_t workspace_bytes,
                           void *stream) {
    if (M < 0 || K <= 0 || N < 0 || group <= 0 || ldx < K || ldy < N) return QMM_ERR_INVALID;
    if (xt != QMM_T_F32 && xt != QMM_T_F16 && xt != QMM_T_BF16) return QMM_ERR_INVALID;
    if (!group_ok(group) || M > kQ4gMaxRows || K > kMaxSize || N > kMaxSize) return QMM_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return QMM_OK;
    const size_t es = (size_t)size_of(xt);
    if (!X || !Wpacked || !Y || !aligned_to(Wpacked, 256) || !aligned_to(X, es) || !aligned_to(Y, es))
        return QMM_ERR_INVALID;
    const Q4gLayout L = q4g_layout(K, N, group);
    if (!q4g_fits(L)) return QMM_ERR_UNSUPPORTED;
    Q4gParams p{};
    p.recs = (const uint8_t *)Wpacked;
    p.words = (const uint32_t *)(p.recs + L.words_off);
    p.X = X;
    p.Y = Y;
    p.ldx = ldx;
    p.ldy = ldy;
    p.M = (int)M;
    p.K = (int)K;
    p.N = (int)N;
    p.NQ = (int)L.NQ;
    p.NS = (int)L.NS;
    p.NG = (int)L.NG;
    p.rpg = group < 128 ? 1 : (int)(group / 128 < L.NQ ? group / 128 : L.NQ);
    p.gpr = (int)L.gpr;
    p.x_vec = aligned_to(X, 16) && (M == 1 || ldx * (int64_t)es % 16 == 0);
    const Q4gShape z = q4g_shape(M, N, xt == QMM_T_F32 ? 3 : 1, p.x_vec && K >= 8, L);
    if (z.total > 0 && (!workspace || !aligned_to(workspace, 256))) return QMM_ERR_WORKSPACE;
    // workgroups read all rows of X while others write their columns of Y
    if (may_overlap({X, {M, 1}, {(int64_t)es * ldx, 0}, (int64_t)es * K}, {Y, {M, 1}, {(int64_t)es * ldy, 0}, (int64_t)es * N}))
        return QMM_ERR_INVALID;
    if (z.total > 0) {
        if (workspace_bytes < (size_t)z.total) return QMM_ERR_WORKSPACE;
        p.xa = workspace;
        p.xs = (float *)((char *)workspace + z.xs_off);
        p.part = (float *)((char *)workspace + z.part_off);
    }
    const char *variant = "";
    const hipError_t e = launch_q4g_matmul(p, xt, (int)L.gpr, z, (hipStream_t)stream, &variant);
    return record_status(e, variant);
}

// ------------------------------------------------------------- paged cache ---

qmm_status kv_plan(const int32_t *ctx_lens, const int32_t *new_lens, int64_t R, int32_t *block_table,
                   int64_t ld_table, int64_t table_width, int64_t page_size, const int32_t *free_pages,
                   int64_t n_free, const int32_t *free_begin, int64_t max_tokens, int32_t *cu_new,
                   int64_t *slots, int32_t *positions, int32_t *info, void *stream) {
    if (R < 0 || table_width < 0 || ld_table < table_width || page_size < 1 || n_free < 0 || max_tokens < 0)
        return QMM_ERR_INVALID;
    if (!cu_new || !info || !aligned_to(cu_new, 4) || !aligned_to(info, 4)) return QMM_ERR_INVALID;
    if (R > 0 && (!ctx_lens || !new_lens || !aligned_to(ctx_lens, 4) || !aligned_to(new_lens, 4)))
        return QMM_ERR_INVALID;
    if (R > 0 && table_width > 0 && (!block_table || !aligned_to(block_table, 4))) return QMM_ERR_INVALID;
    if (n_free > 0 && (!free_pages || !aligned_to(free_pages, 4))) return QMM_ERR_INVALID;
    if (max_tokens > 0 && (!slots || !positions || !aligned_to(slots, 8) || !aligned_to(positions, 4)))
        return QMM_ERR_INVALID;
    if (free_begin && (!aligned_to(free_begin, 4) || (free_begin >= info && free_begin < info + 4)))
        return QMM_ERR_INVALID;
    if (R > kPlanMaxRequests || n_free > kMaxSize || max_tokens > kMaxSize || page_size > INT32_MAX ||
        table_width > INT32_MAX || table_width * page_size > INT32_MAX)
        return QMM_ERR_UNSUPPORTED;
    KvPlanParams p{};
    p.ctx_lens = ctx_lens;
    p.new_lens = new_lens;
    p.table = block_table;
    p.ld_table = ld_table;
    p.free_pages = free_pages;
    p.free_begin = free_begin;
    p.cu_new = cu_new;
    p.positions = positions;
    p.info = info;
    p.slots = slots;
    p.R = (int)R;
    p.width = (int)table_width;
    p.page = (int)page_size;
    p.n_free = (int)n_free;
    p.max_tokens = (int)max_tokens;
    return record_status(launch_kv_plan(p, (hipStream_t)stream), "kv_plan");
}

qmm_status kv_append(const void *K, int64_t k_token_stride, int64_t k_head_stride, const void *V,
                     int64_t v_token_stride, int64_t v_head_stride, qmm_dtype xt, int64_t T,
                     const int64_t *slots, const qmm_kv_cache *c, void *stream) {
    KvAppendParams p{};
    bool vec = false;
    const qmm_status st = kv_rows(K, k_token_stride, k_head_stride, V, v_token_stride, v_head_stride, xt, T, slots, c, p, vec);
    if (st != QMM_OK || T == 0) return st;
    return record_status(launch_kv_append(p, xt, c->type, vec, (hipStream_t)stream), "kv_append");
}

qmm_status kv_gather(const int64_t *slots, int64_t T, const qmm_kv_cache *c, void *K, int64_t k_token_stride,
                     int64_t k_head_stride, void *V, int64_t v_token_stride, int64_t v_head_stride, qmm_dtype xt,
                     void *stream) {
    KvAppendParams p{};
    bool vec = false;
    const qmm_status st = kv_rows(K, k_token_stride, k_head_stride, V, v_token_stride, v_head_stride, xt, T, slots, c, p, vec);
    if (st != QMM_OK || T == 0) return st;
    const int64_t es = size_of(xt), H = c->n_heads;
    if (may_overlap({K, {T, H}, {es * k_token_stride, es * k_head_stride}, es * c->head_dim},
                    {V, {T, H}, {es * v_token_stride, es * v_head_stride}, es * c->head_dim}))
        return QMM_ERR_INVALID;
    return record_status(launch_kv_gather(p, xt, c->type, vec, (hipStream_t)stream), "kv_gather");
}

// ---------------------------------------------------------- tree attention ---

size_t qmm_tree_attention_workspace_bytes(int64_t T, int64_t Hq, int64_t R, int64_t n_heads, int64_t head_dim) {
    if (T <= 0 || R <= 0 || n_heads < 1 || Hq < 1 || Hq % n_heads != 0 || head_dim < 1 || head_dim > 256 ||
        T > kMaxSize || Hq > 65535)
        return 0;
    // the most that a cache of any type and length needs
    size_t most = 0;
    for (bool q4 : {false, true})
        for (int64_t keys : {(int64_t)1, (int64_t)INT32_MAX}) {
            const size_t n = (size_t)tree_shape(T, Hq / n_heads, R, n_heads, head_dim, keys, q4).total;
            if (n > most) most = n;
        }
    return most;
}

qmm_status tree_attention(const void *Q, int64_t q_token_stride, int64_t q_head_stride, qmm_dtype xt, int64_t T,
                          int64_t Hq, const qmm_kv_cache *c, const int32_t *block_table, int64_t ld_table,
                          int64_t table_width, const int32_t *ctx_lens, const int32_t *cu_new, int64_t R,
                          const uint8_t *mask, int64_t ld_mask, int64_t mask_cols, float scale, void *O,
                          int64_t o_token_stride, int64_t o_head_stride, void *workspace, size_t workspace_bytes,
                          void *stream) {
    if (mask && (mask_cols < 0 || ld_mask < mask_cols)) return QMM_ERR_INVALID;
    TreeParams p{};
    TreeShape z;
    const qmm_status st = attention(Q, q_token_stride, q_head_stride, xt, T, Hq, c, block_table, ld_table, table_width, ctx_lens,
                                    cu_new, R, mask_cols, scale, O, o_token_stride, o_head_stride, workspace, workspace_bytes,
                                    INT64_MAX, p, z);
    if (st != QMM_OK || T == 0 || R == 0) return st;
    p.mask = mask;
    p.ld_mask = ld_mask;
    p.mask_cols = (int)mask_cols;
    const char *variant = "";
    const hipError_t e = launch_tree_attention(p, z, c->type, (hipStream_t)stream, &variant);
    return record_status(e, variant);
}

size_t qmm_window_attention_workspace_bytes(int64_t T, int64_t Hq, int64_t R, int64_t n_heads, int64_t head_dim) {
    return qmm_tree_attention_workspace_bytes(T, Hq, R, n_heads, head_dim);
}

qmm_status window_attention(const void *Q, int64_t q_token_stride, int64_t q_head_stride, qmm_dtype xt, int64_t T,
                            int64_t Hq, const qmm_kv_cache *c, const int32_t *block_table, int64_t ld_table,
                            int64_t table_width, const int32_t *ctx_lens, const int32_t *cu_new, int64_t R,
                            int64_t window, int64_t sinks, float scale, void *O, int64_t o_token_stride,
                            int64_t o_head_stride, void *workspace, size_t workspace_bytes, void *stream) {
    if (window < 1 || sinks < 0) return QMM_ERR_INVALID;
    // keys that a request's tokens can see
    const int64_t seen = window < INT32_MAX && sinks < INT32_MAX && T < INT32_MAX ? window + sinks + T : INT64_MAX;
    TreeParams p{};
    TreeShape z;
    const qmm_status st = attention(Q, q_token_stride, q_head_stride, xt, T, Hq, c, block_table, ld_table, table_width, ctx_lens,
                                    cu_new, R, 0, scale, O, o_token_stride, o_head_stride, workspace, workspace_bytes,
                                    seen, p, z);
    if (st != QMM_OK || T == 0 || R == 0) return st;
    p.window = (int)(window < INT32_MAX ? window : INT32_MAX);
    p.sinks = (int)(sinks < INT32_MAX ? sinks : INT32_MAX);
    const char *variant = "";
    const hipError_t e = launch_window_attention(p, z, c->type, (hipStream_t)stream, &variant);
    return record_status(e, variant);
}

}  // extern "C"
