// k_tree_attention.hip -- attention of drafted tokens over a paged cache on
// gfx950.
//
//   O[t,h] = sum_j exp(c s_j - m) v_j / sum_j exp(c s_j - m),  s_j = q[t,h].k_j
//
// over the keys j that t sees, m their running maximum.
#include "serve_internal.h"

namespace qmm {

namespace {

// One wavefront per (query row, head): 64 keys a step, a key per lane for the
// scores, then 4 values of the head dimension per lane for the sum over V.
template <class XT, class CT>
__global__ __launch_bounds__(64) void k_tree_simple(TreeParams p) {
    const int lane = threadIdx.x;
    const int t = blockIdx.x, h = blockIdx.y, hk = h / p.G;
    // the request of row t
    int lo = 0, hi = p.R - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.cu_new[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    const int r = lo, first = p.cu_new[r], last = p.cu_new[r + 1];
    if (t < first || t >= last) return;
    const int ctx = max(p.ctx_lens[r], 0);
    const int64_t cap = (int64_t)p.width * p.page, end = (int64_t)ctx + last - first;
    const int len = (int)(end < cap ? end : cap);
    __shared__ float s_q[256], s_p[64];
    __shared__ int64_t s_row[64];
    __shared__ float s_vs[64];
    const XT *q = (const XT *)p.Q + t * p.q_tok + h * p.q_head;
    for (int d = lane; d < p.D; d += 64) s_q[d] = (float)q[d];
    float m = -INFINITY, l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int j0 = 0; j0 < len; j0 += 64) {
        const int j = j0 + lane;
        bool sees = j < len;
        int page = -1;
        if (sees) {
            page = p.table[(int64_t)r * p.ld_table + j / p.page];
            sees = page >= 0 && page < p.num_pages;
        }
        if (sees && j >= ctx) {
            const int i = j - ctx;
            sees = p.mask ? i < p.mask_cols && p.mask[t * p.ld_mask + i] != 0 : i <= t - first;
        }
        const int64_t row = sees ? (int64_t)page * p.page_stride + (int64_t)(j % p.page) * p.token_stride + hk * p.head_stride : 0;
        const int64_t srow = sees ? (int64_t)page * p.sp_stride + (int64_t)(j % p.page) * p.st_stride + hk * p.sh_stride : 0;
        __syncthreads();
        float s = 0.0f;
        if (sees)
            for (int d = 0; d < p.D; ++d) s = fmaf(s_q[d], (float)((const CT *)p.k)[row + d], s);
        if (sizeof(CT) == 1 && sees) s *= p.k_scale[srow];
        s = sees ? s * p.scale : -INFINITY;
        float top = s;
#pragma unroll
        for (int x = 32; x > 0; x /= 2) top = fmaxf(top, __shfl_xor(top, x));
        const float mn = fmaxf(m, top), base = mn == -INFINITY ? 0.0f : mn;
        const float pj = sees ? exp2f(s - base) : 0.0f, alpha = exp2f(m - base);
        m = mn;
        float sum = pj;
#pragma unroll
        for (int x = 32; x > 0; x /= 2) sum += __shfl_xor(sum, x);
        l = l * alpha + sum;
        s_p[lane] = pj;
        s_row[lane] = sees ? row : -1;
        s_vs[lane] = sizeof(CT) == 1 && sees ? p.v_scale[srow] : 1.0f;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] *= alpha;
        for (int k = 0; k < 64; ++k) {
            const int64_t vr = s_row[k];
            if (vr < 0) continue;
            const float w = s_p[k] * s_vs[k];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int d = lane + 64 * e;
                if (d < p.D) o[e] = fmaf(w, (float)((const CT *)p.v)[vr + d], o[e]);
            }
        }
        __syncthreads();
    }
    XT *out = (XT *)p.O + t * p.o_tok + h * p.o_head;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int d = lane + 64 * e;
        if (d < p.D) out[d] = (XT)(l == 0.0f ? 0.0f : o[e] / l);
    }
}

}  // namespace

hipError_t launch_tree_attention(const TreeParams &p, qmm_dtype xt, qmm_dtype ct, hipStream_t s, const char **variant) {
    const dim3 grid((unsigned)p.T, (unsigned)p.Hq), block(64);
    *variant = "tree_simple";
    if (ct == QMM_T_F16)
        hipLaunchKernelGGL((k_tree_simple<_Float16, _Float16>), grid, block, 0, s, p);
    else if (ct == QMM_T_BF16)
        hipLaunchKernelGGL((k_tree_simple<__bf16, __bf16>), grid, block, 0, s, p);
    else
        hipLaunchKernelGGL((k_tree_simple<__bf16, int8_t>), grid, block, 0, s, p);
    return hipGetLastError();
}

}  // namespace qmm
