// k_kv.hip -- the paged cache's plan (block tables and slot maps from request
// lengths) and append (new rows of K and V to their slots) on gfx950.
#include "serve_internal.h"

namespace qmm {

namespace {

// -------------------------------------------------------------------- plan ---

__device__ __forceinline__ int sat32(int64_t v) { return v > INT32_MAX ? INT32_MAX : (int)v; }

// Every workgroup adds up all requests' lengths (two loads a request, in
// L2 after the first) and then serves its own tokens, so one launch needs no
// order between workgroups.  Sums are 64-bit and saturate to int32 where they
// are kept.  A thread whose requests hold the workgroup's first or last token
// says so, and a token finds its request by bisection between the two in LDS:
// none where one request covers the workgroup.  A page's block table entry is
// written by the token that opens the page.  Latency bounds it: the lengths, one
// two-value scan, and per token a division and the page.  64 requests: 6.0 us, 509
// requests with 783 thousand tokens: 9.7 us (9.6 MB written).  PER tokens a thread:
// 230 thousand tokens take 7.5 us a call with one and 8.6 with four, 780 thousand
// 11.8 and 9.6.
template <int PER>
__global__ __launch_bounds__(256) void k_kv_plan(KvPlanParams p) {
    extern __shared__ int lds[];
    int *s_cu = lds, *s_first = lds + p.R;  // first new token; first place in the free list
    __shared__ int64_t part[4][2];
    __shared__ int s_flags, s_longest, s_lo, s_hi;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const uint32_t P = (uint32_t)p.page;
    const bool lead = blockIdx.x == 0;
    const int64_t begin = p.free_begin ? max(*p.free_begin, 0) : 0;
    const int64_t t0 = (int64_t)blockIdx.x * (256 * PER);
    // each thread takes `per` consecutive requests
    const int per = (p.R + 255) / 256, r0 = min(tid * per, p.R), r1 = min(r0 + per, p.R);
    int64_t toks = 0, pages = 0, longest = 0;
    int flags = 0;
    for (int r = r0; r < r1; ++r) {
        const int c = p.ctx_lens[r], n = p.new_lens[r];
        if (c < 0 || n < 0) flags |= QMM_PLAN_NEGATIVE;
        const uint32_t ctx = (uint32_t)max(c, 0), len = ctx + (uint32_t)max(n, 0);
        uint32_t have = ctx / P + (ctx % P != 0), need = len / P + (len % P != 0);
        if (need > (uint32_t)p.width) flags |= QMM_PLAN_WIDTH;
        if (lead && n > 0 && ctx % P != 0 && ctx / P < (uint32_t)p.width && p.table[(int64_t)r * p.ld_table + ctx / P] < 0)
            flags |= QMM_PLAN_NO_ENTRY;
        have = min(have, (uint32_t)p.width);
        need = min(need, (uint32_t)p.width);
        s_cu[r] = sat32(toks);
        s_first[r] = sat32(pages);
        toks += max(n, 0);
        pages += need - have;
        longest = len > longest ? len : longest;
    }
    int64_t x = toks, y = pages;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int64_t a = __shfl_up(x, d), b = __shfl_up(y, d);
        if (lane >= d) {
            x += a;
            y += b;
        }
    }
    if (lane == 63) {
        part[wave][0] = x;
        part[wave][1] = y;
    }
    if (tid == 0) {
        s_flags = 0;
        s_longest = 0;
        s_lo = 0;
        s_hi = p.R - 1;
    }
    __syncthreads();
    int64_t tok0 = x - toks, page0 = y - pages + begin, all_toks = 0, all_pages = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        if (w < wave) {
            tok0 += part[w][0];
            page0 += part[w][1];
        }
        all_toks += part[w][0];
        all_pages += part[w][1];
    }
    const int64_t t1 = t0 + 256 * PER < all_toks ? t0 + 256 * PER : all_toks;  // past the workgroup's last token
    if (r0 < r1) {
        // the last of the requests before the first (last) token lies at or past
        // these, and the first of those after it at or before them
        if (tok0 <= t0 && t0 < tok0 + toks) s_lo = r0;
        if (tok0 < t1 && t1 <= tok0 + toks) s_hi = r1 - 1;
    }
    for (int r = r0; r < r1; ++r) {
        s_cu[r] = sat32(s_cu[r] + tok0);
        s_first[r] = sat32(s_first[r] + page0);
        if (lead) p.cu_new[r] = s_cu[r];
    }
    if (lead) {
        if (flags) atomicOr(&s_flags, flags);
        atomicMax(&s_longest, sat32(longest));
    }
    __syncthreads();
    if (lead && tid == 0) {
        int f = s_flags;
        if (all_pages > 0 && begin + all_pages > p.n_free) f |= QMM_PLAN_NO_PAGES;
        if (all_toks > p.max_tokens) f |= QMM_PLAN_MAX_TOKENS;
        p.cu_new[p.R] = sat32(all_toks);
        const int64_t end = begin + all_pages;
        p.info[0] = sat32(end < p.n_free ? end : (begin > p.n_free ? begin : p.n_free));
        p.info[1] = sat32(all_toks);
        p.info[2] = f;
        p.info[3] = s_longest;
    }
    const int lo0 = s_lo, hi0 = s_hi;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int64_t t = t0 + 256 * i + tid;
        if (t >= p.max_tokens) break;
        int64_t slot = -1;
        uint32_t pos = 0;
        if (t < all_toks) {
            int lo = lo0, hi = hi0;  // the last request whose first token is <= t
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (s_cu[mid] <= t) lo = mid;
                else hi = mid - 1;
            }
            const int r = lo;
            const uint32_t ctx = (uint32_t)max(p.ctx_lens[r], 0);
            pos = ctx + (uint32_t)(t - s_cu[r]);
            const uint32_t j = pos / P, in = pos - j * P, have = ctx / P + (ctx % P != 0);
            if (j < (uint32_t)p.width) {
                int32_t *entry = p.table + (int64_t)r * p.ld_table + j;
                int page;
                if (j < have) {
                    page = *entry;
                } else {
                    const int64_t at = (int64_t)s_first[r] + (j - have);
                    page = at < p.n_free ? p.free_pages[at] : -1;
                    if (in == 0) *entry = page;
                }
                if (page >= 0) slot = (int64_t)page * P + in;
            }
        }
        p.slots[t] = slot;
        p.positions[t] = sat32(pos);
    }
}

// ------------------------------------------------------------------ append ---

template <class T>
__device__ __forceinline__ float to_f32(T v) { return (float)v; }

// LPR = next power of two >= D/8 lanes per (token, head) row, 8 values a lane;
// blockIdx.y: K or V.  One pass: a row's largest value goes round its lanes, so an
// int8 row is read once.  Memory bounds it: 8190 rows of 8 x 128 fp32 to int8 in
// 20.9 us (84 MB, 4.0 TB/s); 256 bf16 rows in 3.9 us, about the length of a launch.
template <class XT, class CT, bool VEC>
__global__ __launch_bounds__(256) void k_kv_append(KvAppendParams p, int lpr_log2) {
    const int lpr = 1 << lpr_log2, which = blockIdx.y;
    const int64_t row = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> lpr_log2;
    const int d = (threadIdx.x & (lpr - 1)) * 8;
    const bool ok = row < p.rows;
    const int64_t t = (ok ? row : 0) / p.H;
    const int h = (int)((ok ? row : 0) % p.H);
    const int64_t slot = p.slots[t];
    const bool use = ok && slot >= 0 && slot < p.n_slots;
    const XT *src = (const XT *)p.src[which] + t * p.tok[which] + h * p.head[which] + d;
    float x[8];
    const bool mine = use && d < p.D;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.0f;
    if (mine) {
        if (VEC) {
            XT raw[8];
            *(v4i *)raw = *(const v4i *)src;
            if (sizeof(XT) == 4) *(v4i *)(raw + 4) = *(const v4i *)(src + 4);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = to_f32(raw[e]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = to_f32(src[e]);
        }
    }
    const int64_t page = use ? slot / p.page : 0, i = use ? slot % p.page : 0;
    CT *dst = (CT *)p.dst[which] + page * p.page_stride + i * p.token_stride + h * p.head_stride + d;
    if (sizeof(CT) == 1) {
        // largest |x| by its bits: a NaN is above infinity, so it reaches the scale
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(x[e]) & 0x7FFFFFFFu);
        for (int o = lpr / 2; o > 0; o /= 2) m = max(m, (uint32_t)__shfl_xor((int)m, o));
        const float s = __uint_as_float(m) / 127.0f;
        uint64_t codes = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float c = s > 0.0f && m < 0x7F800000u ? fminf(fmaxf(rintf(x[e] / s), -127.0f), 127.0f) : 0.0f;
            codes |= (uint64_t)(uint8_t)(int8_t)(int)c << (8 * e);
        }
        if (mine) *(uint64_t *)dst = codes;
        if (mine && d == 0) p.scale[which][page * p.sp_stride + i * p.st_stride + h * p.sh_stride] = s;
    } else if (mine) {
        CT out[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) out[e] = (CT)x[e];
        *(v4i *)dst = *(v4i *)out;
    }
}

template <class XT, class CT>
hipError_t launch_append(const KvAppendParams &p, bool vec, hipStream_t s) {
    const int l = kv_append_lanes_log2(p.D);
    const dim3 grid((unsigned)ceil_div(p.rows << l, 256), 2);
    if (vec)
        hipLaunchKernelGGL((k_kv_append<XT, CT, true>), grid, dim3(256), 0, s, p, l);
    else
        hipLaunchKernelGGL((k_kv_append<XT, CT, false>), grid, dim3(256), 0, s, p, l);
    return hipGetLastError();
}

template <class XT>
hipError_t launch_append_x(const KvAppendParams &p, qmm_dtype ct, bool vec, hipStream_t s) {
    return ct == QMM_T_F16    ? launch_append<XT, _Float16>(p, vec, s)
           : ct == QMM_T_BF16 ? launch_append<XT, __bf16>(p, vec, s)
                              : launch_append<XT, int8_t>(p, vec, s);
}

}  // namespace

hipError_t launch_kv_plan(const KvPlanParams &p, hipStream_t s) {
    const int64_t tokens = p.max_tokens > 0 ? p.max_tokens : 1;
    if (tokens <= 256 * 1024)
        hipLaunchKernelGGL((k_kv_plan<1>), dim3((unsigned)ceil_div(tokens, 256)), dim3(256), (size_t)p.R * 8, s, p);
    else
        hipLaunchKernelGGL((k_kv_plan<4>), dim3((unsigned)ceil_div(tokens, 1024)), dim3(256), (size_t)p.R * 8, s, p);
    return hipGetLastError();
}

hipError_t launch_kv_append(const KvAppendParams &p, qmm_dtype xt, qmm_dtype ct, bool vec, hipStream_t s) {
    return xt == QMM_T_F32   ? launch_append_x<float>(p, ct, vec, s)
           : xt == QMM_T_F16 ? launch_append_x<_Float16>(p, ct, vec, s)
                             : launch_append_x<__bf16>(p, ct, vec, s);
}

}  // namespace qmm
