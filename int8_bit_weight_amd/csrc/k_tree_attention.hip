// k_tree_attention.hip -- attention of drafted tokens over a paged cache on
// gfx950.
//
//   O[t,h] = sum_j exp(c s_j - m) v_j / sum_j exp(c s_j - m),  s_j = q[t,h].k_j
//
// over the keys j that t sees, m their running maximum, in one pass over K and V.
//
// The rows (drafted token, query head) that read one cache head of one request
// are the columns of a matrix product: S^T = K Q^T puts 16 keys x 16 rows in a
// wavefront with a row's scores in four lanes, and those registers are the
// second operand of O^T = V^T P^T as they stand (the order of the 32 keys of a
// step is free, and V^T is read from LDS with the transposing load in the same
// order), so the weights never leave their registers.
//
// Work is cut evenly over a fixed number of workgroups: the key blocks of all
// (request, cache head, row tile) items stand in one line, and each workgroup takes
// one run of it, whatever the lengths.  An item that several workgroups share
// leaves sums in the workspace, which a second launch joins; the lengths are read
// on the device only, so a captured graph serves any lengths.
//
// Weights enter the second product as two terms of the operand type (16 bits of
// significand and more), so that the output's own rounding is the only one
// that shows.  NaN and infinities reach rows that must not see them through
// 0 * NaN in the matrix products only; rows whose sums are not finite are computed
// again by the second launch with plain fp32 steps that skip hidden keys.
#include "serve_internal.h"

namespace qmm {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef int v2i __attribute__((ext_vector_type(2)));

struct F16 {
    typedef _Float16 T;
    typedef v8h V;
    // weights carry a factor 2^7: with it the second term of a weight of 2^-14
    // is still an fp16 normal's neighbour, and 2^8 (the slack of the maximum)
    // times it stays below the largest fp16
    static constexpr float kLift = 7.0f;
    static __device__ __forceinline__ v4f mfma(V a, V b, v4f c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ void split(float x, float y, int &hi, int &lo) {
        const v2h h = __builtin_bit_cast(v2h, __builtin_amdgcn_cvt_pkrtz(x, y));
        hi = __builtin_bit_cast(int, h);
        lo = __builtin_bit_cast(int, __builtin_amdgcn_cvt_pkrtz(x - (float)h[0], y - (float)h[1]));
    }
};
struct BF16 {
    typedef __bf16 T;
    typedef v8bf V;
    static constexpr float kLift = 0.0f;
    static __device__ __forceinline__ v4f mfma(V a, V b, v4f c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    // cut, not rounded: the rest is exact in fp32 and the second term rounds it
    static __device__ __forceinline__ void split(float x, float y, int &hi, int &lo) {
        const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
        hi = (int)__builtin_amdgcn_perm(b, a, 0x07060302u);
        const v2bf l = {(__bf16)(x - __uint_as_float(a & 0xFFFF0000u)), (__bf16)(y - __uint_as_float(b & 0xFFFF0000u))};
        lo = __builtin_bit_cast(int, l);
    }
};

// The arguments as they lie in memory.  A kernel asks for them again where a part
// of it begins: kept from its start they would fill the scalar registers, and
// what does not fit is parked in vector registers and fetched back in the loop.
typedef const __attribute__((address_space(4))) TreeParams Params;
__device__ __forceinline__ Params &params() {
    int zero = 0;
    asm volatile("" : "+s"(zero));
    return ((Params *)__builtin_amdgcn_kernarg_segment_ptr())[__builtin_amdgcn_readfirstlane(zero)];
}

// max / sum over the four lanes that hold one row (lanes c, c+16, c+32, c+48)
__device__ __forceinline__ float row_max(float x) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float row_sum(float x) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// What every lane holds, as a scalar.
__device__ __forceinline__ int64_t uniform(int64_t x) {
    return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(x >> 32)) << 32 |
                     (uint32_t)__builtin_amdgcn_readfirstlane((int)x));
}
// a / b of non-negative numbers: a 32-bit division where both fit, as nearly always.
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// 16 bytes per lane from global memory to LDS at byte dst + 16 lane.  Written as
// assembly because with the builtin the compiler waits for every copy in flight
// before each transposing read, of whichever buffer; the kernel itself waits
// (vmcnt) and synchronises before it reads a buffer.  The block has no register
// outputs.
__device__ __forceinline__ void copy_to_lds(const void *src, int dst) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "s"(dst) : "m0", "memory");
}
__device__ __forceinline__ int lds_byte(const void *p) {
    return (int)(uintptr_t)(__attribute__((address_space(3))) const char *)p;
}

// Wavefronts of a workgroup, keys of a step and rows of a tile.
template <int DK, int MT>
struct Cut {
    static constexpr int WAVES = 4, KB = tree_keys(DK), ROWT = 16 * WAVES * MT;
};

// A request as the kernels see it: lengths clipped to what there is.
struct Request {
    int first, n, ctx, len;  // first row of Q, drafted tokens, context, keys
    int nb, units, tiles;    // key blocks; what an item counts; row tiles of a cache head
};

template <int KB, int ROWT>
__device__ __forceinline__ Request request(Params &p, int r) {
    Request q;
    const int a = min(max(p.cu_new[r], 0), p.T), b = min(max(p.cu_new[r + 1], 0), p.T);
    q.first = a;
    q.n = max(b - a, 0);
    q.ctx = max(p.ctx_lens[r], 0);
    const int64_t cap = (int64_t)p.width * p.page, end = (int64_t)q.ctx + q.n;
    q.len = (int)(end < cap ? end : cap);
    q.nb = q.len > 0 ? (int)(((uint32_t)q.len + KB - 1) / KB) : 1;
    q.units = q.nb + kTreeItem;
    q.tiles = (int)(((uint32_t)(q.n * p.G) + ROWT - 1) / ROWT);
    return q;
}
__device__ __forceinline__ Request uniform(Request q) {
    return {__builtin_amdgcn_readfirstlane(q.first), __builtin_amdgcn_readfirstlane(q.n), __builtin_amdgcn_readfirstlane(q.ctx),
            __builtin_amdgcn_readfirstlane(q.len), __builtin_amdgcn_readfirstlane(q.nb), __builtin_amdgcn_readfirstlane(q.units),
            __builtin_amdgcn_readfirstlane(q.tiles)};
}

// Rows of one tile: of request q and cache head hk, rows row0 .. row0+nrows-1
// in (drafted token, query head of the group) order.
struct Tile {
    int hk, row0, nrows;
};

// Row i of a request and cache head, in (drafted token, query head of the group)
// order: its token (row of Q) and its query head.
struct Row {
    int t, h;
};
__device__ __forceinline__ Row row_of(Params &p, const Request &q, int hk, int i) {
    const uint32_t k = (uint32_t)i / (uint32_t)p.G;
    return {q.first + (int)k, hk * p.G + (int)((uint32_t)i - k * p.G)};
}

// The plain form of a row, for sums that are not finite: a wavefront, with a
// key per lane for the scores and up to four head elements per lane for the sum.
// s_q: 256 floats of LDS of the wavefront's own.
template <class X, bool S8>
__device__ void plain_row(Params &p, const Request &q, int r, int hk, Row z, float *s_q) {
    typedef typename X::T T;
    const int lane = threadIdx.x & 63;
    const T *src = (const T *)p.Q + z.t * p.q_tok + z.h * p.q_head;
    __builtin_amdgcn_wave_barrier();
    for (int d = lane; d < p.D; d += 64) s_q[d] = (float)src[d];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const float scale = p.q_flip ? -p.scale : p.scale;
    float m = -INFINITY, l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int j0 = 0; j0 < q.len; j0 += 64) {
        const int j = j0 + lane;
        bool sees = j < q.len;
        int page = -1;
        if (sees) {
            page = p.table[(int64_t)r * p.ld_table + j / p.page];
            sees = page >= 0 && page < p.num_pages;
        }
        if (sees && j >= q.ctx) {
            const int k = j - q.ctx;
            sees = p.mask ? k < p.mask_cols && p.mask[z.t * p.ld_mask + k] != 0 : k <= z.t - q.first;
        }
        const int64_t at = sees ? page * p.page_stride + (j % p.page) * p.token_stride + hk * p.head_stride : 0;
        const int64_t sat = S8 && sees ? page * p.sp_stride + (j % p.page) * p.st_stride + hk * p.sh_stride : 0;
        float s = 0.0f, vs = 1.0f;
        if (sees)
            for (int d = 0; d < p.D; ++d)
                s = fmaf(s_q[d], S8 ? (float)((const int8_t *)p.k)[at + d] : (float)((const T *)p.k)[at + d], s);
        if (S8 && sees) {
            s *= p.k_scale[sat];
            vs = p.v_scale[sat];
        }
        s = sees ? s * scale : -INFINITY;
        float top = s;
        for (int x = 32; x > 0; x /= 2) top = fmaxf(top, __shfl_xor(top, x));
        const float mn = fmaxf(m, top), base = mn == -INFINITY ? 0.0f : mn;
        const float pj = sees ? exp2f(s - base) : 0.0f, alpha = exp2f(m - base);
        m = mn;
        float sum = pj;
        for (int x = 32; x > 0; x /= 2) sum += __shfl_xor(sum, x);
        l = l * alpha + sum;
        for (int e = 0; e < 4; ++e) o[e] *= alpha;
        const uint64_t seen = __ballot(sees);
        for (int k = 0; k < 64; ++k) {
            if (!((seen >> k) & 1)) continue;
            const float wk = __shfl(pj, k), sk = __shfl(vs, k);
            const int64_t vr = ((int64_t)__shfl((int)(at >> 32), k) << 32) | (uint32_t)__shfl((int)at, k);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int d = lane + 64 * e;
                if (d < p.D)
                    o[e] = fmaf(wk, S8 ? (float)((const int8_t *)p.v)[vr + d] * sk : (float)((const T *)p.v)[vr + d], o[e]);
            }
        }
    }
    T *out = (T *)p.O + z.t * p.o_tok + z.h * p.o_head;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (lane + 64 * e < p.D) out[lane + 64 * e] = (T)(l == 0.0f ? 0.0f : o[e] / l);
}

// In LDS a key's row is LCH 16-byte chunks, chunk ch at ch ^ swizzle(row): the
// matrix operand reads of K (16 rows, one chunk each) and the transposing reads
// of V (8 rows, two chunks each, per half wavefront) then touch every bank
// evenly.
template <int LCH>
__device__ __forceinline__ int swizzle(int row) {
    return LCH == 8 ? (row >> 1 & 3) << 1 | (row >> 3 & 1) : (row & 7) << 1 | (row >> 3 & 1);
}

// A step works on KB keys in one of two LDS buffers, while the other is being
// filled for the next step: 16-bit rows go straight to LDS, int8 rows through
// registers, where they become bf16 (exactly).  Page entries are read a step
// earlier still.  RW of the wavefronts split the tile's rows (MT 16-row tiles
// each) and KW its keys; the KW parts are joined at the end, lane by lane.
//
// Two workgroups of four wavefronts to a CU: 64 KB of rows are always on their
// way.  64 tokens of one request over 131000 keys (bf16, 537 MB): 127 to 135 us (in
// an earlier build the loads alone took 111, the arithmetic alone 101); eight
// wavefronts of one tile each took 135 to 152 us, 128 keys a step with one
// workgroup to a CU 149.  32 requests of 32 tokens over up to 32768 int8 keys
// (1.41 GB): 451 to 467 us a call with the join; the arithmetic alone took 293
// before.  Forms that do not fit 256 registers: heads of more than 128 (8 spilled,
// int8 46) and int8 with two tiles (12).
template <class X, bool S8, int DK, int MT>
__global__ __launch_bounds__(256, 2) void k_tree(TreeParams) {
    typedef typename X::T T;
    typedef typename X::V V;
    typedef Cut<DK, MT> C;
    constexpr int WAVES = C::WAVES, NT = 64 * WAVES, KB = C::KB, ROWT = C::ROWT, SB = KB / 32;
    constexpr int LCH = DK == 96 ? 16 : DK / 8, LS = LCH * 8;  // an LDS row: chunks, elements
    constexpr int NP = KB * LCH / NT, NK = DK / 32, ND = DK / 16;
    constexpr int kSums = MT * ND * 1024;  // a wavefront's sums, in bytes
    __shared__ __align__(256) char s_mem0[4 * KB * LS], s_mem1[4 * KB * LS];
    __shared__ int64_t s_off[4][KB], s_soff[S8 ? 4 : 1][S8 ? KB : 1];
    __shared__ float s_ks[S8 ? 2 : 1][S8 ? KB : 1], s_vs[S8 ? 2 : 1][S8 ? KB : 1], s_m[WAVES][MT][16], s_l[WAVES][MT][16];
    __shared__ int64_t s_part[WAVES], s_base;
    __shared__ int s_r, s_bad;
    __shared__ Request s_req;
    __shared__ uint64_t s_bits[ROWT];  // the keys of a block that a token sees
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, g = lane >> 4;

    Params &p0 = params();
    // ---- this workgroup's run of key blocks
    int64_t u, u1, each, more;  // all units: `each` a workgroup, one more in the first `more`
    int64_t base_u = 0;         // where the units of request r, now, begin
    int r = 0;
    Request now;
    {
        const int per = (p0.R + NT - 1) / NT, r0 = min(tid * per, p0.R), r1 = min(r0 + per, p0.R);
        int64_t mine = 0, before = 0, U = 0, x = 0;
        Request q;
        const bool alone = p0.R == 1;  // every thread has the one request: nothing to add up or to look for
        for (int r = alone ? 0 : r0; r < (alone ? 1 : r1); ++r) {
            q = request<KB, ROWT>(p0, r);
            mine += (int64_t)q.tiles * q.units * p0.Hkv;
        }
        if (alone) {
            U = mine;
        } else {
            x = mine;
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const int64_t y = __shfl_up(x, d);
                if (lane >= d) x += y;
            }
            if (lane == 63) s_part[wave] = x;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < WAVES; ++i) {
                if (i < wave) before += s_part[i];
                U += s_part[i];
            }
        }
        U = uniform(U);
        if (tid == 0) {
            p0.hdr[blockIdx.x].rows = 0;
            p0.hdr[blockIdx.x].bad = 0;
            s_bad = 0;
        }
        if (blockIdx.x >= U) return;
        each = divide(U, gridDim.x);
        more = U - each * gridDim.x;
        u = blockIdx.x * each + (blockIdx.x < more ? blockIdx.x : more);
        u1 = u + each + (blockIdx.x < more);
        if (alone) {
            now = q;
        } else {
            int64_t at = before + x - mine;
            if (u >= at && u < at + mine) {
                for (int k = r0; k < r1; ++k) {
                    if (per > 1) q = request<KB, ROWT>(p0, k);
                    const int64_t units = (int64_t)q.tiles * q.units * p0.Hkv;
                    if (u < at + units) {
                        s_r = k;
                        s_base = at;
                        s_req = q;
                        break;
                    }
                    at += units;
                }
            }
            __syncthreads();
            r = s_r;
            base_u = s_base;
            now = s_req;
        }
        r = __builtin_amdgcn_readfirstlane(r);
        base_u = uniform(base_u);
    }
    if (tid == 0) {
        p0.hdr[blockIdx.x].r = r;
        p0.hdr[blockIdx.x].base = base_u;
        p0.hdr[blockIdx.x].u = u;
        p0.hdr[blockIdx.x].u1 = u1;
    }

    while (u < u1) {
        Params &p = params();
        const Request q = uniform(now);
        const int64_t per_head = (int64_t)q.tiles * q.units;
        if (u >= base_u + per_head * p.Hkv) {
            base_u += per_head * p.Hkv;
            now = request<KB, ROWT>(p, ++r);
            continue;
        }
        Tile w;
        w.hk = __builtin_amdgcn_readfirstlane((int)divide(u - base_u, per_head));
        const int64_t rest = u - base_u - w.hk * per_head;
        const int tile = __builtin_amdgcn_readfirstlane((int)divide(rest, q.units));
        const int from = __builtin_amdgcn_readfirstlane((int)(rest - (int64_t)tile * q.units));
        const int to = __builtin_amdgcn_readfirstlane((int)(u1 - u < q.units - from ? from + (u1 - u) : q.units));
        const int b0 = max(from - kTreeItem, 0), b1 = max(to - kTreeItem, 0);  // an item's first units are not blocks
        if (b1 == 0) {
            u += to - from;
            continue;
        }
        const bool first_part = b0 == 0, last_part = b1 == q.nb;
        w.row0 = tile * ROWT;
        w.nrows = min(q.n * p.G - w.row0, ROWT);
        const int tiles16 = (w.nrows + 15) / 16;
        const int RW = tiles16 <= WAVES / 2 * MT && SB > 1 ? WAVES / 2 : WAVES, KW = WAVES / RW;
        const int rg = wave & (RW - 1), kg = wave / RW;

        Params &pq = params();
        const int tok0 = row_of(pq, q, w.hk, w.row0).t, ntok = row_of(pq, q, w.hk, w.row0 + w.nrows - 1).t - tok0 + 1;

        // what the steps use, kept
        const int page_size = p.page, num_pages = p.num_pages, D = p.D;
        const int64_t page_stride = p.page_stride, token_stride = p.token_stride, head_at = w.hk * p.head_stride;
        const int64_t sp_stride = S8 ? p.sp_stride : 0, st_stride = S8 ? p.st_stride : 0, shead_at = S8 ? w.hk * p.sh_stride : 0;
        const void *const k_cache = p.k, *const v_cache = p.v;
        const float *const k_scale = S8 ? p.k_scale : nullptr, *const v_scale = S8 ? p.v_scale : nullptr;
        const float p_scale = p.scale;

        // ---- page entries: of this block and the next ones
        const int32_t *table = p.table + (int64_t)r * p.ld_table;
        const auto page_of = [&](int b) {  // of key tid of block b; -1: none
            const uint32_t j = (uint32_t)b * KB + tid;  // a block's first key is below 2^31
            return b < b1 && tid < KB && j < (uint32_t)q.len ? table[j / (uint32_t)page_size] : -1;
        };
        const auto put_off = [&](int b, int page) {
            if (tid < KB) {
                const bool ok = page >= 0 && page < num_pages;
                const int i = (int)(((uint32_t)b * KB + tid) % (uint32_t)page_size), ring = (b - b0) & 3;
                s_off[ring][tid] = ok ? page * page_stride + i * token_stride + head_at : -1;
                if (S8) s_soff[ring][tid] = ok ? page * sp_stride + i * st_stride + shead_at : -1;
            }
        };
        const int page0 = page_of(b0), page1 = page_of(b0 + 1), page2 = S8 ? page_of(b0 + 2) : -1;

        // ---- queries: column c of a 16-row tile, elements 32 kk + 8 g ..
        V qv[MT][NK];
        int self[MT];  // place of the column's token among the tile's
        v4f o[MT][ND];
        float base[MT], thr[MT], l[MT];
        const v4f zero = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int row = 16 * (rg + mt * RW) + c;
            const Row z = row_of(pq, q, w.hk, w.row0 + (row < w.nrows ? row : 0));
            self[mt] = z.t - tok0;
            const T *src = (const T *)pq.Q + z.t * pq.q_tok + z.h * pq.q_head;
#pragma unroll
            for (int kk = 0; kk < NK; ++kk) {
                const int d = 32 * kk + 8 * g;
                v4i v = {0, 0, 0, 0};
                if (row < w.nrows && d < pq.D) {
                    if (pq.q_vec) {
                        v = *(const v4i *)(src + d);
                    } else {
                        T e[8];
#pragma unroll
                        for (int x = 0; x < 8; ++x) e[x] = src[d + x];
                        v = *(v4i *)e;
                    }
                }
#pragma unroll
                for (int x = 0; x < 4; ++x) v[x] ^= pq.q_flip;
                qv[mt][kk] = __builtin_bit_cast(V, v);
            }
#pragma unroll
            for (int dt = 0; dt < ND; ++dt) o[mt][dt] = zero;
            base[mt] = 0.0f;
            thr[mt] = -INFINITY;  // the maximum plus its slack; -inf: none yet
            l[mt] = 0.0f;
        }

        // ---- staging
        // Thread tid's chunks: rows tid / LCH + i * NT / LCH, i < NP, at its own place
        // of the row.  The swizzle repeats every 16 rows; 8 rows on it flips bit 0.
        const int srow = tid / LCH, sd0 = 8 * ((tid % LCH) ^ swizzle<LCH>(srow));
        const auto head_element = [&](int i) { return LCH == 32 ? sd0 ^ (8 * (i & 1)) : sd0; };
        const auto copy = [&](char *buf, int b) {  // 16-bit rows of block b
            const int ring = (b - b0) & 3, to = lds_byte(buf) + 1024 * wave;
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int sd = head_element(i);
                const int64_t off = s_off[ring][srow + i * (NT / LCH)], at = (off < 0 ? 0 : off) + sd;
                if (sd < D) {
                    copy_to_lds((const T *)k_cache + at, to + 16 * NT * i);
                    copy_to_lds((const T *)v_cache + at, to + 16 * NT * i + KB * LS * 2);
                }
            }
        };
        v2i kr[S8 ? NP : 1], vr[S8 ? NP : 1];
        float sc = 0.0f;
        const auto load = [&](int b) {  // int8 rows of block b and their scales
            const int ring = (b - b0) & 3;
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int sd = head_element(i);
                const int64_t off = s_off[ring][srow + i * (NT / LCH)], at = sd < D && off >= 0 ? off + sd : 0;
                kr[i] = *(const v2i *)((const int8_t *)k_cache + at);
                vr[i] = *(const v2i *)((const int8_t *)v_cache + at);
            }
            if (tid < 2 * KB) {
                const int64_t so = s_soff[ring][tid & (KB - 1)];
                sc = so >= 0 ? (tid < KB ? k_scale : v_scale)[so] : 0.0f;
            }
        };
        const auto widen = [](v2i x) {  // eight int8 codes as bf16
            v4i y;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int w2 = x[e / 2] >> (16 * (e & 1));
                y[e] = (int)__builtin_amdgcn_perm(__float_as_uint((float)(int8_t)(w2 >> 8)), __float_as_uint((float)(int8_t)w2),
                                                  0x07060302u);
            }
            return y;
        };
        const auto store = [&](char *buf, int which) {
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                if (head_element(i) < D) {
                    *(v4i *)(buf + (NT * i + tid) * 16) = widen(kr[i]);
                    *(v4i *)(buf + KB * LS * 2 + (NT * i + tid) * 16) = widen(vr[i]);
                }
            }
            if (tid < KB) s_ks[which][tid] = sc * p_scale;
            else if (tid < 2 * KB) s_vs[which][tid - KB] = sc;
        };

        // ---- one 32-key step; clean: every row sees all its keys (else s_bits tells)
        const int kx = swizzle<LCH>(c), vrow = 4 * g + (c >> 2), vx = swizzle<LCH>(vrow);
        const float scale = S8 ? 1.0f : p_scale;  // an int8 cache's key scales carry it
        const auto step = [&](char *buf, int which, int k0, bool clean) __attribute__((always_inline)) {
            const T *const sK = (const T *)buf + k0 * LS;
            T *const sV = (T *)buf + (KB + k0) * LS;
            v4f s[MT][2];
#pragma unroll
            for (int kt = 0; kt < 2; ++kt) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) s[mt][kt] = zero;
            }
            // all of K's operands are asked for before the first is used, and V's
            // before the softmax: left to itself the compiler waits for each
            V ka[NK][2];
#pragma unroll
            for (int kk = 0; kk < NK; ++kk)
#pragma unroll
                for (int kt = 0; kt < 2; ++kt) ka[kk][kt] = *(const V *)(sK + (16 * kt + c) * LS + 8 * ((4 * kk + g) ^ kx));
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int kk = 0; kk < NK; ++kk)
#pragma unroll
                for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) s[mt][kt] = X::mfma(ka[kk][kt], qv[mt][kk], s[mt][kt]);
            typedef __attribute__((address_space(3))) v4s *LdsV;
            V va[ND];
#pragma unroll
            for (int dt = 0; dt < ND; ++dt) {
                // keys 4g .. 4g+3 and 16+4g .. of head element 16 dt + c
                T *at = sV + vrow * LS + 8 * ((2 * dt + (c >> 1 & 1)) ^ vx) + 4 * (c & 1);
                const v4s a0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsV)at);
                const v4s a1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsV)(at + 16 * LS));
                va[dt] = __builtin_bit_cast(V, __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7));
            }
            v4f vs[2];
            if (S8) {
#pragma unroll
                for (int kt = 0; kt < 2; ++kt) {
                    const v4f ks = *(const v4f *)(s_ks[which] + k0 + 16 * kt + 4 * g);
                    vs[kt] = *(const v4f *)(s_vs[which] + k0 + 16 * kt + 4 * g);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int v = 0; v < 4; ++v) s[mt][kt][v] *= ks[v];
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            // hidden keys end as exp2(-inf); x c1 - base in one step below
            if (!clean) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const uint32_t bits = (uint32_t)(s_bits[self[mt]] >> k0) >> (4 * g);
#pragma unroll
                    for (int e = 0; e < 8; ++e) s[mt][e / 4][e % 4] = bits >> (16 * (e / 4) + e % 4) & 1 ? s[mt][e / 4][e % 4] * scale : -INFINITY;
                }
            }
            const float c1 = clean ? scale : 1.0f;
            // The sums move to a new maximum only when a score passes the old one by
            // 2^8: weights up to 2^8 cost fp32 sums nothing.
            float top[MT];
            bool above = false;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const v4f a = s[mt][0], b = s[mt][1];
                top[mt] = fmaxf(fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3])), fmaxf(fmaxf(b[0], b[1]), fmaxf(b[2], b[3]))) * c1;
                above |= top[mt] > thr[mt];
            }
            if (__any(above)) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const float m0 = thr[mt] - 8.0f, m1 = fmaxf(m0, row_max(top[mt]));
                    const float nb = m1 == -INFINITY ? 0.0f : m1 - X::kLift;
                    const float alpha = thr[mt] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(base[mt] - nb);
                    base[mt] = nb;
                    thr[mt] = m1 + 8.0f;
                    l[mt] *= alpha;
#pragma unroll
                    for (int dt = 0; dt < ND; ++dt)
#pragma unroll
                        for (int v = 0; v < 4; ++v) o[mt][dt][v] *= alpha;
                }
            }
            V hi[MT], lo[MT];
            const auto weights = [&](int mt) {
                v4i h4, l4;
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    float a = __builtin_amdgcn_exp2f(fmaf(s[mt][e / 4][e % 4], c1, -base[mt]));
                    float b = __builtin_amdgcn_exp2f(fmaf(s[mt][e / 4][e % 4 + 1], c1, -base[mt]));
                    l[mt] += a;
                    l[mt] += b;
                    if (S8) {
                        a *= vs[e / 4][e % 4];
                        b *= vs[e / 4][e % 4 + 1];
                    }
                    int hh, ll;
                    X::split(a, b, hh, ll);
                    h4[e / 2] = hh;
                    l4[e / 2] = ll;
                }
                hi[mt] = __builtin_bit_cast(V, h4);
                lo[mt] = __builtin_bit_cast(V, l4);
            };
            const auto weigh = [&](int mt) {
#pragma unroll
                for (int dt = 0; dt < ND; ++dt) o[mt][dt] = X::mfma(va[dt], hi[mt], o[mt][dt]);
#pragma unroll
                for (int dt = 0; dt < ND; ++dt) o[mt][dt] = X::mfma(va[dt], lo[mt], o[mt][dt]);
            };
            weights(0);
            if (MT == 2) {  // the second tile's weights between the first one's products
                __builtin_amdgcn_sched_barrier(0);
                weights(MT - 1);
                weigh(0);
#pragma unroll
                for (int i = 0; i < 2 * ND; ++i) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x402, 4, 0);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            weigh(MT - 1);
        };

        // ---- block b, in buffer WHICH
        constexpr int AHEAD = S8 ? 2 : 1;  // blocks whose rows are on their way
        const auto block = [&](auto WHICH, int b) __attribute__((always_inline)) {
            constexpr int which = decltype(WHICH)::value;
            char *const cur = which ? s_mem1 : s_mem0, *const other = which ? s_mem0 : s_mem1;
            __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): the copies of this block
            __syncthreads();                     // and everyone is done with the other buffer
            const int page = page_of(b + AHEAD + 1);
            if constexpr (S8) {
                if (b + 1 < b1) store(other, 1 - which);
                if (b + 2 < b1) load(b + 2);
            } else if (b + 1 < b1) {
                copy(other, b + 1);
            }
            const int64_t *const off = s_off[(b - b0) & 3];
            const uint64_t vis = __ballot(off[lane & (KB - 1)] >= 0);  // the keys there are
            const bool clean = vis == ~0ull && (int64_t)(b + 1) * KB <= q.ctx;
            if (!clean) {
                Params &p = params();
                int first = tok0, me = tid;  // nothing of this is worth keeping over the steps in between
                asm volatile("" : "+s"(first), "+v"(me));
                if (!S8)  // what stands for missing keys must not be NaN
                    for (int x = me; x < KB * LCH; x += NT)
                        if (off[x / LCH] < 0) *(v4i *)(cur + KB * LS * 2 + x * 16) = v4i{0, 0, 0, 0};
                const int k = b * KB + (me & 63) - q.ctx;  // of the drafted token that lane's key is
                const bool in = k >= 0 && k < p.mask_cols;
                for (int i0 = me >> 6; i0 < ntok; i0 += 8 * WAVES) {
                    int m[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int i = min(i0 + WAVES * e, ntok - 1);
                        m[e] = k < 0 || (!p.mask && k <= first - q.first + i);
                        if (p.mask && in) m[e] = p.mask[(first + i) * p.ld_mask + k];
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint64_t bits = __ballot(m[e] != 0) & vis;
                        if ((me & 63) == 0 && i0 + WAVES * e < ntok) s_bits[i0 + WAVES * e] = bits;
                    }
                }
                __syncthreads();
            }
            if (rg < tiles16)
                for (int sb = kg; sb < SB; sb += KW) step(cur, which, 32 * sb, clean);
            put_off(b + AHEAD + 1, page);
        };

        __syncthreads();  // the last item's sums and offsets have been read
        if (D < DK)  // K's chunks past the head: the queries' are zero there
            for (int x = tid; x < KB * LCH; x += NT) {
                const int row = x / LCH;
                if (8 * ((x % LCH) ^ swizzle<LCH>(row)) >= D) *(v4i *)(s_mem0 + x * 16) = *(v4i *)(s_mem1 + x * 16) = v4i{0, 0, 0, 0};
            }
        put_off(b0, page0);
        put_off(b0 + 1, page1);
        if (S8) put_off(b0 + 2, page2);
        __syncthreads();
        if constexpr (S8) {
            load(b0);
            store(s_mem0, 0);
            if (b0 + 1 < b1) load(b0 + 1);
        } else {
            copy(s_mem0, b0);
        }
        for (int b = b0; b < b1; b += 2) {
            block(std::integral_constant<int, 0>(), b);
            if (b + 1 < b1) block(std::integral_constant<int, 1>(), b + 1);
        }

        // ---- join the KW parts: the others leave their sums in LDS for the first
        Params &pe = params();
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) l[mt] = row_sum(l[mt]);
        v4f *const sums = (v4f *)(s_mem0 + rg * kSums) + lane;
        if (KW > 1) {
            __syncthreads();
            if (kg > 0 && rg < tiles16) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    if (g == 0) {
                        s_m[wave][mt][c] = thr[mt] == -INFINITY ? -INFINITY : base[mt];
                        s_l[wave][mt][c] = l[mt];
                    }
#pragma unroll
                    for (int dt = 0; dt < ND; ++dt) sums[64 * (mt * ND + dt)] = o[mt][dt];
                }
            }
            __syncthreads();
        }
        if (kg == 0 && rg < tiles16) {
            const bool final = first_part && last_part;
            float *const slot = pe.part + (2 * (int64_t)blockIdx.x + (first_part ? 1 : 0)) * pe.slot_rows * (DK + 2);
            bool bad = false;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                float m = thr[mt] == -INFINITY ? -INFINITY : base[mt];
                if (KW > 1) {
                    v4f part[ND];
#pragma unroll
                    for (int dt = 0; dt < ND; ++dt) part[dt] = sums[64 * (mt * ND + dt)];
                    const float m2 = s_m[RW + rg][mt][c], l2 = s_l[RW + rg][mt][c];
                    __builtin_amdgcn_sched_barrier(0);
                    const float top = fmaxf(m, m2), b = top == -INFINITY ? 0.0f : top;
                    const float x = __builtin_amdgcn_exp2f(m - b), y = __builtin_amdgcn_exp2f(m2 - b);
                    l[mt] = x * l[mt] + y * l2;
                    m = top;
#pragma unroll
                    for (int dt = 0; dt < ND; ++dt)
#pragma unroll
                        for (int v = 0; v < 4; ++v) o[mt][dt][v] = x * o[mt][dt][v] + y * part[dt][v];
                }
                const int row = 16 * (rg + mt * RW) + c;
                if (row >= w.nrows) continue;
                bad |= !(l[mt] < INFINITY);
#pragma unroll
                for (int dt = 0; dt < ND; ++dt)
                    if (16 * dt + 4 * g < pe.D)
#pragma unroll
                        for (int v = 0; v < 4; ++v) bad |= !(fabsf(o[mt][dt][v]) < INFINITY);
                if (final) {
                    const Row z = row_of(pe, q, w.hk, w.row0 + row);
                    T *const out = (T *)pe.O + z.t * pe.o_tok + z.h * pe.o_head + 4 * g;
                    const float inv = l[mt] == 0.0f ? 0.0f : 1.0f / l[mt];
#pragma unroll
                    for (int dt = 0; dt < ND; ++dt) {
                        if (16 * dt + 4 * g >= pe.D) continue;
                        T e[4];
#pragma unroll
                        for (int v = 0; v < 4; ++v) e[v] = (T)(o[mt][dt][v] * inv);
                        if (pe.o_vec) {
                            *(v2i *)(out + 16 * dt) = *(v2i *)e;
                        } else {
#pragma unroll
                            for (int v = 0; v < 4; ++v) out[16 * dt + v] = e[v];
                        }
                    }
                } else {
                    if (g == 0) {
                        slot[row] = m;
                        slot[pe.slot_rows + row] = l[mt];
                    }
                    float *const to = slot + 2 * pe.slot_rows + row * DK + 4 * g;
#pragma unroll
                    for (int dt = 0; dt < ND; ++dt) *(v4f *)(to + 16 * dt) = o[mt][dt];
                }
            }
            if (bad) s_bad = 1;
        }
        if (!first_part && last_part && tid == 0) {  // the last of an item's parts: what the join needs
            const int64_t a = u - from + kTreeItem, large = more * (each + 1);  // the item's first block
            TreeHeader &h = pe.hdr[blockIdx.x];
            h.rows = w.nrows;
            h.first_wg = (int)(a < large ? divide(a, each + 1) : more + divide(a - large, each));
            h.hk = w.hk;
            h.row0 = w.row0;
            h.first = q.first;
        }
        u += to - from;
    }
    __syncthreads();
    if (tid == 0 && s_bad) params().hdr[blockIdx.x].bad = 1;
}

// One row's sums over parts k, k + step, ... of n, BATCH of them in flight:
// d .. d+3 of the head.  first: its first part's slot; its other parts are every
// second slot from the next one on.
template <int BATCH, int DK>
__device__ __forceinline__ void join_parts(Params &p, const float *first, int row, int d, int k, int step, int n,
                                           float &m, float &l, v4f &acc) {
    const int64_t stride = (int64_t)p.slot_rows * (DK + 2);
    for (int i0 = k; i0 < n; i0 += BATCH * step) {
        float pm[BATCH], pl[BATCH];
        v4f po[BATCH];
#pragma unroll
        for (int e = 0; e < BATCH; ++e) {
            const int i = min(i0 + e * step, n - 1);
            const float *s = first + (2 * i + (i == 0)) * stride;
            pm[e] = s[row];
            pl[e] = s[p.slot_rows + row];
            po[e] = *(const v4f *)(s + 2 * p.slot_rows + (int64_t)row * DK + d);
        }
        float top = m;
#pragma unroll
        for (int e = 0; e < BATCH; ++e) top = fmaxf(top, pm[e]);
        const float base = top == -INFINITY ? 0.0f : top, alpha = __builtin_amdgcn_exp2f(m - base);
        l *= alpha;
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[v] *= alpha;
#pragma unroll
        for (int e = 0; e < BATCH; ++e) {
            const float a = i0 + e * step < n ? __builtin_amdgcn_exp2f(pm[e] - base) : 0.0f;
            l += a * pl[e];
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[v] += a * po[e][v];
        }
        m = top;
    }
}

// What the join needs of a header, kept in LDS.
struct Shared {
    int rows, first_wg, hk, row0, first;
};

// Joins the parts of the items that several workgroups shared.  The rows of all
// items stand in one line, found from the headers.  DK/4 lanes hold a row; a
// wavefront takes SP rows, or one row of many parts whose parts its SP runs of
// lanes share.
template <class X, bool S8, int DK, int MT>
__global__ __launch_bounds__(256) void k_tree_join(TreeParams) {
    Params &p = params();
    typedef typename X::T T;
    typedef Cut<DK, MT> C;
    constexpr int Q = DK / 4, SP = 64 / Q > 0 ? 64 / Q : 1, MANY = 8;
    static_assert(kTreeWorkgroups <= 512, "two headers a thread");
    __shared__ int s_end[512], s_rows[512], s_part[4], s_any;
    __shared__ Shared s_item[512];
    __shared__ float s_q[4][256];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // steps of the line: a header's rows, or its rows / SP
    int steps[2], bad = 0, x = 0;
    if (tid == 0) s_any = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int at = 2 * tid + i;
        Shared h = {};
        if (at < p.wgs) {
            const TreeHeader *from = p.hdr + at;
            h = {from->rows, from->first_wg, from->hk, from->row0, from->first};
            bad |= from->bad;
        }
        s_item[at] = h;
        steps[i] = h.rows == 0 ? 0 : at - h.first_wg + 1 > MANY ? h.rows : (h.rows + SP - 1) / SP;
        x += steps[i];
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int y = __shfl_up(x, d);
        if (lane >= d) x += y;
    }
    if (lane == 63) s_part[wave] = x;
    __syncthreads();
    if (bad) s_any = 1;
    int total = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i < wave) x += s_part[i];
        total += s_part[i];
    }
    s_end[2 * tid] = x - steps[1];
    s_end[2 * tid + 1] = x;
    s_rows[2 * tid] = steps[0];
    s_rows[2 * tid + 1] = steps[1];
    __syncthreads();
    const int d = 4 * (lane % Q), k = lane / Q;
    for (int at = blockIdx.x * 4 + wave; at < total; at += gridDim.x * 4) {
        int lo = 0, hi = 511;  // the first header whose steps end past this one
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (s_end[mid] > at) hi = mid;
            else lo = mid + 1;
        }
        lo = __builtin_amdgcn_readfirstlane(lo);
        const Shared h = s_item[lo];
        const int step = at - (s_end[lo] - s_rows[lo]), n = lo - h.first_wg + 1;
        const float *first = p.part + 2 * (int64_t)h.first_wg * p.slot_rows * (DK + 2);
        const bool many = n > MANY;
        const int row = many ? step : step * SP + k;
        if (s_any) {
            bool again = false;
            for (int i = h.first_wg; i <= lo; ++i) again |= p.hdr[i].bad != 0;
            if (again) {
                const int r = p.hdr[lo].r;
                const Request q = uniform(request<C::KB, C::ROWT>(p, r));
                for (int i = many ? step : step * SP; i < min(many ? step + 1 : (step + 1) * SP, h.rows); ++i)
                    plain_row<X, S8>(p, q, r, h.hk, row_of(p, q, h.hk, h.row0 + i), s_q[wave]);
                continue;
            }
        }
        float m = -INFINITY, l = 0.0f;
        v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
        const bool ok = row < h.rows && k < SP;
        if (many) {
            if (ok) join_parts<16, DK>(p, first, row, d, k, SP, n, m, l, acc);
#pragma unroll
            for (int y = SP / 2; y > 0; y /= 2) {
                const int from = lane + Q * y;
                const float m2 = __shfl(m, from), l2 = __shfl(l, from), top = fmaxf(m, m2);
                const float base = top == -INFINITY ? 0.0f : top;
                const float a = __builtin_amdgcn_exp2f(m - base), b = __builtin_amdgcn_exp2f(m2 - base);
                l = a * l + b * l2;
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[v] = a * acc[v] + b * __shfl(acc[v], from);
                m = top;
            }
        } else if (ok) {
            join_parts<4, DK>(p, first, row, d, 0, 1, n, m, l, acc);
        }
        if (ok && (k == 0 || !many) && d < p.D) {
            Request q;
            q.first = h.first;
            const Row z = row_of(p, q, h.hk, h.row0 + row);
            T *out = (T *)p.O + z.t * p.o_tok + z.h * p.o_head + d;
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            T e[4];
#pragma unroll
            for (int v = 0; v < 4; ++v) e[v] = (T)(acc[v] * inv);
            if (p.o_vec) {
                *(v2i *)out = *(v2i *)e;
            } else {
#pragma unroll
                for (int v = 0; v < 4; ++v) out[v] = e[v];
            }
        }
    }
    if (!s_any) return;
    // rows of whole items of workgroups with sums that are not finite
    for (int x = 0; x < p.wgs; ++x) {
        const TreeHeader h = p.hdr[x];
        if (!h.bad) continue;
        int64_t u = uniform(h.u), base = uniform(h.base);
        int r = __builtin_amdgcn_readfirstlane(h.r);
        while (u < h.u1) {
            const Request q = uniform(request<C::KB, C::ROWT>(p, r));
            const int64_t per_head = (int64_t)q.tiles * q.units;
            if (u >= base + per_head * p.Hkv) {
                base += per_head * p.Hkv;
                ++r;
                continue;
            }
            const int hk = (int)divide(u - base, per_head);
            const int64_t rest = u - base - hk * per_head;
            const int tile = (int)divide(rest, q.units), from = (int)(rest - (int64_t)tile * q.units);
            const int64_t end = u + q.units - from;
            if (from <= kTreeItem && end <= h.u1) {
                const int row0 = tile * C::ROWT, n = min(q.n * p.G - row0, C::ROWT);
                for (int row = blockIdx.x * 4 + wave; row < n; row += gridDim.x * 4)
                    plain_row<X, S8>(p, q, r, hk, row_of(p, q, hk, row0 + row), s_q[wave]);
            }
            u = end;
        }
    }
}
template <class X, bool S8, int DK, int MT>
hipError_t launch(const TreeParams &p, const TreeShape &z, hipStream_t s) {
    hipLaunchKernelGGL((k_tree<X, S8, DK, MT>), dim3((unsigned)z.wgs), dim3(256), 0, s, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // at most one shared item ends in a workgroup
    const int64_t wgs = ceil_div(z.wgs * z.slot_rows, 4);
    hipLaunchKernelGGL((k_tree_join<X, S8, DK, MT>), dim3((unsigned)(wgs < 1024 ? wgs : 1024)), dim3(256), 0, s, p);
    return hipGetLastError();
}

template <class X, bool S8>
hipError_t launch_dk(const TreeParams &p, const TreeShape &z, hipStream_t s) {
    if (z.dk == 256) return launch<X, S8, 256, 1>(p, z, s);
    if (z.mt == 1)
        return z.dk == 64 ? launch<X, S8, 64, 1>(p, z, s) : z.dk == 96 ? launch<X, S8, 96, 1>(p, z, s) : launch<X, S8, 128, 1>(p, z, s);
    return z.dk == 64 ? launch<X, S8, 64, 2>(p, z, s) : z.dk == 96 ? launch<X, S8, 96, 2>(p, z, s) : launch<X, S8, 128, 2>(p, z, s);
}

}  // namespace

hipError_t launch_tree_attention(const TreeParams &p, const TreeShape &z, qmm_dtype ct, hipStream_t s,
                                 const char **variant) {
    *variant = z.mt == 2 ? "tree_rows128" : "tree_rows64";
    return ct == QMM_T_F16 ? launch_dk<F16, false>(p, z, s) : ct == QMM_T_BF16 ? launch_dk<BF16, false>(p, z, s)
                                                                               : launch_dk<BF16, true>(p, z, s);
}

}  // namespace qmm
