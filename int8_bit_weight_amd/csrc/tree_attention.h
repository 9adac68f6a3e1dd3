// tree_attention.h -- attention of new tokens over a paged cache on gfx950: of
// drafted tokens by a mask (k_tree_attention.hip) or behind a window
// (k_window_attention.hip).
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
//
// A 4-bit row's codes q enter both products as 16 + q, which a shift, a mask and an or
// make of a pair of them: with the row's step d and minimum m
//   s_j = d_j sum (16 + q) x + (m_j - 16 d_j) sum x,
//   o   = sum_j (w_j d_j) (16 + q_j) + sum_j w_j (m_j - 16 d_j)
// so the sum of a query's elements and one more weighted sum are all it adds.
//
// Behind a window a tile of rows reads the blocks of the first keys that stay visible
// and those from its first token's window to its last token.  Tiles then cost
// different numbers of blocks, so the line is measured in keys, by a formula whose
// sum over tiles is closed, and a workgroup's share of an item is that part of its blocks.
#pragma once

#include <type_traits>

#include "serve_internal.h"

namespace qmm {

namespace {

// How a cache's rows are held: 16-bit elements, int8 codes with a scale, 4-bit codes
// with a step and a minimum.
enum Held { kWide, kS8, kQ4 };

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

// Wavefronts of a workgroup, keys of a step and rows of a tile; WIN: behind a window.
template <int DK, int MT, bool WINDOW>
struct Cut {
    static constexpr int WAVES = 4, KB = tree_keys(DK), ROWT = 16 * WAVES * MT, ITEM = kTreeItem;
    static constexpr bool WIN = WINDOW, NEAR = WINDOW;
    static constexpr int HEADS = 1;  // cache heads of a workgroup
};
// Groups of cache heads that items are made for.
template <class C>
__device__ __forceinline__ int head_groups(Params &p) {
    return C::HEADS == 1 ? p.Hkv : (int)((uint32_t)p.Hkv / C::HEADS);
}

// A request as the kernels see it: lengths clipped to what there is.
struct Request {
    int first, n, ctx, len;  // first row of Q, drafted tokens, context, keys
    int nb, units, tiles;    // key blocks; what an item counts; row tiles of a cache head
};

template <class C>
__device__ __forceinline__ Request request(Params &p, int r) {
    constexpr int KB = C::KB, ROWT = C::ROWT;
    Request q;
    const int a = min(max(p.cu_new[r], 0), p.T), b = min(max(p.cu_new[r + 1], 0), p.T);
    q.first = a;
    q.n = max(b - a, 0);
    q.ctx = max(p.ctx_lens[r], 0);
    const int64_t cap = (int64_t)p.width * p.page, end = (int64_t)q.ctx + q.n;
    q.len = (int)(end < cap ? end : cap);
    q.nb = q.len > 0 ? (int)(((uint32_t)q.len + KB - 1) / KB) : 1;
    q.units = q.nb + C::ITEM;
    q.tiles = (int)(((uint32_t)(q.n * p.G) + ROWT - 1) / ROWT);
    return q;
}
__device__ __forceinline__ Request uniform(Request q) {
    return {__builtin_amdgcn_readfirstlane(q.first), __builtin_amdgcn_readfirstlane(q.n), __builtin_amdgcn_readfirstlane(q.ctx),
            __builtin_amdgcn_readfirstlane(q.len), __builtin_amdgcn_readfirstlane(q.nb), __builtin_amdgcn_readfirstlane(q.units),
            __builtin_amdgcn_readfirstlane(q.tiles)};
}

// What the tiles of a request and cache head count on the line, one after the other.
// Behind a window tile k counts its keys, as if it began at token k * step: with window
// W, from max(0, a + k * step), a = ctx + 1 - W, to ctx + (k + 1) * step, and what it
// costs beside.
template <class C>
struct Line {
    int tiles, step;
    int64_t each, units, a;  // of a tile; WIN: but for its keys; a as above
    __device__ __forceinline__ Line(Params &p, const Request &q) : tiles(q.tiles) {
        units = q.units;
        if (!C::WIN) return;
        step = max(C::ROWT / p.G, 1);
        a = (int64_t)q.ctx + 1 - p.window;
        // first keys beside the window: none where the window reaches the first key
        each = C::ITEM * C::KB + step + q.ctx + ((int64_t)q.ctx + q.n > p.window ? min(p.sinks, q.len) : 0);
    }
    __device__ __forceinline__ int64_t of(int k) const {  // tile k's units
        if (!C::WIN) return units;
        const int64_t from = a + (int64_t)k * step;
        return each + (int64_t)k * step - (from > 0 ? from : 0);
    }
    __device__ __forceinline__ int64_t before(int k) const {  // units of the tiles before tile k
        if (!C::WIN) return k * units;
        int64_t sum = k * each + (int64_t)step * ((int64_t)k * (k - 1) / 2);
        const int64_t i = a > 0 ? 0 : (uint32_t)-a / (uint32_t)step + 1, m = k - i;  // tiles i .. k-1 begin past the first key
        if (m > 0) sum -= m * a + step * ((i + k - 1) * m / 2);
        return sum;
    }
    __device__ __forceinline__ int64_t all() const { return before(tiles); }
    // the tile that holds unit x
    __device__ __forceinline__ int find(int64_t x) const {
        if (!C::WIN) return (int)divide(x, units);
        int lo = 0, hi = tiles - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (before(mid) <= x) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    }
};

// A tile's key blocks, as the kernels count them: `firsts` blocks of first keys and then
// those from block `from` on, nb in all.  Without a window all of the request's.
template <class C>
struct Blocks {
    int nb, firsts, from;
    __device__ __forceinline__ Blocks(Params &p, const Request &q, int row0, int nrows) : nb(q.nb), firsts(0), from(0) {
        if (!C::WIN) return;
        const int i0 = (uint32_t)row0 / (uint32_t)p.G, i1 = (uint32_t)(row0 + nrows - 1) / (uint32_t)p.G;
        const int64_t lo = max((int64_t)q.ctx + i0 + 1 - p.window, (int64_t)0), end = (int64_t)q.ctx + i1 + 1;
        const int64_t hi = end < q.len ? end : q.len;
        firsts = (min(p.sinks, q.len) + C::KB - 1) / C::KB;
        nb = firsts;
        if (hi > lo) {
            from = (int)(lo / C::KB);
            firsts = min(firsts, from);
            nb = firsts + (int)((hi + C::KB - 1) / C::KB) - from;
        }
        nb = max(nb, 1);
    }
    // the key block that counts as b
    __device__ __forceinline__ int key_block(int b) const { return !C::WIN || b < firsts ? b : b - firsts + from; }
    // how many of the blocks end in the tile's first x units (of `units`)
    __device__ __forceinline__ int within(int64_t x, int64_t units) const {
        return C::WIN ? (int)divide(x * nb, units) : max((int)x - C::ITEM, 0);
    }
    // the unit that the first block ends in
    __device__ __forceinline__ int64_t first_unit(int64_t units) const {
        return C::WIN ? divide(units + nb - 1, nb) - 1 : C::ITEM;
    }
};

// What the token at position pos sees behind the window; all below 2^32.
__device__ __forceinline__ bool in_window(uint32_t j, uint32_t pos, uint32_t window, uint32_t sinks) {
    return j <= pos && (j + window > pos || j < sinks);
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

// A 4-bit row's step and minimum, and one of its codes.
__device__ __forceinline__ float2 pair_of(uint32_t x) {
    return {__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u)};
}
__device__ __forceinline__ float2 pair_of(const float *scales, int64_t at) { return pair_of(((const uint32_t *)scales)[at]); }
__device__ __forceinline__ int code_of(const uint8_t *row, int d) {
    return row[(d & ~7) / 2 + 2 * (d & 1) + (d >> 2 & 1)] >> (4 * (d >> 1 & 1)) & 15;
}

// Pairs of codes as 16 + code: two instructions each, a shift and v_and_or_b32, which takes
// one constant from a scalar register and no second one: the other is kept in a vector
// register (with two literals the compiler makes three instructions).
struct Widen {
    int mask, offset;
    __device__ __forceinline__ Widen(int m, int o) : mask(m), offset(o) { asm("" : "+s"(mask), "+v"(offset)); }
    // the pair in nibble i of each half of x, in bf16 and in fp16
    __device__ __forceinline__ int bf16(uint32_t x, int i) const { return ((int)(i ? x >> (4 * i - 3) : x << 3) & mask) | offset; }
    __device__ __forceinline__ int f16(uint32_t x, int i) const {
        return ((int)(i > 1 ? x >> (4 * i - 6) : x << (6 - 4 * i)) & mask) | offset;
    }
};
constexpr int kMaskBf16 = 0x00780078, kSixteenBf16 = 0x41804180, kMaskF16 = 0x03C003C0, kSixteenF16 = 0x4C004C00;

// The plain form of a row, for sums that are not finite: a wavefront, with a
// key per lane for the scores and up to four head elements per lane for the sum.
// s_q: 256 floats of LDS of the wavefront's own.
template <class X, Held H, bool WIN>
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
    // behind a window: `firsts` first keys and then those from `from` on
    int firsts = 0, from = 0, keys = q.len;
    const uint32_t pos = (uint32_t)q.ctx + (uint32_t)(z.t - q.first);
    if (WIN) {
        const int64_t lo = max((int64_t)pos + 1 - p.window, (int64_t)0), hi = min((int64_t)pos + 1, (int64_t)q.len);
        from = (int)min(lo, (int64_t)q.len);
        firsts = min(p.sinks, from);
        keys = firsts + (int)max(hi - from, (int64_t)0);
    }
    for (int j0 = 0; j0 < keys; j0 += 64) {
        const int at_j = j0 + lane, j = WIN && at_j >= firsts ? at_j - firsts + from : at_j;
        bool sees = at_j < keys;
        int page = -1;
        if (sees) {
            page = p.table[(int64_t)r * p.ld_table + j / p.page];
            sees = page >= 0 && page < p.num_pages;
        }
        if (!WIN && sees && j >= q.ctx) {
            const int k = j - q.ctx;
            sees = p.mask ? k < p.mask_cols && p.mask[z.t * p.ld_mask + k] != 0 : k <= z.t - q.first;
        }
        const int64_t at = sees ? page * p.page_stride + (j % p.page) * p.token_stride + hk * p.head_stride : 0;
        const int64_t sat = H != kWide && sees ? page * p.sp_stride + (j % p.page) * p.st_stride + hk * p.sh_stride : 0;
        float s = 0.0f, vs = 1.0f, vm = 0.0f;
        if (sees) {
            if constexpr (H == kQ4) {
                const float2 ks = pair_of(p.k_scale, sat), v2 = pair_of(p.v_scale, sat);
                vs = v2.x;
                vm = v2.y;
                for (int d = 0; d < p.D; ++d) s = fmaf(s_q[d], fmaf((float)code_of((const uint8_t *)p.k + at, d), ks.x, ks.y), s);
            } else {
                for (int d = 0; d < p.D; ++d)
                    s = fmaf(s_q[d], H == kS8 ? (float)((const int8_t *)p.k)[at + d] : (float)((const T *)p.k)[at + d], s);
                if (H == kS8) {
                    s *= p.k_scale[sat];
                    vs = p.v_scale[sat];
                }
            }
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
            const float wk = __shfl(pj, k), sk = __shfl(vs, k), mk = __shfl(vm, k);
            const int64_t vr = ((int64_t)__shfl((int)(at >> 32), k) << 32) | (uint32_t)__shfl((int)at, k);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int d = lane + 64 * e;
                if (d >= p.D) continue;
                if constexpr (H == kQ4)
                    o[e] = fmaf(wk, fmaf((float)code_of((const uint8_t *)p.v + vr, d), sk, mk), o[e]);
                else
                    o[e] = fmaf(wk, H == kS8 ? (float)((const int8_t *)p.v)[vr + d] * sk : (float)((const T *)p.v)[vr + d], o[e]);
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

// A workgroup's run of units u .. u1-1 (none: u1 = u), which begins in request r, whose
// units begin at base.  Workgroups take `each` units, the first `more` one more.  NEAR:
// neighbouring runs go to one XCD (workgroups are dealt out to the eight in turn), whose
// L2 then serves the heads that share lines of 128 bytes, and the tiles that share keys.
template <class C>
struct Run {
    struct Shared {
        int64_t part[C::WAVES], base;
        int r;
        Request req;
    };
    int64_t u, u1, each, more, base;
    int wg;  // its place among them
    int r;
    Request now;

    // All threads of the workgroup; leaves its header and clears `bad`.
    __device__ __forceinline__ Run(Shared &s, int &bad) : u(0), u1(0), each(0), more(0), base(0), wg(0), r(0) {
        constexpr int NT = 64 * C::WAVES;
        Params &p = params();
        const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int per = (p.R + NT - 1) / NT, r0 = min(tid * per, p.R), r1 = min(r0 + per, p.R);
        int64_t mine = 0, before = 0, U = 0, x = 0;
        Request q;
        const bool alone = p.R == 1;  // every thread has the one request: nothing to add up or to look for
        for (int i = alone ? 0 : r0; i < (alone ? 1 : r1); ++i) {
            q = request<C>(p, i);
            mine += Line<C>(p, q).all() * head_groups<C>(p);
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
            if (lane == 63) s.part[wave] = x;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < C::WAVES; ++i) {
                if (i < wave) before += s.part[i];
                U += s.part[i];
            }
        }
        U = uniform(U);
        // behind a window a unit is a key: a workgroup takes a block's worth at least
        const int64_t share = C::WIN ? max(U / C::KB, (int64_t)1) : U, grid = share < gridDim.x ? share : gridDim.x;
        wg = blockIdx.x;
        if (C::NEAR && wg < grid) {
            const int x = wg & 7, whole = (int)grid >> 3, rest = (int)grid & 7;
            wg = x * whole + min(x, rest) + (wg >> 3);
        }
        if (tid == 0) {
            p.hdr[wg].rows = 0;
            p.hdr[wg].bad = 0;
            bad = 0;
        }
        if (U == 0 || wg >= grid) return;
        each = divide(U, grid);
        more = U - each * grid;
        u = wg * each + (wg < more ? wg : more);
        u1 = u + each + (wg < more);
        if (alone) {
            now = q;
        } else {
            int64_t at = before + x - mine;
            if (u >= at && u < at + mine) {
                for (int k = r0; k < r1; ++k) {
                    if (per > 1) q = request<C>(p, k);
                    const int64_t units = Line<C>(p, q).all() * head_groups<C>(p);
                    if (u < at + units) {
                        s.r = k;
                        s.base = at;
                        s.req = q;
                        break;
                    }
                    at += units;
                }
            }
            __syncthreads();
            r = s.r;
            base = s.base;
            now = s.req;
        }
        r = __builtin_amdgcn_readfirstlane(r);
        base = uniform(base);
        if (tid == 0) {
            p.hdr[wg].r = r;
            p.hdr[wg].base = base;
            p.hdr[wg].u = u;
            p.hdr[wg].u1 = u1;
        }
    }
    // the workgroup that has unit x
    __device__ __forceinline__ int workgroup(int64_t x) const {
        const int64_t large = more * (each + 1);
        return (int)(x < large ? divide(x, each + 1) : more + divide(x - large, each));
    }
};

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
template <class X, Held H, int DK, int MT, bool WIN>
__global__ __launch_bounds__(256, 2) void k_tree(TreeParams) {
    typedef typename X::T T;
    typedef typename X::V V;
    typedef Cut<DK, MT, WIN> C;
    constexpr bool S8 = H != kWide, Q4 = H == kQ4;  // S8: codes, through registers
    constexpr int WAVES = C::WAVES, NT = 64 * WAVES, KB = C::KB, ROWT = C::ROWT, SB = KB / 32;
    constexpr int LCH = DK == 96 ? 16 : DK / 8, LS = LCH * 8;  // an LDS row: chunks, elements
    constexpr int NP = KB * LCH / NT, NK = DK / 32, ND = DK / 16;
    constexpr int kSums = MT * ND * 1024;  // a wavefront's sums, in bytes
    __shared__ __align__(256) char s_mem0[4 * KB * LS], s_mem1[4 * KB * LS];
    __shared__ int64_t s_off[4][KB], s_soff[S8 ? 4 : 1][S8 ? KB : 1];
    __shared__ float s_ks[S8 ? 2 : 1][S8 ? KB : 1], s_vs[S8 ? 2 : 1][S8 ? KB : 1];
    __shared__ float s_km[Q4 ? 2 : 1][Q4 ? KB : 1], s_vm[Q4 ? 2 : 1][Q4 ? KB : 1], s_m[WAVES][MT][16], s_l[WAVES][MT][16];
    __shared__ typename Run<C>::Shared s_run;
    __shared__ int s_bad;
    __shared__ uint64_t s_bits[ROWT];  // the keys of a block that a token sees
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, g = lane >> 4;

    const Run<C> run(s_run, s_bad);
    if (run.u >= run.u1) return;
    int64_t u = run.u, base_u = run.base;
    int r = run.r;
    Request now = run.now;

    while (u < run.u1) {
        Params &p = params();
        const Request q = uniform(now);
        const Line<C> line(p, q);
        const int64_t per_head = uniform(line.all());
        if (u >= base_u + per_head * p.Hkv) {
            base_u += per_head * p.Hkv;
            now = request<C>(p, ++r);
            continue;
        }
        Tile w;
        w.hk = __builtin_amdgcn_readfirstlane((int)divide(u - base_u, per_head));
        const int64_t rest = u - base_u - w.hk * per_head;
        const int tile = __builtin_amdgcn_readfirstlane(line.find(rest));
        const int64_t units = uniform(line.of(tile)), from = uniform(rest - line.before(tile));
        const int64_t to = uniform(run.u1 - u < units - from ? from + (run.u1 - u) : units);
        w.row0 = tile * ROWT;
        w.nrows = min(q.n * p.G - w.row0, ROWT);
        const Blocks<C> at(p, q, w.row0, w.nrows);
        // an item's first units need not hold a block
        const int b0 = __builtin_amdgcn_readfirstlane(at.within(from, units)), b1 = __builtin_amdgcn_readfirstlane(at.within(to, units));
        if (b1 == 0) {
            u += to - from;
            continue;
        }
        const int nb = __builtin_amdgcn_readfirstlane(at.nb), firsts = __builtin_amdgcn_readfirstlane(at.firsts),
                  later = __builtin_amdgcn_readfirstlane(at.from - at.firsts);
        const auto key_block = [&](int b) { return !WIN || b < firsts ? b : b + later; };
        const bool first_part = b0 == 0, last_part = b1 == nb;
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
        const int window = WIN ? p.window : 0, sinks = WIN ? p.sinks : 0;

        // ---- page entries: of this block and the next ones
        const int32_t *table = p.table + (int64_t)r * p.ld_table;
        const auto page_of = [&](int b) {  // of key tid of block b; -1: none
            const uint32_t j = (uint32_t)key_block(b) * KB + tid;  // a block's first key is below 2^31
            return b < b1 && tid < KB && j < (uint32_t)q.len ? table[j / (uint32_t)page_size] : -1;
        };
        const auto put_off = [&](int b, int page) {
            if (tid < KB) {
                const bool ok = page >= 0 && page < num_pages;
                const int i = (int)(((uint32_t)key_block(b) * KB + tid) % (uint32_t)page_size), ring = (b - b0) & 3;
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
        float xs[MT], lm[MT];  // 4-bit rows: the sum of the query's elements, and of the weighted minima
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
            if (Q4) {
                lm[mt] = 0.0f;
                xs[mt] = 0.0f;
#pragma unroll
                for (int kk = 0; kk < NK; ++kk)
#pragma unroll
                    for (int x = 0; x < 8; ++x) xs[mt] += (float)qv[mt][kk][x];
                xs[mt] = row_sum(xs[mt]);
            }
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
        typedef typename std::conditional<Q4, int, v2i>::type Codes;  // of eight elements
        Codes kr[S8 ? NP : 1], vr[S8 ? NP : 1];
        uint32_t sc = 0;  // a scale, or a step and a minimum
        const auto load = [&](int b) {  // rows of codes of block b and their scales
            const int ring = (b - b0) & 3;
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int sd = head_element(i);
                const int64_t off = s_off[ring][srow + i * (NT / LCH)], at = sd < D && off >= 0 ? off + (Q4 ? sd / 2 : sd) : 0;
                kr[i] = *(const Codes *)((const int8_t *)k_cache + at);
                vr[i] = *(const Codes *)((const int8_t *)v_cache + at);
            }
            if (tid < 2 * KB) {
                const int64_t so = s_soff[ring][tid & (KB - 1)];
                sc = so >= 0 ? ((const uint32_t *)(tid < KB ? k_scale : v_scale))[so] : 0;
            }
        };
        const Widen wide16(kMaskBf16, kSixteenBf16);
        const auto widen = [&](Codes x) {  // eight codes as bf16; 4-bit ones as 16 + code
            v4i y;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (Q4) {
                    y[e] = wide16.bf16((uint32_t)x, e);
                } else {
                const int w2 = x[e / 2] >> (16 * (e & 1));
                y[e] = (int)__builtin_amdgcn_perm(__float_as_uint((float)(int8_t)(w2 >> 8)), __float_as_uint((float)(int8_t)w2),
                                                  0x07060302u);
                }
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
            const float2 dm = Q4 ? pair_of(sc) : float2{__uint_as_float(sc), 0.0f};
            if (tid < KB) {
                s_ks[which][tid] = dm.x * p_scale;
                if (Q4) s_km[which][tid] = (dm.y - 16.0f * dm.x) * p_scale;
            } else if (tid < 2 * KB) {
                s_vs[which][tid - KB] = dm.x;
                if (Q4) s_vm[which][tid - KB] = dm.y - 16.0f * dm.x;
            }
        };

        // ---- one 32-key step; clean: every row sees all its keys (else s_bits tells)
        const int kx = swizzle<LCH>(c), vrow = 4 * g + (c >> 2), vx = swizzle<LCH>(vrow);
        const float scale = S8 ? 1.0f : p_scale;  // the key scales of codes carry it
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
            v4f vs[2], vm[2];
            if (S8) {
#pragma unroll
                for (int kt = 0; kt < 2; ++kt) {
                    const v4f ks = *(const v4f *)(s_ks[which] + k0 + 16 * kt + 4 * g);
                    vs[kt] = *(const v4f *)(s_vs[which] + k0 + 16 * kt + 4 * g);
                    v4f km;
                    if (Q4) {
                        km = *(const v4f *)(s_km[which] + k0 + 16 * kt + 4 * g);
                        vm[kt] = *(const v4f *)(s_vm[which] + k0 + 16 * kt + 4 * g);
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int v = 0; v < 4; ++v) s[mt][kt][v] = Q4 ? fmaf(s[mt][kt][v], ks[v], km[v] * xs[mt]) : s[mt][kt][v] * ks[v];
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
                    if (Q4) lm[mt] *= alpha;
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
                    if (Q4) {
                        lm[mt] = fmaf(a, vm[e / 4][e % 4], lm[mt]);
                        lm[mt] = fmaf(b, vm[e / 4][e % 4 + 1], lm[mt]);
                    }
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
            const int kb = key_block(b);
            bool clean = vis == ~0ull;
            if (WIN) {  // every row of the tile sees the block
                const uint32_t k0 = (uint32_t)kb * KB, k1 = k0 + KB - 1, pos = (uint32_t)q.ctx + (uint32_t)(tok0 - q.first);
                clean = clean && k1 <= pos && (k0 + (uint32_t)window > pos + (uint32_t)(ntok - 1) || k1 < (uint32_t)sinks);
            } else {
                clean = clean && (int64_t)(b + 1) * KB <= q.ctx;
            }
            if (!clean) {
                Params &p = params();
                int first = tok0, me = tid;  // nothing of this is worth keeping over the steps in between
                asm volatile("" : "+s"(first), "+v"(me));
                if (!S8)  // what stands for missing keys must not be NaN
                    for (int x = me; x < KB * LCH; x += NT)
                        if (off[x / LCH] < 0) *(v4i *)(cur + KB * LS * 2 + x * 16) = v4i{0, 0, 0, 0};
                const int k = kb * KB + (me & 63) - (WIN ? 0 : q.ctx);  // the lane's key; of the drafted token that it is
                const bool in = !WIN && k >= 0 && k < p.mask_cols;
                for (int i0 = me >> 6; i0 < ntok; i0 += 8 * WAVES) {
                    int m[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int i = min(i0 + WAVES * e, ntok - 1);
                        if (WIN) m[e] = in_window((uint32_t)k, (uint32_t)q.ctx + (uint32_t)(first - q.first + i), (uint32_t)window, (uint32_t)sinks);
                        else m[e] = k < 0 || (!p.mask && k <= first - q.first + i);
                        if (!WIN && p.mask && in) m[e] = p.mask[(first + i) * p.ld_mask + k];
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
        if (WIN && b0 == b1) {
            // a share of an item that no block ends in: empty sums
        } else if constexpr (S8) {
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
        for (int mt = 0; mt < MT; ++mt) {
            l[mt] = row_sum(l[mt]);
            if (Q4) {
                lm[mt] = row_sum(lm[mt]);
#pragma unroll
                for (int dt = 0; dt < ND; ++dt)
#pragma unroll
                    for (int v = 0; v < 4; ++v) o[mt][dt][v] += lm[mt];
            }
        }
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
            float *const slot = pe.part + (2 * (int64_t)run.wg + (first_part ? 1 : 0)) * pe.slot_rows * (DK + 2);
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
            TreeHeader &h = pe.hdr[run.wg];
            h.rows = w.nrows;
            h.first_wg = run.workgroup(u - from + at.first_unit(units));  // of the item's first block
            h.hk = w.hk;
            h.row0 = w.row0;
            h.first = q.first;
        }
        u += to - from;
    }
    __syncthreads();
    if (tid == 0 && s_bad) params().hdr[run.wg].bad = 1;
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
template <class X, Held H, int DK, int MT, bool WIN>
__global__ __launch_bounds__(256) void k_tree_join(TreeParams) {
    Params &p = params();
    typedef typename X::T T;
    typedef Cut<DK, MT, WIN> C;
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
                const Request q = uniform(request<C>(p, r));
                for (int i = many ? step : step * SP; i < min(many ? step + 1 : (step + 1) * SP, h.rows); ++i)
                    plain_row<X, H, WIN>(p, q, r, h.hk, row_of(p, q, h.hk, h.row0 + i), s_q[wave]);
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
            const Request q = uniform(request<C>(p, r));
            const Line<C> line(p, q);
            const int64_t per_head = line.all();
            if (u >= base + per_head * p.Hkv) {
                base += per_head * p.Hkv;
                ++r;
                continue;
            }
            const int hk = (int)divide(u - base, per_head);
            const int64_t rest = u - base - hk * per_head;
            const int tile = line.find(rest), row0 = tile * C::ROWT, n = min(q.n * p.G - row0, C::ROWT);
            const int64_t units = line.of(tile), from = rest - line.before(tile), end = u + units - from;
            if (Blocks<C>(p, q, row0, n).within(from, units) == 0 && end <= h.u1) {
                for (int row = blockIdx.x * 4 + wave; row < n; row += gridDim.x * 4)
                    plain_row<X, H, WIN>(p, q, r, hk, row_of(p, q, hk, row0 + row), s_q[wave]);
            }
            u = end;
        }
    }
}
// The workgroups of the join: at most one shared item ends in a workgroup.
inline dim3 join_grid(const TreeShape &z) {
    const int64_t wgs = ceil_div(z.wgs * z.slot_rows, 4);
    return dim3((unsigned)(wgs < 1024 ? wgs : 1024));
}

template <class X, Held H, int DK, int MT, bool WIN>
hipError_t launch(const TreeParams &p, const TreeShape &z, hipStream_t s) {
    hipLaunchKernelGGL((k_tree<X, H, DK, MT, WIN>), dim3((unsigned)z.wgs), dim3(256), 0, s, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_tree_join<X, H, DK, MT, WIN>), join_grid(z), dim3(256), 0, s, p);
    return hipGetLastError();
}

template <class X, Held H, bool WIN>
hipError_t launch_dk(const TreeParams &p, const TreeShape &z, hipStream_t s) {
    if (z.dk == 256) return launch<X, H, 256, 1, WIN>(p, z, s);
    if (z.mt == 1)
        return z.dk == 64   ? launch<X, H, 64, 1, WIN>(p, z, s)
               : z.dk == 96 ? launch<X, H, 96, 1, WIN>(p, z, s)
                            : launch<X, H, 128, 1, WIN>(p, z, s);
    return z.dk == 64   ? launch<X, H, 64, 2, WIN>(p, z, s)
           : z.dk == 96 ? launch<X, H, 96, 2, WIN>(p, z, s)
                        : launch<X, H, 128, 2, WIN>(p, z, s);
}

}  // namespace

}  // namespace qmm
