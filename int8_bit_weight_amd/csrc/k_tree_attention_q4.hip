// k_tree_attention_q4.hip -- attention over a paged cache of 4-bit rows: of drafted
// tokens, and behind a window.  tree_attention.h has the kernels for many rows a request;
// k_few4 below is for few.
#include "tree_attention.h"

namespace qmm {

namespace {

template <int DK, int MT, bool WINDOW, int HEADS_>
struct Few {
    static constexpr int HEADS = HEADS_, WAVES = few_waves(HEADS), KB = few_keys(HEADS), ROWT = 16 * MT, ITEM = few_item(HEADS);
    static constexpr int WGS = few_workgroups(DK > 128 ? 2 : MT, HEADS);
    static constexpr bool WIN = WINDOW, NEAR = true;
};

// f(0), f(1) ...
template <int N, int I = 0, class F>
__device__ __forceinline__ void for_sets(F f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>());
        for_sets<N, I + 1>(f);
    }
}

typedef int v4iu __attribute__((ext_vector_type(4), aligned(2)));
// N words of a row.
template <int N>
struct Words {
    typedef uint32_t T __attribute__((ext_vector_type(N), aligned(4)));
};

// The line of work is k_tree's, but each wavefront goes through 32 keys at a time on its
// own, from memory to the matrix operands without LDS or barriers:
//   S^T = K Q^T: a lane (c, g) has key c and the W words from W g on of its row; the
//     order of a product's 32 elements is free, so product kk takes word kk of each lane.
//     The sum starts at -16 sum x, and the minima's part, m_j sum x, comes from a product
//     of its own (three bf16 terms of sum x) that starts at minus the running maximum.
//   O^T = V^T P^T: a lane has word c of the eight keys whose weights it holds.  Halves of
//     two keys' words side by side are the pairs that product e (element e of each word)
//     takes, so element e of word c becomes row c of product e.
// Two instructions make a pair of operands of a word.
//
// The weights enter the second product as w_j d_j in fp16, rounded once (2^-12), with d_j
// below a power of two that only grows.  A product with ones gives the sum of the
// rounded weights, so that 24 of it can be taken from the sums of 16 + q: what the
// rounding moves is w d (q - 8), not the offset, and
//   o = sum (w d)~ (q - 8) + sum w (m + 8 d),  the second sum in fp32.
//
// HEADS 4: the wavefronts take a cache head each, so that a workgroup reads 256 bytes of
// a token's row in a cache whose heads stand side by side (one head alone is 64
// bytes, and read by itself moves 4.1 TB/s where 5.3 can be had).  HEADS 1: the wavefronts
// take a quarter of a block's keys each and join their sums where a share of an item ends.
//
// One row a head behind a window of 16384, 61 requests: 230 us, 1.22 GB at 5.3 TB/s, memory bound.
// Two tiles of rows (32 requests of 32 rows, 32768 keys): 192 us; the operands of both
// fill the registers, VALU issue is 62 % and 709 MB come at 3.7 TB/s, so one set of
// loads is in flight: two spill 23 to 48 registers and take as long.
// Heads of 256, one set against two (which spill 4 to 21), us: 32 x 16000 keys of 8 heads 207 / 215,
// 8 x 30000 of 4 heads 56 / 59, 64 x 5000 of 2 heads 45 / 55.
template <int DK, int MT, bool WIN, int HEADS>
__global__ __launch_bounds__(64 * few_waves(HEADS), HEADS == 8 ? 1 : HEADS == 4 && MT == 1 && DK <= 128 ? 3 : 2) void k_few4(TreeParams) {
    typedef __bf16 T;
    typedef v8bf V;
    typedef Few<DK, MT, WIN, HEADS> C;
    constexpr int W = DK / 32, NV = (DK / 8 + 15) / 16, SETS = MT == 2 || NV == 2 ? 1 : HEADS == 8 ? 3 : 2;
    constexpr float kLift = 64.0f;  // weights up to 2^8 stay below 2^14, and those of 2^-20 are fp16 normals
    __shared__ typename Run<C>::Shared s_run;
    __shared__ int s_bad;
    __shared__ int64_t s_off[C::WAVES][SETS][32];
    __shared__ __align__(16) float s_scale[C::WAVES][3][32];
    __shared__ v4f s_sum[HEADS == 1 ? 2 : 1][HEADS == 1 ? MT * NV * 8 : 1][64];
    __shared__ float s_m[4][MT][16], s_l[4][MT][16];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, g = lane >> 4, key = lane & 31;

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
        const int groups = head_groups<C>(p);
        if (u >= base_u + per_head * groups) {
            base_u += per_head * groups;
            now = request<C>(p, ++r);
            continue;
        }
        Tile w;
        w.hk = __builtin_amdgcn_readfirstlane((int)divide(u - base_u, per_head));
        const int64_t rest = u - base_u - w.hk * per_head;
        const int tile = __builtin_amdgcn_readfirstlane(line.find(rest));
        const int64_t units = uniform(line.of(tile)), from = uniform(rest - line.before(tile));
        const int64_t to = uniform(run.u1 - u < units - from ? from + (run.u1 - u) : units);
        w.row0 = tile * C::ROWT;
        w.nrows = min(q.n * p.G - w.row0, C::ROWT);
        const Blocks<C> at(p, q, w.row0, w.nrows);
        const int b0 = __builtin_amdgcn_readfirstlane(at.within(from, units)), b1 = __builtin_amdgcn_readfirstlane(at.within(to, units));
        if (b1 == 0) {
            u += to - from;
            continue;
        }
        const int nb = __builtin_amdgcn_readfirstlane(at.nb), firsts = __builtin_amdgcn_readfirstlane(at.firsts),
                  later = __builtin_amdgcn_readfirstlane(at.from - at.firsts);
        // the wavefront's first key of a block
        const auto first_key = [&](int b) {
            return (uint32_t)(!WIN || b < firsts ? b : b + later) * C::KB + (HEADS == 1 ? 32u * wave : 0u);
        };
        const int hk = HEADS == 1 ? w.hk : w.hk * HEADS + wave;
        const bool first_part = b0 == 0, last_part = b1 == nb;
        const int tok0 = row_of(p, q, w.hk, w.row0).t, ntok = row_of(p, q, w.hk, w.row0 + w.nrows - 1).t - tok0 + 1;

        const uint32_t page_size = p.page, page_mul = p.page_mul;
        const int page_shift = p.page_shift, num_pages = p.num_pages, D = p.D, window = WIN ? p.window : 0, sinks = WIN ? p.sinks : 0;
        const int64_t page_stride = p.page_stride, token_stride = p.token_stride, head_at = hk * p.head_stride;
        const int64_t sp_stride = p.sp_stride, st_stride = p.st_stride, shead_at = hk * p.sh_stride;
        const uint8_t *const k_cache = (const uint8_t *)p.k, *const v_cache = (const uint8_t *)p.v;
        const uint32_t *const scales = (const uint32_t *)(lane < 32 ? p.k_scale : p.v_scale);
        const float p_scale = p.scale;
        const auto page_of = [&](uint32_t j) { return (uint32_t)((uint64_t)j * page_mul >> page_shift); };
        const int32_t *table = p.table + (int64_t)r * p.ld_table;

        // ---- queries: column c, the words from W g on, or the row's last W: those that lane g - 1 has count as zeros
        const int word0 = min(W * g, D / 8 - W);
        V qv[MT][W], xq[MT];  // xq: the sum of a query's elements, times the scale, as three terms
        int token[MT];
        // o: sums of 16 + q; ones: of the weights as they enter them; both in units of `limit`
        v4f o[MT][NV][8], ones[MT], start[MT], against[MT];  // start: -16 sum x; against: minus the maximum
        float base[MT], thr[MT], l[MT], lm[MT], limit = -1.0f, down = 0.0f;
        const v4f zero = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int row = 16 * mt + c;
            const Row z = row_of(p, q, hk, w.row0 + (row < w.nrows ? row : 0));
            token[mt] = z.t;
            const T *src = (const T *)p.Q + z.t * p.q_tok + z.h * p.q_head;
            float sum = 0.0f;
#pragma unroll
            for (int kk = 0; kk < W; ++kk) {
                const int d = 8 * (word0 + kk);
                v4i v = {0, 0, 0, 0};
                if (row < w.nrows && d >= 8 * W * g) v = *(const v4iu *)(src + d);
#pragma unroll
                for (int x = 0; x < 4; ++x) v[x] ^= p.q_flip;
                qv[mt][kk] = __builtin_bit_cast(V, v);
#pragma unroll
                for (int x = 0; x < 8; ++x) sum += (float)qv[mt][kk][x];
            }
            sum = row_sum(sum);
#pragma unroll
            for (int v = 0; v < 4; ++v) start[mt][v] = -16.0f * sum;
            sum *= p_scale;
            const float s1 = __uint_as_float(__float_as_uint(sum) & 0xFFFF0000u), s2 = __uint_as_float(__float_as_uint(sum - s1) & 0xFFFF0000u);
            V terms = {};
            if (g < 2) {  // the lanes whose keys the product's first operand names
                terms[0] = (__bf16)s1;
                terms[1] = (__bf16)s2;
                terms[2] = (__bf16)(sum - s1 - s2);
            }
            xq[mt] = terms;
            ones[mt] = against[mt] = zero;
#pragma unroll
            for (int nv = 0; nv < NV; ++nv)
#pragma unroll
                for (int e = 0; e < 8; ++e) o[mt][nv][e] = zero;
            base[mt] = l[mt] = lm[mt] = 0.0f;
            thr[mt] = -INFINITY;  // 8 once there is a maximum
        }

        // ---- what is on its way: words of K and V, a scale pair, which keys there are.  Keys
        // that there are not have the cache's first row; their pairs are put out when they are used.
        typename Words<W < 4 ? W : 4>::T kw[SETS][2][W < 4 ? 1 : W / 4];
        uint32_t vw[SETS][NV][8], pair[SETS], there[SETS];
        uint32_t v_word[NV];  // past the row's last word: any, its sums are not used
#pragma unroll
        for (int nv = 0; nv < NV; ++nv) v_word[nv] = 4 * min(c + 16 * nv, D / 8 - 1);
        const auto entry = [&](int b) {
            const uint32_t j = first_key(b) + key;
            int page = -1;
            if (b < b1 && j < (uint32_t)q.len) page = table[page_of(j)];
            return page;
        };
        const auto ask = [&](auto SET, int b, int page) __attribute__((always_inline)) {
            constexpr int set = decltype(SET)::value;
            const bool ok = page >= 0 && page < num_pages;
            const uint32_t j = first_key(b) + key, i = j - page_of(j) * page_size;
            there[set] = (uint32_t)__ballot(ok);
            pair[set] = scales[ok ? page * sp_stride + i * st_stride + shead_at : 0];
            __builtin_amdgcn_wave_barrier();
            s_off[wave][set][key] = ok ? page * page_stride + i * token_stride + head_at : 0;
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int kt = 0; kt < 2; ++kt) {
                const uint8_t *row = k_cache + s_off[wave][set][16 * kt + c] + 4 * word0;
#pragma unroll
                for (int y = 0; y < W; y += 4) kw[set][kt][y / 4] = *(const typename Words<W < 4 ? W : 4>::T *)(row + 4 * y);
            }
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const uint8_t *row = v_cache + s_off[wave][set][16 * (x / 4) + 4 * g + x % 4];
#pragma unroll
                for (int nv = 0; nv < NV; ++nv) vw[set][nv][x] = *(const uint32_t *)(row + v_word[nv]);
            }
        };

        const Widen in_k(kMaskBf16, kSixteenBf16), in_v(kMaskF16, kSixteenF16);
        const auto step = [&](auto SET, int b) __attribute__((always_inline)) {
            constexpr int set = decltype(SET)::value;
            const uint32_t j0 = first_key(b);
            if (there[set] == 0) return;
            const uint32_t mine = there[set] >> key & 1 ? pair[set] : 0;
            const float2 dm = pair_of(mine);
            if (__any(lane >= 32 && dm.x > limit)) {
                // a larger step than any: the sums go over to its power of two
                float most = lane >= 32 ? dm.x : 0.0f;
#pragma unroll
                for (int x = 1; x < 64; x *= 2) most = fmaxf(most, __shfl_xor(most, x));
                most = fminf(fmaxf(most, 0x1p-100f), 0x1p126f);
                const float next = __uint_as_float((__float_as_uint(most) & 0x7F800000u) + 0x00800000u);
                const float factor = limit > 0.0f ? limit / next : 0.0f;
                limit = next;
                down = kLift / next;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    ones[mt] *= factor;
#pragma unroll
                    for (int i = 0; i < NV * 8; ++i) o[mt][i / 8][i % 8] *= factor;
                }
            }
            __builtin_amdgcn_wave_barrier();
            if (lane < 32) {
                s_scale[wave][0][key] = dm.x * p_scale;
            } else {
                s_scale[wave][1][key] = dm.x * down;
                s_scale[wave][2][key] = fmaf(8.0f, dm.x, dm.y);
            }
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            v4f s[MT][2], minima[MT][2];
#pragma unroll
            for (int kt = 0; kt < 2; ++kt) {
                // the minimum of key c against each of the three terms: lanes g = kt hold the pairs of tile kt's keys
                const uint32_t m = g == kt ? mine : 0;
                const v4i mins = {(int)__builtin_amdgcn_perm(m, m, 0x03020302u), (int)(m >> 16), 0, 0};
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    minima[mt][kt] = BF16::mfma(__builtin_bit_cast(V, mins), xq[mt], against[mt]);
                    s[mt][kt] = start[mt];
                }
#pragma unroll
                for (int kk = 0; kk < W; ++kk) {
                    v4i a;
#pragma unroll
                    for (int e = 0; e < 4; ++e) a[e] = in_k.bf16(kw[set][kt][kk / 4][kk % 4], e);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) s[mt][kt] = BF16::mfma(__builtin_bit_cast(V, a), qv[mt][kk], s[mt][kt]);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            v4f vs[2], vm[2];
#pragma unroll
            for (int kt = 0; kt < 2; ++kt) {
                const v4f ks = *(const v4f *)&s_scale[wave][0][16 * kt + 4 * g];
                vs[kt] = *(const v4f *)&s_scale[wave][1][16 * kt + 4 * g];
                vm[kt] = *(const v4f *)&s_scale[wave][2][16 * kt + 4 * g];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int v = 0; v < 4; ++v) s[mt][kt][v] = fmaf(s[mt][kt][v], ks[v], minima[mt][kt][v]);
            }
            bool clean = there[set] == ~0u;
            if (WIN) {
                const uint32_t pos = (uint32_t)q.ctx + (uint32_t)(tok0 - q.first);
                clean = clean && j0 + 31 <= pos && (j0 + (uint32_t)window > pos + (uint32_t)(ntok - 1) || j0 + 31 < (uint32_t)sinks);
            } else {
                clean = clean && j0 + 32 <= (uint32_t)q.ctx;
            }
            if (!clean) {
                Params &pm = params();
                uint32_t sees[MT];  // of the lane's eight keys, by row
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    sees[mt] = 0;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t j = j0 + 16 * (e / 4) + 4 * g + e % 4;
                        const int k = (int)(j - (uint32_t)q.ctx);  // the drafted token; below 0: context
                        const bool in = WIN ? in_window(j, (uint32_t)q.ctx + (uint32_t)(token[mt] - q.first), (uint32_t)window, (uint32_t)sinks)
                                            : j < (uint32_t)q.ctx || (!pm.mask && k <= token[mt] - q.first);
                        sees[mt] |= (uint32_t)in << e;
                    }
                    if (!WIN && pm.mask && pm.mask_cols > 0) {
                        const uint8_t *row = pm.mask + token[mt] * pm.ld_mask;
                        uint32_t m[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            m[e] = row[min(max((int)(j0 + 16 * (e / 4) + 4 * g + e % 4 - (uint32_t)q.ctx), 0), pm.mask_cols - 1)];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const uint32_t j = j0 + 16 * (e / 4) + 4 * g + e % 4;
                            const bool in = j >= (uint32_t)q.ctx && (int)(j - (uint32_t)q.ctx) < pm.mask_cols && m[e] != 0;
                            sees[mt] |= (uint32_t)in << e;
                        }
                    }
                    const uint32_t here = there[set] >> (4 * g);
                    sees[mt] &= (here & 15) | (here >> 12 & 0xF0);
#pragma unroll
                    for (int e = 0; e < 8; ++e) s[mt][e / 4][e % 4] = sees[mt] >> e & 1 ? s[mt][e / 4][e % 4] : -INFINITY;
                }
            }
            float top[MT];
            bool above = false;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const v4f a = s[mt][0], b = s[mt][1];
                top[mt] = fmaxf(fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3])), fmaxf(fmaxf(b[0], b[1]), fmaxf(b[2], b[3])));
                above |= top[mt] > thr[mt];
            }
            if (__any(above)) {  // as in k_tree: a new maximum only past the old one's slack of 2^8
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const bool none = thr[mt] == -INFINITY;
                    const float rise = fmaxf(none ? -INFINITY : 0.0f, row_max(top[mt]));  // from the old maximum
                    const float next = rise == -INFINITY ? 0.0f : base[mt] + rise, by = next - base[mt];
                    const float alpha = none ? 0.0f : __builtin_amdgcn_exp2f(-by);
                    base[mt] = next;
                    thr[mt] = rise == -INFINITY ? -INFINITY : 8.0f;
                    l[mt] *= alpha;
                    lm[mt] *= alpha;
                    ones[mt] *= alpha;
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        against[mt][v] = -next;
                        s[mt][0][v] -= by;
                        s[mt][1][v] -= by;
                    }
#pragma unroll
                    for (int i = 0; i < NV * 8; ++i) o[mt][i / 8][i % 8] *= alpha;
                }
            }
            v8h hw[MT];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float a = __builtin_amdgcn_exp2f(s[mt][e / 4][e % 4]);
                    l[mt] += a;
                    lm[mt] = fmaf(a, vm[e / 4][e % 4], lm[mt]);
                    hw[mt][e] = (_Float16)(a * vs[e / 4][e % 4]);
                }
                const _Float16 one = (_Float16)1.0f;
                ones[mt] = F16::mfma(v8h{one, one, one, one, one, one, one, one}, hw[mt], ones[mt]);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int nv = 0; nv < NV; ++nv) {
                uint32_t even[4], odd[4];  // halves of two keys' words: their even elements, and their odd ones
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    even[i] = __builtin_amdgcn_perm(vw[set][nv][2 * i + 1], vw[set][nv][2 * i], 0x05040100u);
                    odd[i] = __builtin_amdgcn_perm(vw[set][nv][2 * i + 1], vw[set][nv][2 * i], 0x07060302u);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    v4i a;
#pragma unroll
                    for (int i = 0; i < 4; ++i) a[i] = in_v.f16(e & 1 ? odd[i] : even[i], e / 2);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) o[mt][nv][e] = F16::mfma(__builtin_bit_cast(v8h, a), hw[mt], o[mt][nv][e]);
                }
            }
        };

        for_sets<SETS>([&](auto SET) { ask(SET, b0 + decltype(SET)::value, entry(b0 + decltype(SET)::value)); });
        int page = entry(b0 + SETS);
        for (int b = b0; b < b1; b += SETS)
            for_sets<SETS>([&](auto SET) __attribute__((always_inline)) {
                const int at = b + decltype(SET)::value, next = entry(at + SETS + 1);
                if (at < b1) step(SET, at);
                ask(SET, at + SETS, page);
                page = next;
            });

        // ---- sums of w (d q + m)
        Params &pe = params();
        float m[MT];
        const float up = limit / kLift;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            m[mt] = thr[mt] == -INFINITY ? -INFINITY : base[mt];
            l[mt] = row_sum(l[mt]);
            lm[mt] = row_sum(lm[mt]);
#pragma unroll
            for (int i = 0; i < NV * 8; ++i)
#pragma unroll
                for (int v = 0; v < 4; ++v) o[mt][i / 8][i % 8][v] = fmaf(fmaf(-24.0f, ones[mt][0], o[mt][i / 8][i % 8][v]), up, lm[mt]);
        }
        if constexpr (HEADS == 1) {
            // join the wavefronts' sums: 2 and 3 leave theirs for 0 and 1, then 1 for 0
#pragma unroll
            for (int half = 2; half > 0; half /= 2) {
                __syncthreads();
                if (wave >= half && wave < 2 * half) {
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        if (g == 0) {
                            s_m[wave][mt][c] = m[mt];
                            s_l[wave][mt][c] = l[mt];
                        }
#pragma unroll
                        for (int i = 0; i < NV * 8; ++i) s_sum[wave - half][mt * NV * 8 + i][lane] = o[mt][i / 8][i % 8];
                    }
                }
                __syncthreads();
                if (wave < half) {
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        const float m2 = s_m[wave + half][mt][c], l2 = s_l[wave + half][mt][c];
                        const float top = fmaxf(m[mt], m2), b = top == -INFINITY ? 0.0f : top;
                        const float x = __builtin_amdgcn_exp2f(m[mt] - b), y = __builtin_amdgcn_exp2f(m2 - b);
                        l[mt] = x * l[mt] + y * l2;
                        m[mt] = top;
#pragma unroll
                        for (int i = 0; i < NV * 8; ++i) {
                            const v4f part = s_sum[wave][mt * NV * 8 + i][lane];
#pragma unroll
                            for (int v = 0; v < 4; ++v) o[mt][i / 8][i % 8][v] = x * o[mt][i / 8][i % 8][v] + y * part[v];
                        }
                    }
                }
            }
        }
        if (HEADS > 1 || wave == 0) {
            const bool final = first_part && last_part;
            float *const slot = pe.part + (2 * (int64_t)run.wg + (first_part ? 1 : 0)) * pe.slot_rows * (DK + 2);
            const int row1 = HEADS > 1 ? wave * w.nrows : 0;  // rows stand one head after the other
            bool bad = false;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const int row = 16 * mt + c;
                if (row >= w.nrows) continue;
                bad |= !(l[mt] < INFINITY);
                const Row z = row_of(pe, q, hk, w.row0 + row);
                T *const out = (T *)pe.O + z.t * pe.o_tok + z.h * pe.o_head;
                const float inv = l[mt] == 0.0f ? 0.0f : 1.0f / l[mt];
                if (!final && g == 0) {
                    slot[row1 + row] = m[mt];
                    slot[pe.slot_rows + row1 + row] = l[mt];
                }
#pragma unroll
                for (int nv = 0; nv < NV; ++nv)
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const int d = 8 * (16 * nv + 4 * g + v);
                        if (d >= pe.D) continue;
                        T x[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            bad |= !(fabsf(o[mt][nv][e][v]) < INFINITY);
                            x[e] = (T)(o[mt][nv][e][v] * inv);
                        }
                        if (final) {
                            *(v4iu *)(out + d) = *(v4i *)x;
                        } else {
                            float *const at = slot + 2 * pe.slot_rows + (row1 + row) * DK + d;
#pragma unroll
                            for (int e = 0; e < 8; e += 4)
                                *(v4f *)(at + e) = v4f{o[mt][nv][e][v], o[mt][nv][e + 1][v], o[mt][nv][e + 2][v], o[mt][nv][e + 3][v]};
                        }
                    }
            }
            if (bad) s_bad = 1;
        }
        if (!first_part && last_part && tid == 0) {  // the last of an item's parts: what the join needs
            TreeHeader &h = pe.hdr[run.wg];
            h.rows = HEADS * w.nrows;
            h.first_wg = run.workgroup(u - from + at.first_unit(units));
            h.hk = w.hk;
            h.row0 = w.row0;
            h.first = q.first;
        }
        u += to - from;
    }
    __syncthreads();
    if (tid == 0 && s_bad) params().hdr[run.wg].bad = 1;
}

// k_tree_join for these: a workgroup takes a step of the line.  Of items of few parts that
// is 4 SP rows, of more a row a wavefront, and of more than 48 one row, whose parts the
// four wavefronts share (16 rows of 256 parts: 7.8 us against 16.8; 128 rows of 16 parts
// 17 against 7.6).  Rows of an item's heads stand one head after the other.
template <int DK, class C>
__global__ __launch_bounds__(256) void k_few_join(TreeParams) {
    constexpr Held H = kQ4;
    constexpr bool WIN = C::WIN;
    typedef BF16 X;
    typedef __bf16 T;
    Params &p = params();
    constexpr int Q = DK / 4, SP = 64 / Q > 0 ? 64 / Q : 1, TEAM = 4, RUN = SP * TEAM, MANY = 8, MOST = 48, PER = (C::WGS + 255) / 256;  // headers a thread
    __shared__ int s_end[256 * PER], s_rows[256 * PER], s_part[4], s_any;
    __shared__ Shared s_item[256 * PER];
    __shared__ float s_q[4][256];
    __shared__ float s_tm[4], s_tl[4];
    __shared__ v4f s_acc[4][Q];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // steps of the line: of RUN rows, TEAM or one, by an item's parts
    int steps[PER], bad = 0, x = 0;
    if (tid == 0) s_any = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int at = PER * tid + i;
        Shared h = {};
        if (at < p.wgs) {
            const TreeHeader *from = p.hdr + at;
            h = {from->rows, from->first_wg, from->hk, from->row0, from->first};
            bad |= from->bad;
        }
        s_item[at] = h;
        const int n = at - h.first_wg + 1;
        steps[i] = n <= MANY ? (h.rows + RUN - 1) / RUN : n <= MOST ? (h.rows + TEAM - 1) / TEAM : h.rows;
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
#pragma unroll
    for (int i = PER - 1; i >= 0; --i) {
        s_end[PER * tid + i] = x;
        s_rows[PER * tid + i] = steps[i];
        x -= steps[i];
    }
    __syncthreads();
    const int d = 4 * (lane % Q), k = lane / Q;
    for (int at = blockIdx.x; at < total; at += gridDim.x) {
        int lo = 0, hi = 256 * PER - 1;  // the first header whose steps end past this one
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (s_end[mid] > at) hi = mid;
            else lo = mid + 1;
        }
        lo = __builtin_amdgcn_readfirstlane(lo);
        const Shared h = s_item[lo];
        const int step = at - (s_end[lo] - s_rows[lo]), n = lo - h.first_wg + 1;
        const float *first = p.part + 2 * (int64_t)h.first_wg * p.slot_rows * (DK + 2);
        const bool many = n > MANY, team = n > MOST;
        const int row = !many ? step * RUN + wave * SP + k : team ? step : step * TEAM + wave;
        // rows of an item's heads stand one head after the other
        const int head_rows = h.rows / C::HEADS;
        const auto place_of = [&](const Request &q, int i) {
            return C::HEADS == 1 ? row_of(p, q, h.hk, h.row0 + i) : row_of(p, q, h.hk * C::HEADS + i / head_rows, h.row0 + i % head_rows);
        };
        if (s_any) {
            bool again = false;
            for (int i = h.first_wg; i <= lo; ++i) again |= p.hdr[i].bad != 0;
            if (again) {
                const int r = p.hdr[lo].r;
                const Request q = uniform(request<C>(p, r));
                const int i0 = row - (many ? 0 : k), i1 = many ? i0 + (!team || wave == 0) : i0 + SP;
                for (int i = i0; i < min(i1, h.rows); ++i)
                    plain_row<X, H, WIN>(p, q, r, C::HEADS == 1 ? h.hk : h.hk * C::HEADS + i / head_rows, place_of(q, i), s_q[wave]);
                continue;
            }
        }
        float m = -INFINITY, l = 0.0f;
        v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
        const bool ok = row < h.rows && k < SP;
        if (many) {
            if (ok) join_parts<16, DK>(p, first, row, d, team ? wave * SP + k : k, team ? RUN : SP, n, m, l, acc);
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
            if (team) {  // then the first wavefront takes the others' sums
                __syncthreads();
                if (lane < Q) {
                    s_acc[wave][lane] = acc;
                    if (lane == 0) {
                        s_tm[wave] = m;
                        s_tl[wave] = l;
                    }
                }
                __syncthreads();
                if (wave > 0) continue;
                float top = m;
#pragma unroll
                for (int i = 1; i < 4; ++i) top = fmaxf(top, s_tm[i]);
                const float base = top == -INFINITY ? 0.0f : top, mine = __builtin_amdgcn_exp2f(m - base);
                l *= mine;
                acc *= mine;
#pragma unroll
                for (int i = 1; i < 4; ++i) {
                    const float a = __builtin_amdgcn_exp2f(s_tm[i] - base);
                    l += a * s_tl[i];
                    acc += a * s_acc[i][lane % Q];
                }
            }
        } else if (ok) {
            join_parts<4, DK>(p, first, row, d, 0, 1, n, m, l, acc);
        }
        if (ok && (k == 0 || !many) && d < p.D) {
            Request q;
            q.first = h.first;
            const Row z = place_of(q, row);
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
            if (u >= base + per_head * head_groups<C>(p)) {
                base += per_head * head_groups<C>(p);
                ++r;
                continue;
            }
            const int hk = (int)divide(u - base, per_head);
            const int64_t rest = u - base - hk * per_head;
            const int tile = line.find(rest), row0 = tile * C::ROWT, n = min(q.n * p.G - row0, C::ROWT);
            const int64_t units = line.of(tile), from = rest - line.before(tile), end = u + units - from;
            if (Blocks<C>(p, q, row0, n).within(from, units) == 0 && end <= h.u1) {
                for (int row = blockIdx.x * 4 + wave; row < C::HEADS * n; row += gridDim.x * 4) {
                    const int head = C::HEADS == 1 ? hk : hk * C::HEADS + row / n, i = C::HEADS == 1 ? row : row % n;
                    plain_row<X, H, WIN>(p, q, r, head, row_of(p, q, head, row0 + i), s_q[wave]);
                }
            }
            u = end;
        }
    }
}
template <int DK, int MT, bool WIN, int HEADS>
hipError_t launch_few(const TreeParams &p, const TreeShape &z, hipStream_t s) {
    hipLaunchKernelGGL((k_few4<DK, MT, WIN, HEADS>), dim3((unsigned)z.wgs), dim3(64 * few_waves(HEADS)), 0, s, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_few_join<DK, Few<DK, MT, WIN, HEADS>>), join_grid(z), dim3(256), 0, s, p);
    return hipGetLastError();
}

template <bool WIN, int HEADS>
hipError_t launch_few_dk(const TreeParams &p, const TreeShape &z, hipStream_t s) {
    if (z.dk == 256) return launch_few<256, 1, WIN, HEADS>(p, z, s);
    if (z.mt == 1)
        return z.dk == 64   ? launch_few<64, 1, WIN, HEADS>(p, z, s)
               : z.dk == 96 ? launch_few<96, 1, WIN, HEADS>(p, z, s)
                            : launch_few<128, 1, WIN, HEADS>(p, z, s);
    return z.dk == 64   ? launch_few<64, 2, WIN, HEADS>(p, z, s)
           : z.dk == 96 ? launch_few<96, 2, WIN, HEADS>(p, z, s)
                        : launch_few<128, 2, WIN, HEADS>(p, z, s);
}

template <bool WIN>
hipError_t launch_q4(const TreeParams &p, const TreeShape &z, hipStream_t s) {
    return !z.few ? launch_dk<BF16, kQ4, WIN>(p, z, s) : z.heads == 8 ? launch_few_dk<WIN, 8>(p, z, s) : z.heads == 4 ? launch_few_dk<WIN, 4>(p, z, s) : launch_few_dk<WIN, 1>(p, z, s);
}

}  // namespace

hipError_t launch_tree_attention_q4(const TreeParams &p, const TreeShape &z, hipStream_t s) { return launch_q4<false>(p, z, s); }
hipError_t launch_window_attention_q4(const TreeParams &p, const TreeShape &z, hipStream_t s) { return launch_q4<true>(p, z, s); }

}  // namespace qmm
