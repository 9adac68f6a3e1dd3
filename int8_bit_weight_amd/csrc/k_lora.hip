// k_lora.hip -- low-rank adapters of many requests at once on gfx950.
//
//   out[t] = base[t] + s_a B_a (A_a x_t),  a = adapters[t]
//
// z = A_a x_t (fp32, in the workspace, in ranges of k), then base + B_a z.
// Rows are taken 16 at a time as the columns of matrix products, whose other operand is
// the adapter's matrix; a tile is gone through once for each adapter that its rows
// name, and only those rows' columns are used.  A column of a product depends on its own
// row alone, so NaN and infinities stay where they are.
//
// Few rows: two launches, 16 rows a workgroup, both matrices straight from memory to the
// operands; latency bounds them (one row, 1024 -> 2048, rank 16, bf16: 3.6 + 3.8 us).
// Many rows: 64 a workgroup, which go through LDS with the adapter's matrix, and
// the ranges of z are added up by a launch of their own, once instead of in
// every tile of columns (4001 rows, 4096 -> 14336, rank 64, bf16: 25 + 5 + 82 us; base and
// output alone are 230 MB, 45 us).
#include <type_traits>

#include "token_internal.h"

namespace qmm {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

// Element types: X of the rows, W of the adapters; TERMS operands make up a row's
// values in the first product, ZTERMS those of z in the second.
struct RowsF16 {
    typedef _Float16 X;
    typedef _Float16 W;
    typedef v8h V;
    static constexpr int TERMS = 1, ZTERMS = 2;
    static __device__ __forceinline__ v4f mfma(V a, V b, v4f c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};
struct RowsBF16 {
    typedef __bf16 X;
    typedef __bf16 W;
    typedef v8bf V;
    static constexpr int TERMS = 1, ZTERMS = 2;
    static __device__ __forceinline__ v4f mfma(V a, V b, v4f c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};
struct RowsF32 : RowsBF16 {
    typedef float X;
    static constexpr int TERMS = 3, ZTERMS = 3;
};

// fp32 values as N operands that add up to them: N - 1 cut to W's bits, the last rounded.
template <class R, int N>
__device__ __forceinline__ void split(const float (&x)[8], typename R::V (&out)[N]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float rest = x[e];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            typename R::W h = (typename R::W)rest;
            if (i < N - 1 && sizeof(typename R::X) != 2) {
                // bf16: cut, so that the rest is exact and no value rounds up to infinity
                const uint32_t b = __float_as_uint(rest);
                if (rest == rest) h = (typename R::W)__uint_as_float(b & 0xFFFF0000u);
            }
            out[i][e] = h;
            rest = fabsf(rest) < INFINITY ? rest - (float)h : 0.0f;
        }
    }
}

// 16 bytes at any element's address.
typedef int v4iu __attribute__((ext_vector_type(4), aligned(2)));

// Elements d .. d+7 of a row of n, zeros past it.  `room` elements can be read from the
// row's start on: where other rows follow, they are read and put out, which costs less
// than element by element.
template <class T>
__device__ __forceinline__ void load8(const T *row, int d, int n, int64_t room, T (&x)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (T)0.0f;
    if (d < n) {
        if (d + 8 <= room) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) / 2; ++i) ((v4i *)x)[i] = ((const v4iu *)(row + d))[i];
            if (d + 8 > n) {
#pragma unroll
                for (int e = 1; e < 8; ++e)
                    if (d + e >= n) x[e] = (T)0.0f;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (d + e < n) x[e] = row[d + e];
        }
    }
}
// The same inside a row.
template <class T>
__device__ __forceinline__ void load8(const T *at, bool have, T (&x)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (T)0.0f;
    if (have) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) ((v4i *)x)[i] = ((const v4iu *)at)[i];
    }
}

// Goes through the adapters that a tile's rows name (ids < -1: no row), in the order of
// their first rows: each(a) for every slots-th from `mine` on.
template <int MT, class F>
__device__ __forceinline__ void each_adapter(const int (&id)[MT], int mine, int slots, F each) {
    uint32_t left[MT], any = 0;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) any |= left[mt] = (uint32_t)__ballot(id[mt] >= -1) & 0xFFFF;
    for (int slot = 0; any; ++slot) {
        int a = 0;
        bool found = false;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
            if (!found && left[mt]) {
                a = __builtin_amdgcn_readlane(id[mt], __builtin_ctz(left[mt]));
                found = true;
            }
        any = 0;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) any |= left[mt] &= ~(uint32_t)__ballot(id[mt] == a);
        if (slot % slots == mine) each(a);
    }
}

template <int MT>
__device__ __forceinline__ void tile_ids(const LoraParams &p, int t0, int (&id)[MT]) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int t = t0 + 16 * mt + (threadIdx.x & 15);
        id[mt] = -2;
        if (t < p.T) {
            const int a = p.adapters[t];
            id[mt] = a >= 0 && a < p.n_adapters ? a : -1;
        }
    }
}

// z[split][t][i] = sum of x[t,k] A[a,i,k] over a range of k, which the four wavefronts
// share step by step, STEPS of each on their way at a time.
template <class R, int MT, int RT>
__global__ __launch_bounds__(256) void k_lora_shrink(LoraParams p) {
    typedef typename R::X X;
    typedef typename R::W W;
    typedef typename R::V V;
    constexpr int STEPS = RT <= 2 ? 4 : 2;
    __shared__ v4f s_sum[4][MT * RT][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 15, g = lane >> 4;
    const int t0 = blockIdx.x * 16 * MT;
    const int begin = blockIdx.y * p.per, end = min(begin + p.per, (p.K + 31) / 32);
    int id[MT];
    tile_ids<MT>(p, t0, id);
    each_adapter<MT>(id, blockIdx.z, gridDim.z, [&](int a) {
        if (a < 0) return;
        const v4f zero = {0.0f, 0.0f, 0.0f, 0.0f};
        v4f acc[MT][RT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) acc[mt][rt] = zero;
        const W *const A = (const W *)p.A + a * p.a_stride + c * p.lda;
        const X *const Xr = (const X *)p.X + (int64_t)(t0 + c) * p.ldx;
        const auto steps = [&](auto COUNT, auto WHOLE, int s0) __attribute__((always_inline)) {
            constexpr int N = decltype(COUNT)::value;
            W w[N][RT][8];
            X x[N][MT][8];
#pragma unroll
            for (int s = 0; s < N; ++s) {
                const int k = 32 * (s0 + 4 * s) + 8 * g;
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    const bool have = 16 * rt + c < p.rank;
                    const W *row = A + 16 * rt * p.lda;
                    if constexpr (decltype(WHOLE)::value) load8<W>(row + k, have, w[s][rt]);
                    else load8<W>(row, k, have ? p.K : 0, (p.rank - 1 - 16 * rt - c) * p.lda + p.K, w[s][rt]);
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const X *row = Xr + 16 * mt * p.ldx;
                    if constexpr (decltype(WHOLE)::value) load8<X>(row + k, id[mt] == a, x[s][mt]);
                    else load8<X>(row, k, id[mt] == a ? p.K : 0, (p.T - 1 - t0 - 16 * mt - c) * p.ldx + p.K, x[s][mt]);
                }
            }
#pragma unroll
            for (int s = 0; s < N; ++s)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    V v[R::TERMS];
                    if constexpr (R::TERMS == 1) v[0] = *(V *)x[s][mt];
                    else split<R, R::TERMS>(x[s][mt], v);
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                        for (int i = 0; i < R::TERMS; ++i) acc[mt][rt] = R::mfma(*(V *)w[s][rt], v[i], acc[mt][rt]);
                }
        };
        const std::integral_constant<int, STEPS> many;
        const std::integral_constant<int, 1> one;
        const int whole = min(end, p.K / 32);
        int s0 = begin + wave;
        for (; s0 + 4 * (STEPS - 1) < whole; s0 += 4 * STEPS) steps(many, std::true_type(), s0);
        for (; s0 < whole; s0 += 4) steps(one, std::true_type(), s0);
        if (s0 < end) steps(one, std::false_type(), s0);  // the last step, which K ends in
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) s_sum[wave][mt * RT + rt][lane] = acc[mt][rt];
        __syncthreads();
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const int i = mt * RT + rt;
                if (i % 4 != wave || id[mt] != a || 16 * rt >= p.rp) continue;
                const v4f z = (s_sum[0][i][lane] + s_sum[1][i][lane]) + (s_sum[2][i][lane] + s_sum[3][i][lane]);
                *(v4f *)(p.z + ((int64_t)blockIdx.y * p.T + t0 + 16 * mt + c) * p.rp + 16 * rt + 4 * g) = z;
            }
        __syncthreads();
    });
}

// The rows' sums over the ranges of k, to LDS, eight ranges on their way at a time.  Rows
// without an adapter get whatever the workspace holds: no column of theirs is used.
template <int ROWS, int STRIDE>
__device__ __forceinline__ void sum_z(const LoraParams &p, int t0, float *s_z) {
    const int quads = p.rp / 4;
    const int64_t stride = (int64_t)p.T * p.rp;
    for (int i = threadIdx.x; i < ROWS * quads; i += 256) {
        const int row = i / quads, q = i % quads;
        const float *from = p.z + (int64_t)min(t0 + row, p.T - 1) * p.rp + 4 * q;
        v4f sum = *(const v4f *)from;
        for (int s0 = 1; s0 < p.splits; s0 += 8) {
            v4f a[8];
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                a[s] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
                if (s0 + s < p.splits) a[s] = *(const v4f *)(from + (s0 + s) * stride);
            }
#pragma unroll
            for (int s = 0; s < 8; ++s) sum += a[s];
        }
        *(v4f *)(s_z + row * STRIDE + 4 * q) = sum;
    }
}

// The terms of a row's z, which four lanes hold, and the power of two that was taken out of it.
template <class R, int RK>
__device__ __forceinline__ int z_terms(float (&x)[RK][8], typename R::V (&z)[RK][R::ZTERMS]) {
    int exponent = 0;
    if (std::is_same<typename R::W, _Float16>::value) {
        // the row's largest goes below 2^14: neither fp16 term leaves its range
        uint32_t top = 0;
#pragma unroll
        for (int kk = 0; kk < RK; ++kk)
#pragma unroll
            for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[kk][e]) & 0x7FFFFFFFu);
        top = max(top, (uint32_t)__shfl_xor((int)top, 16));
        top = max(top, (uint32_t)__shfl_xor((int)top, 32));
        exponent = (int)(top >> 23) - 127 - 13;
#pragma unroll
        for (int kk = 0; kk < RK; ++kk)
#pragma unroll
            for (int e = 0; e < 8; ++e) x[kk][e] = ldexpf(x[kk][e], -exponent);
    }
#pragma unroll
    for (int kk = 0; kk < RK; ++kk) split<R, R::ZTERMS>(x[kk], z[kk]);
    return exponent;
}

// base + s B z, 64 columns of a wavefront at a time.  Which column a product's row is is
// free: row 4 g + v of product nt is column LANE g + 4 (nt % PER) + v of the nt / PER-th
// LANE * 4, so that PER products are 16 bytes of a lane and 64 of a row.  z stays
// in registers while a wavefront goes through its columns.
template <class R, int MT, int RK>
__global__ __launch_bounds__(256) void k_lora_expand(LoraParams p) {
    typedef typename R::X X;
    typedef typename R::W W;
    typedef typename R::V V;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 15, g = lane >> 4;
    constexpr int LANE = 16 / sizeof(X), PER = LANE / 4, STRIDE = 32 * RK + 4;
    __shared__ __align__(16) float s_z[16 * MT * STRIDE];
    const int t0 = blockIdx.x * 16 * MT, n_first = (blockIdx.y * 4 + wave) * 64;
    int id[MT], exponent[MT];
    tile_ids<MT>(p, t0, id);
    sum_z<16 * MT, STRIDE>(p, t0, s_z);
    __syncthreads();
    V z[MT][RK][R::ZTERMS];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        float x[RK][8];
#pragma unroll
        for (int kk = 0; kk < RK; ++kk) {
            const bool have = 32 * kk + 8 * g < p.rp;
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                v4f q = {0.0f, 0.0f, 0.0f, 0.0f};
                if (have) q = *(const v4f *)(s_z + (16 * mt + c) * STRIDE + 32 * kk + 8 * g + e);
#pragma unroll
                for (int v = 0; v < 4; ++v) x[kk][e + v] = q[v];
            }
        }
        exponent[mt] = z_terms<R, RK>(x, z[mt]);
    }
    const int at = n_first + LANE * (c / 4) + c % 4;  // the lane's column of product 0
    const auto column = [](int nt) { return 4 * LANE * (nt / PER) + 4 * (nt % PER); };
    each_adapter<MT>(id, blockIdx.z, gridDim.z, [&](int a) {
        if (a < 0 && p.base == p.out) return;  // rows without an adapter are there already
        const float s = a >= 0 && p.scales ? p.scales[a] : 1.0f;
        float factor[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) factor[mt] = ldexpf(s, exponent[mt]);
        const W *B = (const W *)p.B + (a < 0 ? 0 : a * p.b_stride) + at * p.ldb;
        const X *from = (const X *)p.base + (int64_t)(t0 + c) * p.ld_base + n_first + LANE * g;
        X *to = (X *)p.out + (int64_t)(t0 + c) * p.ld_out + n_first + LANE * g;
        // FAST: all 64 columns are there and the rank is in whole eights
        const auto columns = [&](auto FAST, int n0) __attribute__((always_inline)) {
            constexpr bool fast = decltype(FAST)::value;
            const int col = n0 + LANE * g;
            X out[MT][16 / LANE][LANE];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const X *row = from + 16 * mt * p.ld_base;
#pragma unroll
                for (int i = 0; i < 16 / LANE; ++i) {
                    const bool mine = id[mt] == a && p.base;
                    if (fast) {
                        *(v4i *)out[mt][i] = v4i{0, 0, 0, 0};
                        if (mine) *(v4i *)out[mt][i] = *(const v4iu *)(row + 4 * LANE * i);
                    } else {
#pragma unroll
                        for (int e = 0; e < LANE; ++e) out[mt][i][e] = mine && col + 4 * LANE * i + e < p.N ? row[4 * LANE * i + e] : (X)0.0f;
                    }
                }
            }
            if (a >= 0) {
                W w[4][RK][8];
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
#pragma unroll
                    for (int kk = 0; kk < RK; ++kk) {
                        const int k = 32 * kk + 8 * g, n = at + (n0 - n_first) + column(nt);
                        const W *row = B + column(nt) * p.ldb;
                        if constexpr (fast) load8<W>(row + k, k < p.rank, w[nt][kk]);
                        else load8<W>(row, k, n < p.N ? p.rank : 0, (p.N - 1 - n) * p.ldb + p.rank, w[nt][kk]);
                    }
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int nt = 0; nt < 4; ++nt) {
                        v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int kk = 0; kk < RK; ++kk)
#pragma unroll
                            for (int i = 0; i < R::ZTERMS; ++i) acc = R::mfma(*(V *)w[nt][kk], z[mt][kk][i], acc);
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            X &y = out[mt][nt / PER][4 * (nt % PER) + v];
                            y = (X)fmaf(factor[mt], acc[v], (float)y);
                        }
                    }
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                if (id[mt] != a) continue;
                X *row = to + 16 * mt * p.ld_out;
#pragma unroll
                for (int i = 0; i < 16 / LANE; ++i) {
                    if (fast) {
                        *(v4iu *)(row + 4 * LANE * i) = *(v4i *)out[mt][i];
                    } else {
#pragma unroll
                        for (int e = 0; e < LANE; ++e)
                            if (col + 4 * LANE * i + e < p.N) row[4 * LANE * i + e] = out[mt][i][e];
                    }
                }
            }
        };
        const int step = gridDim.y * 256;
        for (int n0 = n_first; n0 < p.N; n0 += step, B += step * p.ldb, from += step, to += step) {
            if (n0 + 64 <= p.N && p.rank % 8 == 0) columns(std::true_type(), n0);
            else columns(std::false_type(), n0);
        }
    });
}

// The tile of a workgroup of a grid whose x is a whole number of eights: neighbouring
// tiles, whose rows mostly name one adapter, go to one XCD, whose L2 then holds its matrices.
__device__ __forceinline__ int near_tile() { return (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3); }

// The same for many rows, 64 of a workgroup and 16 of a wavefront: both operands go
// through LDS, 64 k at a time.  Straight from memory to the operands neighbouring lanes
// read different rows, 16 bytes of each, which takes a wavefront's load four times as long
// as 1 KB in a row; and a tile's matrix is read once for four tiles of rows.
template <class R, int RT>
__global__ __launch_bounds__(256) void k_lora_shrink_many(LoraParams p) {
    typedef typename R::X X;
    typedef typename R::W W;
    typedef typename R::V V;
    constexpr int KT = 64, P = KT / 8, NX = 64 * P / 256, NA = (16 * RT * P + 255) / 256;  // pieces of a row; of X and A for a thread
    __shared__ X s_x[2][64][P][8];
    __shared__ W s_a[2][16 * RT][P][8];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), c = lane & 15, g = lane >> 4;
    const int t0 = near_tile() * 64;
    if (t0 >= p.T) return;
    const int begin = blockIdx.z * p.per * 32, end = min(begin + p.per * 32, p.K);
    int id[4];
    tile_ids<4>(p, t0, id);
    each_adapter<4>(id, blockIdx.y, gridDim.y, [&](int a) {
        if (a < 0) return;
        const W *const A = (const W *)p.A + a * p.a_stride;
        W wa[NA][8];
        X xa[NX][8];
        const auto load = [&](int k0) {
#pragma unroll
            for (int i = 0; i < NX; ++i) {
                const int row = (tid + 256 * i) / P, t = t0 + row, k = k0 + 8 * (tid % P);
                load8<X>((const X *)p.X + (int64_t)t * p.ldx, k, t < p.T ? end : 0, (p.T - 1 - t) * p.ldx + p.K, xa[i]);
            }
#pragma unroll
            for (int i = 0; i < NA; ++i) {
                const int row = (tid + 256 * i) / P, k = k0 + 8 * (tid % P);
                load8<W>(A + row * p.lda, k, row < p.rank ? end : 0, (p.rank - 1 - row) * p.lda + p.K, wa[i]);
            }
        };
        const auto store = [&](int buf) {
#pragma unroll
            for (int i = 0; i < NX; ++i) {
                const int row = (tid + 256 * i) / P, at = (tid % P) ^ (row & (P - 1));
#pragma unroll
                for (int e = 0; e < (int)sizeof(X) / 2; ++e) ((v4i *)s_x[buf][row][at])[e] = ((v4i *)xa[i])[e];
            }
#pragma unroll
            for (int i = 0; i < NA; ++i) {
                const int row = (tid + 256 * i) / P;
                if (row < 16 * RT) *(v4i *)s_a[buf][row][(tid % P) ^ (row & (P - 1))] = *(v4i *)wa[i];
            }
        };
        v4f acc[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) acc[rt] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        __syncthreads();  // an earlier adapter's operands have been read
        load(begin);
        store(0);
        for (int k0 = begin, buf = 0; k0 < end; k0 += KT, buf ^= 1) {
            __syncthreads();
            if (k0 + KT < end) load(k0 + KT);
#pragma unroll
            for (int kk = 0; kk < KT / 32; ++kk) {
                const int piece = (4 * kk + g) ^ (c & (P - 1));
                V v[R::TERMS];
                X x[8];
#pragma unroll
                for (int e = 0; e < (int)sizeof(X) / 2; ++e) ((v4i *)x)[e] = ((v4i *)s_x[buf][16 * wave + c][piece])[e];
                if constexpr (R::TERMS == 1) v[0] = *(V *)x;
                else split<R, R::TERMS>(x, v);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    const V w = *(const V *)s_a[buf][16 * rt + c][piece];
#pragma unroll
                    for (int i = 0; i < R::TERMS; ++i) acc[rt] = R::mfma(w, v[i], acc[rt]);
                }
            }
            if (k0 + KT < end) store(buf ^ 1);
        }
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
            if (mt == wave && id[mt] == a)
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
                    if (16 * rt < p.rp)
                        *(v4f *)(p.z + ((int64_t)blockIdx.z * p.T + t0 + 16 * mt + c) * p.rp + 16 * rt + 4 * g) = acc[rt];
    });
}

// The sums over the ranges of k, in the first range's place: every workgroup of the next
// launch would add them up again.
__global__ __launch_bounds__(256) void k_lora_sum(LoraParams p) {
    const int64_t n = (int64_t)p.T * p.rp / 4, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    v4f *const z = (v4f *)p.z + i;
    v4f part[16], sum = *z;
#pragma unroll
    for (int s = 1; s < 16; ++s)
        if (s < p.splits) part[s] = z[s * n];
#pragma unroll
    for (int s = 1; s < 16; ++s)
        if (s < p.splits) sum += part[s];
    *z = sum;
}

// base + s B z for many rows: 64 of a workgroup and 16 of a wavefront, as the rows 4 g + v
// of the products, and 128 columns at a time, of which a lane has the eight from 8 c on: a
// quarter wavefront reads and writes 256 bytes of a row.  B goes through LDS.
template <class R, int RK>
__global__ __launch_bounds__(256) void k_lora_expand_many(LoraParams p) {
    typedef typename R::X X;
    typedef typename R::W W;
    typedef typename R::V V;
    constexpr int STRIDE = 32 * RK + 4, P = 4 * RK, COLS = 128, NB = COLS * P / 256;  // pieces of a row; of B for a thread
    __shared__ __align__(16) float s_z[64 * STRIDE];
    __shared__ W s_b[2][COLS][P][8];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), c = lane & 15, g = lane >> 4;
    const int t0 = near_tile() * 64;
    if (t0 >= p.T) return;
    int id[4], mine = -2;
    tile_ids<4>(p, t0, id);
    if (blockIdx.y > 0) {  // most tiles' rows name one adapter: nothing is left for the others
        const int a = __builtin_amdgcn_readfirstlane(id[0]);
        bool other = false;
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) other |= id[mt] >= -1 && id[mt] != a;
        if (!__any(other)) return;
    }
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
        if (mt == wave) mine = id[mt];  // of row c of the wavefront's
    sum_z<64, STRIDE>(p, t0, s_z);
    __syncthreads();
    float x[RK][8];
#pragma unroll
    for (int kk = 0; kk < RK; ++kk) {
        const bool have = 32 * kk + 8 * g < p.rp;
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
            v4f q = {0.0f, 0.0f, 0.0f, 0.0f};
            if (have) q = *(const v4f *)(s_z + (16 * wave + c) * STRIDE + 32 * kk + 8 * g + e);
#pragma unroll
            for (int v = 0; v < 4; ++v) x[kk][e + v] = q[v];
        }
    }
    V z[RK][R::ZTERMS];
    const int exponent = z_terms<R, RK>(x, z);
    int exponents[4];  // of rows 4 g + v
#pragma unroll
    for (int v = 0; v < 4; ++v) exponents[v] = __shfl(exponent, 4 * g + v);
    const int columns = (p.N + COLS - 1) / COLS;
    each_adapter<4>(id, blockIdx.y, gridDim.y, [&](int a) {
        const uint32_t rows = (uint32_t)__ballot(mine == a) & 0xFFFF;  // of the wavefront's 16
        bool has[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) has[v] = rows >> (4 * g + v) & 1;
        if (a < 0 && p.base == p.out) return;  // rows without an adapter are there already
        const float s = a >= 0 && p.scales ? p.scales[a] : 1.0f;
        float factor[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) factor[v] = ldexpf(s, exponents[v]);
        const W *const B = (const W *)p.B + (a < 0 ? 0 : a * p.b_stride);
        W wb[NB][8];
        const auto load = [&](int n0) {
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int n = n0 + (tid + 256 * i) / P;
                load8<W>(B + n * p.ldb, 8 * (tid % P), n < p.N ? p.rank : 0, (p.N - 1 - n) * p.ldb + p.rank, wb[i]);
            }
        };
        const auto store = [&](int buf) {
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int row = (tid + 256 * i) / P;
                *(v4i *)s_b[buf][row][(tid % P) ^ (row / 8 & (P - 1))] = *(v4i *)wb[i];
            }
        };
        const int first = blockIdx.z, step = gridDim.z;
        __syncthreads();  // an earlier adapter's operands have been read
        if (a >= 0) {
            load(first * COLS);
            store(0);
        }
        for (int i = first, buf = 0; i < columns; i += step, buf ^= 1) {
            const int col = i * COLS + 8 * c;
            const bool whole = col + 8 <= p.N;
            X out[4][8];
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const X *from = (const X *)p.base + (int64_t)(t0 + 16 * wave + 4 * g + v) * p.ld_base + col;
#pragma unroll
                for (int e = 0; e < 8; ++e) out[v][e] = (X)0.0f;
                if (has[v] && p.base) {
                    if (whole) {
#pragma unroll
                        for (int e = 0; e < (int)sizeof(X) / 2; ++e) ((v4i *)out[v])[e] = ((const v4iu *)from)[e];
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (col + e < p.N) out[v][e] = from[e];
                    }
                }
            }
            if (a >= 0) {
                __syncthreads();
                if (i + step < columns) load((i + step) * COLS);
                if (rows) {
#pragma unroll
                    for (int nt = 0; nt < 8; ++nt) {
                        v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int kk = 0; kk < RK; ++kk) {
                            const V w = *(const V *)s_b[buf][8 * c + nt][(4 * kk + g) ^ (c & (P - 1))];
#pragma unroll
                            for (int j = 0; j < R::ZTERMS; ++j) acc = R::mfma(z[kk][j], w, acc);
                        }
#pragma unroll
                        for (int v = 0; v < 4; ++v) out[v][nt] = (X)fmaf(factor[v], acc[v], (float)out[v][nt]);
                    }
                }
                if (i + step < columns) store(buf ^ 1);
            }
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                X *to = (X *)p.out + (int64_t)(t0 + 16 * wave + 4 * g + v) * p.ld_out + col;
                if (!has[v]) continue;
                if (whole) {
#pragma unroll
                    for (int e = 0; e < (int)sizeof(X) / 2; ++e) ((v4iu *)to)[e] = ((v4i *)out[v])[e];
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (col + e < p.N) to[e] = out[v][e];
                }
            }
        }
    });
}

template <class R, int RT>
hipError_t launch_shrink(const LoraParams &p, const LoraShape &z, int slots, hipStream_t s) {
    const int64_t tiles = ceil_div(p.T, z.rows);
    if (z.rows == 64)
        hipLaunchKernelGGL((k_lora_shrink_many<R, RT>), dim3((unsigned)round_up(tiles, 8), (unsigned)slots, (unsigned)z.splits), dim3(256), 0, s, p);
    else
        hipLaunchKernelGGL((k_lora_shrink<R, 1, RT>), dim3((unsigned)tiles, (unsigned)z.splits, (unsigned)slots), dim3(256), 0, s, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || z.rows != 64 || z.splits == 1) return e;
    hipLaunchKernelGGL(k_lora_sum, dim3((unsigned)ceil_div((int64_t)p.T * p.rp / 4, 256)), dim3(256), 0, s, p);
    return hipGetLastError();
}

constexpr int64_t kMost = 32768;  // workgroups in a grid's second and third dimension; they go on where columns are left

template <class R, int RK>
hipError_t launch_expand(const LoraParams &p, const LoraShape &z, int slots, hipStream_t s) {
    const int64_t tiles = ceil_div(p.T, z.rows);
    if (z.rows == 64) {
        // short workgroups: those of the few tiles whose rows name two adapters end last
        const int64_t columns = ceil_div(p.N, 128 * 4), most = columns < kMost ? columns : kMost;
        hipLaunchKernelGGL((k_lora_expand_many<R, RK>), dim3((unsigned)round_up(tiles, 8), (unsigned)slots, (unsigned)most), dim3(256), 0, s, p);
    } else {
        const int64_t columns = ceil_div(p.N, 256), most = columns < kMost ? columns : kMost;
        hipLaunchKernelGGL((k_lora_expand<R, 1, RK>), dim3((unsigned)tiles, (unsigned)most, (unsigned)slots), dim3(256), 0, s, p);
    }
    return hipGetLastError();
}

template <class R>
hipError_t launch_type(const LoraParams &p, const LoraShape &z, hipStream_t s) {
    // tiles of 16 rows have a grid column for each adapter that their rows can name; of 64
    // rows, which come in runs, for the two where one run meets the next
    const int slots = z.rows == 64 ? 2 : (int)(p.T < 16 ? p.T : 16);
    hipError_t e = p.rp <= 16   ? launch_shrink<R, 1>(p, z, slots, s)
                   : p.rp <= 32 ? launch_shrink<R, 2>(p, z, slots, s)
                   : p.rp <= 64 ? launch_shrink<R, 4>(p, z, slots, s)
                                : launch_shrink<R, 8>(p, z, slots, s);
    if (e != hipSuccess) return e;
    LoraParams q = p;
    if (z.rows == 64) q.splits = 1;
    return p.rp <= 32   ? launch_expand<R, 1>(q, z, slots, s)
           : p.rp <= 64 ? launch_expand<R, 2>(q, z, slots, s)
                        : launch_expand<R, 4>(q, z, slots, s);
}

}  // namespace

hipError_t launch_lora(const LoraParams &p, const LoraShape &z, qmm_dtype xt, hipStream_t s) {
    return xt == QMM_T_F32   ? launch_type<RowsF32>(p, z, s)
           : xt == QMM_T_F16 ? launch_type<RowsF16>(p, z, s)
                             : launch_type<RowsBF16>(p, z, s);
}

}  // namespace qmm
