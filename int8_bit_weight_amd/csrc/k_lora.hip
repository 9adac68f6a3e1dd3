// k_lora.hip -- low-rank adapters of many requests at once on gfx950.
//
//   out[t] = base[t] + s_a B_a (A_a x_t),  a = adapters[t]
//
// Two launches: z = A_a x_t (fp32, in the workspace, in ranges of k), then base + B_a z.
// Rows are taken 16 at a time as the columns of matrix products, whose other operand is
// the adapter's matrix; a tile is gone through once for each adapter that its rows
// name, and only those rows' columns are used.  A column of a product depends on its own
// row alone, so NaN and infinities stay where they are.  Both matrices go straight
// from memory to the operands: each is read once by a workgroup.
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
// their first rows: each(a) for those of this workgroup, every gridDim.z-th.
template <int MT, class F>
__device__ __forceinline__ void each_adapter(const int (&id)[MT], F each) {
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
        if (slot % gridDim.z == blockIdx.z) each(a);
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
    each_adapter<MT>(id, [&](int a) {
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
    each_adapter<MT>(id, [&](int a) {
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

template <class R, int RT>
hipError_t launch_shrink(const LoraParams &p, const LoraShape &z, int slots, hipStream_t s) {
    const dim3 grid((unsigned)ceil_div(p.T, 16 * z.mt), (unsigned)z.splits, (unsigned)slots);
    if (z.mt > 1) hipLaunchKernelGGL((k_lora_shrink<R, 2, RT>), grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL((k_lora_shrink<R, 1, RT>), grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

template <class R, int RK>
hipError_t launch_expand(const LoraParams &p, const LoraShape &z, int slots, hipStream_t s) {
    const int64_t tiles = ceil_div(p.T, 16 * z.mt), chunks = ceil_div(p.N, 256);
    // as many workgroups as are resident, four to a CU, and then as many columns for each
    const int64_t fit = tiles < 1024 ? 1024 / tiles : 1;
    const int64_t columns = z.mt == 1 ? chunks : ceil_div(chunks, ceil_div(chunks, fit));
    const dim3 grid((unsigned)tiles, (unsigned)columns, (unsigned)slots);
    if (z.mt > 1) hipLaunchKernelGGL((k_lora_expand<R, 2, RK>), grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL((k_lora_expand<R, 1, RK>), grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

template <class R>
hipError_t launch_type(const LoraParams &p, const LoraShape &z, hipStream_t s) {
    // tiles of few rows have a grid column for each adapter that their rows can name; of
    // many rows, which come in runs, for the two where one run meets the next
    const int slots = z.mt > 1 ? 2 : (int)(p.T < 16 ? p.T : 16);
    hipError_t e = p.rp <= 16   ? launch_shrink<R, 1>(p, z, slots, s)
                   : p.rp <= 32 ? launch_shrink<R, 2>(p, z, slots, s)
                   : p.rp <= 64 ? launch_shrink<R, 4>(p, z, slots, s)
                                : launch_shrink<R, 8>(p, z, slots, s);
    if (e != hipSuccess) return e;
    return p.rp <= 32   ? launch_expand<R, 1>(p, z, slots, s)
           : p.rp <= 64 ? launch_expand<R, 2>(p, z, slots, s)
                        : launch_expand<R, 4>(p, z, slots, s);
}

}  // namespace

hipError_t launch_lora(const LoraParams &p, const LoraShape &z, qmm_dtype xt, hipStream_t s) {
    return xt == QMM_T_F32   ? launch_type<RowsF32>(p, z, s)
           : xt == QMM_T_F16 ? launch_type<RowsF16>(p, z, s)
                             : launch_type<RowsBF16>(p, z, s);
}

}  // namespace qmm
