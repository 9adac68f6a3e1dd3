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

// Elements d .. d+7 of a row of n.
template <class T, bool VEC>
__device__ __forceinline__ void load8(const T *row, int d, int n, T (&x)[8]) {
    if (VEC && d + 8 <= n) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) ((v4i *)x)[i] = ((const v4i *)(row + d))[i];
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = d + e < n ? row[d + e] : (T)0.0f;
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
// share step by step.
template <class R, int MT, int RT, bool VEC>
__global__ __launch_bounds__(256) void k_lora_shrink(LoraParams p) {
    typedef typename R::X X;
    typedef typename R::W W;
    typedef typename R::V V;
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
        const W *A = (const W *)p.A + a * p.a_stride;
        for (int step = begin + wave; step < end; step += 4) {
            const int k = 32 * step + 8 * g;
            V w[RT];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const int i = 16 * rt + c;
                W x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = (W)0.0f;
                if (i < p.rank) load8<W, VEC>(A + i * p.lda, k, p.K, x);
                w[rt] = *(V *)x;
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                X x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = (X)0.0f;
                if (id[mt] == a) load8<X, VEC>((const X *)p.X + (int64_t)(t0 + 16 * mt + c) * p.ldx, k, p.K, x);
                V v[R::TERMS];
                if constexpr (R::TERMS == 1) v[0] = *(V *)x;
                else split<R, R::TERMS>(x, v);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int i = 0; i < R::TERMS; ++i) acc[mt][rt] = R::mfma(w[rt], v[i], acc[mt][rt]);
            }
        }
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

// base + s B z for 64 columns a wavefront.  Row i = 4 g + v of product nt is column 16 g
// + 4 nt + v, so that a lane's four products are 16 neighbouring columns of its row.
template <class R, int MT, int RK, bool VEC>
__global__ __launch_bounds__(256) void k_lora_expand(LoraParams p) {
    typedef typename R::X X;
    typedef typename R::W W;
    typedef typename R::V V;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 15, g = lane >> 4;
    const int t0 = blockIdx.x * 16 * MT, n0 = (blockIdx.y * 4 + wave) * 64;
    if (n0 >= p.N) return;
    int id[MT], exponent[MT];
    tile_ids<MT>(p, t0, id);
    V z[MT][RK][R::ZTERMS];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        float x[RK][8];
#pragma unroll
        for (int kk = 0; kk < RK; ++kk)
#pragma unroll
            for (int e = 0; e < 8; ++e) x[kk][e] = 0.0f;
        if (id[mt] >= 0) {
            for (int split = 0; split < p.splits; ++split) {
                const float *from = p.z + ((int64_t)split * p.T + t0 + 16 * mt + c) * p.rp + 8 * g;
#pragma unroll
                for (int kk = 0; kk < RK; ++kk)
                    if (32 * kk + 8 * g < p.rp) {
                        const v4f a = *(const v4f *)(from + 32 * kk), b = *(const v4f *)(from + 32 * kk + 4);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            x[kk][e] += a[e];
                            x[kk][e + 4] += b[e];
                        }
                    }
            }
        }
        exponent[mt] = 0;
        if (sizeof(X) == 2 && sizeof(W) == 2 && std::is_same<W, _Float16>::value) {
            // a power of two takes the row's largest below 2^14: neither fp16 term leaves its range
            uint32_t top = 0;
#pragma unroll
            for (int kk = 0; kk < RK; ++kk)
#pragma unroll
                for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[kk][e]) & 0x7FFFFFFFu);
            top = max(top, (uint32_t)__shfl_xor((int)top, 16));
            top = max(top, (uint32_t)__shfl_xor((int)top, 32));
            exponent[mt] = (int)(top >> 23) - 127 - 13;
#pragma unroll
            for (int kk = 0; kk < RK; ++kk)
#pragma unroll
                for (int e = 0; e < 8; ++e) x[kk][e] = ldexpf(x[kk][e], -exponent[mt]);
        }
#pragma unroll
        for (int kk = 0; kk < RK; ++kk) split<R, R::ZTERMS>(x[kk], z[mt][kk]);
    }
    each_adapter<MT>(id, [&](int a) {
        if (a < 0 && p.base == p.out) return;  // rows without an adapter are there already
        const int col = n0 + 16 * g;
        const bool whole = VEC && col + 16 <= p.N;
        X out[MT][16];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int e = 0; e < 16; ++e) out[mt][e] = (X)0.0f;
            if (id[mt] != a || !p.base) continue;
            const X *from = (const X *)p.base + (int64_t)(t0 + 16 * mt + c) * p.ld_base + col;
            if (whole) {
#pragma unroll
                for (int i = 0; i < (int)sizeof(X); ++i) ((v4i *)out[mt])[i] = ((const v4i *)from)[i];
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (col + e < p.N) out[mt][e] = from[e];
            }
        }
        if (a >= 0) {
            const W *B = (const W *)p.B + a * p.b_stride;
            V w[4][RK];
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
                const int n = n0 + 16 * (c / 4) + 4 * nt + c % 4;
#pragma unroll
                for (int kk = 0; kk < RK; ++kk) {
                    W x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = (W)0.0f;
                    if (n < p.N) load8<W, VEC>(B + n * p.ldb, 32 * kk + 8 * g, p.rank, x);
                    w[nt][kk] = *(V *)x;
                }
            }
            const float s = p.scales ? p.scales[a] : 1.0f;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
                    v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int kk = 0; kk < RK; ++kk)
#pragma unroll
                        for (int i = 0; i < R::ZTERMS; ++i) acc = R::mfma(w[nt][kk], z[mt][kk][i], acc);
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        out[mt][4 * nt + v] = (X)fmaf(s, ldexpf(acc[v], exponent[mt]), (float)out[mt][4 * nt + v]);
                }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            if (id[mt] != a) continue;
            X *to = (X *)p.out + (int64_t)(t0 + 16 * mt + c) * p.ld_out + col;
            if (whole) {
#pragma unroll
                for (int i = 0; i < (int)sizeof(X); ++i) ((v4i *)to)[i] = ((v4i *)out[mt])[i];
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (col + e < p.N) to[e] = out[mt][e];
            }
        }
    });
}

template <class R, int RT>
hipError_t launch_shrink(const LoraParams &p, const LoraShape &z, int slots, hipStream_t s) {
    const dim3 grid((unsigned)ceil_div(p.T, 16 * z.mt), (unsigned)z.splits, (unsigned)slots);
    const bool vec = p.x_vec && p.a_vec;
    if (z.mt == 2) {
        if (vec) hipLaunchKernelGGL((k_lora_shrink<R, 2, RT, true>), grid, dim3(256), 0, s, p);
        else hipLaunchKernelGGL((k_lora_shrink<R, 2, RT, false>), grid, dim3(256), 0, s, p);
    } else {
        if (vec) hipLaunchKernelGGL((k_lora_shrink<R, 1, RT, true>), grid, dim3(256), 0, s, p);
        else hipLaunchKernelGGL((k_lora_shrink<R, 1, RT, false>), grid, dim3(256), 0, s, p);
    }
    return hipGetLastError();
}

template <class R, int RK>
hipError_t launch_expand(const LoraParams &p, const LoraShape &z, int slots, hipStream_t s) {
    const dim3 grid((unsigned)ceil_div(p.T, 16 * z.mt), (unsigned)ceil_div(p.N, 256), (unsigned)slots);
    const bool vec = p.b_vec && p.o_vec;
    if (z.mt == 2) {
        if (vec) hipLaunchKernelGGL((k_lora_expand<R, 2, RK, true>), grid, dim3(256), 0, s, p);
        else hipLaunchKernelGGL((k_lora_expand<R, 2, RK, false>), grid, dim3(256), 0, s, p);
    } else {
        if (vec) hipLaunchKernelGGL((k_lora_expand<R, 1, RK, true>), grid, dim3(256), 0, s, p);
        else hipLaunchKernelGGL((k_lora_expand<R, 1, RK, false>), grid, dim3(256), 0, s, p);
    }
    return hipGetLastError();
}

template <class R>
hipError_t launch_type(const LoraParams &p, const LoraShape &z, hipStream_t s) {
    // tiles of few rows have a grid column for each adapter that their rows can name
    const int slots = z.mt == 2 ? 1 : (int)(p.T < 16 ? p.T : 16);
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
