// k_q4_group.hip -- 4-bit weights with group scales, W = (q - z) * s, on gfx950.
//
//   Y[m,n] = sum_g s[n,g] * ( sum_{k in g} (16 + q[n,k]) * x[m,k]
//                           - (16 + z[n,g]) * sum_{k in g} x[m,k] )
//
// A code becomes a matrix operand as 16 + q: those sixteen integers share one
// exponent, so the code is a field of the mantissa and two codes take one
// shift and one and-or, with no conversion (128 + q, the form with the code
// in the lowest bits, would cost bf16 three more bits to cancellation).  The
// products are exact in fp32; the group's sum of x for the (16 + z) term
// comes from a second MFMA against ones, over the same operand.
#include "serve_internal.h"

namespace qmm {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

// ------------------------------------------------------------------ repack ---

// One thread per (record, lane chunk): four code words.
__global__ __launch_bounds__(256) void k_q4g_codes(const uint8_t *codes, int64_t ldc, Q4gLayout L, uint8_t *packed) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= L.NS * L.NQ * 64) return;
    const int lane = (int)(i & 63);
    const int64_t rec = i >> 6, strip = rec / L.NQ, q = rec % L.NQ;
    const int64_t n = strip * 16 + (lane & 15);
    v4i out = {0, 0, 0, 0};
    if (n < L.N) {
        const uint8_t *row = codes + n * ldc;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int64_t k0 = q * 128 + b * 32 + (lane >> 4) * 8;
            uint32_t w = 0;
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const int64_t k = k0 + 2 * p;
                if (k < L.K) {
                    const uint32_t c = row[k >> 1];
                    w |= (c & 15u) << (4 * p);
                    if (k + 1 < L.K) w |= (c >> 4) << (16 + 4 * p);
                }
            }
            out[b] = (int)w;
        }
    }
    *(v4i *)(packed + i * 16) = out;
}

// One thread per group word.
template <bool BF16>
__global__ __launch_bounds__(256) void k_q4g_words(const uint16_t *scales, int64_t lds, const uint8_t *zeros,
                                                   int64_t ldz, int64_t group, Q4gLayout L, uint32_t *words) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t per_strip = group < 128 ? L.NQ * L.gpr : L.NG;
    if (i >= L.NS * per_strip * 16) return;
    const int64_t strip = i / (per_strip * 16), r = i % (per_strip * 16);
    int64_t g;
    int c;
    if (group < 128) {
        const int64_t q = r / (16 * L.gpr), rr = r % (16 * L.gpr);
        c = (int)(rr / L.gpr);
        g = q * L.gpr + rr % L.gpr;
    } else {
        g = r / 16;
        c = (int)(r & 15);
    }
    const int64_t n = strip * 16 + c;
    uint32_t w = 0;
    if (n < L.N && g < L.NG) {
        const uint16_t h = scales[n * lds + g];
        const float s = BF16 ? __uint_as_float((uint32_t)h << 16) : (float)__builtin_bit_cast(_Float16, h);
        const uint32_t z = zeros ? zeros[n * ldz + g] & 15u : 8u;
        w = (__float_as_uint(s) & ~15u) | z;
    }
    words[i] = w;
}

// ----------------------------------------------------------------- product ---

// Element types: the operand vector, 16 + q in it, and how an activation octet
// becomes TERMS operands that add up to it.
struct F16 {
    typedef _Float16 T;
    typedef v8h V;
    static constexpr int kTerms = 1;
    static constexpr int kShift = 6;  // mantissa bit of the code's lowest bit
    static constexpr uint32_t kBase = 0x4C004C00u, kMask = 0x03C003C0u, kOnes = 0x3C003C00u;
    static __device__ __forceinline__ v4f mfma(V a, V b, v4f c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ void split(const T (&x)[8], V (&a)[1]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) a[0][e] = x[e];
    }
    static __device__ __forceinline__ T from(float v) { return (T)v; }
};
struct BF16 {
    typedef __bf16 T;
    typedef v8bf V;
    static constexpr int kTerms = 1;
    static constexpr int kShift = 3;
    static constexpr uint32_t kBase = 0x41804180u, kMask = 0x00780078u, kOnes = 0x3F803F80u;
    static __device__ __forceinline__ v4f mfma(V a, V b, v4f c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ void split(const T (&x)[8], V (&a)[1]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) a[0][e] = x[e];
    }
    static __device__ __forceinline__ T from(float v) { return (T)v; }
};
// fp32 activations as three bf16 terms: 24 significand bits, the sum is exact.
struct F32 : BF16 {
    typedef float T;
    static constexpr int kTerms = 3;
    static __device__ __forceinline__ void split(const T (&x)[8], V (&a)[3]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            a[0][e] = (__bf16)x[e];
            const float r1 = x[e] - (float)a[0][e];
            a[1][e] = (__bf16)r1;
            a[2][e] = (__bf16)(r1 - (float)a[1][e]);
        }
    }
    static __device__ __forceinline__ T from(float v) { return v; }
};

template <class X>
__device__ __forceinline__ typename X::V decode(uint32_t w) {
    v4i o;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const int sh = 4 * p - X::kShift;
        const uint32_t t = sh >= 0 ? w >> sh : w << -sh;
        o[p] = (int)((t & X::kMask) | X::kBase);
    }
    return __builtin_bit_cast(typename X::V, o);
}

// A workgroup owns one 16-column strip and one 16-row tile; its WAVES
// wavefronts take the strip's records round-robin and add their partial tiles
// in LDS in wavefront order.  GPR: groups per record.  VEC: rows are 16-byte
// aligned and K is a multiple of 8, so an octet is one or two 16-byte loads and
// wholly inside or outside K.
template <class X, int GPR, bool VEC, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void k_q4g_mm(Q4gParams p) {
    typedef typename X::T T;
    typedef typename X::V V;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 15, g = lane >> 4;
    const int strip = blockIdx.x, m0 = blockIdx.y * 16;
    const T *xrow = (const T *)p.X + (int64_t)min(m0 + r, p.M - 1) * p.ldx;
    const uint8_t *recs = p.recs + (int64_t)strip * p.NQ * kQ4gRecBytes + lane * 16;
    const uint32_t *words = p.words + (GPR > 1 ? ((int64_t)strip * p.NQ * 16 + r) * GPR : (int64_t)strip * p.NG * 16 + r);
    const V ones = __builtin_bit_cast(V, v4i{(int)X::kOnes, (int)X::kOnes, (int)X::kOnes, (int)X::kOnes});
    const v4f zero = {0.0f, 0.0f, 0.0f, 0.0f};
    v4f y = zero;
    for (int q = wave; q < p.NQ; q += WAVES) {
        const v4i cw = *(const v4i *)(recs + (int64_t)q * kQ4gRecBytes);
        uint32_t gw[GPR];
#pragma unroll
        for (int w = 0; w < GPR; ++w) gw[w] = GPR > 1 ? words[(int64_t)q * 16 * GPR + w] : words[(int64_t)(q / p.rpg) * 16];
        v4f d = zero, s = zero;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k0 = 128 * q + 32 * i + 8 * g;
            T x[8];
            if (VEC) {
                const T *src = xrow + min(k0, p.K - 8);
                *(v4i *)x = *(const v4i *)src;
                if (sizeof(T) == 4) *(v4i *)(x + 4) = *(const v4i *)(src + 4);
                if (k0 >= p.K)
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = (T)0.0f;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const T v = xrow[min(k0 + e, p.K - 1)];
                    x[e] = k0 + e < p.K ? v : (T)0.0f;
                }
            }
            V a[X::kTerms];
            X::split(x, a);
            const V b = decode<X>((uint32_t)cw[i]);
#pragma unroll
            for (int t = X::kTerms - 1; t >= 0; --t) {
                d = X::mfma(a[t], b, d);
                s = X::mfma(a[t], ones, s);
            }
            if ((i + 1) % (4 / GPR) == 0) {
                const uint32_t w = gw[i / (4 / GPR)];
                const float sc = __uint_as_float(w & ~15u), z = 16.0f + (float)(w & 15u);
#pragma unroll
                for (int v = 0; v < 4; ++v) y[v] = fmaf(sc, fmaf(-z, s[v], d[v]), y[v]);
                d = zero;
                s = zero;
            }
        }
    }
    __shared__ float red[WAVES][16][17];
#pragma unroll
    for (int v = 0; v < 4; ++v) red[wave][4 * g + v][r] = y[v];
    __syncthreads();
    for (int i = threadIdx.x; i < 256; i += WAVES * 64) {
        const int row = i >> 4, n = strip * 16 + (i & 15);
        float acc = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) acc += red[w][row][i & 15];
        if (m0 + row < p.M && n < p.N) ((T *)p.Y)[(int64_t)(m0 + row) * p.ldy + n] = X::from(acc);
    }
}

template <class X, int GPR>
hipError_t launch_gpr(const Q4gParams &p, bool vec, hipStream_t s) {
    const dim3 grid((unsigned)p.NS, (unsigned)((p.M + 15) / 16));
    if (vec)
        hipLaunchKernelGGL((k_q4g_mm<X, GPR, true, 8>), grid, dim3(512), 0, s, p);
    else
        hipLaunchKernelGGL((k_q4g_mm<X, GPR, false, 8>), grid, dim3(512), 0, s, p);
    return hipGetLastError();
}

template <class X>
hipError_t launch_x(const Q4gParams &p, int gpr, hipStream_t s) {
    const int64_t size = sizeof(typename X::T);
    const bool vec = (uintptr_t)p.X % 16 == 0 && p.ldx * size % 16 == 0 && p.K % 8 == 0;
    return gpr == 1 ? launch_gpr<X, 1>(p, vec, s) : gpr == 2 ? launch_gpr<X, 2>(p, vec, s) : launch_gpr<X, 4>(p, vec, s);
}

}  // namespace

hipError_t launch_q4g_repack(const uint8_t *codes, int64_t ldc, const void *scales, bool bf16, int64_t lds,
                             const uint8_t *zeros, int64_t ldz, int64_t group, const Q4gLayout &L,
                             uint8_t *packed, hipStream_t s) {
    const dim3 block(256), g1((unsigned)ceil_div(L.NS * L.NQ * 64, 256));
    hipLaunchKernelGGL(k_q4g_codes, g1, block, 0, s, codes, ldc, L, packed);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    uint32_t *words = (uint32_t *)(packed + L.words_off);
    const dim3 g2((unsigned)ceil_div((L.total - L.words_off) / 4, 256));
    if (bf16)
        hipLaunchKernelGGL((k_q4g_words<true>), g2, block, 0, s, (const uint16_t *)scales, lds, zeros, ldz, group, L, words);
    else
        hipLaunchKernelGGL((k_q4g_words<false>), g2, block, 0, s, (const uint16_t *)scales, lds, zeros, ldz, group, L, words);
    return hipGetLastError();
}

hipError_t launch_q4g_matmul(const Q4gParams &p, qmm_dtype xt, int gpr, hipStream_t s, const char **variant) {
    *variant = "q4g_mm16";
    return xt == QMM_T_F32 ? launch_x<F32>(p, gpr, s) : xt == QMM_T_F16 ? launch_x<F16>(p, gpr, s) : launch_x<BF16>(p, gpr, s);
}

}  // namespace qmm
