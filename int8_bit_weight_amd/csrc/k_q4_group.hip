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
// comes from a second MFMA against ones over the same operand, or is computed once
// where the activations are laid out first.  What the two terms lose to each other,
// a relative 8e-7 to 1.6e-6 at K = 128, lies far below a 16-bit output's rounding
// but not below an fp32 one's: fp32 rows take q - z itself as the operand, some 90
// instructions a record to decode instead of 32 (error 1.0e-7 at K = 128 and 1.3e-7 at K = 4100, where
// a plain fp32 product has 1.0e-7 and 5.4e-7; 4100 x 11003, M = 5: 19.2 us a call
// against 19.5 with 16 + q and its sums).
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
    static constexpr bool kSums = true;  // operands 16 + q, and sums of x for the zeros
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
    static constexpr bool kSums = true;
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
    static constexpr bool kSums = false;  // operands q - z
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

// base: X::kBase kept in a vector register (an and-or takes one constant only).
template <class X>
__device__ __forceinline__ uint32_t decode_base() {
    uint32_t base = X::kBase;
    asm volatile("" : "+v"(base));
    return base;
}
template <class X>
__device__ __forceinline__ typename X::V decode(uint32_t w, uint32_t base) {
    v4i o;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const int sh = 4 * p - X::kShift;
        const uint32_t t = sh >= 0 ? w >> sh : w << -sh;
        o[p] = (int)((t & X::kMask) | base);
    }
    return __builtin_bit_cast(typename X::V, o);
}

// q - z as operands, z in each byte of zzzz: the zeros are taken from bytes 128 + q,
// without a borrow, and the differences become floats whose upper halves are exact.
__device__ __forceinline__ v8bf decode_difference(uint32_t w, uint32_t zzzz) {
    const uint32_t a = (((w & 0x0F0F0F0Fu) | 0x80808080u) - zzzz) ^ 0x80808080u;       // elements 0, 4, 1, 5
    const uint32_t b = (((w >> 4 & 0x0F0F0F0Fu) | 0x80808080u) - zzzz) ^ 0x80808080u;  // 2, 6, 3, 7
    v4i o;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const int x = (int)(p & 1 ? b : a) >> (p & 2 ? 8 : 0);
        o[p] = (int)__builtin_amdgcn_perm(__float_as_uint((float)(int8_t)(x >> 16)), __float_as_uint((float)(int8_t)x), 0x07060302u);
    }
    return __builtin_bit_cast(v8bf, o);
}

// One output term by term, sum_k ((q - z) s) x, for sums that are not finite: an
// infinite activation meets both sums above and leaves inf - inf, and 16 + q times
// an activation of 2^123 and more leaves fp32's range though s brings it back.  (q - z) s
// is exact in fp32 and the sum is kept times 2^-32, so that it cannot leave the
// range on its way (what falls below it is 2^-117 of what brought the output here).
// Every kernel that writes an output checks it.
template <class X>
__device__ __forceinline__ float plain_output(const Q4gParams &p, int row, int n) {
    typedef typename X::T T;
    const T *x = (const T *)p.X + (int64_t)row * p.ldx;
    const int64_t strip = n >> 4;
    const int c = n & 15;
    float acc = 0.0f;
#pragma unroll 1
    for (int at = 0; at < 16 * p.NQ; ++at) {  // octets of k, in order: record, 32-k block, lane group
        const int q = at >> 4, i = at >> 2 & 3, k0 = 8 * at;
        uint32_t codes = *(const uint32_t *)(p.recs + (strip * p.NQ + q) * kQ4gRecBytes + ((at & 3) * 16 + c) * 16 + 4 * i);
        const uint32_t w = p.gpr > 1 ? p.words[((strip * p.NQ + q) * 16 + c) * p.gpr + i * p.gpr / 4]
                                     : p.words[(strip * p.NG + q / p.rpg) * 16 + c];
        const float s = __uint_as_float(w & ~15u);
        const int z = (int)(w & 15u);
#pragma unroll 1
        for (int k = k0; k < k0 + 8 && k < p.K; k += 2) {  // codes 2e and 2e + 1 are nibbles e and 4 + e
            acc = fmaf((float)((int)(codes & 15) - z) * s, 0x1p-32f * (float)x[k], acc);
            if (k + 1 < p.K) acc = fmaf((float)((int)(codes >> 16 & 15) - z) * s, 0x1p-32f * (float)x[k + 1], acc);
            codes >>= 4;
        }
    }
    return acc * 0x1p32f;
}
__device__ __forceinline__ bool finite(float v) { return fabsf(v) < INFINITY; }

// Up to 16 rows.  A workgroup owns one 16-column strip; its WAVES wavefronts take
// the strip's records round-robin, U records' loads in flight at once, and
// add their partial tiles in LDS in wavefront order.  Rows are 16-byte aligned
// and K is at least 8, so an octet is a 16-byte load, but for the last one where
// K is no multiple of 8.  GPR: groups per record.  XLDS: the rows fit LDS and are
// copied there, padded with zeros to whole records, while the first records are
// on their way.  4096 x 14336, M = 1 fp16: 9.2 us on weights that come from HBM
// (3.3 TB/s of codes and words).  With three weights in turn, which the last-level
// cache holds, it takes 8.3; so measured, 8.5 with two records in flight and 9.6
// with four (spills at 64 registers), an earlier build 10.6 with these and 11.3 to
// 12 with four or sixteen wavefronts a strip, and 11.9 a call with the rows read
// from L2 by every wavefront.  Laid out first, M = 1, 4, 16 take 15.5, 15.7 and
// 18.1 us a call, this way 8.4, 12.4 and 18.4: hence up to 16 rows.  Past 29 KiB
// of rows the form that reads them in the loop spills 8 registers for groups of 32.
template <class X, int GPR, int WAVES, int U, bool XLDS>
__global__ __launch_bounds__(WAVES * 64, XLDS ? 8 : 4) void k_q4g_mm16(Q4gParams p) {
    typedef typename X::T T;
    typedef typename X::V V;
    static_assert(X::kTerms == 1, "fp32 rows are laid out first");
    __shared__ __align__(16) char s_x[XLDS ? kQ4gRowsLds : 16];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int strip = blockIdx.x, whole = p.K & ~7;
    const T *xrow = XLDS ? (const T *)s_x + min(r, p.M - 1) * 128 * p.NQ : (const T *)p.X + (int64_t)min(r, p.M - 1) * p.ldx;
    const uint8_t *recs = p.recs + (int64_t)strip * p.NQ * kQ4gRecBytes + lane * 16;
    const uint32_t *words = p.words + (GPR > 1 ? ((int64_t)strip * p.NQ * 16 + r) * GPR : (int64_t)strip * p.NG * 16 + r);
    const V ones = __builtin_bit_cast(V, v4i{(int)X::kOnes, (int)X::kOnes, (int)X::kOnes, (int)X::kOnes});
    const v4f zero = {0.0f, 0.0f, 0.0f, 0.0f};
    const uint32_t code_base = decode_base<X>();
    v4f y = zero;
    for (int q0 = wave; q0 < p.NQ || q0 == wave; q0 += WAVES * U) {
        v4i cw[U], xr[XLDS ? 1 : U][4];
        uint32_t gw[U][GPR];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int q = min(q0 + u * WAVES, p.NQ - 1);
            cw[u] = __builtin_nontemporal_load((const v4i *)(recs + (int64_t)q * kQ4gRecBytes));
#pragma unroll
            for (int w = 0; w < GPR; ++w)
                gw[u][w] = GPR > 1 ? words[(int64_t)q * 16 * GPR + w] : words[(int64_t)(q / p.rpg) * 16];
            if (!XLDS)
#pragma unroll
                for (int i = 0; i < 4; ++i) xr[u][i] = *(const v4i *)(xrow + min(128 * q + 32 * i + 8 * g, whole - 8));
        }
        if (XLDS && q0 == wave) {
            const int octets = 16 * p.NQ;  // of a row
            for (int i = threadIdx.x; i < octets * p.M; i += WAVES * 64) {
                const int m = i / octets, k = 8 * (i - m * octets);
                const T *src = (const T *)p.X + (int64_t)m * p.ldx + k;
                v4i v = {0, 0, 0, 0};
                if (k < whole) {
                    v = *(const v4i *)src;
                } else if (k < p.K) {
                    T e[8] = {};
#pragma unroll
                    for (int j = 0; j < 7; ++j)
                        if (k + j < p.K) e[j] = src[j];
                    v = *(v4i *)e;
                }
                *((v4i *)s_x + i) = v;
            }
            __syncthreads();
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int q = q0 + u * WAVES;
            if (q >= p.NQ) break;
            v4f d = zero, s = zero;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                T x[8];
                const int k0 = 128 * q + 32 * i + 8 * g;
                if (XLDS) {
                    *(v4i *)x = *(const v4i *)(xrow + k0);
                } else {
                    *(v4i *)x = k0 < whole ? xr[XLDS ? 0 : u][i] : v4i{0, 0, 0, 0};
                    if (128 * q + 32 * i + 32 > p.K && whole < p.K && k0 == whole) {  // the octet that K ends in
#pragma unroll
                        for (int e = 0; e < 7; ++e)
                            if (whole + e < p.K) x[e] = xrow[whole + e];
                    }
                }
                const V a = *(const V *)x, b = decode<X>((uint32_t)cw[u][i], code_base);
                d = X::mfma(a, b, d);
                s = X::mfma(a, ones, s);
                if ((i + 1) % (4 / GPR) == 0) {
                    const uint32_t w = gw[u][i / (4 / GPR)];
                    const float sc = __uint_as_float(w & ~15u), z = 16.0f + (float)(w & 15u);
#pragma unroll
                    for (int v = 0; v < 4; ++v) y[v] = fmaf(sc, fmaf(-z, s[v], d[v]), y[v]);
                    d = zero;
                    s = zero;
                }
            }
        }
    }
    __shared__ float red[WAVES][16][17];
#pragma unroll
    for (int v = 0; v < 4; ++v) red[wave][4 * g + v][r] = y[v];
    __syncthreads();
    for (int i = threadIdx.x; i < 256; i += WAVES * 64) {
        const int row = i >> 4, n = strip * 16 + (i & 15);
        if (row >= p.M || n >= p.N) continue;
        float acc = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) acc += red[w][row][i & 15];
        if (!finite(acc)) acc = plain_output<X>(p, row, n);
        ((T *)p.Y)[(int64_t)row * p.ldy + n] = X::from(acc);
    }
}

// More rows, or rows of any alignment: the activations are laid out first.  One
// workgroup per (16-row tile, record of 128 k) writes the matrix operands (per
// term 64 lanes x 16 bytes per 32 k, rows and k past the end zero) and, of 16-bit
// rows, the fp32 sums over every group of at most 128 k, which the zeros multiply.
template <class X, int GPR>
__global__ __launch_bounds__(256) void k_q4g_lay(Q4gParams p) {
    typedef typename X::T T;
    typedef typename X::V V;
    const int lane = threadIdx.x & 63, i = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    const int q = blockIdx.x, mt = blockIdx.y, row = mt * 16 + r, k0 = 128 * q + 32 * i + 8 * g;
    const T *src = (const T *)p.X + (int64_t)min(row, p.M - 1) * p.ldx;
    T x[8];
    float sum = 0.0f;
    if (p.x_vec && k0 + 8 <= p.K) {
#pragma unroll
        for (int h = 0; h < (int)sizeof(T) / 2; ++h) *((v4i *)x + h) = *((const v4i *)(src + k0) + h);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = src[min(k0 + e, p.K - 1)];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (row >= p.M || k0 + e >= p.K) x[e] = (T)0.0f;
        sum += (float)x[e];
    }
    V a[X::kTerms];
    X::split(x, a);
    const int64_t at = (int64_t)q * gridDim.y + mt;
    v4i *out = (v4i *)p.xa + (at * 4 + i) * X::kTerms * 64 + lane;
#pragma unroll
    for (int t = 0; t < X::kTerms; ++t) out[t * 64] = __builtin_bit_cast(v4i, a[t]);
    if (!X::kSums) return;
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    __shared__ float s_sum[4][16];
    if (g == 0) s_sum[i][r] = sum;
    __syncthreads();
    if (threadIdx.x < 16 * GPR) {
        const int w = threadIdx.x >> 4;
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < 4 / GPR; ++e) s += s_sum[w * (4 / GPR) + e][r];
        p.xs[(at * GPR + w) * 16 + r] = s;
    }
}

// 16 bytes per lane from global memory to LDS at byte dst + 16 lane.  As assembly
// because the compiler waits for every copy in flight before any LDS read that
// it cannot tell from them; the kernel itself counts its copies.  The block has
// no register outputs.
__device__ __forceinline__ void copy_to_lds(const void *src, int dst) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "s"(dst) : "m0", "memory");
}
template <int N>
__device__ __forceinline__ void wait_loads() {  // at most N vector memory operations of the wavefront left
    static_assert(N < 16, "low field only");
    __builtin_amdgcn_s_waitcnt(0x0F70 | N);
}

// The product from laid-out activations: a wavefront takes one strip and MT
// 16-row tiles, so a code is decoded once for all rows.  Eight wavefronts share a
// record's operands (and sums), which are copied to a ring of four LDS buffers three
// records ahead, and have their codes and words on the way four records ahead.
// blockIdx.y splits the records: with more than one range the sums go to the
// workspace for k_q4g_sum.  14336 x 4096, M = 64 bf16, group 64: 20.5 us (and 4.8
// and 4.6 of the launches around it), 0.37 PFLOP/s.  A record and strip need 32
// VALU instructions to decode and 64 to scale 16 x 64 sums beside 16 MFMAs: VALU
// issue takes 47 % of the cycles, the matrix units 20 %, LDS 30 %, at about 1.7
// GHz.  4100 x 11003, M = 5 fp32, group 32: 15.7 us (and 3.0 and 4.0), VALU issue
// 50 %, matrix units 16 %.  A second group of wavefronts for every other record, 16 to a CU: 22.3 us.
template <class X, int GPR, int MT>
__global__ __launch_bounds__(512, 2) void k_q4g_mm(Q4gParams p) {
    typedef typename X::T T;
    typedef typename X::V V;
    constexpr int TERMS = X::kTerms, RING = 4;
    constexpr bool SUMS = X::kSums;
    constexpr int CHUNKS = MT * 4 * TERMS, PIECES = CHUNKS + SUMS;  // 1 KiB pieces of a record: operands, sums
    constexpr int COPIES = (PIECES + 7) / 8;                        // of a wavefront
    __shared__ __align__(1024) char s_a[RING][PIECES * 1024];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int strip = blockIdx.x * 8 + wave, mt0 = blockIdx.z * MT, tiles = gridDim.z * MT;
    const int64_t own = min(strip, p.NS - 1);
    const int q0 = (int)((int64_t)blockIdx.y * p.NQ / gridDim.y), q1 = (int)((int64_t)(blockIdx.y + 1) * p.NQ / gridDim.y);
    const int steps = q1 - q0;
    const auto record = [&](int step) { return min(q0 + step, q1 - 1); };
    const uint32_t code_base = SUMS ? decode_base<X>() : 0;
    const v4f zero = {0.0f, 0.0f, 0.0f, 0.0f};
    const int base = (int)(uintptr_t)(__attribute__((address_space(3))) const char *)&s_a[0][0];
    const auto copy = [&](int step) {  // the same number of copies in every wavefront: the last piece repeats
        const int64_t at = (int64_t)record(step) * tiles + mt0;
        const int to = base + step % RING * PIECES * 1024;
#pragma unroll
        for (int i = 0; i < COPIES; ++i) {
            const int chunk = min(wave + 8 * i, PIECES - 1);
            const char *src = !SUMS || chunk < CHUNKS ? (const char *)p.xa + (at * 4 * TERMS + chunk) * 1024 : (const char *)(p.xs + at * GPR * 16);
            copy_to_lds(src + lane * 16, to + chunk * 1024);
        }
    };
    v4i cw[RING];
    uint32_t gw[RING][GPR];
    const auto load = [&](int step, int u) {
        const int q = record(step);
        cw[u] = __builtin_nontemporal_load((const v4i *)(p.recs + (own * p.NQ + q) * kQ4gRecBytes) + lane);
#pragma unroll
        for (int w = 0; w < GPR; ++w)
            gw[u][w] = GPR > 1 ? p.words[((own * p.NQ + q) * 16 + r) * GPR + w] : p.words[(own * p.NG + q / p.rpg) * 16 + r];
    };
    v4f y[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) y[m] = zero;
#pragma unroll
    for (int u = 0; u < RING - 1; ++u) copy(u);
#pragma unroll
    for (int u = 0; u < RING; ++u) load(u, u);
    for (int s0 = 0; s0 < steps; s0 += RING) {
#pragma unroll
        for (int u = 0; u < RING; ++u) {
            const int step = s0 + u;
            if (step >= steps) break;
            // after this step's copies came at least the next two's and, of each of
            // three steps before it, a load of codes
            wait_loads<2 * COPIES + 3>();
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            copy(step + RING - 1);
            const v4i code = cw[u];
            uint32_t word[GPR];
#pragma unroll
            for (int w = 0; w < GPR; ++w) word[w] = gw[u][w];
            load(step + RING, u);
            const char *const buf = s_a[u];
            v4f d[MT];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                V a[MT][TERMS];
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int t = 0; t < TERMS; ++t) a[m][t] = *(const V *)(buf + (((m * 4 + i) * TERMS + t) * 64 + lane) * 16);
                V b;
                if constexpr (SUMS) {
                    b = decode<X>((uint32_t)code[i], code_base);
                } else {
                    const uint32_t z = word[i * GPR / 4] & 15u;
                    b = decode_difference((uint32_t)code[i], __builtin_amdgcn_perm(z, z, 0u));
                }
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    if (i % (4 / GPR) == 0) d[m] = zero;
#pragma unroll
                for (int t = TERMS - 1; t >= 0; --t)
#pragma unroll
                    for (int m = 0; m < MT; ++m) d[m] = X::mfma(a[m][t], b, d[m]);
                if ((i + 1) % (4 / GPR) == 0) {
                    const int w = i / (4 / GPR);
                    const float sc = __uint_as_float(word[w] & ~15u), z = 16.0f + (float)(word[w] & 15u);
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        if (SUMS) {
                            const v4f s = *(const v4f *)(buf + CHUNKS * 1024 + ((m * GPR + w) * 16 + 4 * g) * 4);
#pragma unroll
                            for (int v = 0; v < 4; ++v) d[m][v] = fmaf(-z, s[v], d[m][v]);
                        }
#pragma unroll
                        for (int v = 0; v < 4; ++v) y[m][v] = fmaf(sc, d[m][v], y[m][v]);
                    }
                }
            }
        }
    }
    wait_loads<0>();  // no copy may arrive in LDS that has another owner by then
    const int n = strip * 16 + r;
    if (n >= p.N) return;
    uint32_t again = 0;  // outputs, a bit each
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int row = (mt0 + m) * 16 + 4 * g + v;
            if (row >= p.M) continue;
            if (gridDim.y > 1) {
                p.part[((int64_t)blockIdx.y * p.M + row) * p.N + n] = y[m][v];
            } else {
                ((T *)p.Y)[(int64_t)row * p.ldy + n] = X::from(y[m][v]);
                if (!finite(y[m][v])) again |= 1u << (4 * m + v);
            }
        }
    for (; again != 0; again &= again - 1) {
        const int i = __ffs(again) - 1, row = (mt0 + (i >> 2)) * 16 + 4 * g + (i & 3);
        ((T *)p.Y)[(int64_t)row * p.ldy + n] = X::from(plain_output<X>(p, row, n));
    }
}

template <class X>
__global__ __launch_bounds__(256) void k_q4g_sum(Q4gParams p, int parts) {
    const int64_t size = (int64_t)p.M * p.N, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= size) return;
    float acc = 0.0f;
    for (int k = 0; k < parts; ++k) acc += p.part[k * size + i];
    if (!finite(acc)) acc = plain_output<X>(p, (int)(i / p.N), (int)(i % p.N));
    ((typename X::T *)p.Y)[i / p.N * p.ldy + i % p.N] = X::from(acc);
}

template <class X, int GPR, int MT>
hipError_t launch_laid(const Q4gParams &p, const Q4gShape &z, hipStream_t s) {
    const dim3 grid((unsigned)ceil_div(p.NS, 8), (unsigned)z.parts, (unsigned)(z.tiles / MT));
    hipLaunchKernelGGL((k_q4g_mm<X, GPR, MT>), grid, dim3(512), 0, s, p);
    return hipGetLastError();
}

template <class X, int GPR>
hipError_t launch_gpr(const Q4gParams &p, const Q4gShape &z, hipStream_t s) {
    if (!z.laid) {
        if constexpr (X::kTerms == 1) {  // fp32 rows are always laid out
            if (p.M * (int64_t)p.NQ * 256 <= kQ4gRowsLds)
                hipLaunchKernelGGL((k_q4g_mm16<X, GPR, 8, 2, true>), dim3((unsigned)p.NS), dim3(512), 0, s, p);
            else
                hipLaunchKernelGGL((k_q4g_mm16<X, GPR, 8, 4, false>), dim3((unsigned)p.NS), dim3(512), 0, s, p);
        }
        return hipGetLastError();
    }
    hipLaunchKernelGGL((k_q4g_lay<X, GPR>), dim3((unsigned)p.NQ, (unsigned)z.tiles), dim3(256), 0, s, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if constexpr (X::kTerms == 1) {
        if (z.mt == 4) e = launch_laid<X, GPR, 4>(p, z, s);
    }
    if (z.mt < 4) e = z.mt == 1 ? launch_laid<X, GPR, 1>(p, z, s) : launch_laid<X, GPR, 2>(p, z, s);
    if (e != hipSuccess || z.parts == 1) return e;
    hipLaunchKernelGGL((k_q4g_sum<X>), dim3((unsigned)ceil_div((int64_t)p.M * p.N, 256)), dim3(256), 0, s, p, z.parts);
    return hipGetLastError();
}

template <class X>
hipError_t launch_x(const Q4gParams &p, int gpr, const Q4gShape &z, hipStream_t s) {
    return gpr == 1 ? launch_gpr<X, 1>(p, z, s) : gpr == 2 ? launch_gpr<X, 2>(p, z, s) : launch_gpr<X, 4>(p, z, s);
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

hipError_t launch_q4g_matmul(const Q4gParams &p, qmm_dtype xt, int gpr, const Q4gShape &z, hipStream_t s,
                             const char **variant) {
    *variant = !z.laid ? "q4g_mm16" : z.parts > 1 ? "q4g_mm_split" : "q4g_mm";
    return xt == QMM_T_F32   ? launch_x<F32>(p, gpr, z, s)
           : xt == QMM_T_F16 ? launch_x<F16>(p, gpr, z, s)
                             : launch_x<BF16>(p, gpr, z, s);
}

}  // namespace qmm
