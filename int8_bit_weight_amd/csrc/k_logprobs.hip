// k_logprobs.hip -- log probabilities of given tokens, entropy and the largest
// logits of a row, from logits read once, on gfx950.
//
//   lse = m + log sum exp(z - m),  entropy = log S - sum e (z - m) / S,  e = exp(z - m), S = sum e
//
// The first launch reads the logits: a wavefront keeps its piece of a row in
// registers, finds its maximum and leaves (m, S, sum e (z - m)).  For the
// alternatives it also leaves the largest logit of each group of 32 neighbouring
// tokens: the k largest logits lie in the k groups of the largest maxima (groups of
// equal maxima in their order, as tokens of equal logits), since every other group has
// k logits before all of its own.  The second launch, a workgroup a row, joins the
// pieces, picks those k groups and reads them again.
#include <type_traits>

#include "token_internal.h"

namespace qmm {

namespace {

typedef unsigned long long u64;

constexpr float kLn2 = 0.69314718055994531f;

template <class T>
__device__ __forceinline__ float value(const v4i &raw, int e);
template <>
__device__ __forceinline__ float value<float>(const v4i &raw, int e) {
    return __int_as_float(raw[e]);
}
template <>
__device__ __forceinline__ float value<__bf16>(const v4i &raw, int e) {
    return __uint_as_float(e & 1 ? (uint32_t)raw[e / 2] & 0xFFFF0000u : (uint32_t)raw[e / 2] << 16);
}
template <>
__device__ __forceinline__ float value<_Float16>(const v4i &raw, int e) {
    typedef _Float16 v2h __attribute__((ext_vector_type(2)));
    const int pair = raw[e / 2];  // a bit cast of the element itself takes the first one
    return (float)__builtin_bit_cast(v2h, pair)[e & 1];
}

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
    for (int o = 1; o < 64; o *= 2) x = fmaxf(x, __shfl_xor(x, o));
    return x;
}
__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
    for (int o = 1; o < 64; o *= 2) x += __shfl_xor(x, o);
    return x;
}

// f over the 4 or 8 neighbouring lanes of a group.
template <int LANES, class F>
__device__ __forceinline__ int over_group(int x, F f) {
    x = f(x, __builtin_amdgcn_mov_dpp(x, 0xB1, 0xF, 0xF, true));                  // lanes 1 0 3 2 of four
    x = f(x, __builtin_amdgcn_mov_dpp(x, 0x4E, 0xF, 0xF, true));                  // lanes 2 3 0 1
    if (LANES == 8) x = f(x, __builtin_amdgcn_mov_dpp(x, 0x141, 0xF, 0xF, true));  // lanes 7 .. 0 of eight
    return x;
}
template <int LANES>
__device__ __forceinline__ float group_max(float x) {
    return __int_as_float(over_group<LANES>(__float_as_int(x), [](int a, int b) {
        return __float_as_int(fmaxf(__int_as_float(a), __int_as_float(b)));
    }));
}
template <int LANES>
__device__ __forceinline__ int group_sum(int x) {
    return over_group<LANES>(x, [](int a, int b) { return a + b; });
}

// The order of logits and tokens as one number: larger logits first, of equal ones (0
// and -0, NaN and -inf) the lower token.  0 is below every logit's.
__device__ __forceinline__ u64 order(float x, uint32_t token) {
    if (x != x) x = -INFINITY;
    const uint32_t b = __float_as_uint(x + 0.0f);
    return (u64)(b & 0x80000000u ? ~b : b | 0x80000000u) << 32 | (0xFFFFFFFFu - token);
}
__device__ __forceinline__ uint32_t token_of(u64 key) { return 0xFFFFFFFFu - (uint32_t)key; }
__device__ __forceinline__ float logit_of(u64 key) {
    const uint32_t b = (uint32_t)(key >> 32);
    return __uint_as_float(b & 0x80000000u ? b & 0x7FFFFFFFu : ~b);
}

// A wavefront's piece starts at a multiple of 16 bytes, which may lie before the row.
// Bound by the read of the logits.
template <class T, int LOADS, bool TOP>
__global__ __launch_bounds__(256) void k_logprob_part(LogprobParams p) {
    constexpr int VEC = 16 / sizeof(T), LANES = kTopGroup / VEC;  // lanes of a group
    const int lane = threadIdx.x & 63;
    const int64_t at = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t = at / p.chunks;
    const int chunk = (int)(at - t * p.chunks);
    if (t >= p.T) return;
    const T *row = (const T *)p.logits + t * p.ld;
    const int before = (int)((uintptr_t)row & 15) / (int)sizeof(T);
    const int first = chunk * (64 * VEC * LOADS) - before;
    v4i raw[LOADS];
    bool whole[LOADS];
    T none[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) none[e] = (T)-INFINITY;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int v = first + (64 * i + lane) * VEC;
        whole[i] = v >= 0 && v <= p.V - VEC;
        raw[i] = *(v4i *)none;
        // many rows stream past the caches: 304 MB in 56 us instead of 58
        if (whole[i]) raw[i] = LOADS == 8 ? __builtin_nontemporal_load((const v4i *)(row + v)) : *(const v4i *)(row + v);
    }
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int v = first + (64 * i + lane) * VEC;
        if (!whole[i] && v > -VEC && v < p.V) {  // the row's first and last elements
            T x[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) x[e] = v + e >= 0 && v + e < p.V ? row[v + e] : (T)-INFINITY;
            raw[i] = *(v4i *)x;
        }
    }
    float top = -INFINITY;
    float *gmax = p.gmax + t * p.groups + chunk * (64 * LOADS / LANES);
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        float m = value<T>(raw[i], 0);
#pragma unroll
        for (int e = 1; e < VEC; ++e) m = fmaxf(m, value<T>(raw[i], e));
        top = fmaxf(top, m);
        if (TOP) {
            m = group_max<LANES>(m);
            // NaN alone gives NaN, which stands with -inf
            if (lane % LANES == 0) gmax[(64 * i + lane) / LANES] = m;
        }
    }
    const float m = wave_max(top), base = m == -INFINITY ? 0.0f : m;
    float s = 0.0f, w = 0.0f;
    const auto add = [&](auto DIFFERENCE, float from) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float v = value<T>(raw[i], e);
                float y = decltype(DIFFERENCE)::value ? (v - base) * p.scale : fmaf(v, p.scale, -from);
                const float x = __builtin_amdgcn_exp2f(y);
                y = fmaxf(y, -1000.0f);  // 0 times this, not times -inf; NaN shows in the sum
                s += x;
                w = fmaf(x, y, w);
            }
    };
    const float from = base * p.scale;
    if (fabsf(from) < 65536.0f) {
        // one step an element; every exponent is off by the rounding of `from`, which is put right in the sums
        add(std::false_type(), from);
        const float off = fmaf(base, p.scale, -from), right = __builtin_amdgcn_exp2f(-off);
        w = right * (w - off * s);
        s *= right;
    } else {  // the difference first: a product of large logits would lose it
        add(std::true_type(), 0.0f);
    }
    s = wave_sum(s);
    w = wave_sum(w);
    if (lane == 0) {
        float *part = p.part + at * 3;
        part[0] = m;
        part[1] = s;
        part[2] = w;
    }
}

constexpr int kListed = 1024;  // groups, then logits, that may pass a first bound

// The k-th largest of the largest keys of each four threads: at least k keys are not
// below it, where there are that many (k <= 64).  All threads call it; s_key holds 64.
__device__ __forceinline__ u64 bound(u64 mine, int k, u64 *s_key, u64 *s_bound) {
    const int tid = threadIdx.x;
#pragma unroll
    for (int o = 1; o < 4; o *= 2) {
        const u64 other = __shfl_xor(mine, o);
        mine = other > mine ? other : mine;
    }
    if (tid == 0) *s_bound = 0;
    __syncthreads();
    if (tid % 4 == 0) s_key[tid / 4] = mine;
    __syncthreads();
    int above = 0;  // four lanes hold a key, and compare it with a quarter of the others each
#pragma unroll
    for (int i = 0; i < 64; i += 4) above += s_key[i + tid % 4] > mine;
    above = group_sum<4>(above);
    if (above == k - 1 && mine) *s_bound = mine;  // keys differ but for 0: four lanes at most, of one value
    __syncthreads();
    return *s_bound;
}

// Joins a row's pieces and finds its largest logits.  All of it is latency: what can be
// asked for at the start is, and rows of up to 256 HELD groups keep their maxima in
// registers (HELD 0: any number of them, read again where they are needed).
template <class T, int HELD>
__global__ __launch_bounds__(256) void k_logprob_row(LogprobParams p) {
    __shared__ u64 s_list[kListed], s_key[64], s_bound;
    __shared__ uint32_t s_group[QMM_MAX_TOP];
    __shared__ float s_m[4], s_s[4], s_w[4];
    __shared__ int s_count, s_above[4];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t t = blockIdx.x;
    const T *row = (const T *)p.logits + t * p.ld;
    const int before = (int)((uintptr_t)row & 15) / (int)sizeof(T);
    const int k = p.top, groups_here = (before + p.V + kTopGroup - 1) / kTopGroup;  // groups with a token
    const float *gmax = p.gmax + t * p.groups;
    float held[HELD ? HELD : 1];
#pragma unroll
    for (int i = 0; i < HELD; ++i) held[i] = gmax[min(tid + 256 * i, groups_here - 1)];
    int64_t id = -1;
    float given = 0.0f;
    if (tid < p.n) {
        id = p.tokens[t * p.ld_tokens + tid];
        if (id >= 0 && id < p.V) given = (float)row[id];
    }
    // ---- m, S and sum e (z - m) of the row
    const float *part = p.part + t * p.chunks * 3;
    float m = -INFINITY, s = 0.0f, w = 0.0f;
    const auto join = [&](float m2, float s2, float w2) {
        const float top = fmaxf(m, m2), base = top == -INFINITY ? 0.0f : top;
        // a part with nothing has m = -inf and zeros: its factor's -inf must not meet them
        const float d1 = fmaxf((m - base) * p.scale, -1000.0f), d2 = fmaxf((m2 - base) * p.scale, -1000.0f);
        const float a = __builtin_amdgcn_exp2f(d1), b = __builtin_amdgcn_exp2f(d2);
        w = a * (w + s * d1) + b * (w2 + s2 * d2);
        s = a * s + b * s2;
        m = top;
    };
    for (int i = tid; i < p.chunks; i += 256) join(part[3 * i], part[3 * i + 1], part[3 * i + 2]);
#pragma unroll
    for (int o = 1; o < 64; o *= 2) join(__shfl_xor(m, o), __shfl_xor(s, o), __shfl_xor(w, o));
    if (lane == 0) {
        s_m[wave] = m;
        s_s[wave] = s;
        s_w[wave] = w;
    }
    if (tid == 0) s_count = 0;
    __syncthreads();
    m = s_m[0];
    s = s_s[0];
    w = s_w[0];
#pragma unroll
    for (int i = 1; i < 4; ++i) join(s_m[i], s_s[i], s_w[i]);
    const bool empty = m == -INFINITY && s == 0.0f;  // nothing but -inf
    const float log_s = __builtin_amdgcn_logf(s);    // of two
    const auto logprob = [&](float x) { return empty ? -INFINITY : fmaf(x - m, p.scale_e, -log_s * kLn2); };
    if (tid < p.n) p.logprobs[t * p.n + tid] = id >= 0 && id < p.V ? logprob(given) : -INFINITY;
    for (int i = tid + 256; i < p.n; i += 256) {
        id = p.tokens[t * p.ld_tokens + i];
        p.logprobs[t * p.n + i] = id >= 0 && id < p.V ? logprob((float)row[id]) : -INFINITY;
    }
    if (tid == 0 && p.entropy) p.entropy[t] = empty ? 0.0f : (log_s - w / s) * kLn2;
    if (k == 0) return;

    // ---- the groups of the largest maxima
    const auto each = [&](auto use) {  // use(key) for this thread's groups
        if constexpr (HELD > 0) {
#pragma unroll
            for (int i = 0; i < HELD; ++i)
                if (tid + 256 * i < groups_here) use(order(held[i], (uint32_t)(tid + 256 * i)));
        } else {
            for (int g = tid; g < groups_here; g += 256) use(order(gmax[g], (uint32_t)g));
        }
    };
    u64 mine = 0;
    each([&](u64 x) { mine = x > mine ? x : mine; });
    u64 least = bound(mine, k, s_key, &s_bound);
    each([&](u64 x) {
        if (x >= least) {
            const int i = atomicAdd(&s_count, 1);
            if (i < kListed) s_list[i] = x;
        }
    });
    __syncthreads();
    if (s_count > kListed) {  // a few threads hold most of the largest: bisect for the k-th key
        u64 lo = least, hi = ~0ull;  // at least k keys >= lo, fewer than k >= hi
        while (hi - lo > 1) {
            const u64 mid = lo + (hi - lo) / 2;
            int n = 0;
            each([&](u64 x) { n += x >= mid; });
#pragma unroll
            for (int o = 1; o < 64; o *= 2) n += __shfl_xor(n, o);
            __syncthreads();
            if (lane == 0) s_above[wave] = n;
            __syncthreads();
            if (s_above[0] + s_above[1] + s_above[2] + s_above[3] >= k) lo = mid;
            else hi = mid;
        }
        if (tid == 0) s_count = 0;
        __syncthreads();
        each([&](u64 x) {
            if (x >= lo) s_list[atomicAdd(&s_count, 1)] = x;  // k of them
        });
        __syncthreads();
    }
    // take(place, key) for the k largest of the n listed, whose places eight lanes count together
    const auto largest = [&](int n, auto take) {
        for (int i0 = 0; i0 < n; i0 += 32) {
            const int i = i0 + tid / 8;
            const u64 x = s_list[min(i, n - 1)];
            int above = 0;
#pragma unroll 4
            for (int j = tid % 8; j < n; j += 8) above += s_list[j] > x;
            above = group_sum<8>(above);
            if (i < n && tid % 8 == 0 && above < k) take(above, x);
        }
    };
    int n = s_count;
    const int groups = min(k, n);
    largest(n, [&](int at, u64 x) { s_group[at] = token_of(x); });
    // ---- their logits
    __syncthreads();
    if (tid == 0) s_count = 0;
    u64 key[QMM_MAX_TOP * kTopGroup / 256];
    mine = 0;
#pragma unroll
    for (int j = 0; j < QMM_MAX_TOP * kTopGroup / 256; ++j) {
        const int i = j * 256 + tid;
        key[j] = 0;
        if (i < groups * kTopGroup) {
            const int64_t v = (int64_t)s_group[i / kTopGroup] * kTopGroup + i % kTopGroup - before;
            if (v >= 0 && v < p.V) key[j] = order((float)row[v], (uint32_t)v);
        }
        mine = key[j] > mine ? key[j] : mine;
    }
    least = bound(mine, k, s_key, &s_bound);
#pragma unroll
    for (int j = 0; j < QMM_MAX_TOP * kTopGroup / 256; ++j)
        if (key[j] && key[j] >= least) s_list[atomicAdd(&s_count, 1)] = key[j];
    __syncthreads();
    n = s_count;
    largest(n, [&](int at, u64 x) {
        p.top_ids[t * k + at] = token_of(x);
        p.top_lp[t * k + at] = logprob(logit_of(x));
    });
    for (int i = n + tid; i < k; i += 256) {  // fewer tokens than asked for
        p.top_ids[t * k + i] = -1;
        p.top_lp[t * k + i] = -INFINITY;
    }
}

template <class T, int LOADS>
hipError_t launch(const LogprobParams &p, hipStream_t s) {
    const dim3 grid((unsigned)ceil_div((int64_t)p.T * p.chunks, 4));
    if (p.top > 0)
        hipLaunchKernelGGL((k_logprob_part<T, LOADS, true>), grid, dim3(256), 0, s, p);
    else
        hipLaunchKernelGGL((k_logprob_part<T, LOADS, false>), grid, dim3(256), 0, s, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // 20 groups a thread cover vocabularies of 163 thousand
    if (p.top > 0 && p.groups > 256 * 4 && p.groups <= 256 * 20)
        hipLaunchKernelGGL((k_logprob_row<T, 20>), dim3((unsigned)p.T), dim3(256), 0, s, p);
    else if (p.top > 0 && p.groups <= 256 * 4)
        hipLaunchKernelGGL((k_logprob_row<T, 4>), dim3((unsigned)p.T), dim3(256), 0, s, p);
    else
        hipLaunchKernelGGL((k_logprob_row<T, 0>), dim3((unsigned)p.T), dim3(256), 0, s, p);
    return hipGetLastError();
}

template <class T>
hipError_t launch_type(const LogprobParams &p, const LogprobShape &z, hipStream_t s) {
    return z.loads == 8 ? launch<T, 8>(p, s) : launch<T, 2>(p, s);
}

}  // namespace

hipError_t launch_logprobs(const LogprobParams &p, const LogprobShape &z, qmm_dtype xt, hipStream_t s) {
    return xt == QMM_T_F32   ? launch_type<float>(p, z, s)
           : xt == QMM_T_F16 ? launch_type<_Float16>(p, z, s)
                             : launch_type<__bf16>(p, z, s);
}

}  // namespace qmm
