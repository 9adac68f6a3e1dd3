// api_checks.h -- argument checks that the entry points of api_serve.cpp and
// api_tokens.cpp share.
#pragma once

#include <hip/hip_runtime.h>

#include <initializer_list>
#include <utility>

#include "qmm.h"

namespace qmm {

// Set by every entry point (defined in api.cpp).
qmm_status record_status(hipError_t e, const char *variant);

inline bool aligned_to(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

constexpr int64_t kMaxSize = INT32_MAX / 2;

inline int64_t size_of(qmm_dtype t) { return t == QMM_T_F32 ? 4 : t == QMM_T_S8 ? 1 : 2; }

// Whether no stride is negative and the last row starts below element 2^60.
inline bool span_ok(std::initializer_list<std::pair<int64_t, int64_t>> dims) {
    __int128 at = 0;
    for (const auto &d : dims) {
        if (d.second < 0) return false;
        at += (__int128)(d.first > 0 ? d.first - 1 : 0) * d.second;
    }
    return at < ((__int128)1 << 60);
}

// Rows of `run` bytes at base + i*s[0] + j*s[1], i < n[0], j < n[1] (bytes).
struct Rows {
    const void *base;
    int64_t n[2], s[2], run;
    // Bytes from a row's start to the end of those that lie less than `step` apart.
    int64_t extent(int64_t step) const {
        int64_t e = run;
        for (int i = 0; i < 2; ++i)
            if (s[i] % step != 0) e += (n[i] - 1) * s[i];
        return e;
    }
};

// Whether two sets of rows may share a byte: no where their ranges lie apart, or
// where both repeat with one stride and lie apart within it (slices of one tensor).
inline bool may_overlap(const Rows &a, const Rows &b) {
    const uintptr_t pa = (uintptr_t)a.base, pb = (uintptr_t)b.base;
    const int64_t all = INT64_MAX;
    if (pa + a.extent(all) <= pb || pb + b.extent(all) <= pa) return false;
    for (int64_t step : {a.s[0], a.s[1], b.s[0], b.s[1]}) {
        if (step <= 0) continue;
        const int64_t ea = a.extent(step), eb = b.extent(step);
        const int64_t at = (int64_t)((pb % step + step - pa % step) % step);  // of b's rows after a's
        if (ea <= at && at + eb <= step) return false;
    }
    return true;
}

}  // namespace qmm
