// k_window_attention.hip -- attention behind a window over a paged cache of 16-bit
// or int8 rows (tree_attention.h has the kernels).
#include "tree_attention.h"

namespace qmm {

hipError_t launch_window_attention(const TreeParams &p, const TreeShape &z, qmm_dtype ct, hipStream_t s,
                                   const char **variant) {
    *variant = z.mt == 2 ? "window_rows128" : "window_rows64";
    return ct == QMM_T_F16    ? launch_dk<F16, kWide, true>(p, z, s)
           : ct == QMM_T_BF16 ? launch_dk<BF16, kWide, true>(p, z, s)
           : ct == QMM_T_S8   ? launch_dk<BF16, kS8, true>(p, z, s)
                              : launch_window_attention_q4(p, z, s);
}

}  // namespace qmm
