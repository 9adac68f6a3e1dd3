// k_tree_attention.hip -- attention of drafted tokens over a paged cache of 16-bit
// or int8 rows (tree_attention.h has the kernels).
#include "tree_attention.h"

namespace qmm {

hipError_t launch_tree_attention(const TreeParams &p, const TreeShape &z, qmm_dtype ct, hipStream_t s,
                                 const char **variant) {
    *variant = z.mt == 2 ? "tree_rows128" : "tree_rows64";
    return ct == QMM_T_F16    ? launch_dk<F16, kWide, false>(p, z, s)
           : ct == QMM_T_BF16 ? launch_dk<BF16, kWide, false>(p, z, s)
           : ct == QMM_T_S8   ? launch_dk<BF16, kS8, false>(p, z, s)
                              : launch_tree_attention_q4(p, z, s);
}

}  // namespace qmm
