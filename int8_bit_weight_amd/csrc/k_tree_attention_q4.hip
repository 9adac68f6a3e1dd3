// k_tree_attention_q4.hip -- attention over a paged cache of 4-bit rows: of drafted
// tokens, and behind a window (tree_attention.h has the kernels).
#include "tree_attention.h"

namespace qmm {

hipError_t launch_tree_attention_q4(const TreeParams &p, const TreeShape &z, hipStream_t s) {
    return launch_dk<BF16, kQ4, false>(p, z, s);
}
hipError_t launch_window_attention_q4(const TreeParams &p, const TreeShape &z, hipStream_t s) {
    return launch_dk<BF16, kQ4, true>(p, z, s);
}

}  // namespace qmm
