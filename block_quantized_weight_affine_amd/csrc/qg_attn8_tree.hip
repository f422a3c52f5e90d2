// qg_attn8_tree.hip -- attention for trees of drafted tokens over the 8-bit cache: few rows a K/V head.
#include "qg_attn8_rows.hpp"

namespace qg {

hipError_t launch_attn8_tree(const AttnParams& a, int xt, hipStream_t s) { return launch_rows<true>(a, xt, s); }

}  // namespace qg
