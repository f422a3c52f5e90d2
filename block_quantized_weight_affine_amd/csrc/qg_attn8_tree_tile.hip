// qg_attn8_tree_tile.hip -- attention for trees of drafted tokens over the 8-bit cache: many rows a K/V head.
#include "qg_attn8_tile.hpp"

namespace qg {

hipError_t launch_attn8_tree_tile(const AttnParams& a, int xt, hipStream_t s) { return launch_tiles<true>(a, xt, s); }

}  // namespace qg
