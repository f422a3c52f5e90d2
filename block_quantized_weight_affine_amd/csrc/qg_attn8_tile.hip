// qg_attn8_tile.hip -- attention over the 8-bit cache for many rows a K/V head: tile heights, launch.
#include "qg_attn8_tile.hpp"

namespace qg {

// 256 rows share a stage's decoding where their sums fit the registers and such tiles are enough for all
// CUs; with fewer, tiles of 128 rows, of which a CU takes two (5 chunks of 129 to 384 rows, 6 heads of 64 a
// group, window 1024: 34.7 and 32.2 us; 2 x 4096 prompt tokens, 32 heads of 128: 325 and 415 us).
int attn8_tile_rows(const AttnParams& a, int xt) {
    if (xt == XT_F32 || a.c.dim > 128) return 128;
    const int64_t tiles = ((int64_t)a.q.max_new * a.group + 255) / 256;
    return a.q.seqs * tiles * a.c.heads < 256 ? 128 : 256;
}

hipError_t launch_attn8_tile(const AttnParams& a, int xt, hipStream_t s) { return launch_tiles<false>(a, xt, s); }

}  // namespace qg
