// qg_attn8.hip -- attention over the 8-bit key/value cache: which kernel, tiles and splits a call takes.
#include <algorithm>
#include <cmath>

#include "qg_attn8_rows.hpp"

namespace qg {
namespace {
// Rows a K/V head (query rows times heads of the group) from which the tile kernel takes over.  The rows
// kernel and the tiles over 2000 tokens, bf16, dim 128, us: 16 sequences 48 rows 42 and 37, 64 rows 54 and 38,
// 124 rows 98 and 45; 2 sequences 48 rows 13.5 and 18.6, 96 rows 19.4 and 20.2.  Over 20000, f16, dim 64, 2
// sequences 96 rows 46 and 32; over 8000, f32, dim 128, 4 sequences 48 rows 44 and 44, 96 rows 70 and 47.
constexpr int64_t kTileFrom = 64;
// Tokens a split at least, and tokens that are not split however few the heads are: 1024 of 8 heads of 128 take
// 9.4 us in one launch; 5.8 and 3.8 us in two.
constexpr int64_t kMinChunk = 256, kAlone = 1024;
void set_tiles(AttnParams& a, int xt) {
    const int64_t rows = (int64_t)a.q.max_new * a.group;
    a.tile_rows = rows >= kTileFrom ? attn8_tile_rows(a, xt) : 16;
    a.tiles = (int)((rows + a.tile_rows - 1) / a.tile_rows);
}
// Splits of `span` tokens.  Rows kernel: one where the workgroups that there are take no longer than a second
// kernel would (bf16, dim 128, sequences x heads: 128 of 2048 tokens 15.8 us in one launch, 20.8 us in eight splits,
// of 8192 62.4 and 61.1 us; 216 of 1024 13.5 and 19.3 us; 512 of 4096 98 and 109 us, of lengths up to that 62 and
// 65 us), but of no more than 4096 tokens, as one long sequence among short ones has its heads' workgroups alone.
// Otherwise, of few heads the splits that fill all CUs evenly, the fewest such (8 of 200000 tokens: 32 splits 82 us,
// 64 86 us, 128 92 us), of more some 1024 workgroups and always a few splits, so that sequences of different
// lengths even out (128 of up to 32768 tokens: 8 splits 108 us, 6 splits 123 us; all of 32768: 203 and 196 us).
// Where the registers leave room for one workgroup a CU, no more than the CUs in a turn (f32, dim 256: 24 of 32768
// tokens 8 splits 72 us, 11 splits 97 us; 96 of 32768 5 splits 247 us, 3 splits 350 us, of lengths up to that 119 and
// 167 us; 256 of 3000 one launch 77 us, 3 splits 92 us).
// Tile kernel: a stage of 64 tokens takes about 24 times as long as a tile's part in writing and joining the sums of
// one more split, so at most sqrt(24 stages / workgroups); none once the card is full.
int64_t wanted_splits(const AttnParams& a, int xt, int64_t span) {
    const int64_t base = (int64_t)a.q.seqs * a.c.heads * a.tiles;
    if (a.tile_rows > 16) {
        int64_t k = 1;
        while ((k + 1) * base <= 256 && (k + 1) * (k + 1) * base <= 24 * (span / 64)) k++;
        return k;
    }
    if (rows_late(xt == XT_F32 ? 2 : 1, a.c.dim)) {
        if (base >= 192 && span <= std::min(16 * base, 4 * kAlone)) return 1;
        return base <= 85 ? 256 / base : base <= 102 ? 512 / base : 3;
    }
    if (span <= std::clamp(16 * base, kAlone, 4 * kAlone)) return 1;
    if (base >= 32) return std::max((1024 + base - 1) / base, (int64_t)6);
    int64_t best = 0;
    double least = 0;
    for (int64_t k = 256 / base; k <= 1024 / base; k++) {
        const double turns = k * base / 256.0, cost = std::ceil(turns) / turns + 0.03 * turns;
        if (!best || cost < least) best = k, least = cost;
    }
    return best;
}
}  // namespace

int attn8_max_splits(AttnParams a) {
    const int64_t most = (a.q.max_kv + kMinChunk - 1) / kMinChunk;
    int64_t want = 1;
    for (int xt : {XT_F32, XT_F16}) {
        set_tiles(a, xt);
        const int64_t w = wanted_splits(a, xt, a.q.max_kv);
        if (w > want) want = w;
    }
    return (int)(most < want ? most : want);
}

// Kernel, tiles and splits of a call, from the host's bounds alone.
void attn8_plan(AttnParams& a, int xt) {
    set_tiles(a, xt);
    // tokens that a tile's rows may see: all, or their window, started at a multiple of 64
    int64_t span = a.q.max_kv;
    const int64_t seen = (int64_t)a.window + a.tile_rows / a.group + 65;
    if (a.causal && a.window > 0 && seen < span) span = seen;
    if (a.mask && a.window > 0) span = std::min(span, (int64_t)a.window + a.q.max_new + 64);
    const int64_t want = wanted_splits(a, xt, span);
    int64_t chunk = (span + want - 1) / want;
    // 8 wavefronts a workgroup where its registers let a CU hold one, or there are few (320 workgroups of one
    // launch, dim 192, 2048 tokens: 62 us, with 4 59 us; 4096 of different lengths: 69 and 83 us)
    const int64_t groups = want * a.q.seqs * a.c.heads * a.tiles;
    const bool wide = a.tile_rows == 16 && (want == 1 ? groups < 512 : groups <= 256 && chunk >= 1024);
    a.row_waves = rows_late(xt == XT_F32 ? 2 : 1, a.c.dim) || wide ? 8 : 4;
    const int64_t unit = a.tile_rows > 16 ? 64 : 64 * a.row_waves;
    if (chunk < kMinChunk) chunk = kMinChunk;
    a.chunk = (int)((chunk + unit - 1) / unit * unit);
    a.splits = (int)((span + a.chunk - 1) / a.chunk);
    if (a.splits < 1) a.splits = 1;
}

size_t attn8_workspace(const AttnParams& a) {
    if (a.splits <= 1) return 0;
    return (size_t)a.q.T * a.q_heads * a.splits * (a.c.dim + 2) * sizeof(float);
}

hipError_t launch_attn8(AttnParams a, int xt, float* ws, hipStream_t s) {
    a.part_o = ws;
    a.part_ml = ws ? ws + (size_t)a.q.T * a.q_heads * a.splits * a.c.dim : nullptr;
    return a.mask ? launch_attn8_tree(a, xt, s) : launch_rows<false>(a, xt, s);
}

}  // namespace qg
