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
void set_chunk(AttnParams& a, int64_t span, int64_t chunk) {
    const int64_t unit = a.tile_rows > 16 ? 64 : 64 * a.row_waves;
    if (chunk < kMinChunk) chunk = kMinChunk;
    a.chunk = (int)((chunk + unit - 1) / unit * unit);
    a.splits = (int)((span + a.chunk - 1) / a.chunk);
    if (a.splits < 1) a.splits = 1;
}

// A tree's call: tiles of 16 rows, of 128 or of 256.  16 rows decode the codes for themselves, which takes 5 us for 1000
// tokens on each CU; a tile of 128 rows takes 22 us, and its workgroups longer to start.  Microseconds of 16 rows and of 128,
// each at its best splits, bf16, 32 heads of 128 on 8 (drafted rows times 4 a K/V head): 1 sequence of 1000 tokens, 25 / 100
// drafted rows 10.6 and 18.0 / 11.5 and 21.1; of 8000, 25 / 61: 19.9 and 21.8 / 32.9 and 28.6; 16 of 2000, 16 / 25 / 61: 28 and 36
// / 44 and 41 / 84 and 53; 16 of up to 8191, 16 / 25 / 61: 71 and 74 / 102 and 78 / 208 and 132; 4 of 30000, f32, 20 heads of 96 on
// 4, 9 / 30: 50 and 69 / 132 and 123; 4 of up to 10000, heads of 256, 30: 68 and 56.
bool tree_in_rows(const AttnParams& a, int64_t span) {
    const int64_t rows = (int64_t)a.q.max_new * a.group, r16 = (rows + 15) / 16, r128 = (rows + 127) / 128;
    const double load = std::max((double)a.q.seqs * a.c.heads * span / 256, 1.0);  // tokens a CU of one tile
    return r16 < 4.5 * r128 + 2400 / load;
}
// Tokens of a tree's tiles of 16 rows that are not split: for heads of up to 128 values up to 1280, wider ones 1024, half as many
// more where CUs get two splits at most.  Several splits and one, us, bf16 heads of 128: 8 workgroups 1152 tokens 10.3 and 10.1, 1280 10.3
// and 10.3, 1408 10.7 and 11.7, 1536 10.4 and 11.7; 56 of 1280 10.6 and 10.5, of 1536 11.0 and 12.0; 104 of 1152 13.1 and 10.4, of
// 1792 13.3 and 12.7, of 2048 13.6 and 14.4.  f32, 96: 8 of 1280 11.6 and 11.7, of 1536 11.6 and 13.4; 120 of 1536 14.9 and 13.6, of 2048
// 15.2 and 16.2.  bf16, 256: 40 of 896 14.4 and 14.9, of 1152 14.7 and 16.3, 104 of 1152 19.6 and 16.5, of 1536 19.7 and 19.2, of 2048
// 20.3 and 22.9; f32: 24 of 896 18.0 and 19.7, 72 of 1024 19.3 and 19.9, 104 of 1152 23.9 and 21.4, of 1408 24.1 and 24.9.
int64_t tree_alone(const AttnParams& a, int64_t base) { return (a.c.dim <= 128 ? 1280 : 1024) * (256 / base > 2 ? 2 : 3) / 2; }
// Splits that fill the card, and more of them where the tokens are many, as their lengths may differ: tiles of 16 rows 5
// sequences of up to 120000 tokens 4 splits 79 us, 8 86, 17 70, 32 76 (f32, 45 rows on 4 heads of 96), 16 of up to 8191 (512
// workgroups) 1 split 71 us, 2 72, 4 81; 128 rows, 25 drafted, 5 of up to 30000 6 splits 57 us, 16 49, 24 62, 16 of up to 8191 2 splits 95
// us, 4 78, 8 79; 256 rows, 61 drafted, 16 of up to 8191 1 split 198 us, 2 121, 4 136, 5 of up to 30000 4 splits 94 us, 6 76, 8 69, 12 94.
// wide: two workgroups a CU.
int64_t tree_splits(const AttnParams& a, int tile_rows, bool wide, int64_t span) {
    const int64_t rows = (int64_t)a.q.max_new * a.group;
    const int64_t base = (int64_t)a.q.seqs * a.c.heads * ((rows + tile_rows - 1) / tile_rows);
    const bool two = wide && tile_rows == 128;
    const int64_t full = tile_rows == 16 || two ? 1024 : 256, tokens = two ? 2048 : 4096;
    if (tile_rows == 16 && (base >= 256 || span <= tree_alone(a, base))) return 1;
    return std::max<int64_t>({256 / base, std::min(full / base, (span + tokens - 1) / tokens), 1});
}
bool tree_wide(const AttnParams& a, int xt) { return xt != XT_F32 && a.c.dim <= 128; }
// Rows a tile of a tree's call; never fewer over more tokens.
int tree_tile_rows(const AttnParams& a, int xt, int64_t span) {
    if (tree_in_rows(a, span)) return 16;
    const int64_t rows = (int64_t)a.q.max_new * a.group, pairs = (int64_t)a.q.seqs * a.c.heads;
    // 256 rows share a stage's decoding where every CU has some 24 stages (16 of 2000 tokens, 244 rows: 53 us of 128, 64 of 256;
    // of up to 8191: 132 and 121)
    if (tree_wide(a, xt) && rows > 128 &&
        (a.q.max_new > kPairTreeRows || pairs * span / 64 * ((rows + 255) / 256) >= 24 * 256))
        return 256;
    return 128;
}
void plan_tree(AttnParams& a, int xt) {
    int64_t span = a.q.max_kv;
    if (a.window > 0) span = std::min(span, (int64_t)a.window + a.q.max_new + 64);
    const int64_t rows = (int64_t)a.q.max_new * a.group, pairs = (int64_t)a.q.seqs * a.c.heads;
    a.tile_rows = tree_tile_rows(a, xt, span);
    a.tiles = (int)((rows + a.tile_rows - 1) / a.tile_rows);
    const int64_t want = tree_splits(a, a.tile_rows, tree_wide(a, xt), span);
    // 8 wavefronts a workgroup, or 4 where there are enough of few tokens (512 of 2000: 28.7 us, of 8 29.5; 2048: 105 and 123)
    a.row_waves = rows_late(xt == XT_F32 ? 2 : 1, a.c.dim) || pairs * a.tiles < 512 || span > 4 * kAlone ? 8 : 4;
    set_chunk(a, span, (span + want - 1) / want);
}
// Splits of any tree's call: a tile's height has most of them over the most tokens that it is taken for.
int64_t most_tree_splits(const AttnParams& a, int xt) {
    int64_t most = 1;
    for (int rows : {16, 128, 256}) {
        int64_t lo = 0, hi = a.q.max_kv;  // the most tokens of tiles of no more rows
        while (lo < hi) {
            const int64_t mid = (lo + hi + 1) / 2;
            tree_tile_rows(a, xt, mid) <= rows ? lo = mid : hi = mid - 1;
        }
        if (lo > 0 && tree_tile_rows(a, xt, lo) == rows) most = std::max(most, tree_splits(a, rows, tree_wide(a, xt), lo));
    }
    return most;
}
}  // namespace

int attn8_max_splits(AttnParams a) {
    const int64_t most = (a.q.max_kv + kMinChunk - 1) / kMinChunk;
    int64_t want = 1;
    for (int xt : {XT_F32, XT_F16}) {
        set_tiles(a, xt);
        const int64_t w = wanted_splits(a, xt, a.q.max_kv);
        if (w > want) want = w;
        if (a.q.max_new > 1 && a.q.max_new <= kMaxTreeRows) want = std::max(want, most_tree_splits(a, xt));
    }
    return (int)(most < want ? most : want);
}

// Kernel, tiles and splits of a call, from the host's bounds alone.
void attn8_plan(AttnParams& a, int xt) {
    if (a.mask && a.q.max_new > 1) return plan_tree(a, xt);
    set_tiles(a, xt);
    // tokens that a tile's rows may see: all, or their window, started at a multiple of 64
    int64_t span = a.q.max_kv;
    const int64_t seen = (int64_t)a.window + a.tile_rows / a.group + 65;
    if ((a.causal || a.mask) && a.window > 0 && seen < span) span = seen;
    const int64_t want = wanted_splits(a, xt, span);
    int64_t chunk = (span + want - 1) / want;
    // 8 wavefronts a workgroup where its registers let a CU hold one, or there are few (320 workgroups of one
    // launch, dim 192, 2048 tokens: 62 us, with 4 59 us; 4096 of different lengths: 69 and 83 us)
    const int64_t groups = want * a.q.seqs * a.c.heads * a.tiles;
    const bool wide = a.tile_rows == 16 && (want == 1 ? groups < 512 : groups <= 256 && chunk >= 1024);
    a.row_waves = rows_late(xt == XT_F32 ? 2 : 1, a.c.dim) || wide ? 8 : 4;
    set_chunk(a, span, chunk);
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
