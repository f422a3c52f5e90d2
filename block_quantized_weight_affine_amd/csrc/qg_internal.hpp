// qg_internal.hpp -- launch parameters shared by the host entry points and the kernel files.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "qg_kv8.hpp"

namespace qg {

struct ExpertPtr {
    const void* codes;
    const void* scales;
    const uint16_t* offsets;
};

// One matmul launch: either dense (one weight matrix, rows 0..R-1 of X) or grouped (an expert
// table and the row segments seg_off[e]..seg_off[e+1]-1 of each expert).
struct GemmParams {
    const void* codes;           // dense weights
    const void* scales;
    const uint16_t* offs;
    const ExpertPtr* experts;    // grouped: device table [E]
    const int32_t* seg_off;      // grouped: device [E+1]
    const int32_t* row_src;      // optional: X row of output row r
    const void* X;
    const float* rs;             // optional per-row output scale
    float* Y;                    // [R][N]
    int group;
    int N, K;
    int R;                       // output rows (dense: T)
    int E;                       // grouped: experts
    int x_rows;                  // rows of X (bounds for row_src)
};

// Convolution as an implicit GEMM (page "oxinfer 0.0.5 src/metal.rs", SHADER_SRC conv_body / CP):
// output row r of the GEMM is output pixel r = oy * ow + ox, K runs over (ky, kx, ci), and X is the
// image [H][W][cin] in f32.  norm 1: group norm with stats[c / cpg]; 2: layer norm with stats[input
// pixel]; stats are (mean, rstd) f32 pairs, gb gamma[cin] then beta[cin]; silu applies SiLU after.
struct ConvParams {
    int H, W, cin, ksz, stride, pad, ow;
    int norm, cpg, silu;
    const float* stats;
    const float* gb;
};

// Several weight matrices sharing one X row in one T = 1 launch: job j owns the global output rows
// [start[j], start[j+1]) and writes them to Y[j] (page "oxinfer 0.0.5 src/metal.rs",
// Backend::matmul, whose jobs share X).  Passed by value in the kernel arguments.
constexpr int kMaxBatchJobs = 8;
struct BatchJobs {
    int J;
    int start[kMaxBatchJobs + 1];
    const void* codes[kMaxBatchJobs];
    const void* scales[kMaxBatchJobs];
    const uint16_t* offs[kMaxBatchJobs];
    float* Y[kMaxBatchJobs];
};

// Kernel launchers; each returns a hipError_t from hipGetLastError after the launch.
hipError_t launch_gemm_fast(int fmt, int st, const GemmParams& p, bool grouped, hipStream_t s);
hipError_t launch_gemm_exact(int fmt, int xt, const GemmParams& p, bool grouped, hipStream_t s);
// The convolution through the exact kernel (f32 X gathered per tap; Q4 / Q8 weights); p.R = oh * ow
// output pixels, p.N output channels, p.K = ksz * ksz * cin.
hipError_t launch_conv_exact(int fmt, const GemmParams& p, const ConvParams& cv, hipStream_t s);
// (mean, rstd) pairs of the image [npix][cin]: groups > 0 per group (all pixels, cin / groups
// channels), groups == 0 per pixel.
hipError_t launch_conv_stats(const float* X, int npix, int cin, int groups, float eps, float* stats, hipStream_t s);
// Dense fast matmul with the weights kept exact (Q4 / Q8 codes as f16, f16 X, block scale on the f32
// block partial); hipErrorInvalidValue for another format.
hipError_t launch_gemm_fast_wexact(int fmt, const GemmParams& p, hipStream_t s);
hipError_t launch_gemv(int fmt, int xt, const GemmParams& p, bool grouped, hipStream_t s);
// T = 1, K <= 16384: every job of bj in one launch (p.N = bj.start[bj.J]); false if not applicable.
bool launch_gemv1_batch(int fmt, int xt, const GemmParams& p, const BatchJobs& bj, hipStream_t s, hipError_t& err);
// T = p.R = 2..8, K within the K-split kernel's limit: every job of bj in one launch; false if not
// applicable.
bool launch_gemv_batch(int fmt, int xt, const GemmParams& p, const BatchJobs& bj, hipStream_t s, hipError_t& err);
// Grouped matmul with short segments streamed per expert row (epi 0: Y = X W^T; epi 1: gate|up
// matrices of N = 2I rows, Y[r][j] = SiLU(g) * u with pitch I).  fast: f16 X through v_dot2, or f32
// X scaled to f16 per row in the kernel; otherwise f32 arithmetic.  grouped_rows_fits tells whether
// the shape is taken.
bool grouped_rows_fits(int fmt, int K, int N, int epi);
hipError_t launch_grouped_rows(int fmt, int xt, bool fast, int epi, const GemmParams& p, hipStream_t s);
hipError_t launch_dequant_dump(int fmt, const void* codes, const void* scales, const uint16_t* offs, int group,
                               int N, int K, int n0, int k0, int rows, int cols, int staged, void* out,
                               hipStream_t s);
hipError_t launch_x_half(const float* X, int x_rows, const int32_t* row_src, int R, int K, int guard, uint16_t* Xh,
                         float* rs, hipStream_t s);
hipError_t launch_swiglu(const float* GU, int R, int I, void* A, int at, float* rs, hipStream_t s);
hipError_t launch_moe_plan(const float* logits, int T, int E, int k, int32_t* seg_off, int32_t* row_src,
                           int32_t* slot_row, float* slot_w, int32_t* slot_expert, int32_t* status, int err_code,
                           hipStream_t s);
hipError_t launch_repack_gguf(int q8, const void* src, size_t nblocks, void* codes, void* scales, hipStream_t s);
hipError_t launch_repack_q8f(const void* blob, int N, int K, bool has_col, float* scales, float* col, hipStream_t s);
hipError_t launch_col_scale(const void* X, int xt, int T, int K, const float* col, void* Xs, int st, hipStream_t s);
hipError_t launch_repack_gguf_q8a(int type, const void* src, size_t nblocks, void* codes, float* scales,
                                  float* offs, hipStream_t s);
hipError_t launch_repack_gguf_q8a16(int type, const void* src, size_t nblk16, void* codes, float* scales,
                                    float* offs, hipStream_t s);
// Device address of this GPU's copy of the fixed scratch array (qg_moe_ffn_noalloc), looked up once
// per device with that device current.
hipError_t noalloc_scratch(void** ptr);
hipError_t launch_moe_combine(const float* O, int R, const int32_t* slot_row, const float* slot_w, float* Y, int H,
                              int T, int k, int accumulate, hipStream_t s);


// Workgroups of a launch at most, of up to 512 work items, which a launch counts in 32 bits: larger grids take
// several launches.
constexpr int64_t kLaunchGroups = 1 << 22;

// ---- 8-bit serving operators ------------------------------------------------------------------------
// Elements between tokens and between heads of K and V rows.
struct KvStrides {
    int64_t k_row, k_head, v_row, v_head;
};
// New tokens into the cache (write), or a sequence's last tokens out of it.
hipError_t launch_kv8(bool write, const KvCache& c, const KvSeqs& q, void* k, void* v, int xt, const KvStrides& st,
                      hipStream_t s);

// Rotary positions: radians a position of each pair, of the first `rot` values of a head.
struct Rotary {
    const double* freqs;  // [rot / 2]
    int rot, inter;
    float mscale;
};
// Rows x [T][heads][dim] turned into y; the rest is set by the launcher: how a head's values are shared out, tokens a
// workgroup.
struct RopeRows {
    const void* x;
    void* y;
    int64_t x_row, x_head, y_row, y_head;
    int heads, units, mode, per;
};
hipError_t launch_rope(const RopeRows& a, const Rotary& r, const int32_t* pos, int T, int dim, int xt, hipStream_t s);
// New tokens turned into the cache, row r from row src[r] (src NULL: r) of k and v, at positions pos (NULL: those in the
// sequence); q's rows (q.x NULL: none) turned beside them.  kv_groups is set by the launcher.
struct KvRope {
    Rotary rot;
    const void *k, *v;
    KvStrides st;
    const int32_t *pos, *src;
    int src_rows;
    RopeRows q;
    int kv_groups;
};
hipError_t launch_kv8_rope(const KvCache& c, const KvSeqs& q, const KvRope& a, int xt, hipStream_t s);

// Masks [T][words] and positions [T] of trees; window > 0: masks end that many rows up.
hipError_t launch_tree_plan(const KvSeqs& q, const int32_t* parents, uint32_t* mask, int words, int32_t* pos, int window,
                            hipStream_t s);

// Drafted tokens against the target's probabilities.  Set by the launcher: pieces a row, pieces a wavefront takes, and
// the workspace's parts.
struct VerifyPart {
    double sum;  // of exp((l - top) / temperature) over a piece of a row; NaN where it has a NaN
    float top;
    int at;      // the first index that holds it
};
struct VerifyParams {
    KvSeqs q;
    const int32_t *parents, *tokens;
    const void *target, *draft;
    int64_t t_row, d_row;
    int xt, vocab;
    const float *temps, *accept, *sample;
    int32_t *accepted, *next, *rows_out, *path, *kv_out;
    int pieces, per;
    VerifyPart* part;     // [target, draft][T][pieces]
    double* mass;         // [seqs][pieces]
    int32_t *drawn, *line; // [T]
    uint32_t* tickets;    // [seqs + 1]
    int rows;             // rows of a sequence that a launch takes, by their number or
    const int32_t *list, *listed;       // from a list [T], so many of each sequence [seqs]
    int32_t *list_out, *listed_out;
};
size_t verify_workspace(const KvSeqs& q, int vocab);
hipError_t launch_draft_verify(VerifyParams p, void* ws, hipStream_t s);

constexpr int kMaxTreeRows = 1024;  // drafted rows of a sequence

struct AttnParams {
    KvCache c;
    KvSeqs q;
    const void* Q;
    void* O;
    int64_t q_row, q_head, o_row, o_head;  // elements
    int q_heads, group;
    float scale;
    int causal, window;
    int tile_rows, tiles, splits, chunk;   // rows a tile, tiles a K/V head, splits of the tokens, tokens a split
    int row_waves;                         // wavefronts a workgroup of 16 rows
    int first;                             // a launch's first workgroup
    float *part_o, *part_ml;               // splits > 1: means [row][head][split][dim], (maximum, weight sum)
    // last, as the others' first loads wait for what lies together (before `tile_rows`: one token over 1024 9.15 us for 8.95)
    const uint32_t* mask;                  // a tree's rows: [T][words], which of its sequence's rows each sees (or NULL)
    const int32_t* pos;                    // and their positions, for the window
    int words;
};
void attn8_plan(AttnParams& a, int xt);
int attn8_max_splits(AttnParams a);  // of any window and type
size_t attn8_workspace(const AttnParams& a);
hipError_t launch_attn8(AttnParams a, int xt, float* ws, hipStream_t s);

// Y [T][N] = X [T][K] w^T in 8-bit integers; set by the launcher: X's codes and row scales, and where K is
// split over workgroups their sums [splits][T][N], `per` pieces of 128 k a split.
struct W8A8Params {
    const int8_t* w;
    const float* ws;
    const void* X;
    const int8_t* xq;
    const float* xs;
    void* Y;
    int N, K, T, xt, yt;
    int* part;
    int splits, per;
};
size_t w8a8_workspace(int N, int K, int T);
hipError_t launch_w8a8(W8A8Params p, void* ws, hipStream_t s);

}  // namespace qg
