// qg_capi8.cpp -- the C ABI of the 8-bit serving operators declared in include/qgemm.h: argument
// validation on the host, before any HIP call, then the launch.
#include <cmath>
#include <cstdint>

#include "qgemm.h"
#include "qg_internal.hpp"

using qg::AttnParams;
using qg::KvCache;
using qg::KvSeqs;
using qg::KvStrides;

namespace {

constexpr int kMaxKv = 1 << 24;
constexpr int kMaxRows = 1 << 21;
constexpr int kMaxTree = qg::kMaxTreeRows;
constexpr int kMaxDim = 1024;   // of rows that are turned
constexpr int kMaxVocab = 1 << 24;
constexpr int64_t kMaxStride = (int64_t)1 << 40;

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
bool xt_ok(int x) { return x == QG_X_F32 || x == QG_X_F16 || x == QG_X_BF16; }
int64_t xt_bytes(int x) { return x == QG_X_F32 ? 4 : 2; }
qg_status launched(hipError_t e) { return e == hipSuccess ? QG_OK : QG_ELAUNCH; }
bool empty(const KvSeqs& q) { return q.seqs == 0 || q.T == 0 || q.max_new == 0; }

// The batch's descriptor; its pointers where there is anything to do.
qg_status check_seqs(const qg_kv8_seqs* q, KvSeqs& ks) {
    if (q->seqs < 0 || q->seqs > 65535 || q->width < 1 || q->width > kMaxKv / 16 || q->T < 0 || q->T > kMaxRows)
        return QG_ESHAPE;
    if (q->max_new < 0 || q->max_new > q->T || q->max_kv < q->max_new || q->max_kv > kMaxKv) return QG_ESHAPE;
    ks.table = q->table;
    ks.rows = q->rows;
    ks.kv_len = q->kv_len;
    ks.seqs = q->seqs;
    ks.width = q->width;
    ks.T = q->T;
    ks.max_new = q->max_new;
    ks.max_kv = q->max_kv;
    return QG_OK;
}
qg_status check_seqs_pointers(const qg_kv8_seqs* q) {
    if (!q->table || !q->rows || !q->kv_len) return QG_EINVAL;
    return aligned(q->table, 4) && aligned(q->rows, 4) && aligned(q->kv_len, 4) ? QG_OK : QG_EALIGN;
}

// The cache's and the batch's descriptors.
qg_status check_kv8(const qg_kv8_cache* c, const qg_kv8_seqs* q, KvCache& kc, KvSeqs& ks) {
    if (!c || !q) return QG_EINVAL;
    if (c->dim != 64 && c->dim != 96 && c->dim != 128 && c->dim != 192 && c->dim != 256) return QG_ESHAPE;
    if (c->page < 16 || c->page > 65536 || c->page % 16 != 0 || c->heads < 1 || c->heads > 1024 || c->pages < 1)
        return QG_ESHAPE;
    if ((int64_t)c->pages * c->heads * (c->page / 16) >= ((int64_t)1 << 31)) return QG_ESHAPE;
    const qg_status st = check_seqs(q, ks);
    if (st != QG_OK) return st;
    kc = qg::kv8_cache_of(c->k_codes, c->k_scales, c->v_codes, c->v_scales, c->pages, c->page, c->heads, c->dim);
    if (empty(ks)) return QG_OK;
    if (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales) return QG_EINVAL;
    const qg_status ptrs = check_seqs_pointers(q);
    if (ptrs == QG_EINVAL) return ptrs;
    if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scales, 4) || !aligned(c->v_scales, 4))
        return QG_EALIGN;
    return ptrs;
}

// A [T][heads][dim] operand: rows and heads apart by any multiple of 16 bytes, in either order; an
// output's must not overlap.
qg_status check_rows(const void* p, int xt, int64_t row, int64_t head, int T, int heads, int dim, bool out) {
    if (!p) return QG_EINVAL;
    if (row < 0 || head < 0 || row > kMaxStride || head > kMaxStride) return QG_ESHAPE;
    const bool by_row = head >= dim && row >= (heads - 1) * head + dim;
    const bool by_head = row >= dim && head >= (T - 1) * row + dim;
    if (out && !by_row && !by_head) return QG_ESHAPE;
    if (!aligned(p, 16) || row * xt_bytes(xt) % 16 != 0 || head * xt_bytes(xt) % 16 != 0) return QG_EALIGN;
    return QG_OK;
}

qg_status run_kv8(bool write, const qg_kv8_cache* cache, const qg_kv8_seqs* seqs, void* k, int64_t k_row,
                  int64_t k_head, void* v, int64_t v_row, int64_t v_head, int xt, hipStream_t stream) {
    KvCache c;
    KvSeqs q;
    if (!xt_ok(xt)) return QG_EINVAL;
    qg_status st = check_kv8(cache, seqs, c, q);
    if (st != QG_OK || empty(q)) return st;
    st = check_rows(k, xt, k_row, k_head, q.T, c.heads, c.dim, !write);
    if (st != QG_OK) return st;
    st = check_rows(v, xt, v_row, v_head, q.T, c.heads, c.dim, !write);
    if (st != QG_OK) return st;
    return launched(qg::launch_kv8(write, c, q, k, v, xt, KvStrides{k_row, k_head, v_row, v_head}, stream));
}

// Shared by qg_attn_kv8 and its workspace query.
qg_status attn_params(const qg_kv8_cache* cache, const qg_kv8_seqs* seqs, int q_heads, int causal, int window,
                      int xt, AttnParams& a) {
    const qg_status st = check_kv8(cache, seqs, a.c, a.q);
    if (st != QG_OK) return st;
    if (q_heads < a.c.heads || q_heads > 65536 || q_heads % a.c.heads != 0) return QG_ESHAPE;
    a.q_heads = q_heads;
    a.group = q_heads / a.c.heads;
    a.causal = causal != 0;
    a.window = window > 0 ? window : 0;
    if (empty(a.q)) return QG_OK;
    if ((int64_t)a.q.max_new * q_heads >= ((int64_t)1 << 31)) return QG_ESHAPE;
    // workgroups stay below 2^31: tiles of 128 rows at least, or at most 4 tiles of 16 rows in 6 splits a head
    if ((int64_t)a.q.seqs * a.q.max_new * q_heads >= ((int64_t)1 << 37)) return QG_ESHAPE;
    qg::attn8_plan(a, xt);
    return QG_OK;
}

// qg_attn_kv8, and with a mask in `a` qg_attn_kv8_tree.
qg_status run_attn(AttnParams& a, const qg_kv8_cache* cache, const qg_kv8_seqs* seqs, const void* q, int64_t q_row,
                   int64_t q_head, void* o, int64_t o_row, int64_t o_head, int xt, int q_heads, float scale, int causal,
                   int window, void* workspace, size_t ws_bytes, hipStream_t stream) {
    if (!xt_ok(xt)) return QG_EINVAL;
    qg_status st = attn_params(cache, seqs, q_heads, causal, window, xt, a);
    if (st != QG_OK || empty(a.q)) return st;
    st = check_rows(q, xt, q_row, q_head, a.q.T, q_heads, a.c.dim, false);
    if (st != QG_OK) return st;
    st = check_rows(o, xt, o_row, o_head, a.q.T, q_heads, a.c.dim, true);
    if (st != QG_OK) return st;
    const size_t need = qg::attn8_workspace(a);
    if (need > 0) {
        if (!workspace || ws_bytes < need) return QG_EWORKSPACE;
        if (!aligned(workspace, 16)) return QG_EALIGN;
    }
    a.Q = q;
    a.O = o;
    a.q_row = q_row;
    a.q_head = q_head;
    a.o_row = o_row;
    a.o_head = o_head;
    a.scale = scale;
    return launched(qg::launch_attn8(a, xt, (float*)workspace, stream));
}

// Rotary positions of a head's first `rot` values.
qg_status check_rotary(const qg_rotary* r, int dim, qg::Rotary& out) {
    if (!r) return QG_EINVAL;
    if (r->rot < 0 || r->rot > dim || r->rot % 2 != 0) return QG_ESHAPE;
    if (r->rot > 0 && !r->freqs) return QG_EINVAL;
    if (!aligned(r->freqs, 8)) return QG_EALIGN;
    out.freqs = r->freqs;
    out.rot = r->rot;
    out.inter = r->interleaved != 0;
    out.mscale = r->mscale;
    return QG_OK;
}

// Rows x turned into y, which may be x in the same places.
qg_status check_turned(const void* x, int64_t x_row, int64_t x_head, void* y, int64_t y_row, int64_t y_head, int xt, int T,
                       int heads, int dim, qg::RopeRows& a) {
    qg_status st = check_rows(x, xt, x_row, x_head, T, heads, dim, false);
    if (st != QG_OK) return st;
    st = check_rows(y, xt, y_row, y_head, T, heads, dim, true);
    if (st != QG_OK) return st;
    if (x == y && (x_row != y_row || x_head != y_head)) return QG_ESHAPE;
    a = qg::RopeRows{};
    a.x = x;
    a.y = y;
    a.x_row = x_row;
    a.x_head = x_head;
    a.y_row = y_row;
    a.y_head = y_head;
    a.heads = heads;
    return QG_OK;
}

// The batch of a tree's or a chain's rows.
qg_status check_drafts(const qg_kv8_seqs* seqs, KvSeqs& q) {
    if (!seqs) return QG_EINVAL;
    const qg_status st = check_seqs(seqs, q);
    if (st != QG_OK) return st;
    if (q.max_new > kMaxTree) return QG_ESHAPE;
    return empty(q) ? QG_OK : check_seqs_pointers(seqs);
}

}  // namespace

extern "C" {

qg_status qg_kv8_write(const qg_kv8_cache* cache, const qg_kv8_seqs* seqs, const void* k, int64_t k_row,
                       int64_t k_head, const void* v, int64_t v_row, int64_t v_head, qg_xtype xt,
                       hipStream_t stream) {
    return run_kv8(true, cache, seqs, const_cast<void*>(k), k_row, k_head, const_cast<void*>(v), v_row, v_head, xt,
                   stream);
}

qg_status qg_kv8_read(const qg_kv8_cache* cache, const qg_kv8_seqs* seqs, void* k, int64_t k_row, int64_t k_head,
                      void* v, int64_t v_row, int64_t v_head, qg_xtype yt, hipStream_t stream) {
    return run_kv8(false, cache, seqs, k, k_row, k_head, v, v_row, v_head, yt, stream);
}

size_t qg_attn_kv8_workspace(const qg_kv8_cache* cache, const qg_kv8_seqs* seqs, int q_heads) {
    AttnParams a{};
    if (attn_params(cache, seqs, q_heads, 1, 0, QG_X_F32, a) != QG_OK || empty(a.q)) return 0;
    a.splits = qg::attn8_max_splits(a);
    return qg::attn8_workspace(a);
}

qg_status qg_attn_kv8(const qg_kv8_cache* cache, const qg_kv8_seqs* seqs, const void* q, int64_t q_row,
                      int64_t q_head, void* o, int64_t o_row, int64_t o_head, qg_xtype xt, int q_heads, float scale,
                      int causal, int window, void* workspace, size_t ws_bytes, hipStream_t stream) {
    AttnParams a{};
    return run_attn(a, cache, seqs, q, q_row, q_head, o, o_row, o_head, xt, q_heads, scale, causal, window, workspace,
                    ws_bytes, stream);
}

qg_status qg_attn_kv8_tree(const qg_kv8_cache* cache, const qg_kv8_seqs* seqs, const uint32_t* mask, int words,
                           const int32_t* pos, const void* q, int64_t q_row, int64_t q_head, void* o, int64_t o_row,
                           int64_t o_head, qg_xtype xt, int q_heads, float scale, int window, void* workspace,
                           size_t ws_bytes, hipStream_t stream) {
    if (!seqs) return QG_EINVAL;
    if (seqs->max_new > kMaxTree || words < 1 || words > kMaxTree / 32 || (int64_t)words * 32 < seqs->max_new) return QG_ESHAPE;
    if (seqs->seqs != 0 && seqs->T != 0 && seqs->max_new != 0) {
        if (!mask || (window > 0 && !pos)) return QG_EINVAL;
        if (!aligned(mask, 4) || !aligned(pos, 4)) return QG_EALIGN;
    }
    AttnParams a{};
    a.mask = mask;
    a.pos = pos;
    a.words = words;
    return run_attn(a, cache, seqs, q, q_row, q_head, o, o_row, o_head, xt, q_heads, scale, 0, window, workspace, ws_bytes,
                    stream);
}

size_t qgemm_w8a8_workspace(int N, int K, int T) {
    if (N < 1 || K < 16 || K % 16 != 0 || T < 1) return 0;
    return qg::w8a8_workspace(N, K, T);
}

qg_status qgemm_w8a8(const int8_t* w_codes, const float* w_scales, const void* X, qg_xtype xt, void* Y, qg_xtype yt,
                     int N, int K, int T, void* workspace, size_t ws_bytes, hipStream_t stream) {
    if (!xt_ok(xt) || !xt_ok(yt)) return QG_EINVAL;
    if (N < 1 || N > (1 << 24) || K < 16 || K > (1 << 17) || K % 16 != 0 || T < 0 || T > kMaxRows) return QG_ESHAPE;
    if (T == 0) return QG_OK;
    if (!w_codes || !w_scales || !X || !Y) return QG_EINVAL;
    if (!aligned(w_codes, 16) || !aligned(X, 16) || !aligned(w_scales, 4) || !aligned(Y, (size_t)xt_bytes(yt)))
        return QG_EALIGN;
    const size_t need = qg::w8a8_workspace(N, K, T);
    if (need > 0) {
        if (!workspace || ws_bytes < need) return QG_EWORKSPACE;
        if (!aligned(workspace, 16)) return QG_EALIGN;
    }
    qg::W8A8Params p{};
    p.w = w_codes;
    p.ws = w_scales;
    p.X = X;
    p.Y = Y;
    p.xt = xt;
    p.yt = yt;
    p.N = N;
    p.K = K;
    p.T = T;
    return launched(qg::launch_w8a8(p, workspace, stream));
}

qg_status qg_rope_freqs(qg_rope_scaling scaling, int rot, double base, double factor, double context, double low,
                        double high, double* freqs, float* mscale) {
    const double kTurn = 6.283185307179586;
    if (!freqs || !mscale) return QG_EINVAL;
    if (scaling < QG_ROPE_PLAIN || scaling > QG_ROPE_YARN) return QG_EINVAL;
    if (rot < 2 || rot > kMaxDim || rot % 2 != 0 || (scaling == QG_ROPE_NTK && rot < 4)) return QG_ESHAPE;
    if (!(base > 1.0) || !std::isfinite(base)) return QG_EINVAL;
    if (scaling != QG_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return QG_EINVAL;
    const bool ramped = scaling == QG_ROPE_BANDS || scaling == QG_ROPE_YARN;
    if (ramped && (!(context > 0.0) || !std::isfinite(context) || !(low > 0.0) || !(high > low) || !std::isfinite(high)))
        return QG_EINVAL;
    if (scaling == QG_ROPE_NTK) base *= std::pow(factor, rot / (rot - 2.0));
    // the pair whose angle makes so many turns over the context
    auto pair_of = [&](double turns) { return rot * std::log(context / (turns * kTurn)) / (2.0 * std::log(base)); };
    double first = 0.0, last = 1.0;
    if (scaling == QG_ROPE_YARN) {
        first = std::fmax(std::floor(pair_of(high)), 0.0);
        last = std::fmin(std::ceil(pair_of(low)), rot - 1.0);
        if (last <= first) last = first + 0.001;
    }
    for (int i = 0; i < rot / 2; i++) {
        const double f = std::pow(base, -2.0 * i / rot);
        double keep = 1.0;  // share of the frequency that is not slowed down
        if (scaling == QG_ROPE_LINEAR) keep = 0.0;
        if (scaling == QG_ROPE_BANDS) keep = (context * f / kTurn - low) / (high - low);
        if (scaling == QG_ROPE_YARN) keep = 1.0 - (i - first) / (last - first);
        keep = std::fmin(std::fmax(keep, 0.0), 1.0);
        freqs[i] = scaling == QG_ROPE_PLAIN || scaling == QG_ROPE_NTK ? f : f * keep + f / factor * (1.0 - keep);
    }
    *mscale = scaling == QG_ROPE_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
    return QG_OK;
}

qg_status qg_rope(const qg_rotary* rot, const int32_t* pos, const void* x, int64_t x_row, int64_t x_head, void* y,
                  int64_t y_row, int64_t y_head, qg_xtype xt, int T, int heads, int dim, hipStream_t stream) {
    if (!xt_ok(xt)) return QG_EINVAL;
    if (T < 0 || T > kMaxRows || heads < 1 || heads > 65536 || dim < 8 || dim > kMaxDim || dim % 8 != 0) return QG_ESHAPE;
    qg::Rotary r;
    qg_status st = check_rotary(rot, dim, r);
    if (st != QG_OK || T == 0) return st;
    if (!pos) return QG_EINVAL;
    if (!aligned(pos, 4)) return QG_EALIGN;
    qg::RopeRows a;
    st = check_turned(x, x_row, x_head, y, y_row, y_head, xt, T, heads, dim, a);
    if (st != QG_OK) return st;
    return launched(qg::launch_rope(a, r, pos, T, dim, xt, stream));
}

qg_status qg_kv8_write_rope(const qg_kv8_cache* cache, const qg_kv8_seqs* seqs, const qg_rotary* rot, const int32_t* pos,
                            const void* k, int64_t k_row, int64_t k_head, const void* v, int64_t v_row, int64_t v_head,
                            const int32_t* src, int src_rows, const void* q, int64_t q_row, int64_t q_head, void* q_out,
                            int64_t qo_row, int64_t qo_head, int q_heads, qg_xtype xt, hipStream_t stream) {
    KvCache c;
    KvSeqs s;
    if (!xt_ok(xt)) return QG_EINVAL;
    qg_status st = check_kv8(cache, seqs, c, s);
    if (st != QG_OK) return st;
    qg::KvRope a{};
    st = check_rotary(rot, c.dim, a.rot);
    if (st != QG_OK) return st;
    if (src_rows < 0 || src_rows > kMaxRows || q_heads < 0 || q_heads > 65536) return QG_ESHAPE;
    if (empty(s)) return QG_OK;
    if (q_heads > 0 && src) return QG_EUNSUPPORTED;
    if (!aligned(pos, 4) || !aligned(src, 4)) return QG_EALIGN;
    st = check_rows(k, xt, k_row, k_head, s.T, c.heads, c.dim, false);
    if (st != QG_OK) return st;
    st = check_rows(v, xt, v_row, v_head, s.T, c.heads, c.dim, false);
    if (st != QG_OK) return st;
    if (q_heads > 0) {
        st = check_turned(q, q_row, q_head, q_out, qo_row, qo_head, xt, s.T, q_heads, c.dim, a.q);
        if (st != QG_OK) return st;
    }
    a.k = k;
    a.v = v;
    a.st = KvStrides{k_row, k_head, v_row, v_head};
    a.pos = pos;
    a.src = src;
    a.src_rows = src_rows;
    return launched(qg::launch_kv8_rope(c, s, a, xt, stream));
}

qg_status qg_tree_plan(const qg_kv8_seqs* seqs, const int32_t* parents, uint32_t* mask, int words, int32_t* pos, int window,
                       hipStream_t stream) {
    KvSeqs q;
    const qg_status st = check_drafts(seqs, q);
    if (st != QG_OK) return st;
    if (words < 1 || words > kMaxTree / 32 || words * 32 < q.max_new) return QG_ESHAPE;
    if (empty(q)) return QG_OK;
    if (!parents || !mask || !pos) return QG_EINVAL;
    if (!aligned(parents, 4) || !aligned(mask, 4) || !aligned(pos, 4)) return QG_EALIGN;
    return launched(qg::launch_tree_plan(q, parents, mask, words, pos, window > 0 ? window : 0, stream));
}

size_t qg_draft_verify_workspace(const qg_kv8_seqs* seqs, int vocab) {
    KvSeqs q;
    if (check_drafts(seqs, q) != QG_OK || empty(q) || vocab < 1 || vocab > kMaxVocab) return 0;
    return qg::verify_workspace(q, vocab);
}

qg_status qg_draft_verify(const qg_kv8_seqs* seqs, const int32_t* parents, const int32_t* tokens, const void* target,
                          int64_t t_row, const void* draft, int64_t d_row, qg_xtype xt, int vocab, const float* temps,
                          const float* accept, const float* sample, int32_t* accepted, int32_t* next, int32_t* rows_out,
                          int32_t* path, int32_t* kv_out, void* workspace, size_t ws_bytes, hipStream_t stream) {
    if (!xt_ok(xt)) return QG_EINVAL;
    qg::VerifyParams p{};
    const qg_status st = check_drafts(seqs, p.q);
    if (st != QG_OK) return st;
    if (vocab < 1 || vocab > kMaxVocab || t_row < vocab || t_row > kMaxStride) return QG_ESHAPE;
    if (draft && (d_row < vocab || d_row > kMaxStride)) return QG_ESHAPE;
    if (draft && parents) return QG_EUNSUPPORTED;
    if (empty(p.q)) return QG_OK;
    if (!tokens || !target || !accepted || !next || !rows_out || !path || !kv_out || (draft && sample && !accept)) return QG_EINVAL;
    for (const void* i : {(const void*)parents, (const void*)tokens, (const void*)temps, (const void*)accept,
                          (const void*)sample, (const void*)accepted, (const void*)next, (const void*)rows_out,
                          (const void*)path, (const void*)kv_out})
        if (!aligned(i, 4)) return QG_EALIGN;
    if (!aligned(target, (size_t)xt_bytes(xt)) || !aligned(draft, (size_t)xt_bytes(xt))) return QG_EALIGN;
    if (rows_out == p.q.rows) return QG_EINVAL;  // read while the other is written
    if (!workspace || ws_bytes < qg::verify_workspace(p.q, vocab)) return QG_EWORKSPACE;
    if (!aligned(workspace, 16)) return QG_EALIGN;
    p.parents = parents;
    p.tokens = tokens;
    p.target = target;
    p.draft = sample ? draft : nullptr;  // the largest logit alone decides: the draft's are not asked
    p.t_row = t_row;
    p.d_row = d_row;
    p.xt = xt;
    p.vocab = vocab;
    p.temps = temps;
    p.accept = accept;
    p.sample = sample;
    p.accepted = accepted;
    p.next = next;
    p.rows_out = rows_out;
    p.path = path;
    p.kv_out = kv_out;
    return launched(qg::launch_draft_verify(p, workspace, stream));
}

}  // extern "C"
