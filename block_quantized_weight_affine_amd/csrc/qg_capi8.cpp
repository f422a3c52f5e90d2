// qg_capi8.cpp -- the C ABI of the 8-bit serving operators declared in include/qgemm.h: argument
// validation on the host, before any HIP call, then the launch.
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

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
bool xt_ok(int x) { return x == QG_X_F32 || x == QG_X_F16 || x == QG_X_BF16; }
int64_t xt_bytes(int x) { return x == QG_X_F32 ? 4 : 2; }
qg_status launched(hipError_t e) { return e == hipSuccess ? QG_OK : QG_ELAUNCH; }
bool empty(const KvSeqs& q) { return q.seqs == 0 || q.T == 0 || q.max_new == 0; }

// The cache's and the batch's descriptors.
qg_status check_kv8(const qg_kv8_cache* c, const qg_kv8_seqs* q, KvCache& kc, KvSeqs& ks) {
    if (!c || !q) return QG_EINVAL;
    if (c->dim != 64 && c->dim != 96 && c->dim != 128 && c->dim != 192 && c->dim != 256) return QG_ESHAPE;
    if (c->page < 16 || c->page > 65536 || c->page % 16 != 0 || c->heads < 1 || c->heads > 1024 || c->pages < 1)
        return QG_ESHAPE;
    if ((int64_t)c->pages * c->heads * (c->page / 16) >= ((int64_t)1 << 31)) return QG_ESHAPE;
    if (q->seqs < 0 || q->seqs > 65535 || q->width < 1 || q->width > kMaxKv / 16 || q->T < 0 || q->T > kMaxRows)
        return QG_ESHAPE;
    if (q->max_new < 0 || q->max_new > q->T || q->max_kv < q->max_new || q->max_kv > kMaxKv) return QG_ESHAPE;
    kc = qg::kv8_cache_of(c->k_codes, c->k_scales, c->v_codes, c->v_scales, c->pages, c->page, c->heads, c->dim);
    ks.table = q->table;
    ks.rows = q->rows;
    ks.kv_len = q->kv_len;
    ks.seqs = q->seqs;
    ks.width = q->width;
    ks.T = q->T;
    ks.max_new = q->max_new;
    ks.max_kv = q->max_kv;
    if (empty(ks)) return QG_OK;
    if (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales || !q->table || !q->rows || !q->kv_len)
        return QG_EINVAL;
    if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scales, 4) || !aligned(c->v_scales, 4) ||
        !aligned(q->table, 4) || !aligned(q->rows, 4) || !aligned(q->kv_len, 4))
        return QG_EALIGN;
    return QG_OK;
}

// A [T][heads][dim] operand: rows and heads apart by any multiple of 16 bytes, in either order; an
// output's must not overlap.
qg_status check_rows(const void* p, int xt, int64_t row, int64_t head, int T, int heads, int dim, bool out) {
    constexpr int64_t kMax = (int64_t)1 << 40;
    if (!p) return QG_EINVAL;
    if (row < 0 || head < 0 || row > kMax || head > kMax) return QG_ESHAPE;
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
    if (!xt_ok(xt)) return QG_EINVAL;
    AttnParams a{};
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

}  // extern "C"
