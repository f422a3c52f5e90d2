// qg_kv8.hpp -- the 8-bit key/value cache: where a token lies, and which tokens a sequence has.
//
// Plain C++, shared by the kernels and by host code.  Every index that comes from device memory (block
// table, row offsets, lengths) passes through kv8_span and kv8_index, which turn what does not fit
// into "no rows" and "no block", so no kernel address depends on an unchecked value.
#pragma once

#include <stdint.h>

#ifdef __HIPCC__
#include <hip/hip_runtime.h>
#define QG_HD __host__ __device__ __forceinline__
#else
#define QG_HD inline
#endif

namespace qg {

constexpr int kKvBlock = 16;  // tokens that share a scale

// A page holds `page` tokens of every head; block b of head h in page p has index
// (p * heads + h) * nb + b, its codes 16 * dim bytes: K [dim/16][16 tokens][16 dims], V [dim][16 tokens].
struct KvCache {
    int8_t* kc;
    float* ks;
    int8_t* vc;
    float* vs;
    int pages, heads, dim;
    int nb;          // blocks of a page and head
    uint32_t magic;  // ceil(2^32 / nb) for nb >= 2: blk / nb = (blk * magic) >> 32 while blk * nb < 2^32
};

struct KvSeqs {
    const int32_t* table;   // [seqs][width] pages
    const int32_t* rows;    // [seqs + 1] first row of each sequence
    const int32_t* kv_len;  // [seqs] tokens of each sequence, its new rows included
    int seqs, width, T, max_new, max_kv;
};

// Rows r0 .. r0 + n - 1 are the last n of the sequence's len tokens.
struct KvSpan {
    int r0, n, len;
};

QG_HD KvSpan kv8_span_of(int r0, int r1, int len, int T, int max_new, int max_kv) {
    const bool ok = r0 >= 0 && r1 >= r0 && r1 <= T && r1 - r0 <= max_new && len <= max_kv && r1 - r0 <= len;
    KvSpan v;
    v.r0 = ok ? r0 : 0;
    v.n = ok ? r1 - r0 : 0;
    v.len = ok ? len : 0;
    return v;
}

QG_HD KvSpan kv8_span(const KvSeqs& q, int s) {
    return kv8_span_of(q.rows[s], q.rows[s + 1], q.kv_len[s], q.T, q.max_new, q.max_kv);
}

QG_HD uint32_t kv8_div(uint32_t blk, int nb, uint32_t magic) {
    return nb == 1 ? blk : (uint32_t)(((uint64_t)blk * magic) >> 32);
}

// Index of token block blk (tokens 16 blk ..) of head h in `page`, the table's entry pi = blk / nb, or -1 where
// that is no page (or `there` is false).
QG_HD int kv8_index(const KvCache& c, int h, int blk, uint32_t pi, int page, bool there) {
    const bool ok = there & ((uint32_t)page < (uint32_t)c.pages);
    return ok ? (int)(((uint32_t)page * c.heads + h) * c.nb + ((uint32_t)blk - pi * (uint32_t)c.nb)) : -1;
}

// Index of token block blk of sequence s and head h, or -1 where the table has no page for it.
QG_HD int kv8_block(const KvCache& c, const KvSeqs& q, int s, int h, int blk) {
    if (blk < 0) return -1;
    const uint32_t pi = kv8_div((uint32_t)blk, c.nb, c.magic);
    if (pi >= (uint32_t)q.width) return -1;
    return kv8_index(c, h, blk, pi, q.table[(int64_t)s * q.width + pi], true);
}

QG_HD KvCache kv8_cache_of(int8_t* kc, float* ks, int8_t* vc, float* vs, int pages, int page, int heads, int dim) {
    KvCache c;
    c.kc = kc;
    c.ks = ks;
    c.vc = vc;
    c.vs = vs;
    c.pages = pages;
    c.heads = heads;
    c.dim = dim;
    c.nb = page / kKvBlock;
    c.magic = c.nb < 2 ? 0u : (uint32_t)((0x100000000ull + (uint64_t)c.nb - 1) / (uint64_t)c.nb);
    return c;
}

// Tokens that query row r of a tile may see: [lo, hi).
struct KvSight {
    int lo, hi;
};
QG_HD KvSight kv8_sight(const KvSpan& v, int i, int causal, int window) {
    const int p = v.len - v.n + i;  // position of the sequence's row i
    KvSight g;
    g.lo = window > 0 && p - window + 1 > 0 ? p - window + 1 : 0;
    g.hi = causal ? p + 1 : v.len;
    return g;
}

}  // namespace qg
