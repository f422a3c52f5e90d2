// qg_attn8_rows.hpp -- attention over the 8-bit key/value cache: the kernel of few rows a K/V head, and the one that
// joins splits.  TREE: the batch's rows see each other by a mask (qg_attn_kv8_tree) and not by causality.
//
//   o = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale q . k_j) over the tokens j that the row may see.
//
// K and V codes are integers of at most 8 bits, exact in f16, so the products run on the f16 matrix
// instructions with f32 sums: q enters as f16 after an exact power of two per row (f32 q as two such
// f16 pieces), the weights as f16 after the block's V scale.  Nothing of the cache is decoded into
// memory.
#pragma once

#include <algorithm>

#include <hip/hip_runtime.h>

#include "qg_attn8.hpp"

namespace qg {
namespace {

// Maximum / sum over the four lane groups of 16 (lanes l, l ^ 16, l ^ 32, l ^ 48).
__device__ __forceinline__ float groups_max(float v) {
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float groups_sum(float v) {
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// Registers a lane that q, two loads and the sums of the rows kernel take; in its largest forms the two loads
// share theirs, and a CU takes one workgroup, of 8 wavefronts.
constexpr int rows_registers(int pieces, int dim) { return (3 + pieces) * dim / 4; }
constexpr bool rows_late(int pieces, int dim) { return rows_registers(pieces, dim) > 200; }

// One workgroup takes 16 rows (query rows times the heads that share a K/V head, counted together) and
// one split of the tokens they see; its W wavefronts take 64 tokens in turn and are joined at the end.
//
// Layout of a wavefront's 64 tokens (four blocks): the first product is K Q^T with A row r of its
// m-th instruction = token 4m + r % 4 of block r / 4, so result lane (row l % 16, group g = l / 16)
// holds all 16 tokens of block g.  That is what the second product V^T P^T wants as its B operand, so
// the weights never move between lanes, every lane has one K and one V scale, and both code loads are
// 16 bytes a lane as the cache holds them.  The next tokens' K is loaded as soon as the first product is
// done with this one's registers, V after the second, the table's entry one turn earlier.
//
// One row a head reads 2 D bytes a token for 4 D G operations (G heads a K/V head), far below the matrix
// instructions' rate for G <= 16: bound by memory.  3 x 200002 tokens, 64 heads of 128 on 8: 219 us, 5.6 TB/s
// of the 1.23 GB that it cannot do without (a copy of this card: 4.8 TB/s read and written); 64 users of up
// to 8192 tokens: 105 us, 4.7 TB/s.  Short calls are bound by the chain of loads (lengths, table, codes) and
// the decoding of one wavefront: 1024 tokens of one user 9.0 us.  Splits that end their own kernel cost 4 us.
template <bool TREE, int XT, int D, int W>
__global__ __launch_bounds__(64 * W, W == 4 && rows_registers(XT == XT_F32 ? 2 : 1, D) <= 128 ? 3 : 2) void attn8_rows_kernel(AttnParams a) {
    constexpr int NP = XT == XT_F32 ? 2 : 1;  // f16 pieces of a q value and of a weight
    constexpr int NH = (D + 63) / 64;         // 16-byte K loads a token
    constexpr int NT = D / 16;
    constexpr int DH = D > 128 ? D / 2 : D;   // dims joined at a time
    constexpr bool kLate = rows_late(NP, D);
    __shared__ float sh_o[W][16][DH + 4];
    __shared__ float sh_m[W][16], sh_l[W][16];
    __shared__ float2 sh_all[16];
    __shared__ FarSum sh_far[W][64];

    const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // The tiles of a head and split read the same codes: eight workgroups apart, they share a die's cache (trees of 8 sequences
    // of 20000 tokens, 48 rows on each of 8 heads of 128: 146 -> 105 us; qg_attn_kv8, bf16, 64 sequences of 2000 on 8 heads of
    // 128, 20 rows each 79 -> 48, 48 114 -> 65, 60 150 -> 83; one sequence of 200 within 0.1 us).
    int b = a.first + blockIdx.x;
    const int tile = b / 8 % a.tiles;
    b = b / 8 / a.tiles * 8 + b % 8;
    const int h = b % a.c.heads;
    b /= a.c.heads;
    const int split = b % a.splits, s = b / a.splits;
    if (s >= a.q.seqs) return;
    const KvSpan sp = kv8_span(a.q, s);
    const int rows = sp.n * a.group;
    if (tile * 16 >= rows) return;
    const TileRange tr = tile_range<TREE>(a, sp, tile * 16, 16);
    if (split > 0 && split >= tr.nact) return;
    const int t0 = tr.lo + split * a.chunk, t1 = min(t0 + a.chunk, tr.hi);

    // this lane's row
    const int r = tile * 16 + col, ri = min(r, rows - 1) / a.group;
    const int head = h * a.group + min(r, rows - 1) % a.group;
    const KvSight see = row_sight<TREE>(a, sp, ri);
    const KvSight first_row = edge_sight<TREE>(a, sp, tile * 16 / a.group, false);
    const int lo_any = first_row.lo, hi_all = first_row.hi;
    const int lo_all = edge_sight<TREE>(a, sp, (min(tile * 16 + 16, rows) - 1) / a.group, true).lo;

    // block of this lane's group in the 64 tokens from tb, and of the group whose K it loads
    auto entry = [&](int tb) {
        const uint32_t pi = kv8_div((uint32_t)((tb >> 4) + g), a.c.nb, a.c.magic);
        return a.q.table[(int64_t)s * a.q.width + min(pi, (uint32_t)a.q.width - 1)];
    };
    auto index = [&](int tb, int page) {
        const int blk = (tb >> 4) + g;
        const uint32_t pi = kv8_div((uint32_t)blk, a.c.nb, a.c.magic);
        return kv8_index(a.c, h, blk, pi, page, (16 * blk < t1) & (16 * blk + 16 > lo_any) & (pi < (uint32_t)a.q.width));
    };
    uint4 kw[4][NH], vw[NT];
    auto load_k = [&](int bi) {
        const int kbi = max(0, __shfl(bi, (lane & 12) * 4));
        const int8_t* kp = a.c.kc + (int64_t)kbi * (16 * D) + (lane & 3) * 16;
#pragma unroll
        for (int mi = 0; mi < 4; mi++)
#pragma unroll
            for (int i = 0; i < NH; i++)
                kw[mi][i] = *(const uint4*)(kp + ((min(4 * i + g, NT - 1) * 16) + 4 * mi) * 16);
    };
    auto load_v = [&](int bi) {
        const int8_t* vp = a.c.vc + (int64_t)max(bi, 0) * (16 * D) + col * 16;
#pragma unroll
        for (int i = 0; i < NT; i++) vw[i] = *(const uint4*)(vp + i * 256);
    };
    const int first = t0 + 64 * wave;
    const int page0 = entry(first), page1 = entry(first + 64 * W);

    float x[NH][16];
    const int64_t at = (int64_t)(sp.r0 + ri) * a.q_row + head * a.q_head;
#pragma unroll
    for (int i = 0; i < NH; i++) {
        const int ch = 4 * i + g;
        float lo[8] = {}, hi[8] = {};
        if (ch < NT) {
            x_load8<XT>(a.Q, at + 16 * ch, lo);
            x_load8<XT>(a.Q, at + 16 * ch + 8, hi);
        }
#pragma unroll
        for (int e = 0; e < 8; e++) x[i][e] = lo[e], x[i][8 + e] = hi[e];
    }
    int bi = index(first, page0), page = page1;
    load_k(bi);
    if (!kLate) load_v(bi);
    float ks = a.c.ks[max(bi, 0)], vs = a.c.vs[max(bi, 0)];

    // q as f16 pieces, scaled so that the row's largest lies in [2^14, 2^15)
    half8_t qf[NP][NH][2];
    float qs;
    {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < NH; i++)
#pragma unroll
            for (int e = 0; e < 16; e++) top = max(top, __float_as_uint(x[i][e]) & 0x7fffffffu);
        top = max(top, (uint32_t)__shfl_xor((int)top, 16));
        top = max(top, (uint32_t)__shfl_xor((int)top, 32));
        const int ex = q_exponent(top);
        qs = ldexpf(a.scale * kLog2e, -ex);
#pragma unroll
        for (int i = 0; i < NH; i++)
#pragma unroll
            for (int e = 0; e < 16; e++) {
                const float v = ldexpf(x[i][e], ex);
                const _Float16 hi = (_Float16)v;
                qf[0][i][e >> 3][e & 7] = hi;
                if constexpr (NP == 2) qf[1][i][e >> 3][e & 7] = (_Float16)(v - (float)hi);
            }
    }

    f32x4_t o[NT];
#pragma unroll
    for (int i = 0; i < NT; i++) o[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    float m = kNegInf, l = 0.f;
    bool any_far = false;  // sh_far holds sums
    int e0 = bi < 0 ? -1000 : v_exponent(vs);
    e0 = max(e0, __shfl_xor(e0, 16));
    e0 = __builtin_amdgcn_readfirstlane(max(e0, __shfl_xor(e0, 32)));
    if (e0 < -500) e0 = 0;

    for (int tb = first; tb < t1; tb += 64 * W) {
        f32x4_t acc[4];
#pragma unroll
        for (int mi = 0; mi < 4; mi++) {
            acc[mi] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < NH; i++) {
                const half8_t k0 = codes8_f16(kw[mi][i].x, kw[mi][i].y), k1 = codes8_f16(kw[mi][i].z, kw[mi][i].w);
#pragma unroll
                for (int n = 0; n < NP; n++) {
                    acc[mi] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, qf[n][i][0], acc[mi], 0, 0, 0);
                    acc[mi] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k1, qf[n][i][1], acc[mi], 0, 0, 0);
                }
            }
        }
        const int was = bi;
        const float vnow = vs, kf = finite_scales(ks, vs) ? ks * qs : __builtin_nanf("");
        const bool more = tb + 64 * W < t1;
        if (kLate) {
            __builtin_amdgcn_sched_barrier(0);
            load_v(bi);
        }
        if (more) {
            bi = index(tb + 64 * W, page);
            if (!kLate) load_k(bi);
            ks = a.c.ks[max(bi, 0)];
            vs = a.c.vs[max(bi, 0)];
            page = entry(tb + 128 * W);
        }
        const float lv = v_power(vnow, e0);
        float p[16];
#pragma unroll
        for (int j = 0; j < 16; j++) p[j] = acc[j >> 2][j & 3] * kf;
        if (tb < lo_all || tb + 64 > hi_all || __any(was < 0)) {
            // tokens of this lane's block that its row sees: [jl, jh)
            const int jl = see.lo - tb - 16 * g, jh = was < 0 ? 0 : see.hi - tb - 16 * g;
            if constexpr (TREE) {
                uint32_t vis = bits_between(jl, jh);
                if (tb + 64 > see.hi) vis |= (uint32_t)drafted_bits(a, sp, ri, tb + 16 * g);
                if (was < 0) vis = 0;
#pragma unroll
                for (int j = 0; j < 16; j++) p[j] = vis >> j & 1 ? p[j] : kNegInf;
            } else {
#pragma unroll
                for (int j = 0; j < 16; j++) p[j] = ((j >= jl) & (j < jh)) ? p[j] : kNegInf;
            }
        }
        if (__any(is_far(lv))) {
            FarSum f = {kNegInf, 0.f};
            if (any_far) f = sh_far[wave][lane];
            if (is_far(lv)) {
                far_add(f, p);
                const float rest = v_power_rest(vnow, e0, lv);
#pragma unroll
                for (int j = 0; j < 16; j++) p[j] += rest;
            }
            sh_far[wave][lane] = f;
            any_far = true;
        }
        float top = p[0];
#pragma unroll
        for (int j = 1; j < 16; j++) top = fmaxf(top, p[j]);
        top += lv;
        if (__any(top > m + kLag)) {
            const float mn = fmaxf(m, groups_max(top));
            const float f = m == kNegInf ? 0.f : __builtin_amdgcn_exp2f(m - mn);
            l *= f;
#pragma unroll
            for (int i = 0; i < NT; i++) o[i] *= f;
            m = mn;
        }
        const float c = lv + above_m(m);
        half8_t pf[NP][2];
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 16; j++) {
            const float w = __builtin_amdgcn_exp2f(p[j] + c);
            sum += w;
            const _Float16 hi = (_Float16)w;
            pf[0][j >> 3][j & 7] = hi;
            if constexpr (NP == 2) pf[1][j >> 3][j & 7] = (_Float16)(w - (float)hi);
        }
        l = fmaf(sum, v_reciprocal(lv), l);
        const half2_t f = __builtin_bit_cast(half2_t, v_sign(vnow)), fc = f * (half2_t){(_Float16)-1152.f, (_Float16)-1152.f};
#pragma unroll
        for (int i = 0; i < NT; i++) {
            const half8_t v0 = codes8_f16(vw[i].x, vw[i].y, f, fc), v1 = codes8_f16(vw[i].z, vw[i].w, f, fc);
#pragma unroll
            for (int n = 0; n < NP; n++) {
                o[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, pf[n][0], o[i], 0, 0, 0);
                o[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, pf[n][1], o[i], 0, 0, 0);
            }
        }
        if (more) {
            if (kLate) {
                __builtin_amdgcn_sched_barrier(0);
                load_k(bi);
            } else {
                load_v(bi);
            }
        }
    }

    // join the wavefronts
    FarSum far = {kNegInf, 0.f};
    if (any_far) {
        far = sh_far[wave][lane];
        far_add(far, __shfl_xor(far.m, 16), __shfl_xor(far.l, 16));
        far_add(far, __shfl_xor(far.m, 32), __shfl_xor(far.l, 32));
    }
    const RowEnd end = row_end(groups_sum(l), m, far, e0);
    if (g == 0) {
        sh_m[wave][col] = end.m;
        sh_l[wave][col] = end.l;
    }
    __syncthreads();
    // each wavefront's sums as its share of the split's mean: no larger than the values, which may lie anywhere in
    // f32's range
    float mt = kNegInf, lt = 0.f;
#pragma unroll
    for (int w = 0; w < W; w++) mt = fmaxf(mt, sh_m[w][col]);
#pragma unroll
    for (int w = 0; w < W; w++)
        lt += sh_l[w][col] * (sh_m[w][col] == kNegInf ? 1.f : __builtin_amdgcn_exp2f(sh_m[w][col] - mt));
    const float share = end.m == kNegInf ? 0.f : __builtin_amdgcn_exp2f(end.m - mt) / lt;
    if (threadIdx.x < 16) sh_all[col] = make_float2(mt, lt);
#pragma unroll
    for (int d0 = 0; d0 < D; d0 += DH) {
        if (d0) __syncthreads();
#pragma unroll
        for (int i = 0; i < DH / 16; i++) {
            const f32x4_t v = ldexp4(o[d0 / 16 + i] * share, end.e);
            *(f32x4_t*)&sh_o[wave][col][16 * i + 4 * g] = v;
        }
        __syncthreads();
        for (int x = threadIdx.x; x < 16 * (DH / 4); x += 64 * W) {
            const int row = x / (DH / 4), d = 4 * (x % (DH / 4));
            const int rr = tile * 16 + row;
            if (rr >= rows) continue;
            f32x4_t v = *(const f32x4_t*)&sh_o[0][row][d];
#pragma unroll
            for (int w = 1; w < W; w++) v += *(const f32x4_t*)&sh_o[w][row][d];
            const int64_t trow = sp.r0 + rr / a.group;
            const int hd = h * a.group + rr % a.group;
            if (tr.nact > 1) {
                const int64_t pi = (trow * a.q_heads + hd) * a.splits + split;
                *(f32x4_t*)(a.part_o + pi * D + d0 + d) = v;
                if (d0 + d == 0) *(float2*)(a.part_ml + pi * 2) = sh_all[row];
            } else {
                const int64_t at = trow * a.o_row + hd * a.o_head + d0 + d;
                if constexpr (XT == XT_F32)
                    *(f32x4_t*)((float*)a.O + at) = v;
                else {
                    u32x2_t y;
                    y[0] = (uint32_t)f32_to_16<XT>(v[0]) | (uint32_t)f32_to_16<XT>(v[1]) << 16;
                    y[1] = (uint32_t)f32_to_16<XT>(v[2]) | (uint32_t)f32_to_16<XT>(v[3]) << 16;
                    *(u32x2_t*)((uint16_t*)a.O + at) = y;
                }
            }
        }
    }
}

template <int XT>
__device__ __forceinline__ void store2(void* o, int64_t at, float a, float b) {
    if constexpr (XT == XT_F32)
        *(float2*)((float*)o + at) = make_float2(a, b);
    else
        *(uint32_t*)((uint16_t*)o + at) = (uint32_t)f32_to_16<XT>(keep_f32(a)) | (uint32_t)f32_to_16<XT>(keep_f32(b)) << 16;
}

// Joins the splits of a row and head, each a mean with its weight: W wavefronts take the splits in turn, 4 / W
// rows a workgroup.  The order of the sums is fixed, so results repeat bit for bit.
template <bool TREE, int XT, int D, int W>
__global__ __launch_bounds__(256) void attn8_join_kernel(AttnParams a) {
    constexpr int NV = (D + 127) / 128;  // pairs of dims a lane
    __shared__ float sh_o[W > 1 ? 4 : 1][D];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int s = blockIdx.y;
    const uint32_t x = W > 1 ? blockIdx.x : 4 * blockIdx.x + wave;
    const int i = x / (uint32_t)a.q_heads, head = x % (uint32_t)a.q_heads;
    const KvSpan sp = kv8_span(a.q, s);
    if (i >= sp.n) return;
    const int r = i * a.group + head % a.group;
    const TileRange tr = tile_range<TREE>(a, sp, r / a.tile_rows * a.tile_rows, a.tile_rows);
    if (tr.nact <= 1) return;
    const int64_t p0 = ((int64_t)(sp.r0 + i) * a.q_heads + head) * a.splits;
    float2 ml = make_float2(kNegInf, 0.f);
    if (lane < tr.nact) ml = *(const float2*)(a.part_ml + (p0 + lane) * 2);
    float mt = ml.x, l = ml.y;
    for (int x = lane + 64; x < tr.nact; x += 64) {
        const float2 next = *(const float2*)(a.part_ml + (p0 + x) * 2);
        const float mn = fmaxf(mt, next.x);
        l = fmaf(l, mt == kNegInf ? 1.f : __builtin_amdgcn_exp2f(mt - mn),
                 next.y * (next.x == kNegInf ? 1.f : __builtin_amdgcn_exp2f(next.x - mn)));
        mt = mn;
    }
    float mu = mt;
#pragma unroll
    for (int e = 1; e < 64; e <<= 1) mu = fmaxf(mu, __shfl_xor(mu, e));
    if (mt != kNegInf) l *= __builtin_amdgcn_exp2f(mt - mu);
#pragma unroll
    for (int e = 1; e < 64; e <<= 1) l += __shfl_xor(l, e);
    if (mu == kNegInf) mu = 0.f;
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    float2 o[NV];
#pragma unroll
    for (int e = 0; e < NV; e++) o[e] = make_float2(0.f, 0.f);
    for (int x0 = 0; x0 < tr.nact; x0 += 64) {
        // a lane has a split's share; the sums take eight splits' loads at a time
        if (x0 > 0) {
            ml = make_float2(kNegInf, 0.f);
            if (x0 + lane < tr.nact) ml = *(const float2*)(a.part_ml + (p0 + x0 + lane) * 2);
        }
        const float w = ml.y == 0.f ? 0.f : __builtin_amdgcn_exp2f(ml.x - mu) * (ml.y * inv);
        const int n = min(tr.nact - x0, 64);
        for (int y = W > 1 ? wave : 0; y < n; y += 8 * W) {
            float2 v[8][NV];
#pragma unroll
            for (int k = 0; k < 8; k++)
#pragma unroll
                for (int e = 0; e < NV; e++) {
                    const int d = 2 * lane + 128 * e;
                    v[k][e] = *(const float2*)(a.part_o + (p0 + x0 + min(y + k * W, n - 1)) * D + (d < D ? d : 0));
                }
#pragma unroll
            for (int k = 0; k < 8; k++) {
                const float f = y + k * W < n ? __shfl(w, y + k * W) : 0.f;
#pragma unroll
                for (int e = 0; e < NV; e++)
                    if (y + k * W < n) o[e].x = fmaf(v[k][e].x, f, o[e].x), o[e].y = fmaf(v[k][e].y, f, o[e].y);
            }
        }
    }
    const int64_t at = (int64_t)(sp.r0 + i) * a.o_row + head * a.o_head;
    if constexpr (W == 1) {
#pragma unroll
        for (int e = 0; e < NV; e++) {
            const int d = 2 * lane + 128 * e;
            if (d < D) store2<XT>(a.O, at + d, o[e].x, o[e].y);
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < NV; e++) {
        const int d = 2 * lane + 128 * e;
        if (d < D) *(float2*)&sh_o[wave][d] = o[e];
    }
    __syncthreads();
    const int d = 2 * threadIdx.x;
    if (d >= D) return;
    float y[2];
#pragma unroll
    for (int e = 0; e < 2; e++)
        y[e] = sh_o[0][d + e] + sh_o[W > 1 ? 1 : 0][d + e] + sh_o[W > 1 ? 2 : 0][d + e] + sh_o[W > 1 ? 3 : 0][d + e];
    store2<XT>(a.O, at + d, y[0], y[1]);
}

constexpr int64_t kJoinWide = 2048;  // rows that are joined by a workgroup each, where a wavefront has more than 8 splits to read

template <bool TREE, int XT, int D>
hipError_t launch_one(AttnParams a, hipStream_t s) {
    const int64_t grid = ((int64_t)a.q.seqs * a.splits * a.c.heads + 7) / 8 * 8 * a.tiles;
    if (a.tile_rows > 16) {
        const hipError_t e = TREE ? launch_attn8_tree_tile(a, XT, s) : launch_attn8_tile(a, XT, s);
        if (e != hipSuccess) return e;
    } else {
        for (int64_t first = 0; first < grid; first += kLaunchGroups) {
            a.first = (int)first;
            const dim3 part((uint32_t)std::min(grid - first, kLaunchGroups));
            if (a.row_waves == 8)
                attn8_rows_kernel<TREE, XT, D, 8><<<part, 512, 0, s>>>(a);
            else if constexpr (!rows_late(XT == XT_F32 ? 2 : 1, D))
                attn8_rows_kernel<TREE, XT, D, 4><<<part, 256, 0, s>>>(a);
        }
    }
    if (a.splits > 1) {
        const uint32_t rows = (uint32_t)a.q.max_new * (uint32_t)a.q_heads;
        if (a.splits > 8 && (int64_t)rows * a.q.seqs <= kJoinWide)
            attn8_join_kernel<TREE, XT, D, 4><<<dim3(rows, a.q.seqs), 256, 0, s>>>(a);
        else
            attn8_join_kernel<TREE, XT, D, 1><<<dim3((rows + 3) / 4, a.q.seqs), 256, 0, s>>>(a);
    }
    return hipGetLastError();
}

template <bool TREE, int XT>
hipError_t launch_dim(const AttnParams& a, hipStream_t s) {
    switch (a.c.dim) {
        case 64: return launch_one<TREE, XT, 64>(a, s);
        case 96: return launch_one<TREE, XT, 96>(a, s);
        case 128: return launch_one<TREE, XT, 128>(a, s);
        case 192: return launch_one<TREE, XT, 192>(a, s);
        case 256: return launch_one<TREE, XT, 256>(a, s);
    }
    return hipErrorInvalidValue;
}

template <bool TREE>
hipError_t launch_rows(const AttnParams& a, int xt, hipStream_t s) {
    if (xt == XT_F32) return launch_dim<TREE, XT_F32>(a, s);
    if (xt == XT_F16) return launch_dim<TREE, XT_F16>(a, s);
    return launch_dim<TREE, XT_BF16>(a, s);
}

}  // namespace
}  // namespace qg
