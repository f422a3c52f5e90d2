// qg_attn8_tile.hpp -- attention over the 8-bit cache for many rows a K/V head: prompts, chunks and large trees.  TREE:
// the batch's rows see each other by a mask (qg_attn_kv8_tree) and not by causality.
#pragma once

#include <algorithm>

#include <hip/hip_runtime.h>

#include "qg_attn8.hpp"

namespace qg {
namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

constexpr int kInfo = 256;  // blocks looked up at a time
// Two workgroups of the kernel of 128 rows share a CU.
template <int XT, int D, int NW>
constexpr bool kPair = NW == 4 && XT != XT_F32 && D <= 128;

// All lanes' LDS reads and writes so far are done, in every wavefront; loads from memory stay in flight.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Keeps a value's computation where it stands.
__device__ __forceinline__ half2_t stay(half2_t v) {
    asm volatile("" : "+v"(v));
    return v;
}

__device__ __forceinline__ float stay(float v) {
    asm volatile("" : "+v"(v));
    return v;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}

// A workgroup of NW wavefronts takes 32 CT NW rows (query rows times the heads that share a K/V head,
// counted together), each wavefront 32 CT of them, and walks over the tokens they see in stages of 64.
// A stage's codes are decoded once for all rows, into f16 in shared memory in the order in which the
// matrix instructions take them, so every read is 1 KiB without conflicts:
//   K  [dim/8][64 tokens][8 dims]        A operand of S = K Q^T (32 tokens x 32 rows a product)
//   V  [block][half g][dim][8 tokens]    A operand of O = V^T P^T, tokens 4g..4g+3, 4g+8..4g+11
// which is the order in which lane (row l % 32, half g = l / 32) holds its weights after S, so they
// never move between lanes.  Stage t + 1's S is multiplied between the weights of stage t, and O of stage t
// between the maxima and the decoding; an instruction stream is laid out by hand for it (sched_barrier).
//
// Bound by the instructions between the products and by power.  2 x 4096 prompt tokens, 32 heads of 128:
// 293 us, 0.94 PFLOP/s (a product of 8192^3 in f16: 1.46).  A stage of 256 rows takes 3550 cycles, 2048 of
// them products and about 2300 vector instructions of two wavefronts a SIMD; the clock falls to 1.8 GHz from
// the 2.4 GHz that the same kernel has on zeros.  A workgroup's start (lengths, table, scales, first codes)
// takes 5-6 us, its end 2 us.  Measured against it: 64 rows a wavefront and one wavefront a SIMD 25 % slower
// a stage (one wavefront issues an instruction every 6.5 cycles), 32-token stages 10 %, half of the
// wavefronts half a stage behind the others the same.
template <bool TREE, int XT, int D, int NW, int CT>
__global__ __launch_bounds__(64 * NW, (kPair<XT, D, NW> ? 2 : 1)) void attn8_tile_kernel(AttnParams a) {
    constexpr int NP = XT == XT_F32 ? 2 : 1;  // f16 pieces of a q value and of a weight
    constexpr int NK = D / 16, NT = D / 32;
    constexpr int UN = (D / 16 + NW - 1) / NW;  // 1 KiB pieces of K, and of V, that a wavefront decodes
    constexpr int BR = 32 * CT * NW;
    constexpr int KB = D > 192 || (D == 128 && NW == 4) ? 2 : 3;  // stages of K in shared memory
    constexpr bool kEven = NK % NW == 0;
    __shared__ __attribute__((aligned(16))) uint4 sk[KB * 8 * D], sv[2][8 * D];
    __shared__ __attribute__((aligned(16))) int in_bi[2 * kInfo];
    __shared__ __attribute__((aligned(16))) float in_ks[2 * kInfo], in_lv[2 * kInfo], in_rv[2 * kInfo];
    __shared__ uint32_t in_sg[2 * kInfo];
    __shared__ int in_top[NW];
    __shared__ FarSum sh_far[NW][CT][64];
    // A tree's rows: the first token that each may see, and which tokens of the last stages it does; n drafted tokens lie
    // in no more than (n + 62) / 64 + 1 stages.
    constexpr int kEdge = ((kPair<XT, D, NW> ? kPairTreeRows : kMaxTreeRows) + 62) / 64 + 1;
    __shared__ uint64_t sh_vis[TREE ? kEdge : 1][TREE ? 32 * CT * NW : 1];
    __shared__ int sh_lo[TREE ? 32 * CT * NW : 1];
    bool any_far = false;  // sh_far holds sums

    const int lane = threadIdx.x & 63, col = lane & 31, g = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // sequences and heads first, so that the workgroups of one K/V head share a die's cache; of each sequence
    // the last tile, which sees the most, first, so that the workgroups with nothing to do come last
    int b = a.first + blockIdx.x;
    const int pairs = a.q.seqs * a.c.heads;
    const int h = b % pairs % a.c.heads, s = b % pairs / a.c.heads;
    b /= pairs;
    const int split = b % a.splits;
    const KvSpan sp = kv8_span(a.q, s);
    const int rows = sp.n * a.group;
    const int tile = (rows + BR - 1) / BR - 1 - b / a.splits;
    if (tile < 0) return;
    const TileRange tr = tile_range<TREE>(a, sp, tile * BR, BR);
    if (split > 0 && split >= tr.nact) return;
    const int t0 = tr.lo + split * a.chunk, t1 = min(t0 + a.chunk, tr.hi);
    const int stages = (t1 - t0 + 63) / 64;

    // rows of this wavefront, and what all of them see
    const int w0 = tile * BR + wave * 32 * CT;
    const int lo_all = edge_sight<TREE>(a, sp, min(w0 + 32 * CT, rows) <= w0 ? 0 : (min(w0 + 32 * CT, rows) - 1) / a.group, true).lo;
    const int hi_all = edge_sight<TREE>(a, sp, min(w0, rows - 1) / a.group, false).hi;
    const int lo_any = edge_sight<TREE>(a, sp, tile * BR / a.group, false).lo;

    // What the kernel has to know of each block, looked up by a thread each for 64 stages at a time: its
    // index (-1: hidden from all), the K scale, and the V scale relative to 2^e0 as a power of two, its
    // reciprocal and its sign.  A NaN or infinite scale, K's or V's, becomes a K scale of NaN: rows that see
    // the block are NaN, others whole.
    const int tid = threadIdx.x;
    auto page_of = [&](int blk) {
        const uint32_t pi = kv8_div((uint32_t)blk, a.c.nb, a.c.magic);
        return a.q.table[(int64_t)s * a.q.width + min(pi, (uint32_t)a.q.width - 1)];
    };
    auto index_of = [&](int blk, int page) {
        const uint32_t pi = kv8_div((uint32_t)blk, a.c.nb, a.c.magic);
        return kv8_index(a.c, h, blk, pi, page, (16 * blk < t1) & (16 * blk + 16 > lo_any) & (pi < (uint32_t)a.q.width));
    };
    const int my_blk = (t0 >> 4) + tid;  // plus kInfo a segment
    // the first stages' codes set out before anything waits for their scales
    int page0 = 0, first[KB + 1];
    if (tid < kInfo) page0 = page_of(my_blk);
#pragma unroll
    for (int i = 0; i <= KB; i++) first[i] = page_of((t0 >> 4) + 4 * i + (lane >> 4));

    // q sets out too, and is made operands of when everything else is on its way
    constexpr int QW = XT == XT_F32 ? 2 : 1;
    uint4 qraw[CT][NK][QW];
    KvSight see[CT];
#pragma unroll
    for (int c = 0; c < CT; c++) {
        const int r = min(w0 + 32 * c + col, rows - 1), ri = r / a.group, head = h * a.group + r % a.group;
        if constexpr (!TREE) see[c] = row_sight<TREE>(a, sp, ri);
        const int64_t at = (int64_t)(sp.r0 + ri) * a.q_row + head * a.q_head + 8 * g;
#pragma unroll
        for (int k = 0; k < NK; k++)
#pragma unroll
            for (int i = 0; i < QW; i++) qraw[c][k][i] = ((const uint4*)((const char*)a.Q + (at + 16 * k) * (2 * QW)))[i];
    }
    __builtin_amdgcn_sched_barrier(0);

    if constexpr (TREE) {
        for (int x = tid; x < BR; x += 64 * NW) {
            const int i = min(tile * BR + x, rows - 1) / a.group;
            sh_lo[x] = row_sight<TREE>(a, sp, i).lo;
            // the first stage that holds a token behind hi_all, and those that follow
            int tb = t0 + (max(hi_all - t0, 0) & ~63);
#pragma unroll 1
            for (int k = 0; k < kEdge && tb < t1; k++, tb += 64)
                sh_vis[min((tb + 63 - hi_all) >> 6, kEdge - 1)][x] = ones64(hi_all - tb) | drafted_bits(a, sp, i, tb);
        }
    }
    int bi0 = -1, e0 = 0, eb = -1000;
    float ks0 = 0.f, vs0 = 0.f;
    if (tid < kInfo) {
        bi0 = index_of(my_blk, page0);
        ks0 = a.c.ks[max(bi0, 0)];
        vs0 = a.c.vs[max(bi0, 0)];
    }
#pragma unroll
    for (int i = 0; i <= KB; i++) first[i] = index_of((t0 >> 4) + 4 * i + (lane >> 4), first[i]);
    auto note = [&](int seg, int bi, float ks, float vs) {
        const int x = (kInfo * seg + tid) & (2 * kInfo - 1);
        const float lv = bi < 0 ? 0.f : v_power(vs, e0);
        in_bi[x] = bi;
        // a far block's K scale is below 0 here, and its sign that of the zero beside it: scale_and_hide tells far
        // blocks by what it looks at for negative scales
        const float k = is_far(lv) ? -fabsf(ks) : ks;
        in_ks[x] = bi < 0 ? -1.f : finite_scales(ks, vs) ? k : __builtin_nanf("");
        in_lv[x] = lv;
        in_rv[x] = is_far(lv) ? copysignf(0.f, ks) : v_reciprocal(lv);
        in_sg[x] = v_sign(vs);
    };

    auto block_k = [&](int st) { return max(in_bi[(4 * st + (lane >> 4)) & (2 * kInfo - 1)], 0); };
    auto load_k = [&](int bi, uint4 (&raw)[UN]) {
        const int8_t* p = a.c.kc + (int64_t)bi * (16 * D) + (lane & 15) * 16;
#pragma unroll
        for (int i = 0; i < UN; i++)
            if (kEven || wave + NW * i < NK) raw[i] = *(const uint4*)(p + (wave + NW * i) * 256);
    };
    // half x % 2 of piece x / 2, of K or V
    auto store_k = [&](int x, const uint4 (&raw)[UN], uint4* to) {
        const int i = x >> 1;
        if (kEven || wave + NW * i < NK)
            to[(wave + NW * i) * 128 + 64 * (x & 1) + lane] =
                __builtin_bit_cast(uint4, x & 1 ? codes8_f16(raw[i].z, raw[i].w) : codes8_f16(raw[i].x, raw[i].y));
    };
    // V piece u: the 64 (block, dim) pairs from 64 u
    auto piece_v = [&](int i) { return NW - 1 - wave + NW * i; };
    auto place_v = [&](int i, int& j, int& d) {
        const int x = 64 * piece_v(i) + lane;
        j = x / D;
        d = x - j * D;
    };
    auto load_v = [&](int st, uint4 (&raw)[UN]) {
#pragma unroll
        for (int i = 0; i < UN; i++)
            if (kEven || piece_v(i) < NK) {
                int j, d;
                place_v(i, j, d);
                const int bi = in_bi[(4 * st + j) & (2 * kInfo - 1)];
                raw[i] = *(const uint4*)(a.c.vc + (int64_t)max(bi, 0) * (16 * D) + d * 16);
            }
    };
    auto sign_v = [&](int st, half2_t (&sign)[UN]) {
#pragma unroll
        for (int i = 0; i < UN; i++)
            if (kEven || piece_v(i) < NK) {
                int j, d;
                place_v(i, j, d);
                sign[i] = __builtin_bit_cast(half2_t, in_sg[(4 * st + j) & (2 * kInfo - 1)]);
            }
    };
    auto store_v = [&](int x, const uint4 (&raw)[UN], const half2_t (&sign)[UN], uint4* to) {
        const int i = x >> 1;
        if (kEven || piece_v(i) < NK) {
            int j, d;
            place_v(i, j, d);
            const half2_t f = sign[i], c = f * (half2_t){(_Float16)-1152.f, (_Float16)-1152.f};
            u32x4 w;
            uint32_t p, q;
            codes4_f16(x & 1 ? raw[i].y : raw[i].x, f, c, p, q);
            w[0] = p, w[1] = q;
            codes4_f16(x & 1 ? raw[i].w : raw[i].z, f, c, p, q);
            w[2] = p, w[3] = q;
            to[2 * j * D + (x & 1) * D + d] = __builtin_bit_cast(uint4, w);
        }
    };

    half8_t qf[CT][NP][NK];
    float qs[CT];

    // A weight is exp2(score + V scale's power - m + kBase), m the running maximum of what comes before
    // it: it has the V scale in it, and its sum for the denominator is taken times the reciprocal.
    f32x16_t o[CT][NT] = {};
    float m[CT], l[CT], limit[CT], mu[CT];  // mu: kBase - m
#pragma unroll
    for (int c = 0; c < CT; c++) m[c] = limit[c] = kNegInf, l[c] = 0.f, mu[c] = (float)kBase;
    float kf[CT][4], cf[CT][4];  // factor and addend of a score

    // Stage st's scales; where a row does not see all of it, or a scale is negative, NaN, infinite or far, the
    // scores are scaled and hidden one by one.
    f32x4_t kb, lv, rv, rn;
    auto read_scales = [&](int st) {
        const int x = (4 * st) & (2 * kInfo - 1);
        kb = *(const f32x4_t*)&in_ks[x];
        lv = *(const f32x4_t*)&in_lv[x];
        rn = *(const f32x4_t*)&in_rv[x];
    };
    auto scale_and_hide = [&](int st, f32x16_t (&sc)[CT][2]) {
        const int tb = t0 + 64 * st, x = (4 * st) & (2 * kInfo - 1);
        uint32_t odd = 0;
#pragma unroll
        for (int q = 0; q < 4; q++) odd = max(odd, __float_as_uint(kb[q]));
#pragma unroll
        for (int c = 0; c < CT; c++)
#pragma unroll
            for (int q = 0; q < 4; q++) kf[c][q] = kb[q] * qs[c];
        if ((tb < lo_all) | (tb + 64 > hi_all) | (__builtin_amdgcn_readfirstlane((int)(odd >> 23)) >= 255)) {
            const i32x4_t bi = *(const i32x4_t*)&in_bi[x];
#pragma unroll
            for (int c = 0; c < CT; c++) {
                int jl = 0, jh = 0;
                uint64_t vis = 0;
                if constexpr (TREE) {
                    const int row = wave * 32 * CT + 32 * c + col, edge = (tb + 63 - hi_all) >> 6;
                    vis = tb + 64 > hi_all ? sh_vis[min(edge, kEdge - 1)][row] : ~0ull;
                    vis = (vis & ~ones64(sh_lo[row] - tb)) >> (4 * g);
                } else {
                    jl = see[c].lo - tb - 4 * g, jh = see[c].hi - tb - 4 * g;
                }
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    if (is_far(lv[q])) kf[c][q] = copysignf(kb[q], rn[q]) * qs[c];
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        const int j = 16 * q + 8 * (e >> 2) + (e & 3);
                        const bool on = (bi[q] >= 0) & (TREE ? (bool)(vis >> j & 1) : (j >= jl) & (j < jh));
                        sc[c][q >> 1][8 * (q & 1) + e] = on ? sc[c][q >> 1][8 * (q & 1) + e] * kf[c][q] : kNegInf;
                    }
                    kf[c][q] = 1.f;
                }
            }
            float far = 0.f;
#pragma unroll
            for (int q = 0; q < 4; q++) far = fmaxf(far, fabsf(lv[q]));
            if (is_far(__uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(far))))) {
#pragma unroll
                for (int c = 0; c < CT; c++) {
                    FarSum f = {kNegInf, 0.f};
                    if (any_far) f = sh_far[wave][c][lane];
#pragma unroll
                    for (int q = 0; q < 4; q++) {
                        if (!is_far(lv[q])) continue;
                        float s[8];
#pragma unroll
                        for (int e = 0; e < 8; e++) s[e] = sc[c][q >> 1][8 * (q & 1) + e];
                        far_add(f, s);
                        const float rest = v_power_rest(a.c.vs[max(bi[q], 0)], e0, lv[q]);
#pragma unroll
                        for (int e = 0; e < 8; e++) sc[c][q >> 1][8 * (q & 1) + e] += rest;
                    }
                    sh_far[wave][c][lane] = f;
                }
                any_far = true;
            }
        }
    };
    float top[CT], part[CT];
    auto top_pair = [&](int x, const f32x16_t (&sc)[CT][2]) {  // scores 2x, 2x + 1 of the 32 of a column
        const int q = x >> 2;
#pragma unroll
        for (int c = 0; c < CT; c++) {
            const float u = sc[c][x >> 3][2 * x & 15], v = sc[c][x >> 3][(2 * x & 15) + 1];
            part[c] = x & 3 ? max3(part[c], u, v) : max3(u, v, v);
            if ((x & 3) == 3) {
                const float t = fmaf(part[c], kf[c][q], lv[q]);
                top[c] = q ? fmaxf(top[c], t) : t;
            }
        }
    };
    // The sums are rescaled where a maximum grew by more than kLag.
    auto settle = [&]() {
        bool grew = false;
#pragma unroll
        for (int c = 0; c < CT; c++) grew |= top[c] > limit[c];
        if (__any(grew)) {
#pragma unroll
            for (int c = 0; c < CT; c++) {
                const float mn = fmaxf(m[c], fmaxf(top[c], __shfl_xor(top[c], 32)));
                const float f = m[c] == kNegInf ? 0.f : __builtin_amdgcn_exp2f(m[c] - mn);
                l[c] *= f;
#pragma unroll
                for (int i = 0; i < NT; i++)
#pragma unroll
                    for (int e = 0; e < 16; e++) o[c][i][e] *= f;
                m[c] = mn;
                limit[c] = mn + kLag;
                mu[c] = above_m(mn);
            }
        }
        rv = rn;
#pragma unroll
        for (int c = 0; c < CT; c++)
#pragma unroll
            for (int q = 0; q < 4; q++) cf[c][q] = lv[q] + mu[c];
    };
    // The weights of scores 2x, 2x + 1 in three steps that different pairs take at the same time, so that no
    // instruction waits for the one before it.
    half8_t pf[CT][NP][4];
    float sum[CT], arg[CT][16][2], wt[CT][16][2];
    auto weigh_1 = [&](int x, const f32x16_t (&sc)[CT][2]) {
        const int q = x >> 2;
#pragma unroll
        for (int c = 0; c < CT; c++)
#pragma unroll
            for (int e = 0; e < 2; e++) arg[c][x][e] = stay(fmaf(sc[c][x >> 3][(2 * x & 15) + e], kf[c][q], cf[c][q]));
    };
    auto weigh_2 = [&](int x) {
#pragma unroll
        for (int c = 0; c < CT; c++)
#pragma unroll
            for (int e = 0; e < 2; e++) wt[c][x][e] = stay(__builtin_amdgcn_exp2f(arg[c][x][e]));
    };
    auto weigh_3 = [&](int x) {
        const int q = x >> 2, e = 2 * x & 7;
#pragma unroll
        for (int c = 0; c < CT; c++) {
            const float u = wt[c][x][0], v = wt[c][x][1];
            sum[c] = x & 3 ? sum[c] + u + v : u + v;
            if ((x & 3) == 3) l[c] = stay(fmaf(sum[c], rv[q], l[c]));
            const half2_t hi = stay(__builtin_convertvector((f32x2_t){u, v}, half2_t));
            pf[c][0][q][e] = hi[0];
            pf[c][0][q][e + 1] = hi[1];
            if constexpr (NP == 2) {
                const half2_t lo = stay(__builtin_convertvector((f32x2_t){u - (float)hi[0], v - (float)hi[1]}, half2_t));
                pf[c][1][q][e] = lo[0];
                pf[c][1][q][e + 1] = lo[1];
            }
        }
    };
    auto weigh = [&](int step, const f32x16_t (&sc)[CT][2], int steps) {
#pragma unroll
        for (int y = 0; y < 16; y++) {
            if (y >= 16 * step / steps && y < 16 * (step + 1) / steps) weigh_1(y, sc);
            if (y >= 16 * (step - 1) / steps && y < 16 * step / steps) weigh_2(y);
            if (y >= 16 * (step - 2) / steps && y < 16 * (step - 1) / steps) weigh_3(y);
        }
    };

    constexpr int P1 = 2 * NK, P2 = 4 * NT, kDeep = 4;  // operands of a stage's two products, read kDeep ahead
    auto operand = [&](int x, const uint4* k, const uint4* v) {
        const int y = x - P1;
        return __builtin_bit_cast(half8_t, x < P1 ? k[(2 * (x >> 1) + g) * 64 + 32 * (x & 1) + col]
                                                  : v[(2 * (y / NT) + g) * D + 32 * (y % NT) + col]);
    };
    auto score = [&](int x, half8_t k, f32x16_t (&sc)[CT][2]) {
#pragma unroll
        for (int c = 0; c < CT; c++)
#pragma unroll
            for (int n = 0; n < NP; n++) {
                f32x16_t& to = sc[c][x & 1];
                if (x < 2 && n == 0)
                    to = __builtin_amdgcn_mfma_f32_32x32x16_f16(k, qf[c][n][x >> 1], f32x16_t{}, 0, 0, 0);
                else
                    to = __builtin_amdgcn_mfma_f32_32x32x16_f16(k, qf[c][n][x >> 1], to, 0, 0, 0);
            }
    };

    // q's row as operands, scaled so that its largest value lies in [2^14, 2^15)
    auto make_q = [&]() {
#pragma unroll
        for (int c = 0; c < CT; c++) {
            float x[NK][8];
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < NK; k++) {
                x_load8<XT>(qraw[c][k], 0, x[k]);
#pragma unroll
                for (int e = 0; e < 8; e++) top = max(top, __float_as_uint(x[k][e]) & 0x7fffffffu);
            }
            top = max(top, (uint32_t)__shfl_xor((int)top, 32));
            const int ex = q_exponent(top);
            qs[c] = fabsf(ldexpf(a.scale * kLog2e, -ex));
#pragma unroll
            for (int k = 0; k < NK; k++)
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const float v = a.scale < 0.f ? -ldexpf(x[k][e], ex) : ldexpf(x[k][e], ex);
                    const _Float16 hi = (_Float16)v;
                    qf[c][0][k][e] = hi;
                    if constexpr (NP == 2) qf[c][1][k][e] = (_Float16)(v - (float)hi);
                }
        }
    };

    uint4 rk[UN], rw[UN];
    half2_t sign[UN];
    f32x16_t s0[CT][2], s1[CT][2];
    {
        uint4 fk[KB][UN], fv[UN];
#pragma unroll
        for (int i = 0; i < KB; i++) load_k(max(first[i], 0), fk[i]);
        load_k(max(first[KB], 0), rk);
#pragma unroll
        for (int i = 0; i < UN; i++)
            if (kEven || piece_v(i) < NK) {
                int j, d;
                place_v(i, j, d);
                fv[i] = *(const uint4*)(a.c.vc + (int64_t)max(__shfl(first[0], 16 * j), 0) * (16 * D) + d * 16);
                rw[i] = *(const uint4*)(a.c.vc + (int64_t)max(__shfl(first[1], 16 * j), 0) * (16 * D) + d * 16);
            }
        __builtin_amdgcn_sched_barrier(0);
        make_q();
        if (bi0 >= 0) eb = v_exponent(vs0);
#pragma unroll
        for (int x = 1; x < 64; x <<= 1) eb = max(eb, __shfl_xor(eb, x));
        if (lane == 0) in_top[wave] = eb;
        lds_barrier();
        eb = in_top[0];
#pragma unroll
        for (int w = 1; w < NW; w++) eb = max(eb, in_top[w]);
        e0 = eb < -500 ? 0 : __builtin_amdgcn_readfirstlane(eb);
        if (tid < kInfo) note(0, bi0, ks0, vs0);
        lds_barrier();
        sign_v(0, sign);
#pragma unroll
        for (int x = 0; x < 2 * UN; x++) store_k(x, fk[0], sk);
        lds_barrier();
        // the first S between the decoding of the next stages
#pragma unroll
        for (int x = 0; x < P1; x++) {
            score(x, operand(x, sk, sv[0]), s0);
#pragma unroll
            for (int y = 2 * UN * KB * x / P1; y < 2 * UN * KB * (x + 1) / P1; y++) {
                if (y < 2 * UN * (KB - 1))
                    store_k(y % (2 * UN), fk[1 + y / (2 * UN)], sk + (1 + y / (2 * UN)) * 8 * D);
                else
                    store_v(y % (2 * UN), fv, sign, sv[0]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        sign_v(1, sign);
    }
    read_scales(0);
    scale_and_hide(0, s0);
#pragma unroll
    for (int x = 0; x < 16; x++) top_pair(x, s0);
    settle();
    lds_barrier();
    // Iteration t: S of stage t + 1 between the weights of stage t; then O of stage t between the maxima
    // of stage t + 1 and the decoding of stage t + KB's K and stage t + 1's V, whose successors' loads set
    // out as soon as their registers are free.  Stages past the last are hidden.
    int page = 0, nbi = -1;
    float nks = 0.f, nvs = 0.f;
    half8_t f[kDeep];
    if constexpr (KB == 3) {
#pragma unroll
        for (int x = 0; x < kDeep; x++) f[x] = operand(x, sk + 8 * D, sv[0]);
    }
    const uint4 *kr = sk + 8 * D, *kr2 = sk + (KB - 1) * 8 * D;  // K of stages t + 1 and (of three buffers) t + 2
    uint4* kw = sk;
    auto body = [&](int t, f32x16_t (&now)[CT][2], f32x16_t (&next)[CT][2], uint4* vr, uint4* vw) {
        if constexpr (KB == 2) {
#pragma unroll
            for (int x = 0; x < kDeep; x++) f[x] = operand(x, kr, vr);
        }
        const int bk = block_k(t + KB + 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int x = 0; x < P1; x++) {
            score(x, f[x % kDeep], next);
            f[x % kDeep] = operand(x + kDeep, kr, vr);
            if (x == P1 - 4) read_scales(t + 1);
            weigh(x, now, P1);
            __builtin_amdgcn_sched_barrier(0);
        }
        scale_and_hide(t + 1, next);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int x = 0; x < P2; x++) {
#pragma unroll
            for (int c = 0; c < CT; c++)
#pragma unroll
                for (int n = 0; n < NP; n++)
                    o[c][x % NT] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f[(P1 + x) % kDeep], pf[c][n][x / NT], o[c][x % NT], 0, 0, 0);
            if (x + kDeep < P2)
                f[(P1 + x) % kDeep] = operand(P1 + x + kDeep, kr, vr);
            else if (KB == 3)
                f[(P1 + x) % kDeep] = operand(x + kDeep - P2, kr2, vr);
            if (x < 2) weigh(P1 + x, now, P1);
#pragma unroll
            for (int y = 8 * UN * x / P2; y < 8 * UN * (x + 1) / P2; y++) {
                if (y < 2 * UN) store_k(y, rk, kw);
                if (y == 2 * UN - 1) load_k(bk, rk);
                if (y >= 2 * UN && y < 4 * UN) store_v(y - 2 * UN, rw, sign, vw);
                if (y == 4 * UN - 1) {
                    load_v(t + 2, rw);
                    sign_v(t + 2, sign);
                }
            }
#pragma unroll
            for (int y = 16 * x / P2; y < 16 * (x + 1) / P2; y++) top_pair(y, next);
            __builtin_amdgcn_sched_barrier(0);
        }
        settle();
        uint4* k = kw;
        kw = (uint4*)kr;
        kr = KB == 3 ? kr2 : k;
        kr2 = k;
        lds_barrier();
    };
    for (int t = 0; t < stages; t += 2) {
        body(t, s0, s1, sv[0], sv[1]);
        body(t + 1, s1, s0, sv[1], sv[0]);
        // the next 64 stages' blocks, in three steps so that no load is waited for
        const int seg = t / 64 + 1, at = t & 63;
        if (at >= 8 && at < 26 && seg * 64 < stages + 6 && tid < kInfo) {
            if (at == 8) page = page_of(my_blk + kInfo * seg);
            if (at == 16) {
                nbi = index_of(my_blk + kInfo * seg, page);
                nks = a.c.ks[max(nbi, 0)];
                nvs = a.c.vs[max(nbi, 0)];
            }
            if (at == 24) note(seg, nbi, nks, nvs);
        }
    }

#pragma unroll
    for (int c = 0; c < CT; c++) {
        const int r = w0 + 32 * c + col;
        FarSum far = {kNegInf, 0.f};
        if (any_far) {
            far = sh_far[wave][c][lane];
            far_add(far, __shfl_xor(far.m, 32), __shfl_xor(far.l, 32));
        }
        const RowEnd end = row_end(l[c] + __shfl_xor(l[c], 32), m[c], far, e0);
        if (r >= rows) continue;
        const int64_t trow = sp.r0 + r / a.group;
        const int hd = h * a.group + r % a.group;
        // divided before the V scales' power: the values may lie anywhere in f32's range
        const float inv = end.l == 0.f ? 0.f : 1.0f / end.l;
        auto mean = [&](int i, int e) {
            return ldexp4(f32x4_t{o[c][i][4 * e], o[c][i][4 * e + 1], o[c][i][4 * e + 2], o[c][i][4 * e + 3]} * inv, end.e);
        };
        if (tr.nact > 1) {
            const int64_t pi = (trow * a.q_heads + hd) * a.splits + split;
            float* to = a.part_o + pi * D + 4 * g;
#pragma unroll
            for (int i = 0; i < NT; i++)
#pragma unroll
                for (int e = 0; e < 4; e++) *(f32x4_t*)(to + 32 * i + 8 * e) = mean(i, e);
            if (g == 0) *(float2*)(a.part_ml + pi * 2) = make_float2(end.m, end.l);
        } else {
            const int64_t at = trow * a.o_row + hd * a.o_head + 4 * g;
#pragma unroll
            for (int i = 0; i < NT; i++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const f32x4_t y = mean(i, e);
                    if constexpr (XT == XT_F32)
                        *(f32x4_t*)((float*)a.O + at + 32 * i + 8 * e) = y;
                    else {
                        u32x2_t p;
                        p[0] = (uint32_t)f32_to_16<XT>(y[0]) | (uint32_t)f32_to_16<XT>(y[1]) << 16;
                        p[1] = (uint32_t)f32_to_16<XT>(y[2]) | (uint32_t)f32_to_16<XT>(y[3]) << 16;
                        *(u32x2_t*)((uint16_t*)a.O + at + 32 * i + 8 * e) = p;
                    }
                }
        }
    }
}

template <bool TREE, int XT, int D>
hipError_t launch_one(AttnParams a, hipStream_t s) {
    const int64_t grid = (int64_t)a.q.seqs * a.splits * a.c.heads * a.tiles;
    for (int64_t first = 0; first < grid; first += kLaunchGroups) {
        a.first = (int)first;
        const uint32_t part = (uint32_t)std::min(grid - first, kLaunchGroups);
        if (a.tile_rows == 128)
            attn8_tile_kernel<TREE, XT, D, 4, 1><<<part, 256, 0, s>>>(a);
        else if constexpr (XT != XT_F32 && D <= 128)
            attn8_tile_kernel<TREE, XT, D, 8, 1><<<part, 512, 0, s>>>(a);
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
hipError_t launch_tiles(const AttnParams& a, int xt, hipStream_t s) {
    if (xt == XT_F32) return launch_dim<TREE, XT_F32>(a, s);
    if (xt == XT_F16) return launch_dim<TREE, XT_F16>(a, s);
    return launch_dim<TREE, XT_BF16>(a, s);
}

}  // namespace
}  // namespace qg
