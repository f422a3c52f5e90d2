// qg_attn8_tile.hip -- attention over the 8-bit cache for many rows a K/V head: prompts and chunks.
#include <hip/hip_runtime.h>

#include "qg_attn8.hpp"

namespace qg {
namespace {

// All lanes' LDS reads and writes so far are done, in every wavefront; loads from memory stay in flight.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

__device__ __forceinline__ float lane_value(float v, int l) {
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), l));
}

// Four codes times f (0, 1 or -1; c = -1152 f) as f16.
__device__ __forceinline__ void codes4_f16(uint32_t w, half2_t f, half2_t c, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = w ^ 0x80808080u;
    const half2_t a = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u));
    const half2_t b = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u));
    lo = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(a, f, c));
    hi = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(b, f, c));
}

// A workgroup of NW wavefronts takes 32 CT NW rows (query rows times the heads that share a K/V head,
// counted together), each wavefront 32 CT of them, and walks over the tokens they see in stages of 64.
// A stage's codes are decoded once for all rows, into f16 in shared memory in the order in which the
// matrix instructions take them, so every read is 1 KiB without conflicts:
//   K  [dim/8][64 tokens][8 dims]        A operand of S = K Q^T (32 tokens x 32 rows a product)
//   V  [block][half g][dim][8 tokens]    A operand of O = V^T P^T, tokens 4g..4g+3, 4g+8..4g+11
// which is the order in which lane (row l % 32, half g = l / 32) holds its weights after S, so they
// never move between lanes.  Stage t + 1's S is multiplied while stage t's weights are computed.
template <int XT, int D, int NW, int CT>
__global__ __launch_bounds__(64 * NW) void attn8_tile_kernel(AttnParams a) {
    constexpr int NP = XT == XT_F32 ? 2 : 1;  // f16 pieces of a q value and of a weight
    constexpr int NK = D / 16, NT = D / 32;
    constexpr int UN = (D / 16 + NW - 1) / NW;  // 1 KiB pieces of K, and of V, that a wavefront decodes
    constexpr int BR = 32 * CT * NW;
    __shared__ __attribute__((aligned(16))) uint4 sk[2][8 * D], sv[2][8 * D];

    const int lane = threadIdx.x & 63, col = lane & 31, g = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // sequences and heads first, so that the workgroups of one K/V head share a die's cache; the last
    // tiles, which see the most, first
    int b = blockIdx.x;
    const int pairs = a.q.seqs * a.c.heads;
    const int h = b % pairs % a.c.heads, s = b % pairs / a.c.heads;
    b /= pairs;
    const int split = b % a.splits, tile = a.tiles - 1 - b / a.splits;
    const KvSpan sp = kv8_span(a.q, s);
    const int rows = sp.n * a.group;
    if (tile * BR >= rows) return;
    const TileRange tr = tile_range(a, sp, tile * BR, BR);
    if (split > 0 && split >= tr.nact) return;
    const int t0 = tr.lo + split * a.chunk, t1 = min(t0 + a.chunk, tr.hi);
    const int stages = (t1 - t0 + 63) / 64;

    // rows of this wavefront, and what all of them see
    const int w0 = tile * BR + wave * 32 * CT;
    const int lo_all = kv8_sight(sp, min(w0 + 32 * CT, rows) <= w0 ? 0 : (min(w0 + 32 * CT, rows) - 1) / a.group, a.causal, a.window).lo;
    const int hi_all = kv8_sight(sp, min(w0, rows - 1) / a.group, a.causal, a.window).hi;
    const int lo_any = kv8_sight(sp, tile * BR / a.group, a.causal, a.window).lo;

    half8_t qf[CT][NP][NK];
    float qs[CT];
    KvSight see[CT];
#pragma unroll
    for (int c = 0; c < CT; c++) {
        const int r = min(w0 + 32 * c + col, rows - 1), ri = r / a.group, head = h * a.group + r % a.group;
        see[c] = kv8_sight(sp, ri, a.causal, a.window);
        const int64_t at = (int64_t)(sp.r0 + ri) * a.q_row + head * a.q_head + 8 * g;
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < NK; k++) {
            float x[8];
            x_load8<XT>(a.Q, at + 16 * k, x);
#pragma unroll
            for (int e = 0; e < 8; e++) top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
        }
        top = max(top, (uint32_t)__shfl_xor((int)top, 32));
        const int ex = q_exponent(top);
        qs[c] = ldexpf(a.scale * kLog2e, -ex);
#pragma unroll
        for (int k = 0; k < NK; k++) {
            float x[8];
            x_load8<XT>(a.Q, at + 16 * k, x);
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const float v = a.scale < 0.f ? -ldexpf(x[e], ex) : ldexpf(x[e], ex);
                const _Float16 hi = (_Float16)v;
                qf[c][0][k][e] = hi;
                if constexpr (NP == 2) qf[c][1][k][e] = (_Float16)(v - (float)hi);
            }
        }
        qs[c] = fabsf(qs[c]);
    }

    // the table's entry of this lane's block of a stage, and the block's index (-1: hidden from all)
    auto blk_of = [&](int st) { return ((t0 + 64 * st) >> 4) + (lane >> 4); };
    auto entry = [&](int st) {
        const uint32_t pi = kv8_div((uint32_t)blk_of(st), a.c.nb, a.c.magic);
        return a.q.table[(int64_t)s * a.q.width + min(pi, (uint32_t)a.q.width - 1)];
    };
    auto index = [&](int st, int page) {
        const int blk = blk_of(st);
        const uint32_t pi = kv8_div((uint32_t)blk, a.c.nb, a.c.magic);
        const bool ok = (st < stages) & (16 * blk < tr.hi) & (16 * blk + 16 > lo_any) & (pi < (uint32_t)a.q.width) &
                        ((uint32_t)page < (uint32_t)a.c.pages);
        return ok ? (int)(((uint32_t)page * a.c.heads + h) * a.c.nb + ((uint32_t)blk - pi * (uint32_t)a.c.nb)) : -1;
    };
    auto load_k = [&](int bi, uint4 (&raw)[UN]) {
        const int8_t* p = a.c.kc + (int64_t)max(bi, 0) * (16 * D) + (lane & 15) * 16;
#pragma unroll
        for (int i = 0; i < UN; i++)
            if (NK % NW == 0 || wave + NW * i < NK) raw[i] = *(const uint4*)(p + (wave + NW * i) * 256);
    };
    auto store_k = [&](const uint4 (&raw)[UN], uint4* to) {
#pragma unroll
        for (int i = 0; i < UN; i++)
            if (NK % NW == 0 || wave + NW * i < NK) {
                uint4* p = to + (wave + NW * i) * 128 + lane;
                p[0] = __builtin_bit_cast(uint4, codes8_f16(raw[i].x, raw[i].y));
                p[64] = __builtin_bit_cast(uint4, codes8_f16(raw[i].z, raw[i].w));
            }
    };
    // V piece u: the 64 (block, dim) pairs from 64 u
    auto piece_v = [&](int i) { return NW - 1 - wave + NW * i; };
    auto load_v = [&](int bi, uint4 (&raw)[UN]) {
#pragma unroll
        for (int i = 0; i < UN; i++)
            if (NK % NW == 0 || piece_v(i) < NK) {
                const int x = 64 * piece_v(i) + lane, j = x / D;
                const int vb = D % 64 == 0 ? __builtin_amdgcn_readlane(bi, 16 * (64 * piece_v(i) / D)) : __shfl(bi, 16 * j);
                raw[i] = *(const uint4*)(a.c.vc + (int64_t)max(vb, 0) * (16 * D) + (x - j * D) * 16);
            }
    };
    auto store_v = [&](const uint4 (&raw)[UN], float vs, uint4* to) {
#pragma unroll
        for (int i = 0; i < UN; i++)
            if (NK % NW == 0 || piece_v(i) < NK) {
                const int x = 64 * piece_v(i) + lane, j = x / D, d = x - j * D;
                const float sc = D % 64 == 0 ? lane_value(vs, 16 * (64 * piece_v(i) / D)) : __shfl(vs, 16 * j);
                const float sg = sc == 0.f ? 0.f : sc < 0.f ? -1.f : 1.f;
                const half2_t f = {(_Float16)sg, (_Float16)sg}, c = {(_Float16)(-1152.f * sg), (_Float16)(-1152.f * sg)};
                u32x4 lo, hi;
                uint32_t p, q;
                codes4_f16(raw[i].x, f, c, p, q);
                lo[0] = p, lo[1] = q;
                codes4_f16(raw[i].z, f, c, p, q);
                lo[2] = p, lo[3] = q;
                codes4_f16(raw[i].y, f, c, p, q);
                hi[0] = p, hi[1] = q;
                codes4_f16(raw[i].w, f, c, p, q);
                hi[2] = p, hi[3] = q;
                to[2 * j * D + d] = __builtin_bit_cast(uint4, lo);
                to[2 * j * D + D + d] = __builtin_bit_cast(uint4, hi);
            }
    };

    f32x16_t o[CT][NT] = {};
    float m[CT], l[CT];
#pragma unroll
    for (int c = 0; c < CT; c++) m[c] = kNegInf, l[c] = 0.f;
    int ev = -1000;           // exponent that the V scales are taken relative to
    float kf[CT][4], cf[CT][4], rv[4];  // factor and addend of a score in powers of two, 1 / V scale

    auto scores = [&](const uint4* k, f32x16_t (&s)[CT][2]) {
#pragma unroll
        for (int c = 0; c < CT; c++)
#pragma unroll
            for (int t = 0; t < 2; t++)
#pragma unroll
                for (int e = 0; e < 16; e++) s[c][t][e] = 0.f;
#pragma unroll
        for (int i = 0; i < NK; i++)
#pragma unroll
            for (int t = 0; t < 2; t++) {
                const half8_t kk = __builtin_bit_cast(half8_t, k[(2 * i + g) * 64 + 32 * t + col]);
#pragma unroll
                for (int c = 0; c < CT; c++)
#pragma unroll
                    for (int n = 0; n < NP; n++)
                        s[c][t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kk, qf[c][n][i], s[c][t], 0, 0, 0);
            }
    };
    // Stage st's maxima; the sums are rescaled where a maximum or the V scales' exponent grew.
    auto maxima = [&](int st, int bi, float ks, float vs, f32x16_t (&sc)[CT][2]) {
        const int tb = t0 + 64 * st;
        // what a row sees of a block with a NaN or infinite V scale is NaN
        if (bi < 0) vs = 0.f;
        const bool odd = !(fabsf(vs) < __builtin_inff());
        if (odd) ks = __builtin_nanf("");
        const uint64_t there = __ballot(bi >= 0);
        const bool whole = tb >= lo_all && tb + 64 <= hi_all && !__any(bi < 0 || !(ks >= 0.f));
        const float va = odd ? 0.f : fabsf(vs);
        float kb[4];
#pragma unroll
        for (int q = 0; q < 4; q++) kb[q] = lane_value(ks, 16 * q);
        float top[CT];
        if (whole) {
#pragma unroll
            for (int c = 0; c < CT; c++) {
                float best = kNegInf;
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    kf[c][q] = kb[q] * qs[c];
                    float t = sc[c][q >> 1][8 * (q & 1)];
#pragma unroll
                    for (int e = 1; e < 8; e++) t = fmaxf(t, sc[c][q >> 1][8 * (q & 1) + e]);
                    best = fmaxf(best, t * kf[c][q]);
                }
                top[c] = best;
            }
        } else {
#pragma unroll
            for (int c = 0; c < CT; c++) {
                float best = kNegInf;
                const int jl = see[c].lo - tb - 4 * g, jh = see[c].hi - tb - 4 * g;
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    const float f = kb[q] * qs[c];
                    const bool here = (there >> (16 * q)) & 1;
                    kf[c][q] = 1.f;
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        const int j = 16 * q + 8 * (e >> 2) + (e & 3);
                        const float v = here && j >= jl && j < jh ? sc[c][q >> 1][8 * (q & 1) + e] * f : kNegInf;
                        sc[c][q >> 1][8 * (q & 1) + e] = v;
                        best = fmaxf(best, v);
                    }
                }
                top[c] = best;
            }
        }
        bool grew = false;
#pragma unroll
        for (int c = 0; c < CT; c++) {
            top[c] = fmaxf(top[c], __shfl_xor(top[c], 32));
            grew |= top[c] > m[c] + kLag;
        }
        float vm = va;
        vm = fmaxf(vm, __shfl_xor(vm, 16));
        vm = fmaxf(vm, __shfl_xor(vm, 32));
        const int eb = __builtin_amdgcn_readfirstlane((int)(__float_as_uint(vm) >> 23)) - 126;
        if (eb > ev || __any(grew)) {
            const int en = max(ev, eb);
#pragma unroll
            for (int c = 0; c < CT; c++) {
                const float mn = fmaxf(m[c], top[c]);
                const float f = m[c] == kNegInf ? 0.f : __builtin_amdgcn_exp2f(m[c] - mn);
                l[c] *= f;
                const float fo = ldexpf(f, ev - en);
#pragma unroll
                for (int i = 0; i < NT; i++)
#pragma unroll
                    for (int e = 0; e < 16; e++) o[c][i][e] *= fo;
                m[c] = mn;
            }
            ev = en;
        }
        // the block's V scale relative to 2^(ev - kBase), as a power of two; 0: its codes count as 0
        const float lv = va == 0.f ? 0.f : fmaxf(__builtin_amdgcn_logf(ldexpf(va, kBase - ev)), -60.f);
        const float iv = __builtin_amdgcn_exp2f(-lv);
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const float lq = lane_value(lv, 16 * q);
            rv[q] = lane_value(iv, 16 * q);
#pragma unroll
            for (int c = 0; c < CT; c++) cf[c][q] = lq - (m[c] == kNegInf ? 0.f : m[c]);
        }
    };
    half8_t pf[CT][NP][4];
    auto weights = [&](const f32x16_t (&sc)[CT][2]) {
#pragma unroll
        for (int c = 0; c < CT; c++)
#pragma unroll
            for (int q = 0; q < 4; q++) {
                float sum = 0.f;
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    float w[2];
#pragma unroll
                    for (int x = 0; x < 2; x++)
                        w[x] = __builtin_amdgcn_exp2f(fmaf(sc[c][q >> 1][8 * (q & 1) + e + x], kf[c][q], cf[c][q]));
                    sum += w[0] + w[1];
                    const half2_t hi = __builtin_convertvector((__attribute__((ext_vector_type(2))) float){w[0], w[1]}, half2_t);
                    pf[c][0][q][e] = hi[0];
                    pf[c][0][q][e + 1] = hi[1];
                    if constexpr (NP == 2) {
                        pf[c][1][q][e] = (_Float16)(w[0] - (float)hi[0]);
                        pf[c][1][q][e + 1] = (_Float16)(w[1] - (float)hi[1]);
                    }
                }
                l[c] = fmaf(sum, rv[q], l[c]);
            }
    };
    auto values = [&](const uint4* v) {
#pragma unroll
        for (int q = 0; q < 4; q++)
#pragma unroll
            for (int i = 0; i < NT; i++) {
                const half8_t vv = __builtin_bit_cast(half8_t, v[(2 * q + g) * D + 32 * i + col]);
#pragma unroll
                for (int c = 0; c < CT; c++)
#pragma unroll
                    for (int n = 0; n < NP; n++)
                        o[c][i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vv, pf[c][n][q], o[c][i], 0, 0, 0);
            }
    };

    // ids and scales of stages t + 1, t + 2, t + 3 (t: the loop's stage), the entry of stage t + 4
    int b1, b2, b3, e4;
    float k1, v1, k2, v2, k3, v3;
    uint4 rk[UN], rw[UN];
    auto load_scales = [&](int bi, float& ks, float& vs) {
        ks = a.c.ks[max(bi, 0)];
        vs = a.c.vs[max(bi, 0)];
    };
    f32x16_t s0[CT][2], s1[CT][2];
    {
        const int e0 = entry(0), e1 = entry(1), e2 = entry(2), e3 = entry(3);
        const int b0 = index(0, e0);
        float k0, v0;
        load_scales(b0, k0, v0);
        load_k(b0, rk);
        load_v(b0, rw);
        b1 = index(1, e1);
        b2 = index(2, e2);
        b3 = index(3, e3);
        e4 = entry(4);
        load_scales(b1, k1, v1);
        load_scales(b2, k2, v2);
        store_k(rk, sk[0]);
        store_v(rw, v0, sv[0]);
        load_k(b1, rk);
        store_k(rk, sk[1]);
        load_k(b2, rk);
        load_v(b1, rw);
        lds_barrier();
        scores(sk[0], s0);
        maxima(0, b0, k0, v0, s0);
    }
    // Iteration t: S of stage t + 1 and the weights of stage t; then O of stage t, while stage t + 2's K
    // and stage t + 1's V are decoded and the loads after those set out.
    auto body = [&](int t, f32x16_t (&now)[CT][2], f32x16_t (&next)[CT][2], uint4* kn, uint4* ko, uint4* vo, uint4* vn) {
        scores(kn, next);
        weights(now);
        values(vo);
        store_k(rk, ko);
        store_v(rw, v1, vn);
        load_k(b3, rk);
        load_v(b2, rw);
        load_scales(b3, k3, v3);
        if (t + 1 < stages) maxima(t + 1, b1, k1, v1, next);
        b1 = b2, k1 = k2, v1 = v2;
        b2 = b3, k2 = k3, v2 = v3;
        b3 = index(t + 4, e4);
        e4 = entry(t + 5);
        lds_barrier();
    };
    for (int t = 0; t < stages; t += 2) {
        body(t, s0, s1, sk[1], sk[0], sv[0], sv[1]);
        if (t + 1 >= stages) break;
        body(t + 1, s1, s0, sk[0], sk[1], sv[1], sv[0]);
    }

#pragma unroll
    for (int c = 0; c < CT; c++) {
        const int r = w0 + 32 * c + col;
        const float lt = l[c] + __shfl_xor(l[c], 32);
        if (r >= rows) continue;
        const int64_t trow = sp.r0 + r / a.group;
        const int hd = h * a.group + r % a.group;
        if (tr.nact > 1) {
            const float un = m[c] == kNegInf ? 0.f : ldexpf(1.f, ev - kBase);
            const int64_t pi = (trow * a.q_heads + hd) * a.splits + split;
            float* to = a.part_o + pi * D + 4 * g;
#pragma unroll
            for (int i = 0; i < NT; i++)
#pragma unroll
                for (int e = 0; e < 4; e++)
                    *(f32x4_t*)(to + 32 * i + 8 * e) = f32x4_t{o[c][i][4 * e] * un, o[c][i][4 * e + 1] * un,
                                                             o[c][i][4 * e + 2] * un, o[c][i][4 * e + 3] * un};
            if (g == 0) *(float2*)(a.part_ml + pi * 2) = make_float2(m[c], lt);
        } else {
            const float inv = lt == 0.f ? 0.f : 1.0f / lt;
            const int64_t at = trow * a.o_row + hd * a.o_head + 4 * g;
#pragma unroll
            for (int i = 0; i < NT; i++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    float y[4];
#pragma unroll
                    for (int x = 0; x < 4; x++) y[x] = ldexpf(o[c][i][4 * e + x] * inv, ev - kBase);
                    if constexpr (XT == XT_F32)
                        *(f32x4_t*)((float*)a.O + at + 32 * i + 8 * e) = f32x4_t{y[0], y[1], y[2], y[3]};
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

// Rows a wavefront (32 CT) and wavefronts for a type and dim.
template <int XT, int D>
struct Shape {
    static constexpr int NW = XT == XT_F32 || D > 128 ? 4 : 8, CT = 1;
};

template <int XT, int D>
hipError_t launch_one(const AttnParams& a, hipStream_t s) {
    using S = Shape<XT, D>;
    const int64_t grid = (int64_t)a.q.seqs * a.splits * a.c.heads * a.tiles;
    attn8_tile_kernel<XT, D, S::NW, S::CT><<<dim3((uint32_t)grid), 64 * S::NW, 0, s>>>(a);
    return hipGetLastError();
}

template <int XT>
hipError_t launch_dim(const AttnParams& a, hipStream_t s) {
    switch (a.c.dim) {
        case 64: return launch_one<XT, 64>(a, s);
        case 96: return launch_one<XT, 96>(a, s);
        case 128: return launch_one<XT, 128>(a, s);
        case 192: return launch_one<XT, 192>(a, s);
        case 256: return launch_one<XT, 256>(a, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace

int attn8_tile_rows(int xt, int dim) {
    return xt == XT_F32 || dim > 128 ? 128 : 256;
}

hipError_t launch_attn8_tile(const AttnParams& a, int xt, hipStream_t s) {
    if (xt == XT_F32) return launch_dim<XT_F32>(a, s);
    if (xt == XT_F16) return launch_dim<XT_F16>(a, s);
    return launch_dim<XT_BF16>(a, s);
}

}  // namespace qg
