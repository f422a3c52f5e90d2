// qg_attn8.hpp -- what the kernels of the attention over the 8-bit cache share.
//
//   o = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale q . k_j) over the tokens j that the row may see.
//
// K and V codes are integers of at most 8 bits, exact in f16, so the products run on the f16 matrix
// instructions with f32 sums: q enters as f16 after an exact power of two per row (f32 q as two such
// f16 pieces), the weights as f16 after the block's V scale.
#pragma once

#include "qg_device.hpp"
#include "qg_internal.hpp"

namespace qg {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -__builtin_inff();
// A weight enters the second product as f16 with the block's V scale in it:
//   w = exp2(s + log2(vs 2^-e0) - m + kBase),  m a running maximum of what stands before it in the row,
// and the denominator takes w times the reciprocal, so a row's precision is set by the blocks that it sees
// and by no others.  m may lag by kLag before the sums are rescaled: weights stay at or below 2^15 and keep
// f16's full precision down to 2^-23 of the row's largest.  16-bit rows take one f16 piece of a weight, f32 rows
// two: an error of at most 2^-11 (2^-22) of the weighted mean of |v|, where values do not cancel no more than the
// rounding of an f16 result, and one piece halves the second product.  e0, an exponent of V scales near by, keeps the
// powers small.
constexpr float kLag = 6.f;
constexpr int kBase = 9;
// kBase - m; before a row has a maximum, kBase.
__device__ __forceinline__ float above_m(float m) { return m == kNegInf ? (float)kBase : (float)kBase - m; }

// Four codes as four f16 values, exactly: byte ^ 0x80 below 0x64 is 1024 + (code + 128).
__device__ __forceinline__ void codes4_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = w ^ 0x80808080u;
    const half2_t bias = {(_Float16)1152.f, (_Float16)1152.f};
    const half2_t a = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u)) - bias;
    const half2_t b = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u)) - bias;
    lo = __builtin_bit_cast(uint32_t, a);
    hi = __builtin_bit_cast(uint32_t, b);
}
__device__ __forceinline__ half8_t codes8_f16(uint32_t w0, uint32_t w1) {
    u32x4 r;
    uint32_t a, b;
    codes4_f16(w0, a, b);
    r[0] = a, r[1] = b;
    codes4_f16(w1, a, b);
    r[2] = a, r[3] = b;
    return __builtin_bit_cast(half8_t, r);
}

// Four codes times f (0, 1 or -1; c = -1152 f) as f16.
__device__ __forceinline__ void codes4_f16(uint32_t w, half2_t f, half2_t c, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = w ^ 0x80808080u;
    const half2_t a = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u));
    const half2_t b = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u));
    lo = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(a, f, c));
    hi = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(b, f, c));
}
__device__ __forceinline__ half8_t codes8_f16(uint32_t w0, uint32_t w1, half2_t f, half2_t c) {
    u32x4 r;
    uint32_t a, b;
    codes4_f16(w0, f, c, a, b);
    r[0] = a, r[1] = b;
    codes4_f16(w1, f, c, a, b);
    r[2] = a, r[3] = b;
    return __builtin_bit_cast(half8_t, r);
}
// Both scales of a block are finite.  Else its scores become NaN: an infinite K scale by itself would score tokens
// of negative products -inf, as if they were hidden.
__device__ __forceinline__ bool finite_scales(float ks, float vs) { return (ks - ks) + (vs - vs) == 0.f; }
// The factor of a block's V codes: the V scale's sign.
__device__ __forceinline__ uint32_t v_sign(float vs) { return vs == 0.f ? 0u : vs < 0.f ? 0xbc00bc00u : 0x3c003c00u; }
// log2(|vs| 2^-e0): -inf where the scale is 0, 0 where it is not finite (its K scale becomes NaN).
__device__ __forceinline__ float v_power(float vs, int e0) {
    const float va = fabsf(vs);
    if (va == 0.f) return kNegInf;
    if (!(va < __builtin_inff())) return 0.f;
    return __builtin_amdgcn_logf(__builtin_amdgcn_frexp_mantf(va)) + (float)(__builtin_amdgcn_frexp_expf(va) - e0);
}
// What a far block's power lost to rounding: its scores take it once they are in FarSum.
__device__ __forceinline__ float v_power_rest(float vs, int e0, float lv) {
    if (lv == kNegInf) return 0.f;
    const float va = fabsf(vs);
    const float whole = (float)(__builtin_amdgcn_frexp_expf(va) - e0);
    return (whole - lv) + __builtin_amdgcn_logf(__builtin_amdgcn_frexp_mantf(va));
}
// A far block's weights say nothing about its part of the denominator: it has an own sum for that, FarSum, and the
// factor 0 in the other.  Far are V scales of 0, whose tokens weigh nothing in the numerator (whatever they score, the
// running maximum of what stands there must not rise for them), and those so far from 2^e0 that the reciprocal or the
// sum could leave f32's range: e0 comes from blocks that a row need not see.  With 2^32 a row's other blocks keep
// theirs while its V scales lie within 2^100 of each other.
constexpr float kFar = 32.f;
__device__ __forceinline__ bool is_far(float lv) { return fabsf(lv) > kFar; }
__device__ __forceinline__ float v_reciprocal(float lv) { return is_far(lv) ? 0.f : __builtin_amdgcn_exp2f(-lv); }
struct FarSum {
    float m, l;  // sum of exp2(s - m), m the largest s
};
template <int N>
__device__ __forceinline__ void far_add(FarSum& f, const float (&s)[N]) {
    float m = f.m;
#pragma unroll
    for (int i = 0; i < N; i++) m = fmaxf(m, s[i]);
    if (m == kNegInf) return;
    f.l *= __builtin_amdgcn_exp2f(f.m - m);
#pragma unroll
    for (int i = 0; i < N; i++) f.l += __builtin_amdgcn_exp2f(s[i] - m);
    f.m = m;
}
__device__ __forceinline__ void far_add(FarSum& f, float m, float l) {
    const float mn = fmaxf(f.m, m);
    if (mn == kNegInf) return;
    f.l = f.l * __builtin_amdgcn_exp2f(f.m - mn) + l * __builtin_amdgcn_exp2f(m - mn);
    f.m = mn;
}
// A row's weights at the end: their sum is l 2^m, and o / l has to be taken times 2^e.
struct RowEnd {
    float l, m;
    int e;
};
// From the sum l of the other blocks' weights below the maximum m (-inf: there are none), and that of the far ones.
__device__ __forceinline__ RowEnd row_end(float l, float m, const FarSum& f, int e0) {
    const float mu = above_m(m);
    float k = 0.f;  // a whole power, so that nothing is rounded by it
    if (f.m > kNegInf) {
        k = __builtin_rintf(f.m + mu);
        if (m > kNegInf) k = fmaxf(k, 0.f);
        float rest = (mu - k) + f.m;
        if (k != 0.f) rest = fminf(fmaxf(rest, -1.f), 1.f);
        l = (l == 0.f ? 0.f : l * __builtin_amdgcn_exp2f(-k)) + f.l * __builtin_amdgcn_exp2f(rest);
    }
    return RowEnd{l, l == 0.f ? kNegInf : k - mu, e0 - (int)fminf(fmaxf(k, -5000.f), 5000.f)};
}
// Exponent of |vs|, -1000 where it is 0 or not finite.
__device__ __forceinline__ int v_exponent(float vs) {
    const float va = fabsf(vs);
    return va > 0.f && va < __builtin_inff() ? (int)(__float_as_uint(va) >> 23) - 126 : -1000;
}

// Tokens [lo, hi) that row i of a sequence sees.  TREE: those before the batch's rows; of these it sees the ones that
// its mask has, however small the window.
template <bool TREE>
__device__ __forceinline__ KvSight row_sight(const AttnParams& a, const KvSpan& sp, int i) {
    if constexpr (!TREE) return kv8_sight(sp, i, a.causal, a.window);
    const int hist = sp.len - sp.n;
    int p = sp.len - 1;
    if (a.window > 0) p = min(max(a.pos[sp.r0 + i], hist), sp.len - 1);
    return KvSight{a.window > 0 ? min(max(p - a.window + 1, 0), hist) : 0, hist};
}
// The same for the first or last row of some, so that every one of them sees lo and what follows it from `last` on, and
// none sees what lies before `first`'s lo.  A tree's rows have positions in no order.
template <bool TREE>
__device__ __forceinline__ KvSight edge_sight(const AttnParams& a, const KvSpan& sp, int i, bool last) {
    if constexpr (!TREE) return kv8_sight(sp, i, a.causal, a.window);
    const int hist = sp.len - sp.n, p = last ? sp.len - 1 : hist;
    return KvSight{a.window > 0 ? max(p - a.window + 1, 0) : 0, hist};
}
// Ones at lo .. hi - 1, limited to 16 and to 64 bits.
__device__ __forceinline__ uint32_t bits_between(int lo, int hi) {
    const uint32_t below = (1u << min(max(lo, 0), 16)) - 1, upto = (1u << min(max(hi, 0), 16)) - 1;
    return upto & ~below;
}
__device__ __forceinline__ uint64_t ones64(int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1; }
__device__ __forceinline__ uint64_t bits_between64(int lo, int hi) { return ones64(hi) & ~ones64(lo); }
// Which of the tokens t .. t + 63 row i sees by its mask: bit j for token t + j.
__device__ __forceinline__ uint64_t drafted_bits(const AttnParams& a, const KvSpan& sp, int i, int t) {
    const int off = t - (sp.len - sp.n), w = off >> 5, sh = off & 31;  // row of token t, in words and bits
    const uint32_t* m = a.mask + (int64_t)(sp.r0 + i) * a.words;
    auto word = [&](int x) { return (uint32_t)x < (uint32_t)a.words ? m[x] : 0u; };
    const uint64_t lo = word(w) | (uint64_t)word(w + 1) << 32, hi = word(w + 2);
    const uint64_t bits = sh ? lo >> sh | hi << (64 - sh) : lo;
    return bits & ones64(sp.len - t);
}

// What the rows r0 .. r0 + rows - 1 of a tile see together, and how the splits divide it.
struct TileRange {
    int lo, hi, nact;  // tokens [lo, hi), lo a multiple of 64; splits that have any of them
};
template <bool TREE>
__device__ __forceinline__ TileRange tile_range(const AttnParams& a, const KvSpan& sp, int r0, int rows) {
    const int i0 = r0 / a.group, i1 = (min(r0 + rows, sp.n * a.group) - 1) / a.group;
    TileRange t;
    t.lo = edge_sight<TREE>(a, sp, i0, false).lo & ~63;
    t.hi = TREE ? sp.len : edge_sight<TREE>(a, sp, i1, true).hi;
    t.nact = (t.hi - t.lo + a.chunk - 1) / a.chunk;
    return t;
}

__device__ __forceinline__ f32x4_t ldexp4(f32x4_t v, int e) {
    return f32x4_t{ldexpf(v[0], e), ldexpf(v[1], e), ldexpf(v[2], e), ldexpf(v[3], e)};
}

// Power of two that brings the largest of a row's values (its bits without the sign) into [2^14, 2^15).
__device__ __forceinline__ int q_exponent(uint32_t top) {
    const int eb = top >> 23;
    return eb == 0 || eb == 255 ? 0 : 141 - eb;
}

// The kernel of tiles of 128 or 256 rows (qg_attn8_tile.hpp), and which of them a call takes.
int attn8_tile_rows(const AttnParams& a, int xt);
hipError_t launch_attn8_tile(const AttnParams& a, int xt, hipStream_t s);
constexpr int kPairTreeRows = 128;  // drafted rows of a sequence that two workgroups a CU have shared memory for
// The same kernels with masks among the batch's rows.
hipError_t launch_attn8_tree(const AttnParams& a, int xt, hipStream_t s);
hipError_t launch_attn8_tree_tile(const AttnParams& a, int xt, hipStream_t s);

}  // namespace qg
