// qg_draft.hip -- drafted tokens: the plan of a tree, and the verification against the target's probabilities.
#include <algorithm>

#include <hip/hip_runtime.h>

#include "qg_device.hpp"
#include "qg_internal.hpp"

namespace qg {
namespace {

// ---- the plan of a tree -------------------------------------------------------------------------------------------
constexpr int kMaxRows = kMaxTreeRows;

// A workgroup a sequence.  A parent's index is below its row's, so rows go in groups of 64, of which a wavefront first finds
// what a row's ancestors within the group are, a lane a row, doubling the steps that all of them know (6 turns at most), and
// the row that those follow; groups then take the rest of that row's mask, one after the other.  A row's depth is the number
// of its mask's bits, and a window keeps the last ones.  Bound by latency: lengths, parents, turns.  A tree of 25 rows 2.2
// us; 64 trees of 255 rows, each following one of two before it, 5.3, and 8 chains of 1000 16.7, by 256 threads 33 (a thread a row
// that walks up all of its parents: 2.7, 20 and 264).
template <int N>
__global__ __launch_bounds__(N) void tree_plan_kernel(KvSeqs q, const int32_t* parents, uint32_t* mask, int words, int32_t* pos,
                                                     int window) {
    constexpr int kThreads = N;
    __shared__ uint32_t bits[N][N / 32 + 1];  // of row r the words up to its group's
    __shared__ int follows[N], lowest[N];     // the earlier group's row that a row descends from, -1; the first row of its window
    const KvSpan sp = kv8_span(q, blockIdx.x);
    const int lane = threadIdx.x & 63;
    for (int r = threadIdx.x; r < (sp.n + 63 & ~63); r += kThreads) {
        const int g = r & ~63, p = r < sp.n ? parents[sp.r0 + r] : -1;
        int up = p >= g && p < r ? p - g : -1, from = p >= 0 && p < g ? p : -1;
        uint32_t lo = lane < 32 ? 1u << lane : 0, hi = lane < 32 ? 0 : 1u << (lane - 32);
        while (__any(up >= 0)) {
            const int at = max(up, 0);
            const uint32_t l = __shfl(lo, at), h = __shfl(hi, at);
            const int u = __shfl(up, at), f = __shfl(from, at);
            if (up >= 0) lo |= l, hi |= h, up = u, from = f;
        }
        bits[r][g / 32] = lo;
        bits[r][g / 32 + 1] = hi;
        follows[r] = from;
    }
    __syncthreads();
    for (int g = 64; g < sp.n; g += 64) {
        for (int x = threadIdx.x; x < 64 * (g / 32); x += kThreads) {
            const int r = g + (x & 63), w = x >> 6, from = follows[r];
            bits[r][w] = from >= 0 && w <= (from >> 5 | 1) ? bits[from][w] : 0;
        }
        __syncthreads();
    }
    for (int r = threadIdx.x; r < sp.n; r += kThreads) {
        int depth = 0, low = 0;
        for (int w = r >> 5; w >= 0; w--) {
            const uint32_t x = bits[r][w];
            const int need = window - depth;  // the window's first row is the one that has so many from it on
            depth += __builtin_popcount(x);
            if (window > 0 && need > 0 && depth >= window) {
                int at = 0;
#pragma unroll
                for (int b = 16; b > 0; b >>= 1)
                    if (__builtin_popcount(x >> (at + b)) >= need) at += b;
                low = 32 * w + at;
            }
        }
        lowest[r] = low;
        pos[sp.r0 + r] = sp.len - sp.n + depth - 1;
    }
    __syncthreads();
    for (int x = threadIdx.x; x < sp.n * words; x += kThreads) {
        const int r = x / words, w = x - r * words, low = lowest[r];
        uint32_t out = w <= r >> 5 ? bits[r][w] : 0;
        if (w <= low >> 5) out = w < low >> 5 ? 0 : out & ~0u << (low & 31);
        mask[(int64_t)sp.r0 * words + x] = out;
    }
}

// ---- verification -------------------------------------------------------------------------------------------------
// Probabilities in 64 bits throughout: this card's 64-bit rate is that of 32, and a draw falls on a border between two
// tokens of a vocabulary of 10^5 in one call of a hundred if sums are off by 2^-24.
//
// A row is cut into pieces of kPiece values, 16 a lane of a wavefront.
constexpr int kStep = 512, kPiece = 2 * kStep;

// 2^t, -1100 <= t <= 1, off by less than 2^-51 of it.  Series of e^x to x^12.
__device__ __forceinline__ double exp2_64(double t) {
    const double n = __builtin_rint(t), x = (t - n) * 0.69314718055994531;
    double y = 2.08767569878681e-9;
    y = fma(y, x, 2.50521083854417188e-8);
    y = fma(y, x, 2.75573192239858907e-7);
    y = fma(y, x, 2.75573192239858907e-6);
    y = fma(y, x, 2.48015873015873016e-5);
    y = fma(y, x, 1.98412698412698413e-4);
    y = fma(y, x, 1.38888888888888889e-3);
    y = fma(y, x, 8.33333333333333333e-3);
    y = fma(y, x, 4.16666666666666667e-2);
    y = fma(y, x, 1.66666666666666667e-1);
    y = fma(y, x, 0.5);
    y = fma(y, x, 1.0);
    y = fma(y, x, 1.0);
    return __builtin_amdgcn_ldexp(y, (int)n);
}
// The same for t = -a / 256, 0 <= a <= 281600, with 2^(j / 256) from a table, as two factors.  A series of 2^(-f / 256)
// about f = 1/2 to the fourth power: off by less than 2^-53 for 0 <= f < 1.  9 64-bit instructions with the sum of products
// that follows, and 3 of 32 bits; 64 entries take one more of each.
constexpr int kTable = 256;
__device__ __forceinline__ void exp2_64(double a, const double* table, double& u, double& v) {
    const double f = __builtin_amdgcn_fract(a);
    const int k = (int)-a;
    double y = 2.2363655419893987e-12;
    y = fma(y, f, -3.3082996515760766e-09);
    y = fma(y, f, 3.6655655953957943e-06);
    y = fma(y, f, -0.0027076061740619077);
    u = fma(y, f, 1.0);
    v = __builtin_amdgcn_ldexp(table[k & (kTable - 1)], k >> 8);
}
// The table, by all threads of a workgroup, for use behind their next barrier.
__device__ __forceinline__ void make_table(double* table) {
    for (int i = threadIdx.x; i < kTable; i += blockDim.x) table[i] = exp2_64(i / (double)kTable);
}

// A logit's weight below the row's largest; c = log2(e) / temperature.  0 where nothing is left to compare (both
// infinite), or the logit is a NaN: pieces note those apart.
__device__ __forceinline__ double weight(float l, float top, double c) {
    return exp2_64(fmax(((double)l - (double)top) * c, -1100.0));
}
// The same for many values up to one top: 2^(-(m - 256 l c) / 256), m = 256 top c rounded up so that no difference falls
// below 0, and what m gained by that as a factor e^x of all of them.  m stays below 2^44, c halved as often as that takes: from
// 2^43 on logits that differ do so by 2^-24 of them, 2^19 in the exponent, so that the lower one weighs nothing whatever c, and x,
// 2^-16 at most, needs no more than its square (a larger m gained so much that the largest logit itself weighed nothing).
// 0 for a NaN: pieces note those apart.
struct Weigh {
    double c, m, rest;
    const double* table;
    __device__ __forceinline__ Weigh(float top, double c_, const double* t) : c(256.0 * c_), table(t) {
        m = (double)top * c;
        const int over = min(44 - __builtin_amdgcn_frexp_exp(m), 0);
        c = __builtin_amdgcn_ldexp(c, over);
        m = __builtin_amdgcn_ldexp(m, over);
        m = fma(fabs(m), 2.220446049250313e-16, m);
        const double x = fma(-(double)top, c, m) * (0.69314718055994531 / 256);
        rest = fma(fma(x, 0.5, 1.0), x, 1.0);
    }
    __device__ __forceinline__ void operator()(float l, double& u, double& v) const {
        exp2_64(fmin(fma(-(double)l, c, m), 281600.0), table, u, v);
    }
};

template <int XT>
__device__ __forceinline__ float logit(const void* x, int64_t i) {
    if constexpr (XT == XT_F32) return ((const float*)x)[i];
    const uint16_t u = ((const uint16_t*)x)[i];
    return XT == XT_F16 ? f16_to_f32(u) : bf16_to_f32(u);
}
// Eight values of a row, as they lie: rows may begin at any element.
struct __attribute__((packed, aligned(2))) Loose16 {
    uint32_t w[4];
};
template <int XT>
struct Raw8 {
    Loose16 a[XT == XT_F32 ? 2 : 1];
};
// Values first .. first + 7 of a row of n; where those would end past it they begin earlier, and open_raw hides the ones
// before `first`.  Rows of fewer than 8 values are padded.
template <int XT>
__device__ __forceinline__ int row_start(int first, int n) { return n < 8 ? first : min(first, n - 8); }
template <int XT>
__device__ __forceinline__ Raw8<XT> load_raw(const void* x, int64_t at, int first, int n) {
    if (n >= 8) return *(const Raw8<XT>*)((const char*)x + (at + row_start<XT>(first, n)) * (XT == XT_F32 ? 4 : 2));
    Raw8<XT> r;
#pragma unroll
    for (int e = 0; e < 8; e++) {
        const bool on = first + e < n;
        if constexpr (XT == XT_F32) {
            r.a[e >> 2].w[e & 3] = on ? ((const uint32_t*)x)[at + first + e] : 0xff800000u;
        } else {
            const uint32_t u = on ? ((const uint16_t*)x)[at + first + e] : XT == XT_F16 ? 0xfc00u : 0xff80u;
            r.a[0].w[e >> 1] = e & 1 ? r.a[0].w[e >> 1] | u << 16 : u;
        }
    }
    return r;
}
// last: whether some of the wavefront's values may have to be hidden.
template <int XT>
__device__ __forceinline__ void open_raw(const Raw8<XT>& r, int first, int n, bool last, float* v) {
#pragma unroll
    for (int e = 0; e < 8; e++) {
        if constexpr (XT == XT_F32) {
            v[e] = __uint_as_float(r.a[e >> 2].w[e & 3]);
        } else {
            const uint16_t u = (uint16_t)(r.a[0].w[e >> 1] >> (16 * (e & 1)));
            v[e] = XT == XT_F16 ? f16_to_f32(u) : bf16_to_f32(u);
        }
    }
    if (last) {
        const int hide = first - row_start<XT>(first, n);
#pragma unroll
        for (int e = 0; e < 8; e++) v[e] = e < hide ? -__builtin_inff() : v[e];
    }
}

// Over a wavefront by lane shifts: within rows of 16 lanes, then from row to row.  CTRL: shift right by 1, 2, 4, 8
// (0x111 ..), row 0's and 2's last lane to the next row (0x142), lane 31 to the upper half (0x143).
template <int CTRL, int ROWS>
__device__ __forceinline__ double shifted(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xf, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xf, false);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_scan(double v) {  // inclusive
    v += shifted<0x111, 0xf>(v);
    v += shifted<0x112, 0xf>(v);
    v += shifted<0x114, 0xf>(v);
    v += shifted<0x118, 0xf>(v);
    v += shifted<0x142, 0xa>(v);
    v += shifted<0x143, 0xc>(v);
    return v;
}
__device__ __forceinline__ double lane_of(double v, int lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_sum(double v) { return lane_of(wave_scan(v), 63); }
template <int CTRL, int ROWS>
__device__ __forceinline__ float max_shifted(float v) {
    return fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(v), __float_as_int(v), CTRL, ROWS, 0xf, false)));
}
__device__ __forceinline__ float wave_max(float v) {
    v = max_shifted<0x111, 0xf>(v);
    v = max_shifted<0x112, 0xf>(v);
    v = max_shifted<0x114, 0xf>(v);
    v = max_shifted<0x118, 0xf>(v);
    v = max_shifted<0x142, 0xa>(v);
    v = max_shifted<0x143, 0xc>(v);
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ int min_shifted(int v) {
    return min(v, __builtin_amdgcn_update_dpp(v, v, CTRL, ROWS, 0xf, false));
}
__device__ __forceinline__ int wave_min(int v) {
    v = min_shifted<0x111, 0xf>(v);
    v = min_shifted<0x112, 0xf>(v);
    v = min_shifted<0x114, 0xf>(v);
    v = min_shifted<0x118, 0xf>(v);
    v = min_shifted<0x142, 0xa>(v);
    v = min_shifted<0x143, 0xc>(v);
    return __builtin_amdgcn_readlane(v, 63);
}

// How a sequence draws: c > 0: from the probabilities of temperature log2(e) / c; 0: the largest logit; NaN: not at all.
__device__ __forceinline__ double draw_factor(const VerifyParams& p, int s) {
    if (!p.sample) return 0.0;
    const float t = p.temps ? p.temps[s] : 1.f;
    return t == 0.f ? 0.0 : t > 0.f && t < __builtin_inff() ? 1.4426950408889634 / (double)t : __builtin_nan("");
}

// A row's parts, joined by a wavefront: lane l holds those of pieces l, l + 64, .., kHeld of them at most.
constexpr int kHeld = 4;
struct Row {
    VerifyPart all;
    double mass[kHeld];  // of the pieces held, below all.top (temperature above 0)
};
__device__ __forceinline__ Row row_of(const VerifyPart* part, int pieces, double c) {
    const int lane = threadIdx.x & 63;
    VerifyPart a[kHeld];
    float top = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < kHeld; i++) {
        a[i] = VerifyPart{0.0, -__builtin_inff(), 0x7fffffff};
        if (64 * i + lane < pieces) a[i] = part[64 * i + lane];
    }
#pragma unroll
    for (int i = 0; i < kHeld; i++) top = fmaxf(top, a[i].top);
    for (int i = 64 * kHeld + lane; i < pieces; i += 64) top = fmaxf(top, part[i].top);
    Row r;
    r.all.top = top = wave_max(top);
    double sum = 0.0;
    int at = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < kHeld; i++) {
        r.mass[i] = a[i].sum;
        if (64 * i < pieces && c > 0.0) r.mass[i] *= weight(a[i].top, top, c);
        sum += r.mass[i];
        if (a[i].top == top) at = min(at, a[i].at);
    }
    for (int i = 64 * kHeld + lane; i < pieces; i += 64) {
        const VerifyPart b = part[i];
        sum += c > 0.0 ? b.sum * weight(b.top, top, c) : b.sum;
        if (b.top == top) at = min(at, b.at);
    }
    r.all.sum = wave_sum(sum);
    r.all.at = c > 0.0 ? 0 : wave_min(at);
    return r;
}
// Whether a row has a distribution, or a largest logit.
__device__ __forceinline__ bool row_ok(const VerifyPart& a, double c) {
    if (c == 0.0) return a.sum == a.sum && a.top > -__builtin_inff();
    return c > 0.0 && a.sum > 0.0 && a.sum < __builtin_inf();
}

// The r-th row listed of a sequence; one that overlaps another may find the other's.
__device__ __forceinline__ int listed_row(const VerifyParams& p, const KvSpan& sp, int r) {
    return min(p.list[sp.r0 + r], sp.n - 1);
}

// Pieces of a row by a wavefront, p.per of them one after the other, the next one's values on their way: each piece's
// largest logit, where that stands first (temperature 0), and the sum of weights below it.  32 users' seven drafts, 128000 bf16
// logits a row, 25 us: 20 vector instructions for each of a lane's logits issue in 16 of them, the rest waits for a piece's loads, its largest
// logit, its weights and their sum, one after the other.  One user's five of 32000 4.4 us, a launch and its loads.
template <int XT>
__global__ __launch_bounds__(256) void verify_part_kernel(VerifyParams p, uint32_t group0) {
    __shared__ double table[kTable];
    const int s = blockIdx.y, lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const KvSpan sp = kv8_span(p.q, s);
    const int count = p.listed ? min(p.listed[s], sp.n) : sp.n;
    const uint32_t waves = (p.pieces + p.per - 1) / p.per;
    uint32_t b = (group0 + blockIdx.x) * 4 + wave;
    if (b == 0 && lane == 0) {
        p.tickets[s] = 0;
        if (s == 0) p.tickets[p.q.seqs] = 0;
    }
    if (!p.draft && (b - wave) / waves >= (uint32_t)count) return;  // nothing for any of the four
    if (p.sample) {
        make_table(table);
        __syncthreads();
    }
    const int k0 = b % waves * p.per, k1 = min(k0 + p.per, p.pieces);
    b /= waves;
    int r = b % p.rows;
    b /= p.rows;
    const bool of_draft = b == 1;
    if (b > (p.draft ? 1 : 0) || r >= count || (of_draft && r == sp.n - 1)) return;
    if (p.listed) r = listed_row(p, sp, r);
    const double c = draw_factor(p, s);
    if (of_draft && c == 0.0) return;
    const int64_t row = sp.r0 + r;
    const void* x = of_draft ? p.draft : p.target;
    const int64_t at = row * (of_draft ? p.d_row : p.t_row);
    VerifyPart* part = p.part + ((of_draft ? (int64_t)p.q.T : 0) + row) * p.pieces;
    const int i0 = 8 * lane;
    Raw8<XT> raw[2] = {load_raw<XT>(x, at, k0 * kPiece + i0, p.vocab), load_raw<XT>(x, at, k0 * kPiece + kStep + i0, p.vocab)};
    for (int k = k0; k < k1; k++) {
        float v[16];
        const bool last = (k + 1) * kPiece > p.vocab;
#pragma unroll
        for (int h = 0; h < 2; h++) open_raw<XT>(raw[h], k * kPiece + h * kStep + i0, p.vocab, last, v + 8 * h);
        if (k + 1 < k1)
#pragma unroll
            for (int h = 0; h < 2; h++) raw[h] = load_raw<XT>(x, at, (k + 1) * kPiece + h * kStep + i0, p.vocab);
        float top = v[0];
        bool nan = false;
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
            top = fmaxf(top, fmaxf(v[e], v[e + 1]));
            nan |= __builtin_isunordered(v[e], v[e + 1]);
        }
        top = wave_max(top);
        VerifyPart a = {0.0, top, 0x7fffffff};
        if (c > 0.0) {
            if (top > -__builtin_inff()) {
                const Weigh w(top, c, table);
#pragma unroll
                for (int e = 0; e < 16; e++) {
                    double f, g;
                    w(v[e], f, g);
                    a.sum = fma(f, g, a.sum);
                }
                a.sum *= w.rest;
            }
            a.sum = wave_sum(a.sum);
        } else {
#pragma unroll
            for (int e = 15; e >= 0; e--)
                if (v[e] == top) a.at = row_start<XT>(k * kPiece + (e >> 3) * kStep + i0, p.vocab) + (e & 7);
            a.at = wave_min(a.at);
        }
        if (__any(nan)) a.sum = __builtin_nan("");
        if (lane == 0) part[k] = a;
    }
}

// The probabilities in a draw of the tokens of a piece, 16 a lane: the target's, less the draft's.
template <int XT>
struct Mass {
    const void *target, *draft;
    int64_t t_at, d_at;
    Weigh t, d;
    double t_inv, d_inv;  // 1 / sum times the weights' common factor; d_inv 0: the target's alone
    int vocab;
    __device__ __forceinline__ int start(int i) const { return row_start<XT>(i, vocab); }
    __device__ __forceinline__ void operator()(int k, double (&m)[2][8]) const {
        const int i0 = k * kPiece + 8 * (threadIdx.x & 63);
        const bool last = (k + 1) * kPiece > vocab, both = d_inv != 0.0;
        Raw8<XT> rt[2], rd[2];
#pragma unroll
        for (int h = 0; h < 2; h++) rt[h] = load_raw<XT>(target, t_at, i0 + h * kStep, vocab);
        if (both)
#pragma unroll
            for (int h = 0; h < 2; h++) rd[h] = load_raw<XT>(draft, d_at, i0 + h * kStep, vocab);
#pragma unroll
        for (int h = 0; h < 2; h++) {
            float v[8];
            open_raw<XT>(rt[h], i0 + h * kStep, vocab, last, v);
#pragma unroll
            for (int e = 0; e < 8; e++) {
                double f, g;
                t(v[e], f, g);
                m[h][e] = f * g * t_inv;
            }
        }
        if (!both) return;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            float v[8];
            open_raw<XT>(rd[h], i0 + h * kStep, vocab, last, v);
#pragma unroll
            for (int e = 0; e < 8; e++) {
#pragma clang fp contract(off)  // equal probabilities leave nothing
                double f, g;
                d(v[e], f, g);
                const double q = f * g * d_inv;
                m[h][e] = fmax(m[h][e] - q, 0.0);
            }
        }
    }
};

// The first token of piece k at which the running sum of the masses exceeds goal; where rounding leaves none, the last
// that has a mass; -1 if none has.  By a wavefront.
template <class M>
__device__ __forceinline__ int find_in_piece(const M& mass, int k, double goal) {
    const int lane = threadIdx.x & 63, i0 = k * kPiece + 8 * lane;
    double m[2][8], before = 0.0;
    int last = -1;
    mass(k, m);
#pragma unroll
    for (int h = 0; h < 2; h++) {
        double own = 0.0;
#pragma unroll
        for (int e = 0; e < 8; e++) own += m[h][e];
        const double run = wave_scan(own);
        const uint64_t some = __ballot(own > 0.0), hit = __ballot(own > 0.0 && before + run > goal);
        if (some) {
            // the lane of the first hit, else the last that has a mass
            const int at = hit ? __builtin_ctzll(hit) : 63 - __builtin_clzll(some);
            int found = -1;
            double sum = before + (run - own);
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const bool over = sum > goal;  // an earlier one already was
                sum += m[h][e];
                if (m[h][e] > 0.0 && !(over && found >= 0)) found = mass.start(i0 + h * kStep) + e;
            }
            last = __builtin_amdgcn_readlane(found, at);
            if (hit) return last;
        }
        before += lane_of(run, 63);
    }
    return last;
}

// The piece in which the running sum of `mass` (each piece's, in order) exceeds goal, and the sum before it; where rounding
// leaves none, the last that has a mass.  By a wavefront.
struct PieceAt {
    int k;
    double before;
};
template <class F>
__device__ __forceinline__ PieceAt find_piece(const F& mass, int pieces, double goal) {
    const int lane = threadIdx.x & 63;
    PieceAt found = {-1, 0.0};
    double sum = 0.0;
    for (int k0 = 0; k0 < pieces; k0 += 64) {
        const double own = k0 + lane < pieces ? mass(k0 + lane) : 0.0;
        const double run = wave_scan(own);
        const uint64_t hit = __ballot(own > 0.0 && sum + run > goal), some = __ballot(own > 0.0);
        const int at = hit ? __builtin_ctzll(hit) : some ? 63 - __builtin_clzll(some) : -1;
        if (at >= 0) found = PieceAt{k0 + at, sum + lane_of(run - own, at)};
        if (hit) break;
        sum += lane_of(run, 63);
    }
    return found;
}

// The same over pieces that are held, and over a row's own.
__device__ __forceinline__ PieceAt find_held(const Row& row, int pieces, double goal) {
    PieceAt found = {-1, 0.0};
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < kHeld; i++) {
        if (64 * i >= pieces) break;
        const double run = wave_scan(row.mass[i]);
        const uint64_t hit = __ballot(row.mass[i] > 0.0 && sum + run > goal), some = __ballot(row.mass[i] > 0.0);
        const int at = hit ? __builtin_ctzll(hit) : some ? 63 - __builtin_clzll(some) : -1;
        if (at >= 0) found = PieceAt{64 * i + at, sum + lane_of(run - row.mass[i], at)};
        if (hit) break;
        sum += lane_of(run, 63);
    }
    return found;
}
__device__ __forceinline__ PieceAt find_piece(const Row& row, const VerifyPart* part, int pieces, double c, double goal) {
    if (pieces <= 64 * kHeld) return find_held(row, pieces, goal);
    return find_piece([&](int k) { return part[k].sum * weight(part[k].top, row.all.top, c); }, pieces, goal);
}

// What workgroups hand to each other within a launch: stores and loads that go past the dies' caches, so that no cache has
// to be written back or emptied for them.
template <class T>
__device__ __forceinline__ void hand_over(T* p, T v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <class T>
__device__ __forceinline__ T handed(const T* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// Whether this is the last of n wavefronts to come here; it then sees what all of them handed over.  A wavefront's stores
// have arrived before it counts itself.
__device__ __forceinline__ bool last_of(uint32_t* ticket, uint32_t n) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    uint32_t got = 0;
    if ((threadIdx.x & 63) == 0) got = __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const bool last = __builtin_amdgcn_readfirstlane(got) == n - 1;
    asm volatile("" ::: "memory");
    return last;
}
// The same for workgroups, of which the first wavefront goes on: counting at one address goes one after the other.
__device__ __forceinline__ bool last_group_of(uint32_t* ticket, uint32_t n) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    return threadIdx.x < 64 && last_of(ticket, n);
}

// Ends a sequence of span sp whose rows line[0 .. count - 1] stay (counted from its first; NULL: 0 .. count - 1): the last
// sequence to end packs the rows of all, T at most, as sequences that overlap could have more.  By a wavefront.
__device__ __forceinline__ void finish(const VerifyParams& p, int s, const KvSpan& sp, int count, int next, const int* line) {
    const int lane = threadIdx.x & 63;
    if (lane == 0) p.next[s] = next;
    if (p.q.seqs == 1) {
        if (lane == 0) {
            p.accepted[0] = max(count - 1, 0);
            p.rows_out[0] = 0;
            p.rows_out[1] = count;
            p.kv_out[0] = p.q.kv_len[0] - sp.n + count;
        }
        for (int i = lane; i < p.q.T; i += 64) p.path[i] = i < count ? sp.r0 + (line ? line[i] : i) : -1;
        return;
    }
    if (lane == 0) hand_over(&p.accepted[s], max(count - 1, 0));
    if (line)
        for (int i = lane; i < count; i += 64) hand_over(&p.line[sp.r0 + i], line[i]);
    KvSpan first = {0, 0, 0};  // the first sequences', while the others are waited for
    int first_kv = 0;
    if (lane < p.q.seqs) first = kv8_span(p.q, lane), first_kv = p.q.kv_len[lane];
    if (!last_of(&p.tickets[p.q.seqs], p.q.seqs)) return;
    int total = 0;
    for (int s0 = 0; s0 < p.q.seqs; s0 += 64) {
        const int s = s0 + lane;
        KvSpan sp = first;
        int count = 0, kv = first_kv;
        if (s < p.q.seqs) {
            if (s0 > 0) sp = kv8_span(p.q, s), kv = p.q.kv_len[s];
            count = sp.n ? handed(&p.accepted[s]) + 1 : 0;
        }
        int run = count;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int u = __shfl_up(run, o);
            if (lane >= o) run += u;
        }
        if (s < p.q.seqs) {
            const int to = min(total + run - count, p.q.T), end = min(to + count, p.q.T);
            p.rows_out[s] = to;
            p.kv_out[s] = kv - sp.n + count;
            for (int i = 0; i < count; i += 8) {
                int r[8];  // eight loads on their way
#pragma unroll
                for (int j = 0; j < 8; j++) r[j] = line ? handed(&p.line[sp.r0 + min(i + j, count - 1)]) : i + j;
#pragma unroll
                for (int j = 0; j < 8; j++)
                    if (to + i + j < end) p.path[to + i + j] = sp.r0 + r[j];
            }
        }
        total += __shfl(run, 63);
    }
    if (lane == 0) p.rows_out[p.q.seqs] = min(total, p.q.T);
    for (int i = total + lane; i < p.q.T; i += 64) p.path[i] = -1;
}

// What follows a row of the target, whose parts are joined, by its own probabilities: the token drawn, or the largest; -1 if
// there is none.
template <int XT>
__device__ __forceinline__ int draw_row(const VerifyParams& p, const Row& all, int64_t row, double u, double c, const double* table) {
    if (!row_ok(all.all, c)) return -1;
    if (c == 0.0) return all.all.at;
    const double goal = u * all.all.sum;
    const PieceAt at = find_piece(all, p.part + row * p.pieces, p.pieces, c, goal);
    Mass<XT> mass = {p.target, nullptr, row * p.t_row, 0, Weigh(all.all.top, c, table), Weigh(0.f, c, table), 0.0, 0.0, p.vocab};
    mass.t_inv = mass.t.rest;
    return find_in_piece(mass, at.k, goal - at.before);
}
__device__ __forceinline__ Row row_of(const VerifyParams& p, int64_t row, double c) {
    return row_of(p.part + row * p.pieces, p.pieces, c);
}
__device__ __forceinline__ int parent_of(const VerifyParams& p, const KvSpan& sp, int i) {
    const int u = p.parents ? p.parents[sp.r0 + i] : i - 1;
    return u >= 0 && u < i ? u : -1;
}
// The first of rows up[] / tok[] that follows `row` and holds `token`; n if none does.  By a wavefront.
__device__ __forceinline__ int follower(const int* up, const int* tok, int n, int row, int token) {
    if (token < 0) return n;
    for (int i0 = row + 1; i0 < n; i0 += 64) {
        const int i = min(i0 + (int)(threadIdx.x & 63), n - 1);
        const uint64_t hit = __ballot(i >= i0 && up[i] == row && tok[i] == token);
        if (hit) return i0 + __builtin_ctzll(hit);
    }
    return n;
}

// The first rows of large trees by themselves, a wavefront a sequence: what follows row 0, and the rows that descend from the
// one that holds it.  No other can be reached, so only those are looked at afterwards: of 45 rows some ten.  16 trees 6.9 us, one
// wavefront's chain of loads.
template <int XT>
__global__ __launch_bounds__(64) void verify_first_kernel(VerifyParams p) {
    __shared__ double table[kTable];
    __shared__ int up[kMaxRows], tok[kMaxRows];
    __shared__ volatile int in[kMaxRows];
    const int s = blockIdx.x, lane = threadIdx.x;
    const KvSpan sp = kv8_span(p.q, s);
    int listed = 0;
    if (sp.n > 0) {
        const double c = draw_factor(p, s);
        const double u = p.sample ? p.sample[sp.r0] : 0.f;
        const Row first = row_of(p, sp.r0, c);
        for (int i = lane; i < sp.n; i += 64) up[i] = parent_of(p, sp, i), tok[i] = p.tokens[sp.r0 + i];
        if (c > 0.0) make_table(table);
        __syncthreads();
        const int token = draw_row<XT>(p, first, sp.r0, u, c, table);
        if (lane == 0) p.drawn[sp.r0] = token;
        __syncthreads();
        const int child = follower(up, tok, sp.n, 0, token);
        for (int i0 = 0; i0 < sp.n && child < sp.n; i0 += 64) {
            const int i = i0 + lane;
            const bool row = i >= child && i < sp.n;
            const int parent = row ? up[i] : -1;
            bool on = row && i == child;
            in[min(i, kMaxRows - 1)] = on;
            for (;;) {  // parents come before their rows: a turn for each step down within these 64
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
                const bool more = row && !on && parent >= child && in[parent];
                if (!__any(more)) break;
                if (more) on = true, in[i] = 1;
            }
            const uint64_t all = __ballot(on);
            if (on) p.list_out[sp.r0 + listed + __builtin_popcountll(all & ((1ull << lane) - 1))] = i;
            listed += __builtin_popcountll(all);
        }
    }
    if (lane == 0) p.listed_out[s] = listed;
}

// Tokens that were chosen: every row, or every one listed, draws its own next token, and the sequence follows the rows that
// hold what was drawn.  A wavefront a row, four of them a workgroup; the last workgroup of a sequence follows it.  Bound by latency:
// 16 trees 9.9 us.
template <int XT>
__global__ __launch_bounds__(256) void verify_tree_kernel(VerifyParams p) {
    __shared__ double table[kTable];
    __shared__ int up[kMaxRows], tok[kMaxRows], drew[kMaxRows], line[kMaxRows];
    const int s = blockIdx.y, lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int r = blockIdx.x * 4 + wave;
    const KvSpan sp = kv8_span(p.q, s);
    const int rows = p.listed ? min(p.listed[s], sp.n) : sp.n;
    if (blockIdx.x * 4 >= max(rows, 1)) return;
    const double c = draw_factor(p, s);
    const bool some = r < rows;
    Row row;
    double u = 0.0;
    if (some) {
        if (p.listed) r = listed_row(p, sp, r);
        if (p.sample) u = p.sample[sp.r0 + r];
        row = row_of(p, sp.r0 + r, c);
    }
    if (c > 0.0) make_table(table);
    __syncthreads();
    if (some) {
        const int token = draw_row<XT>(p, row, sp.r0 + r, u, c, table);
        if (lane == 0) hand_over(&p.drawn[sp.r0 + r], token);
    }
    if (!last_group_of(&p.tickets[s], (max(rows, 1) + 3) / 4)) return;
    for (int i = lane; i < sp.n; i += 64) {
        up[i] = parent_of(p, sp, i);
        tok[i] = p.tokens[sp.r0 + i];
        drew[i] = handed(&p.drawn[sp.r0 + i]);  // of those that can be reached
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");  // one wavefront is left
    int count = 0, next = -1;
    for (int cur = 0; cur < sp.n;) {  // cur grows
        next = drew[cur];
        if (lane == 0) line[count] = cur;
        count++;
        cur = follower(up, tok, sp.n, cur, next);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
    finish(p, s, sp, count, next, line);
}

// Tokens that were drawn from the draft's probabilities, one after the other: row r + 1's token x stays where
// accept[r + 1] q(x) < p(x), p and q at row r; the first that does not ends the sequence with a draw from
// max(p - q, 0), and where all stay the draw is from p at the last row.  Every workgroup finds the row at which the
// sequence ends, eight rows at a time, a wavefront each for p and for q; for max(p - q, 0) the first p.per wavefronts then sum a
// piece each, and the last workgroup draws, else one alone does.  One user 6.4 us, 3 of them until the row is found, 1.4 for the last piece;
// 32 users of 128000 logits 15.7 us, 5 of them 64-bit instructions of the masses.
constexpr int kChainWaves = 16;
template <int XT>
__global__ __launch_bounds__(64 * kChainWaves) void verify_chain_kernel(VerifyParams p) {
    __shared__ double table[kTable];
    __shared__ VerifyPart sh_all[kChainWaves];
    __shared__ double sh_x[kChainWaves];  // p(x), q(x); temperature 0: whether x stays
    const int s = blockIdx.y, lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int k = wave < p.per ? blockIdx.x * p.per + wave : p.pieces;  // its piece, if it has one
    const KvSpan sp = kv8_span(p.q, s);
    const double c = draw_factor(p, s);
    if (sp.n == 0) {
        if (k == 0) finish(p, s, sp, 0, -1, nullptr);
        return;
    }
    constexpr int kRows = kChainWaves / 2;
    const bool draws = c > 0.0;
    int e;
    for (int r0 = 0;; r0 += kRows) {
        const int r = r0 + wave % kRows;
        const bool of_draft = wave >= kRows;
        const float limit = draws && lane < kRows && r0 + lane < sp.n - 1 ? p.accept[sp.r0 + r0 + lane + 1] : 0.f;
        if (r < sp.n && !(of_draft && (r == sp.n - 1 || c == 0.0))) {
            const int64_t row = sp.r0 + r;
            const int x = r < sp.n - 1 ? p.tokens[row + 1] : -1;
            const bool there = (uint32_t)x < (uint32_t)p.vocab;
            float l = 0.f;
            if (there) l = of_draft ? logit<XT>(p.draft, row * p.d_row + x) : logit<XT>(p.target, row * p.t_row + x);
            const Row a = row_of(p.part + ((of_draft ? (int64_t)p.q.T : 0) + row) * p.pieces, p.pieces, c);
            if (lane == 0) {
                sh_all[wave] = a.all;
                sh_x[wave] = c == 0.0 ? (double)(x == a.all.at) : there ? weight(l, a.all.top, c) / a.all.sum : 0.0;
            }
        }
        if (draws && r0 == 0) make_table(table);
        __syncthreads();
        bool stays = false;
        const int ri = r0 + lane;
        if (lane < kRows && ri < sp.n - 1 && row_ok(sh_all[lane], c)) {
            stays = sh_x[lane] > 0.0;
            if (c > 0.0) stays = row_ok(sh_all[lane + kRows], c) && (double)limit * sh_x[lane + kRows] < sh_x[lane];
        }
        const uint64_t ends = __ballot(lane < kRows && !stays);
        if (ends) {
            e = r0 + __builtin_ctzll(ends);
            break;
        }
        __syncthreads();
    }
    const int64_t row = sp.r0 + e;
    const VerifyPart t = sh_all[e % kRows];
    const bool ok = row_ok(t, c), drawn = ok && c > 0.0;
    float d_top = 0.f;
    double d_inv = 0.0;
    if (drawn && e < sp.n - 1) {
        const VerifyPart d = sh_all[e % kRows + kRows];
        if (row_ok(d, c)) d_top = d.top, d_inv = 1.0 / d.sum;
    }
    const bool shared = d_inv != 0.0;  // all wavefronts have a part in the draw
    if (!shared && k > 0) return;
    Mass<XT> mass = {p.target, p.draft, row * p.t_row, row * p.d_row, Weigh(t.top, c, table), Weigh(d_top, c, table), 0.0, 0.0,
                     p.vocab};
    mass.t_inv = mass.t.rest * (1.0 / t.sum);  // rounded like the draft's, as equal probabilities have to leave nothing
    if (shared) mass.d_inv = mass.d.rest * d_inv;
    double* m = p.mass + (int64_t)s * p.pieces;
    const double u = drawn ? (double)p.sample[row] : 0.0;
    if (shared) {
        if (k < p.pieces) {
            double v[2][8], sum = 0.0;
            mass(k, v);
#pragma unroll
            for (int x = 0; x < 16; x++) sum += v[x >> 3][x & 7];
            sum = wave_sum(sum);
            if (lane == 0) hand_over(&m[k], sum);
        }
        if (!last_group_of(&p.tickets[s], gridDim.x)) return;
    }
    int token = -1;
    if (ok) {
        token = t.at;
        if (drawn) {
            double goal = 0.0;
            PieceAt at = {-1, 0.0};
            if (shared) {
                Row pieces;
                pieces.all = t;
                double all = 0.0;
#pragma unroll
                for (int i = 0; i < kHeld; i++) {
                    pieces.mass[i] = 64 * i + lane < p.pieces ? handed(&m[64 * i + lane]) : 0.0;
                    all += pieces.mass[i];
                }
                for (int i = 64 * kHeld + lane; i < p.pieces; i += 64) all += handed(&m[i]);
                goal = u * wave_sum(all);
                at = p.pieces > 64 * kHeld ? find_piece([&](int i) { return handed(&m[i]); }, p.pieces, goal)
                                           : find_held(pieces, p.pieces, goal);
            }
            if (at.k < 0) {  // or the draft's probabilities are nowhere below the target's
                const VerifyPart* part = p.part + row * p.pieces;
                mass.d_inv = 0.0;
                mass.t_inv = mass.t.rest;
                goal = u * t.sum;
                at = find_piece(row_of(part, p.pieces, c), part, p.pieces, c, goal);
            }
            token = find_in_piece(mass, at.k, goal - at.before);
        }
    }
    finish(p, s, sp, e + 1, token, nullptr);
}

template <int XT>
void launch_parts(VerifyParams p, hipStream_t s) {
    const int64_t rows = (int64_t)p.rows * (p.draft ? 2 : 1);
    // a wavefront's start is worth some pieces where all SIMDs have several, but longer ones even out worse (whole calls of 1 / 3 / 8
    // pieces, bf16, 128000 logits: 32 users of up to 8 rows 45.5 / 40.5 / 54 us, of 8 rows 62 / 57 / 58, 8 users 30.6 / 30.5 / 33);
    // of listed rows there are a quarter or so
    p.per = (int)std::clamp<int64_t>(rows * p.q.seqs * p.pieces / (p.listed ? 4 * 8192 : 8192), 1, 3);
    const int64_t groups = (rows * ((p.pieces + p.per - 1) / p.per) + 3) / 4;
    for (int64_t first = 0; first < groups; first += kLaunchGroups)
        verify_part_kernel<XT><<<dim3((uint32_t)std::min(groups - first, kLaunchGroups), p.q.seqs), 256, 0, s>>>(p, (uint32_t)first);
}

// Pieces of max(p - q, 0) a workgroup: 16, or fewer where that leaves no more workgroups than CUs, as the wavefronts of one wait
// for each other (16 a workgroup and by this rule: one user of 32000 logits 13.9 and 12.4 us a call, 8 of 128000 30.2 and 28.5, 32 of
// 32000 29.5 and 27.1; 32 of 128000 by twice as many workgroups 64, by 256 57).
template <int XT>
void launch_chains(VerifyParams p, hipStream_t s) {
    p.per = kChainWaves;
    while (p.per > 1 && (int64_t)p.q.seqs * ((p.pieces + p.per / 2 - 1) / (p.per / 2)) <= 256) p.per /= 2;
    verify_chain_kernel<XT><<<dim3((p.pieces + p.per - 1) / p.per, p.q.seqs), 64 * kChainWaves, 0, s>>>(p);
}

// Pieces of a batch of trees from which the first rows go before the others, in two launches more.  All rows at once and the
// first before the others, half of the tokens drawn, bf16: 8 trees of 45 rows of 32000 values (11520 pieces) 21 and 22 us, 16
// (23040) 29 and 26, 16 of 25 of 131072 (51200) 46 and 30, 64 of 61 of 32000 (124928) 97 and 45.
constexpr int64_t kFirstFrom = 20000;

template <int XT>
hipError_t launch_one(VerifyParams p, hipStream_t s) {
    p.rows = p.q.max_new;
    if (p.parents && (int64_t)p.q.max_new * p.q.seqs * p.pieces >= kFirstFrom) {
        p.rows = 1;
        launch_parts<XT>(p, s);
        verify_first_kernel<XT><<<p.q.seqs, 64, 0, s>>>(p);
        p.rows = p.q.max_new;
        p.listed = p.listed_out;
        p.list = p.list_out;
    }
    launch_parts<XT>(p, s);
    if (p.draft)
        launch_chains<XT>(p, s);
    else
        verify_tree_kernel<XT><<<dim3((p.q.max_new + 3) / 4, p.q.seqs), 256, 0, s>>>(p);
    return hipGetLastError();
}

size_t up16(size_t n) { return (n + 15) / 16 * 16; }

}  // namespace

hipError_t launch_tree_plan(const KvSeqs& q, const int32_t* parents, uint32_t* mask, int words, int32_t* pos, int window,
                            hipStream_t s) {
    if (q.max_new <= 64)
        tree_plan_kernel<64><<<q.seqs, 64, 0, s>>>(q, parents, mask, words, pos, window);
    else if (q.max_new <= 256)
        tree_plan_kernel<256><<<q.seqs, 256, 0, s>>>(q, parents, mask, words, pos, window);
    else
        tree_plan_kernel<kMaxRows><<<q.seqs, kMaxRows, 0, s>>>(q, parents, mask, words, pos, window);
    return hipGetLastError();
}

size_t verify_workspace(const KvSeqs& q, int vocab) {
    const size_t pieces = (vocab + kPiece - 1) / kPiece, T = q.T, seqs = q.seqs;
    return 2 * T * pieces * sizeof(VerifyPart) + up16(seqs * pieces * 8) + 3 * up16(T * 4) + up16(seqs * 4) + up16((seqs + 1) * 4);
}

hipError_t launch_draft_verify(VerifyParams p, void* ws, hipStream_t s) {
    p.pieces = (p.vocab + kPiece - 1) / kPiece;
    const size_t T = p.q.T, seqs = p.q.seqs;
    char* at = (char*)ws;
    p.part = (VerifyPart*)at;
    at += 2 * T * p.pieces * sizeof(VerifyPart);
    p.mass = (double*)at;
    at += up16(seqs * p.pieces * 8);
    p.drawn = (int32_t*)at;
    at += up16(T * 4);
    p.line = (int32_t*)at;
    at += up16(T * 4);
    p.list_out = (int32_t*)at;
    at += up16(T * 4);
    p.listed_out = (int32_t*)at;
    at += up16(seqs * 4);
    p.tickets = (uint32_t*)at;
    if (p.xt == XT_F32) return launch_one<XT_F32>(p, s);
    if (p.xt == XT_F16) return launch_one<XT_F16>(p, s);
    return launch_one<XT_BF16>(p, s);
}

}  // namespace qg
