// qg_draft.hip -- drafted tokens: the plan of a tree, and the verification against the target's probabilities.
#include <algorithm>

#include <hip/hip_runtime.h>

#include "qg_device.hpp"
#include "qg_internal.hpp"

namespace qg {
namespace {

// ---- the plan of a tree -------------------------------------------------------------------------------------------
constexpr int kMaxRows = 1024;  // rows of a sequence

// A workgroup a sequence, a thread a row: it walks up its parents, whose indices fall, and so writes its mask's words
// from the last to the first.  Bound by latency: lengths, parents, then a step of the walk after the other.
__global__ __launch_bounds__(256) void tree_plan_kernel(KvSeqs q, const int32_t* parents, uint32_t* mask, int words,
                                                        int32_t* pos, int window) {
    __shared__ int up[kMaxRows];
    const KvSpan sp = kv8_span(q, blockIdx.x);
    for (int r = threadIdx.x; r < sp.n; r += 256) {
        const int p = parents[sp.r0 + r];
        up[r] = p >= 0 && p < r ? p : -1;
    }
    __syncthreads();
    for (int r = threadIdx.x; r < sp.n; r += 256) {
        uint32_t* out = mask + (int64_t)(sp.r0 + r) * words;
        int depth = 0, w = words - 1;
        uint32_t bits = 0;
        for (int a = r; a >= 0; a = up[a], depth++) {
            if (window > 0 && depth >= window) continue;
            for (; w > a >> 5; w--) out[w] = bits, bits = 0;
            bits |= 1u << (a & 31);
        }
        for (; w >= 0; w--) out[w] = bits, bits = 0;
        pos[sp.r0 + r] = sp.len - sp.n + depth - 1;
    }
}

// ---- verification -------------------------------------------------------------------------------------------------
// Probabilities in 64 bits throughout: this card's 64-bit rate is that of 32, and a draw falls on a border between two
// tokens of a vocabulary of 10^5 in one call of a hundred if sums are off by 2^-24.
constexpr int kThreads = 256, kRun = 16;  // values a thread takes at a time

// 2^t for t <= 0, off by less than 2^-52 of it.  Series of e^x to x^12.
__device__ __forceinline__ double exp2_64(double t) {
    t = fmax(t, -1100.0);
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
// A logit's weight below the row's largest; c = log2(e) / temperature.
__device__ __forceinline__ double weight(float l, float top, double c) {
    if (l == -__builtin_inff()) return 0.0;
    const double t = ((double)l - (double)top) * c;
    return t == t ? exp2_64(t) : t;
}

template <int XT>
__device__ __forceinline__ float logit(const void* x, int64_t i) {
    if constexpr (XT == XT_F32) return ((const float*)x)[i];
    const uint16_t u = ((const uint16_t*)x)[i];
    return XT == XT_F16 ? f16_to_f32(u) : bf16_to_f32(u);
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// How a sequence draws: c > 0: from the probabilities of temperature log2(e) / c; 0: the largest logit; NaN: not at all.
__device__ __forceinline__ double draw_factor(const VerifyParams& p, int s) {
    if (!p.sample) return 0.0;
    const float t = p.temps ? p.temps[s] : 1.f;
    return t == 0.f ? 0.0 : t > 0.f && t < __builtin_inff() ? 1.4426950408889634 / (double)t : __builtin_nan("");
}

__device__ __forceinline__ bool better(float a, int i, float b, int j) { return a > b || (a == b && i < j); }

// Joins two chunks' parts.
__device__ __forceinline__ void join(VerifyPart& a, const VerifyPart& b, double c) {
    const bool first = better(a.top, a.at, b.top, b.at);
    const float top = first ? a.top : b.top;
    const int at = first ? a.at : b.at;
    double sum = a.sum + b.sum;  // a NaN of either
    if (c > 0.0) sum = (a.sum == 0.0 ? 0.0 : a.sum * weight(a.top, top, c)) + (b.sum == 0.0 ? 0.0 : b.sum * weight(b.top, top, c));
    a = VerifyPart{sum, top, at};
}

// A row's parts, joined by a wavefront.
__device__ __forceinline__ VerifyPart row_part(const VerifyPart* part, int chunks, double c) {
    const int lane = threadIdx.x & 63;
    VerifyPart a = {0.0, -__builtin_inff(), 0x7fffffff};
    for (int i = lane; i < chunks; i += 64) join(a, part[i], c);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const VerifyPart b = {__shfl_xor(a.sum, o), __shfl_xor(a.top, o), __shfl_xor(a.at, o)};
        join(a, b, c);
    }
    return a;
}
// Whether a row has a distribution, or a largest logit.
__device__ __forceinline__ bool row_ok(const VerifyPart& a, double c) {
    if (c == 0.0) return a.sum == a.sum && a.top > -__builtin_inff();
    return c > 0.0 && a.sum > 0.0 && a.sum < __builtin_inf();
}

// Chunk blockIdx.x % chunks of a row: its largest logit, where that stands first, and the sum of weights below it.
template <int XT>
__global__ __launch_bounds__(kThreads) void verify_part_kernel(VerifyParams p, uint32_t group0) {
    __shared__ VerifyPart sh[kThreads / 64];
    const int s = blockIdx.y;
    const KvSpan sp = kv8_span(p.q, s);
    uint32_t b = group0 + blockIdx.x;
    if (b == 0 && threadIdx.x == 0) {
        p.tickets[s] = 0;
        if (s == 0) p.tickets[p.q.seqs] = 0;
    }
    const int k = b % p.chunks;
    b /= p.chunks;
    const int r = b % p.q.max_new;
    const bool of_draft = b / p.q.max_new;
    if (r >= sp.n || (of_draft && r == sp.n - 1)) return;
    const double c = draw_factor(p, s);
    if (of_draft && c == 0.0) return;
    const int64_t row = sp.r0 + r;
    const void* x = of_draft ? p.draft : p.target;
    const int64_t at = row * (of_draft ? p.d_row : p.t_row);
    const int lo = k * p.chunk, hi = min(lo + p.chunk, p.vocab);
    VerifyPart a = {0.0, -__builtin_inff(), 0x7fffffff};
    for (int i0 = lo + threadIdx.x; i0 < hi; i0 += kThreads * kRun) {
        float v[kRun];
#pragma unroll
        for (int e = 0; e < kRun; e++) {
            const int i = i0 + e * kThreads;
            v[e] = i < hi ? logit<XT>(x, at + i) : -__builtin_inff();
        }
        VerifyPart n = {0.0, -__builtin_inff(), 0x7fffffff};
#pragma unroll
        for (int e = 0; e < kRun; e++) {
            if (better(v[e], i0 + e * kThreads, n.top, n.at)) n.top = v[e], n.at = i0 + e * kThreads;
            if (v[e] != v[e]) n.sum = __builtin_nan("");
        }
        if (c > 0.0)
#pragma unroll
            for (int e = 0; e < kRun; e++) n.sum += weight(v[e], n.top, c);
        join(a, n, c);
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const VerifyPart n = {__shfl_xor(a.sum, o), __shfl_xor(a.top, o), __shfl_xor(a.at, o)};
        join(a, n, c);
    }
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = a;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kThreads / 64; w++) join(a, sh[w], c);
        p.part[((of_draft ? (int64_t)p.q.T : 0) + row) * p.chunks + k] = a;
    }
}

// The weight that token i has in a draw.
template <int XT>
struct Mass {
    const void *target, *draft;
    int64_t t_at, d_at;
    float t_top, d_top;
    double c, t_inv, d_inv;  // 1 / sum; d_inv 0: the target's probabilities alone
    __device__ __forceinline__ double operator()(int i) const {
#pragma clang fp contract(off)  // equal probabilities leave nothing
        const double t = weight(logit<XT>(target, t_at + i), t_top, c) * t_inv;
        if (d_inv == 0.0) return t;
        return fmax(t - weight(logit<XT>(draft, d_at + i), d_top, c) * d_inv, 0.0);
    }
};

// Sum over a workgroup, to all threads; sh: 4 values.
__device__ __forceinline__ double group_sum(double v, double* sh) {
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
    return sh[0] + sh[1] + sh[2] + sh[3];
}

// The first i of lo .. hi - 1 at which the running sum of the masses exceeds goal; where rounding leaves none, the last
// that has a mass; -1 if none has.  All threads of a workgroup call it.
template <class M>
__device__ __forceinline__ int find_in_chunk(const M& mass, int lo, int hi, double goal, double* sh, int* sh_at) {
    const int per = (hi - lo + kThreads - 1) / kThreads, t = threadIdx.x, lane = t & 63;
    const int i0 = min(lo + t * per, hi), i1 = min(i0 + per, hi);
    double own = 0.0;
    int last = -1;
    for (int i = i0; i < i1; i++) {
        const double m = mass(i);
        own += m;
        if (m > 0.0) last = i;
    }
    double run = own;  // inclusive, over the wavefront
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const double u = __shfl_up(run, o);
        if (lane >= o) run += u;
    }
    __syncthreads();
    if (lane == 63) sh[t >> 6] = run;
    if (t == 0) sh_at[0] = 0x7fffffff, sh_at[1] = -1;
    __syncthreads();
    double before = run - own;
    for (int w = 0; w < t >> 6; w++) before += sh[w];
    if (last >= 0) {
        atomicMax(&sh_at[1], last);
        // a thread whose run may hold it looks; of several the first index counts
        double sum = before;
        if (before + own > goal)
            for (int i = i0; i < i1; i++) {
                const double m = mass(i);
                sum += m;
                if (m > 0.0 && sum > goal) {
                    atomicMin(&sh_at[0], i);
                    break;
                }
            }
    }
    __syncthreads();
    return sh_at[0] == 0x7fffffff ? sh_at[1] : sh_at[0];
}

// The chunk in which the running sum of `mass` (each chunk's, in order) exceeds goal, and the sum before it.
struct ChunkAt {
    int k;
    double before;
};
template <class F>
__device__ __forceinline__ ChunkAt find_chunk(const F& mass, int chunks, double goal) {
    const int lane = threadIdx.x & 63;
    ChunkAt found = {-1, 0.0};
    double sum = 0.0;
    for (int k0 = 0; k0 < chunks; k0 += 64) {
        const double own = k0 + lane < chunks ? mass(k0 + lane) : 0.0;
        double run = own;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const double u = __shfl_up(run, o);
            if (lane >= o) run += u;
        }
        const uint64_t hit = __ballot(own > 0.0 && sum + run > goal), any = __ballot(own > 0.0);
        const int at = hit ? __builtin_ctzll(hit) : any ? 63 - __builtin_clzll(any) : -1;
        if (at >= 0) found = ChunkAt{k0 + at, sum + __shfl(run - own, at)};
        if (hit) break;
        sum += __shfl(run, 63);
    }
    return found;
}

// Whether this is the last of n workgroups to come here; it then sees what the first wavefronts of all of them wrote.
__device__ __forceinline__ bool last_of(uint32_t* ticket, uint32_t n, int* sh) {
    __syncthreads();
    if (threadIdx.x == 0) {
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent");
        *sh = __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == n - 1;
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
    }
    __syncthreads();
    return *sh;
}

// The last sequence to end packs the rows of all: p.accepted and p.line are theirs.
__device__ __forceinline__ void finish(const VerifyParams& p, int* sh) {
    if (!last_of(&p.tickets[p.q.seqs], p.q.seqs, sh)) return;
    __shared__ int run[kThreads];
    int total = 0;
    for (int s0 = 0; s0 < p.q.seqs; s0 += kThreads) {
        const int s = s0 + threadIdx.x;
        KvSpan sp = {0, 0, 0};
        int count = 0;
        if (s < p.q.seqs) {
            sp = kv8_span(p.q, s);
            count = sp.n ? p.accepted[s] + 1 : 0;
        }
        __syncthreads();
        run[threadIdx.x] = count;
        __syncthreads();
        for (int o = 1; o < kThreads; o <<= 1) {
            const int u = threadIdx.x >= o ? run[threadIdx.x - o] : 0;
            __syncthreads();
            run[threadIdx.x] += u;
            __syncthreads();
        }
        if (s < p.q.seqs) {
            const int to = total + run[threadIdx.x] - count;
            p.rows_out[s] = to;
            for (int i = 0; i < count; i++) p.path[to + i] = p.line[sp.r0 + i];
            p.kv_out[s] = p.q.kv_len[s] - sp.n + count;
        }
        total += run[kThreads - 1];
    }
    if (threadIdx.x == 0) p.rows_out[p.q.seqs] = total;
    for (int i = total + threadIdx.x; i < p.q.T; i += kThreads) p.path[i] = -1;
}

// Tokens that were chosen: every row draws its own next token, and the sequence follows the rows that hold what was
// drawn.  A workgroup a row; the last one of a sequence follows it.
template <int XT>
__global__ __launch_bounds__(kThreads) void verify_tree_kernel(VerifyParams p) {
    __shared__ double sh[4];
    __shared__ int sh_at[2], sh_last, up[kMaxRows], tok[kMaxRows], drew[kMaxRows];
    const int s = blockIdx.y, r = blockIdx.x;
    const KvSpan sp = kv8_span(p.q, s);
    if (r >= max(sp.n, 1)) return;
    const double c = draw_factor(p, s);
    if (sp.n > 0) {
        const int64_t row = sp.r0 + r;
        const VerifyPart* part = p.part + row * p.chunks;
        const VerifyPart all = row_part(part, p.chunks, c);
        int token = -1;
        if (row_ok(all, c)) {
            token = all.at;
            if (c > 0.0) {
                const double goal = (double)p.sample[row] * all.sum;
                const ChunkAt ch = find_chunk([&](int k) { return part[k].sum == 0.0 ? 0.0 : part[k].sum * weight(part[k].top, all.top, c); }, p.chunks, goal);
                const Mass<XT> mass = {p.target, nullptr, row * p.t_row, 0, all.top, 0.f, c, 1.0, 0.0};
                const int lo = ch.k * p.chunk;
                token = find_in_chunk(mass, lo, min(lo + p.chunk, p.vocab), goal - ch.before, sh, sh_at);
            }
        }
        if (threadIdx.x == 0) __hip_atomic_store(&p.drawn[row], token, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (!last_of(&p.tickets[s], max(sp.n, 1), &sh_last)) return;
    for (int i = threadIdx.x; i < sp.n; i += kThreads) {
        const int u = p.parents ? p.parents[sp.r0 + i] : i - 1;
        up[i] = u >= 0 && u < i ? u : -1;
        tok[i] = p.tokens[sp.r0 + i];
        drew[i] = p.drawn[sp.r0 + i];
    }
    __syncthreads();
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x;
        int cur = 0, count = 0, next = -1;
        while (cur < sp.n) {  // cur grows
            if (lane == 0) p.line[sp.r0 + count] = sp.r0 + cur;
            count++;
            next = drew[cur];
            int to = sp.n;
            for (int i0 = cur + 1; i0 < sp.n && next >= 0; i0 += 64) {
                const int i = i0 + lane;
                const uint64_t hit = __ballot(i < sp.n && up[min(i, sp.n - 1)] == cur && tok[min(i, sp.n - 1)] == next);
                if (hit) {
                    to = i0 + __builtin_ctzll(hit);
                    break;
                }
            }
            cur = to;
        }
        if (lane == 0) {
            p.accepted[s] = max(count - 1, 0);
            p.next[s] = next;
        }
    }
    finish(p, &sh_last);
}

// Tokens that were drawn from the draft's probabilities, one after the other: row r + 1's token x stays where
// accept[r + 1] q(x) < p(x), p and q at row r; the first that does not ends the sequence with a draw from
// max(p - q, 0), and where all stay the draw is from p at the last row.  A workgroup a chunk: each finds the row at which
// the sequence ends, and sums its chunk of that row's masses; the last one draws.
template <int XT>
__global__ __launch_bounds__(kThreads) void verify_chain_kernel(VerifyParams p) {
    __shared__ double sh[4];
    __shared__ int sh_at[2], sh_last, sh_end;
    __shared__ VerifyPart sh_t, sh_d;
    const int s = blockIdx.y, k = blockIdx.x;
    const KvSpan sp = kv8_span(p.q, s);
    const double c = draw_factor(p, s);
    if (sp.n == 0 && k > 0) return;
    if (sp.n > 0) {
        if (threadIdx.x == 0) sh_end = sp.n - 1;
        __syncthreads();
        for (int r0 = 0; r0 < sp.n - 1; r0 += kThreads / 64) {
            const int r = r0 + (threadIdx.x >> 6);
            if (r < sp.n - 1) {
                const int64_t row = sp.r0 + r;
                const VerifyPart t = row_part(p.part + row * p.chunks, p.chunks, c);
                const int x = p.tokens[row + 1];
                bool stays = false;
                if (row_ok(t, c) && (uint32_t)x < (uint32_t)p.vocab) {
                    if (c == 0.0) {
                        stays = x == t.at;
                    } else {
                        const VerifyPart d = row_part(p.part + (p.q.T + row) * p.chunks, p.chunks, c);
                        if (row_ok(d, c)) {
                            const double pt = weight(logit<XT>(p.target, row * p.t_row + x), t.top, c) / t.sum;
                            const double qt = weight(logit<XT>(p.draft, row * p.d_row + x), d.top, c) / d.sum;
                            stays = (double)p.accept[row + 1] * qt < pt;
                        }
                    }
                }
                if (!stays && (threadIdx.x & 63) == 0) atomicMin(&sh_end, r);
            }
            __syncthreads();
            if (sh_end <= r0 + kThreads / 64 - 1) break;
        }
        const int e = sh_end;
        const int64_t row = sp.r0 + e;
        if (threadIdx.x < 64) {
            const VerifyPart t = row_part(p.part + row * p.chunks, p.chunks, c);
            if (threadIdx.x == 0) sh_t = t;
        } else if (threadIdx.x < 128) {
            VerifyPart d = {0.0, 0.f, 0};
            if (e < sp.n - 1) d = row_part(p.part + (p.q.T + row) * p.chunks, p.chunks, c);
            if (threadIdx.x == 64) sh_d = d;
        }
        __syncthreads();
    }
    const int e = sp.n > 0 ? sh_end : 0;
    const int64_t row = sp.r0 + e;
    const bool ok = sp.n > 0 && row_ok(sh_t, c), drawn = ok && c > 0.0;
    Mass<XT> mass = {p.target, p.draft, row * p.t_row, row * p.d_row, ok ? sh_t.top : 0.f, 0.f, c, 0.0, 0.0};
    if (drawn) {
        mass.t_inv = 1.0 / sh_t.sum;
        if (e < sp.n - 1 && row_ok(sh_d, c)) mass.d_top = sh_d.top, mass.d_inv = 1.0 / sh_d.sum;
        double sum = 0.0;
        const int lo = k * p.chunk, hi = min(lo + p.chunk, p.vocab);
        for (int i = lo + threadIdx.x; i < hi; i += kThreads) sum += mass(i);
        sum = group_sum(sum, sh);
        if (threadIdx.x == 0) __hip_atomic_store(&p.mass[(int64_t)s * p.chunks + k], sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (!last_of(&p.tickets[s], sp.n > 0 ? p.chunks : 1, &sh_last)) return;
    int token = -1;
    if (ok) {
        token = sh_t.at;
        if (drawn) {
            const double* m = p.mass + (int64_t)s * p.chunks;
            double all = 0.0;
            for (int i = threadIdx.x & 63; i < p.chunks; i += 64) all += m[i];
            all = wave_sum(all);
            const double u = (double)p.sample[row];
            ChunkAt ch;
            if (all > 0.0) {
                ch = find_chunk([&](int i) { return m[i]; }, p.chunks, u * all);
            } else {  // the draft's probabilities are nowhere below the target's
                mass.d_inv = 0.0;
                const VerifyPart* part = p.part + row * p.chunks;
                all = 1.0;
                ch = find_chunk([&](int i) { return part[i].sum == 0.0 ? 0.0 : part[i].sum * weight(part[i].top, sh_t.top, c) * mass.t_inv; }, p.chunks, u);
            }
            const int lo = ch.k * p.chunk;
            token = find_in_chunk(mass, lo, min(lo + p.chunk, p.vocab), u * all - ch.before, sh, sh_at);
        }
    }
    if (threadIdx.x < 64)  // what other workgroups read is written by the wavefront that ends with the fence
        for (int i = threadIdx.x; sp.n > 0 && i <= e; i += 64) p.line[sp.r0 + i] = sp.r0 + i;
    if (threadIdx.x == 0) {
        p.accepted[s] = e;
        p.next[s] = token;
    }
    finish(p, &sh_last);
}

// Chunks of a row: 64 at most, so that a wavefront joins them at once, and no less than 4096 values.
int chunk_of(int vocab) {
    const int64_t per = ((int64_t)vocab + 63) / 64, unit = 4096;
    return (int)std::max(unit, (per + unit - 1) / unit * unit);
}

template <int XT>
hipError_t launch_one(const VerifyParams& p, hipStream_t s) {
    const int64_t groups = (int64_t)p.chunks * p.q.max_new * (p.draft ? 2 : 1);
    for (int64_t first = 0; first < groups; first += kLaunchGroups)
        verify_part_kernel<XT><<<dim3((uint32_t)std::min(groups - first, kLaunchGroups), p.q.seqs), kThreads, 0, s>>>(p, (uint32_t)first);
    if (p.draft)
        verify_chain_kernel<XT><<<dim3(p.chunks, p.q.seqs), kThreads, 0, s>>>(p);
    else
        verify_tree_kernel<XT><<<dim3(p.q.max_new, p.q.seqs), kThreads, 0, s>>>(p);
    return hipGetLastError();
}

size_t up16(size_t n) { return (n + 15) / 16 * 16; }

}  // namespace

hipError_t launch_tree_plan(const KvSeqs& q, const int32_t* parents, uint32_t* mask, int words, int32_t* pos, int window,
                            hipStream_t s) {
    tree_plan_kernel<<<q.seqs, 256, 0, s>>>(q, parents, mask, words, pos, window);
    return hipGetLastError();
}

size_t verify_workspace(const KvSeqs& q, int vocab) {
    const size_t chunks = (vocab + chunk_of(vocab) - 1) / chunk_of(vocab), T = q.T, seqs = q.seqs;
    return 2 * T * chunks * sizeof(VerifyPart) + up16(seqs * chunks * 8) + 2 * up16(T * 4) + up16((seqs + 1) * 4);
}

hipError_t launch_draft_verify(VerifyParams p, void* ws, hipStream_t s) {
    p.chunk = chunk_of(p.vocab);
    p.chunks = (p.vocab + p.chunk - 1) / p.chunk;
    const size_t T = p.q.T, seqs = p.q.seqs;
    char* at = (char*)ws;
    p.part = (VerifyPart*)at;
    at += 2 * T * p.chunks * sizeof(VerifyPart);
    p.mass = (double*)at;
    at += up16(seqs * p.chunks * 8);
    p.drawn = (int32_t*)at;
    at += up16(T * 4);
    p.line = (int32_t*)at;
    at += up16(T * 4);
    p.tickets = (uint32_t*)at;
    if (p.xt == XT_F32) return launch_one<XT_F32>(p, s);
    if (p.xt == XT_F16) return launch_one<XT_F16>(p, s);
    return launch_one<XT_BF16>(p, s);
}

}  // namespace qg
