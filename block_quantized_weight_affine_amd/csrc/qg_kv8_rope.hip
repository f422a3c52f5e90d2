// qg_kv8_rope.hip -- rotary positions of rows, and on the way into the 8-bit key/value cache.
#include <algorithm>

#include <hip/hip_runtime.h>

#include "qg_kv8_block.hpp"
#include "qg_rope.hpp"

namespace qg {
namespace {

constexpr int kTurns = 2048;  // (cos, sin) pairs that a workgroup keeps

// How a thread takes the values of a head: 16 bytes of either half of the turned part, or 16 bytes of adjacent pairs;
// kSingle: a pair at a time, where halves do not begin at a multiple of 16 bytes (8191 rows of 40 heads, bf16, 24 of 96 turned: 64
// us, with 32 of 96 26).
enum { kHalf = 0, kAdjacent = 1, kSingle = 2 };

template <int XT>
constexpr int kPer16 = XT == XT_F32 ? 4 : 8;

template <int XT>
int rope_mode(const Rotary& r) {
    return r.inter ? kAdjacent : r.rot / 2 % kPer16<XT> == 0 ? kHalf : kSingle;
}
template <int XT>
int rope_units(const Rotary& r, int mode, int dim) {
    const int v = kPer16<XT>;
    return mode == kAdjacent ? dim / v : mode == kHalf ? r.rot / 2 / v + (dim - r.rot) / v : r.rot / 2 + dim - r.rot;
}

template <int XT>
__device__ __forceinline__ void load16(const void* x, int64_t i, float (&v)[kPer16<XT>]) {
    if constexpr (XT == XT_F32) {
        const float4 t = *(const float4*)((const float*)x + i);
        v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
    } else {
        x_load8<XT>(x, i, v);
    }
}
template <int XT>
__device__ __forceinline__ void store16(void* y, int64_t i, const float (&v)[kPer16<XT>]) {
    if constexpr (XT == XT_F32) {
        *(float4*)((float*)y + i) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; e++)
            w[e] = (uint32_t)f32_to_16<XT>(keep_f32(v[2 * e])) | (uint32_t)f32_to_16<XT>(keep_f32(v[2 * e + 1])) << 16;
        *(uint4*)((uint16_t*)y + i) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}
template <int XT>
__device__ __forceinline__ float load1(const void* x, int64_t i) {
    if constexpr (XT == XT_F32) return ((const float*)x)[i];
    const uint16_t u = ((const uint16_t*)x)[i];
    return XT == XT_F16 ? f16_to_f32(u) : bf16_to_f32(u);
}
template <int XT>
__device__ __forceinline__ void store1(void* y, int64_t i, float v) {
    if constexpr (XT == XT_F32)
        ((float*)y)[i] = v;
    else
        ((uint16_t*)y)[i] = f32_to_16<XT>(keep_f32(v));
}

// Rows x of `rows` tokens (the first at row0), all heads, into y; tab: the tokens' turns, rot / 2 each.  Every thread
// reads what it writes before it writes, so y may be x.
template <int XT, int MODE>
__device__ __forceinline__ void rope_rows(const RopeRows& a, const Rotary& rt, int64_t row0, int rows, const float2* tab) {
    constexpr int V = kPer16<XT>, B = 4;  // units on their way at a time
    const uint32_t n = (uint32_t)rows * a.heads * a.units;
    const int half = rt.rot / 2;
    for (uint32_t u0 = threadIdx.x; u0 < n; u0 += 256 * B) {
        float x[B][2][V];
        int64_t from[B], to[B];
        int d[B], e2[B], tok[B];  // first dim, the other half's distance (0: none)
#pragma unroll
        for (int b = 0; b < B; b++) {
            const uint32_t u = min(u0 + 256 * b, n - 1), head = u / a.units % a.heads;
            const int unit = u % a.units;
            tok[b] = u / a.units / a.heads;
            if constexpr (MODE == kAdjacent) {
                d[b] = unit * V, e2[b] = 0;
            } else if constexpr (MODE == kHalf) {
                d[b] = unit * V < half ? unit * V : unit * V + half, e2[b] = unit * V < half ? half : 0;
            } else {
                d[b] = unit < half ? unit : unit + half, e2[b] = unit < half ? half : 0;
            }
            from[b] = (row0 + tok[b]) * a.x_row + head * a.x_head + d[b];
            to[b] = (row0 + tok[b]) * a.y_row + head * a.y_head + d[b];
            if constexpr (MODE == kSingle) {
                x[b][0][0] = load1<XT>(a.x, from[b]);
                x[b][1][0] = load1<XT>(a.x, from[b] + e2[b]);
            } else {
                load16<XT>(a.x, from[b], x[b][0]);
                if constexpr (MODE == kHalf) load16<XT>(a.x, from[b] + e2[b], x[b][1]);
            }
        }
#pragma unroll
        for (int b = 0; b < B; b++) {
            if (u0 + 256 * b >= n) break;
            const float2* t = tab + tok[b] * half;
            float y[2][V];
            if constexpr (MODE == kAdjacent) {
#pragma unroll
                for (int e = 0; e < V; e += 2) {
                    const bool on = d[b] + e < rt.rot;
                    const float2 c = t[on ? (d[b] + e) / 2 : 0];
                    y[0][e] = on ? turned_a(x[b][0][e], x[b][0][e + 1], c) : x[b][0][e];
                    y[0][e + 1] = on ? turned_b(x[b][0][e], x[b][0][e + 1], c) : x[b][0][e + 1];
                }
                store16<XT>(a.y, to[b], y[0]);
            } else if constexpr (MODE == kHalf) {
                if (e2[b] == 0) {
                    store16<XT>(a.y, to[b], x[b][0]);
                    continue;
                }
#pragma unroll
                for (int e = 0; e < V; e++) {
                    const float2 c = t[d[b] + e];
                    y[0][e] = turned_a(x[b][0][e], x[b][1][e], c);
                    y[1][e] = turned_b(x[b][0][e], x[b][1][e], c);
                }
                store16<XT>(a.y, to[b], y[0]);
                store16<XT>(a.y, to[b] + half, y[1]);
            } else {
                if (e2[b] == 0) {
                    store1<XT>(a.y, to[b], x[b][0][0]);
                    continue;
                }
                const float2 c = t[d[b]];
                store1<XT>(a.y, to[b], turned_a(x[b][0][0], x[b][1][0], c));
                store1<XT>(a.y, to[b] + half, turned_b(x[b][0][0], x[b][1][0], c));
            }
        }
    }
}

template <int XT>
__device__ __forceinline__ void rope_rows(const RopeRows& a, const Rotary& rt, int64_t row0, int rows, const float2* tab) {
    if (a.mode == kHalf) return rope_rows<XT, kHalf>(a, rt, row0, rows, tab);
    if (a.mode == kAdjacent) return rope_rows<XT, kAdjacent>(a, rt, row0, rows, tab);
    rope_rows<XT, kSingle>(a, rt, row0, rows, tab);
}

// A workgroup takes a.per tokens: their turns once into shared memory, then all heads, four units a thread on their way.
// Bound by memory: 8191 rows of 40 heads of 128 in f32 60 us, 5.6 TB/s (a copy of this card reaches 4.6 to 4.8; some of the
// rows stay in the last cache); 48 rows 4.5 us, a launch and two rounds of loads.
template <int XT>
__global__ __launch_bounds__(256) void rope_kernel(RopeRows a, Rotary rt, const int32_t* pos, int T) {
    __shared__ float2 tab[kTurns];
    const int64_t row0 = (int64_t)blockIdx.x * a.per;
    const int rows = (int)min((int64_t)a.per, T - row0), half = rt.rot / 2;
    for (int i = threadIdx.x; i < rows * half; i += 256) tab[i] = turn_of(pos[row0 + i / half], rt.freqs[i % half], rt.mscale);
    __syncthreads();
    rope_rows<XT>(a, rt, row0, rows, tab);
}

// qg_kv8.hip's blocks, K turned before it is coded.  A workgroup takes one block of 16 tokens and four heads of K or of
// V, a wavefront each; the block's turns are computed once by all of them.  Further workgroups turn q's rows, so that a step has one
// launch where it had two.  Bound by memory: 7 sequences of up to 4096 rows, 32 heads of q and 8 of K and V, f16, 77 us for
// 350 MB; a single row of 48 users 5.4 us, as long as qg_kv8.hip's without q; the
// rows that stay of 16 users' 8, read through src, 4.6 us.  8192 rows of 8 heads of 96, bf16, 32 values turned 16.4 us, 24 of them, whose
// halves begin off 16 bytes, 23.6.
//   K  a lane takes two groups of 8 dims of a token: the halves of 8 pairs, or what lies side by side.
template <int XT, int D>
__global__ __launch_bounds__(64 * kWaves) void kv8_write_rope_kernel(KvCache c, KvSeqs q, KvRope a, uint32_t group0) {
    __shared__ float2 tab[kTurns];
    const int lane = threadIdx.x & 63, s = blockIdx.y;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Rotary& rt = a.rot;
    const int half = rt.rot / 2;
    const KvSpan sp = kv8_span(q, s);
    const int p0 = sp.len - sp.n;  // first new position
    const int hg = (c.heads + kWaves - 1) / kWaves;
    uint32_t b = group0 + blockIdx.x;
    if (b >= (uint32_t)a.kv_groups) {
        const int i0 = (int)(b - a.kv_groups) * a.q.per, rows = min(a.q.per, sp.n - i0);
        if (rows <= 0) return;
        for (int i = threadIdx.x; i < rows * half; i += 256) {
            const int r = i0 + i / half;
            tab[i] = turn_of(a.pos ? a.pos[sp.r0 + r] : p0 + r, rt.freqs[i % half], rt.mscale);
        }
        __syncthreads();
        rope_rows<XT>(a.q, rt, sp.r0 + i0, rows, tab);
        return;
    }
    Item t;
    t.h = (int)(b % hg) * kWaves + wave;
    b /= hg;
    t.is_v = b & 1;
    t.blk = (p0 >> 4) + (int)(b >> 1);
    t.none = sp.n == 0 || 16 * t.blk >= sp.len;
    if (t.none) return;
    t.j0 = max(p0 - 16 * t.blk, 0);
    t.j1 = min(sp.len - 16 * t.blk, 16);
    t.row = (int64_t)sp.r0 + 16 * t.blk - p0;
    const bool begun = t.j0 > 0, head = t.h < c.heads;
    // the row that each token is read from, -1: zeros
    int from = lane >= t.j0 && lane < t.j1 ? (int)(t.row + lane) : -1;
    if (a.src && from >= 0) {
        from = a.src[from];
        if ((uint32_t)from >= (uint32_t)a.src_rows) from = -1;
    }
    if (!t.is_v) {
        constexpr int CH = D / 16, NI = (D + 63) / 64, QW = XT == XT_F32 ? 2 : 1, EB = XT == XT_F32 ? 4 : 2;
        const bool paired = !rt.inter && half % 8 == 0;  // a lane's two groups are the halves of 8 pairs
        uint4 raw[NI][2][QW];
        int dim[NI][2], row[NI];
#pragma unroll
        for (int i = 0; i < NI; i++) {
            const int it = min(lane + 64 * i, D - 1), tok = it / CH, p = it % CH;
            const bool far = paired && p < rt.rot / 16;
            dim[i][0] = far ? 8 * p : 16 * p;
            dim[i][1] = far ? 8 * p + half : 16 * p + 8;
            const int r = row[i] = __shfl(from, tok);
#pragma unroll
            for (int g = 0; g < 2; g++)
#pragma unroll
                for (int w = 0; w < QW; w++) raw[i][g][w] = make_uint4(0, 0, 0, 0);
            if (r >= 0 && head) {
                const char* at = (const char*)a.k + (r * a.st.k_row + t.h * a.st.k_head) * EB;
#pragma unroll
                for (int g = 0; g < 2; g++)
#pragma unroll
                    for (int w = 0; w < QW; w++) raw[i][g][w] = ((const uint4*)(at + dim[i][g] * EB))[w];
            }
        }
        const int bi = head ? kv8_block(c, q, s, t.h, t.blk) : -1;
        for (int i = threadIdx.x; i < (t.j1 - t.j0) * half; i += 64 * kWaves) {
            const int j = t.j0 + i / half;
            tab[j * half + i % half] =
                turn_of(a.pos ? a.pos[t.row + j] : 16 * t.blk + j, rt.freqs[i % half], rt.mscale);
        }
        __syncthreads();
        if (bi < 0) return;
        int8_t* out = c.kc + (int64_t)bi * (16 * D);
        auto place = [&](int i, int g) { return (uint2*)(out + (dim[i][g] / 16 * 16 + (lane + 64 * i) / CH) * 16 + dim[i][g] % 16); };
        float d_old = 0.f;
        uint2 old[NI][2];
        if (begun) {
            d_old = c.ks[bi];
#pragma unroll
            for (int i = 0; i < NI; i++)
                if (lane + 64 * i < D)
#pragma unroll
                    for (int g = 0; g < 2; g++) old[i][g] = *place(i, g);
        }
        float x[NI][2][8];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < NI; i++) {
            const int it = lane + 64 * i, tok = it / CH;
            if (it >= D || tok < t.j0 || tok >= t.j1) continue;
#pragma unroll
            for (int g = 0; g < 2; g++) x_load8<XT>(raw[i][g], 0, x[i][g]);
            const float2* turn = tab + tok * half;
            if (rt.inter) {
#pragma unroll
                for (int g = 0; g < 2; g++)
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        if (dim[i][g] + e >= rt.rot) continue;
                        const float2 cs = turn[(dim[i][g] + e) / 2];
                        const float u = x[i][g][e], v = x[i][g][e + 1];
                        x[i][g][e] = turned_a(u, v, cs);
                        x[i][g][e + 1] = turned_b(u, v, cs);
                    }
            } else if (paired) {
                if (dim[i][0] < half) {
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        const float2 cs = turn[dim[i][0] + e];
                        const float u = x[i][0][e], v = x[i][1][e];
                        x[i][0][e] = turned_a(u, v, cs);
                        x[i][1][e] = turned_b(u, v, cs);
                    }
                }
            } else {
                const int r = row[i];
                const int64_t at = r * a.st.k_row + t.h * a.st.k_head;
#pragma unroll
                for (int g = 0; g < 2; g++)
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        const int dd = dim[i][g] + e;
                        if (dd >= rt.rot) continue;
                        const bool low = dd < half;
                        const float2 cs = turn[low ? dd : dd - half];
                        const float u = x[i][g][e], v = r < 0 ? 0.f : load1<XT>(a.k, at + (low ? dd + half : dd - half));
                        x[i][g][e] = low ? turned_a(u, v, cs) : turned_b(v, u, cs);
                    }
            }
#pragma unroll
            for (int g = 0; g < 2; g++)
#pragma unroll
                for (int e = 0; e < 8; e++) top = max(top, abs_bits(x[i][g][e]));
        }
        const Coding cd = coding(wave_max(top), d_old, begun);
        if (lane == 0) c.ks[bi] = cd.d;
#pragma unroll
        for (int i = 0; i < NI; i++) {
            const int it = lane + 64 * i, tok = it / CH;
            if (it >= D || tok >= t.j1 || (tok < t.j0 && cd.ratio == 1.f)) continue;
#pragma unroll
            for (int g = 0; g < 2; g++) {
                uint32_t w[2] = {0, 0};
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const float v = tok >= t.j0 ? x[i][g][e] * cd.inv : byte_s8(e < 4 ? old[i][g].x : old[i][g].y, e & 3) * cd.ratio;
                    w[e >> 2] |= code8(v) << (8 * (e & 3));
                }
                *place(i, g) = make_uint2(w[0], w[1]);
            }
        }
    } else {
        using Share = VShare<D>;
        constexpr int TOK = Share::TOK;
        if (!head) return;
        const int dim = 4 * (lane % Share::groups), first = lane / Share::groups * TOK;
        const bool on = lane < Share::groups * Share::parts;
        float x[TOK][4];
#pragma unroll
        for (int j = 0; j < TOK; j++) {
#pragma unroll
            for (int e = 0; e < 4; e++) x[j][e] = 0.f;
            const int r = __shfl(from, min(first + j, 15));
            if (on && r >= 0) load4<XT>(a.v, r * a.st.v_row + t.h * a.st.v_head + dim, x[j]);
        }
        const int bi = kv8_block(c, q, s, t.h, t.blk);
        if (bi < 0) return;
        int8_t* out = c.vc + (int64_t)bi * (16 * D) + dim * 16 + first;
        float d_old = 0.f;
        uint32_t old[4][TOK / 4] = {};
        if (begun) {
            d_old = c.vs[bi];
#pragma unroll
            for (int e = 0; e < 4; e++)
                if (on) load_run<TOK>(out + 16 * e, old[e]);
        }
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < TOK; j++)
#pragma unroll
            for (int e = 0; e < 4; e++) top = max(top, abs_bits(x[j][e]));
        const Coding cd = coding(wave_max(top), d_old, begun);
        if (lane == 0) c.vs[bi] = cd.d;
        if (!on) return;
        // earlier tokens, the new ones, and zeros past the sequence's end
#pragma unroll
        for (int e = 0; e < 4; e++) {
            uint32_t w[TOK / 4] = {};
#pragma unroll
            for (int j = 0; j < TOK; j++) {
                uint32_t code = code8(x[j][e] * cd.inv);
                if (begun && first + j < t.j0) code = code8(byte_s8(old[e][j >> 2], j & 3) * cd.ratio);
                w[j >> 2] |= code << (8 * (j & 3));
            }
            store_run<TOK>(out + 16 * e, w);
        }
    }
}

// Tokens a workgroup of turned rows: some 4 units a thread, turns within shared memory.
template <int XT>
void plan_rows(RopeRows& a, const Rotary& rt, int dim) {
    a.mode = rope_mode<XT>(rt);
    a.units = rope_units<XT>(rt, a.mode, dim);
    const int64_t want = 1024 / std::max<int64_t>((int64_t)a.heads * a.units, 1);
    a.per = (int)std::clamp<int64_t>(std::min<int64_t>(want, rt.rot ? kTurns / (rt.rot / 2) : 16), 1, 16);
}

template <int XT, int D>
void launch_write(const KvCache& c, const KvSeqs& q, KvRope a, hipStream_t s) {
    const int64_t blocks = (q.max_new + 30) / 16;  // that n consecutive tokens touch at most
    a.kv_groups = (int)(blocks * 2 * ((c.heads + kWaves - 1) / kWaves));
    int64_t groups = a.kv_groups;
    if (a.q.x) {
        plan_rows<XT>(a.q, a.rot, D);
        groups += (q.max_new + a.q.per - 1) / a.q.per;
    }
    for (int64_t first = 0; first < groups; first += kLaunchGroups)
        kv8_write_rope_kernel<XT, D><<<dim3((uint32_t)std::min(groups - first, kLaunchGroups), q.seqs), 64 * kWaves, 0, s>>>(
            c, q, a, (uint32_t)first);
}

template <int XT>
hipError_t launch_dim(const KvCache& c, const KvSeqs& q, const KvRope& a, hipStream_t s) {
    switch (c.dim) {
        case 64: launch_write<XT, 64>(c, q, a, s); break;
        case 96: launch_write<XT, 96>(c, q, a, s); break;
        case 128: launch_write<XT, 128>(c, q, a, s); break;
        case 192: launch_write<XT, 192>(c, q, a, s); break;
        case 256: launch_write<XT, 256>(c, q, a, s); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

template <int XT>
hipError_t launch_rope_rows(RopeRows a, const Rotary& rt, const int32_t* pos, int T, int dim, hipStream_t s) {
    plan_rows<XT>(a, rt, dim);
    rope_kernel<XT><<<(T + a.per - 1) / a.per, 256, 0, s>>>(a, rt, pos, T);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv8_rope(const KvCache& c, const KvSeqs& q, const KvRope& a, int xt, hipStream_t s) {
    if (xt == XT_F32) return launch_dim<XT_F32>(c, q, a, s);
    if (xt == XT_F16) return launch_dim<XT_F16>(c, q, a, s);
    return launch_dim<XT_BF16>(c, q, a, s);
}

hipError_t launch_rope(const RopeRows& a, const Rotary& rt, const int32_t* pos, int T, int dim, int xt, hipStream_t s) {
    if (xt == XT_F32) return launch_rope_rows<XT_F32>(a, rt, pos, T, dim, s);
    if (xt == XT_F16) return launch_rope_rows<XT_F16>(a, rt, pos, T, dim, s);
    return launch_rope_rows<XT_BF16>(a, rt, pos, T, dim, s);
}

}  // namespace qg
