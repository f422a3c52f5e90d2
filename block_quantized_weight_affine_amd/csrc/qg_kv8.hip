// qg_kv8.hip -- the 8-bit key/value cache: new tokens coded into their blocks, and read back.
//
// A block is 16 tokens of one head with one scale for K and one for V:
//   d = amax / 127 over the block, code = rint(x / d), value = code * d.
// A block that held tokens before keeps the larger of its scale and the new tokens'; where it grows,
// the earlier codes are coded again as rint(code * d_old / d).
#include <algorithm>

#include <hip/hip_runtime.h>

#include "qg_device.hpp"
#include "qg_internal.hpp"

namespace qg {
namespace {

constexpr float kPer127 = 1.0f / 127.0f;
constexpr int kWaves = 4;

// Four adjacent elements.
template <int XT>
__device__ __forceinline__ void load4(const void* x, int64_t i, float (&v)[4]) {
    if constexpr (XT == XT_F32) {
        const float4 t = *(const float4*)((const float*)x + i);
        v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
    } else {
        const uint2 t = *(const uint2*)((const uint16_t*)x + i);
        const uint32_t w[2] = {t.x, t.y};
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const uint16_t u = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
            v[e] = XT == XT_F16 ? f16_to_f32(u) : bf16_to_f32(u);
        }
    }
}

// How a wavefront shares a V block out: a lane takes four dims of TOK tokens.
template <int D>
struct VShare {
    static constexpr int groups = D / 4, parts = groups <= 16 ? 4 : groups <= 32 ? 2 : 1, TOK = 16 / parts;
};
// TOK codes of a dim, as the cache holds them.
template <int TOK>
__device__ __forceinline__ void load_run(const int8_t* p, uint32_t (&w)[TOK / 4]) {
#pragma unroll
    for (int i = 0; i < TOK / 4; i++) w[i] = ((const uint32_t*)p)[i];
}
template <int TOK>
__device__ __forceinline__ void store_run(int8_t* p, const uint32_t (&w)[TOK / 4]) {
    if constexpr (TOK == 16)
        *(uint4*)p = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (TOK == 8)
        *(uint2*)p = make_uint2(w[0], w[1]);
    else
        *(uint32_t*)p = w[0];
}

// |x| as bits: an unsigned maximum of these carries a NaN through to the scale.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t w = (uint32_t)__shfl_xor((int)v, o);
        v = w > v ? w : v;
    }
    return v;
}

// rint, limited to +-127, as the low byte.
__device__ __forceinline__ uint32_t code8(float x) {
    const float r = __builtin_rintf(x);
    return (uint32_t)(int)__builtin_amdgcn_fmed3f(r, -127.f, 127.f) & 0xffu;
}

__device__ __forceinline__ float byte_s8(uint32_t w, int i) { return (float)(int8_t)(w >> (8 * i)); }

// Scale of a block, the factor that new values are coded with, and that of the earlier codes.
struct Coding {
    float d, inv, ratio;
};
__device__ __forceinline__ Coding coding(uint32_t amax_bits, float d_old, bool begun) {
    Coding c;
    // an infinity would leave codes of 0 and of +-127 behind: its block becomes NaN as a whole
    const float d_new = amax_bits >= 0x7f800000u ? __builtin_nanf("") : __uint_as_float(amax_bits) * kPer127;
    c.d = begun && (d_old > d_new || d_old != d_old) ? d_old : d_new;
    // a subnormal scale has no finite reciprocal: the largest finite value takes its place
    c.inv = c.d > 0.f ? fminf(1.0f / c.d, 3.402823466e+38f) : 0.f;
    c.ratio = begun && c.d > d_old ? d_old / c.d : 1.f;
    return c;
}

// Where a wavefront's block lies: the block of the item-th that the sequence's rows touch.
struct Item {
    int h, blk, j0, j1;  // tokens j0 .. j1 - 1 of the block are the sequence's rows
    bool is_v, none;
    int64_t row;         // row of the block's token 0
};
__device__ __forceinline__ Item kv8_item(const KvCache& c, const KvSpan& sp, int item) {
    Item t;
    t.h = item % c.heads;
    item /= c.heads;
    t.is_v = item & 1;
    const int p0 = sp.len - sp.n;  // first new position
    t.blk = (p0 >> 4) + (item >> 1);
    t.none = sp.n == 0 || 16 * t.blk >= sp.len;
    t.j0 = p0 > 16 * t.blk ? p0 - 16 * t.blk : 0;
    t.j1 = sp.len - 16 * t.blk < 16 ? sp.len - 16 * t.blk : 16;
    t.row = (int64_t)sp.r0 + 16 * t.blk - p0;
    return t;
}

// This wavefront's item; group0: the launch's first workgroup.
__device__ __forceinline__ int wave_item(uint32_t group0) {
    return (int)((group0 + blockIdx.x) * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6));
}

// One wavefront codes one block of one head, K or V.  It holds the block in registers (16 dim values),
// so the new tokens are read once and nothing goes through shared memory:
//   K  a lane takes 16 dims of a token (16 codes = the 16 bytes that lie together in the cache);
//   V  a lane takes four dims of 4, 8 or 16 tokens (a run of the cache for each dim).
// The rows are read before the table's answer is there, the earlier scale and codes together: bound by
// memory traffic for prompts (24576 tokens of 8 heads of 128, bf16: 151 MB in 35 us, 4.3 TB/s) and by three
// loads' latency for single tokens (48 sequences: 5.3 us).  Four dims a lane for V rather than two halves
// its loads: 13 x 701 f32 tokens of 5 heads of 96 9.2 -> 8.7 us.
template <int XT, int D>
__global__ __launch_bounds__(64 * kWaves) void kv8_write_kernel(KvCache c, KvSeqs q, const void* k, const void* v,
                                                                KvStrides st, uint32_t group0) {
    const int lane = threadIdx.x & 63, s = blockIdx.y;
    const Item t = kv8_item(c, kv8_span(q, s), wave_item(group0));
    if (t.none) return;
    const bool begun = t.j0 > 0;
    if (!t.is_v) {
        constexpr int CH = D / 16, NI = (D + 63) / 64;
        float x[NI][16];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < NI; i++) {
            const int it = lane + 64 * i, tok = it / CH, ch = it % CH;
            if (it < D && tok >= t.j0 && tok < t.j1) {
                const int64_t at = (t.row + tok) * st.k_row + t.h * st.k_head + 16 * ch;
                float a[8], b[8];
                x_load8<XT>(k, at, a);
                x_load8<XT>(k, at + 8, b);
#pragma unroll
                for (int e = 0; e < 8; e++) x[i][e] = a[e], x[i][8 + e] = b[e];
            }
        }
        const int bi = kv8_block(c, q, s, t.h, t.blk);
        if (bi < 0) return;
        uint4* out = (uint4*)(c.kc + (int64_t)bi * (16 * D));
        float d_old = 0.f;
        uint4 old[NI];
        if (begun) {
            d_old = c.ks[bi];
#pragma unroll
            for (int i = 0; i < NI; i++) {
                const int it = min(lane + 64 * i, D - 1);
                old[i] = out[(it % CH) * 16 + it / CH];
            }
        }
#pragma unroll
        for (int i = 0; i < NI; i++) {
            const int it = lane + 64 * i, tok = it / CH;
            if (it < D && tok >= t.j0 && tok < t.j1) {
#pragma unroll
                for (int e = 0; e < 16; e++) top = max(top, abs_bits(x[i][e]));
            }
        }
        const Coding cd = coding(wave_max(top), d_old, begun);
        if (lane == 0) c.ks[bi] = cd.d;
#pragma unroll
        for (int i = 0; i < NI; i++) {
            const int it = lane + 64 * i, tok = it / CH, ch = it % CH;
            uint4* dst = out + ch * 16 + tok;
            if (it < D && tok >= t.j0 && tok < t.j1) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; e++)
                    w[e] = code8(x[i][4 * e] * cd.inv) | code8(x[i][4 * e + 1] * cd.inv) << 8 |
                           code8(x[i][4 * e + 2] * cd.inv) << 16 | code8(x[i][4 * e + 3] * cd.inv) << 24;
                *dst = make_uint4(w[0], w[1], w[2], w[3]);
            } else if (it < D && tok < t.j0 && cd.ratio != 1.f) {
                uint32_t w[4] = {old[i].x, old[i].y, old[i].z, old[i].w};
#pragma unroll
                for (int e = 0; e < 4; e++)
                    w[e] = code8(byte_s8(w[e], 0) * cd.ratio) | code8(byte_s8(w[e], 1) * cd.ratio) << 8 |
                           code8(byte_s8(w[e], 2) * cd.ratio) << 16 | code8(byte_s8(w[e], 3) * cd.ratio) << 24;
                *dst = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    } else {
        using Share = VShare<D>;
        constexpr int TOK = Share::TOK;
        const int dim = 4 * (lane % Share::groups), first = lane / Share::groups * TOK;
        const bool on = lane < Share::groups * Share::parts;
        float x[TOK][4];
#pragma unroll
        for (int j = 0; j < TOK; j++) {
#pragma unroll
            for (int e = 0; e < 4; e++) x[j][e] = 0.f;
            if (on && first + j >= t.j0 && first + j < t.j1)
                load4<XT>(v, (t.row + first + j) * st.v_row + t.h * st.v_head + dim, x[j]);
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

template <int YT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    return (uint32_t)f32_to_16<YT>(a) | (uint32_t)f32_to_16<YT>(b) << 16;
}

// Each value code * scale, rounded once to the output's type.  One wavefront a block, with the lane
// layout of the write kernel, so the stores of a token are one contiguous run.  Bound as the write kernel:
// 24576 tokens back as bf16 in 25 us (6 TB/s, the codes are still in the cache), 48 tokens in 4.2 us.
template <int YT, int D>
__global__ __launch_bounds__(64 * kWaves) void kv8_read_kernel(KvCache c, KvSeqs q, void* k, void* v, KvStrides st,
                                                               uint32_t group0) {
    const int lane = threadIdx.x & 63, s = blockIdx.y;
    const Item t = kv8_item(c, kv8_span(q, s), wave_item(group0));
    if (t.none) return;
    const int bi = kv8_block(c, q, s, t.h, t.blk);
    const float d = bi < 0 ? 0.f : (t.is_v ? c.vs : c.ks)[bi];  // no page: zeros
    const int8_t* in = (t.is_v ? c.vc : c.kc) + (int64_t)(bi < 0 ? 0 : bi) * (16 * D);
    if (!t.is_v) {
        constexpr int CH = D / 16, NI = (D + 63) / 64;
#pragma unroll
        for (int i = 0; i < NI; i++) {
            const int it = lane + 64 * i, tok = it / CH, ch = it % CH;
            if (it >= D || tok < t.j0 || tok >= t.j1) continue;
            const uint4 o = *(const uint4*)(in + (ch * 16 + tok) * 16);
            const uint32_t w[4] = {o.x, o.y, o.z, o.w};
            const int64_t at = (t.row + tok) * st.k_row + t.h * st.k_head + 16 * ch;
            if constexpr (YT == XT_F32) {
                float4* y = (float4*)((float*)k + at);
#pragma unroll
                for (int e = 0; e < 4; e++)
                    y[e] = make_float4(byte_s8(w[e], 0) * d, byte_s8(w[e], 1) * d, byte_s8(w[e], 2) * d,
                                       byte_s8(w[e], 3) * d);
            } else {
                uint4* y = (uint4*)((uint16_t*)k + at);
                uint32_t r[8];
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    r[2 * e] = pack2<YT>(keep_f32(byte_s8(w[e], 0) * d), keep_f32(byte_s8(w[e], 1) * d));
                    r[2 * e + 1] = pack2<YT>(keep_f32(byte_s8(w[e], 2) * d), keep_f32(byte_s8(w[e], 3) * d));
                }
                y[0] = make_uint4(r[0], r[1], r[2], r[3]);
                y[1] = make_uint4(r[4], r[5], r[6], r[7]);
            }
        }
    } else {
        using Share = VShare<D>;
        constexpr int TOK = Share::TOK;
        const int dim = 4 * (lane % Share::groups), first = lane / Share::groups * TOK;
        if (lane >= Share::groups * Share::parts) return;
        uint32_t w[4][TOK / 4];
#pragma unroll
        for (int e = 0; e < 4; e++) load_run<TOK>(in + dim * 16 + first + 16 * e, w[e]);
#pragma unroll
        for (int j = 0; j < TOK; j++) {
            if (first + j < t.j0 || first + j >= t.j1) continue;
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; e++) x[e] = byte_s8(w[e][j >> 2], j & 3) * d;
            const int64_t at = (t.row + first + j) * st.v_row + t.h * st.v_head + dim;
            if constexpr (YT == XT_F32)
                *(float4*)((float*)v + at) = make_float4(x[0], x[1], x[2], x[3]);
            else
                *(uint2*)((uint16_t*)v + at) = make_uint2(pack2<YT>(keep_f32(x[0]), keep_f32(x[1])),
                                                          pack2<YT>(keep_f32(x[2]), keep_f32(x[3])));
        }
    }
}

template <int XT, int D>
void launch_one(bool write, const KvCache& c, const KvSeqs& q, void* k, void* v, const KvStrides& st, hipStream_t s) {
    // blocks that n consecutive tokens touch at most
    const int nblk = (q.max_new + 30) / 16;
    const int64_t groups = ((int64_t)nblk * 2 * c.heads + kWaves - 1) / kWaves;
    for (int64_t first = 0; first < groups; first += kLaunchGroups) {
        const dim3 grid((uint32_t)std::min(groups - first, kLaunchGroups), q.seqs);
        if (write)
            kv8_write_kernel<XT, D><<<grid, 64 * kWaves, 0, s>>>(c, q, k, v, st, (uint32_t)first);
        else
            kv8_read_kernel<XT, D><<<grid, 64 * kWaves, 0, s>>>(c, q, k, v, st, (uint32_t)first);
    }
}

template <int XT>
hipError_t launch_dim(bool write, const KvCache& c, const KvSeqs& q, void* k, void* v, const KvStrides& st,
                      hipStream_t s) {
    switch (c.dim) {
        case 64: launch_one<XT, 64>(write, c, q, k, v, st, s); break;
        case 96: launch_one<XT, 96>(write, c, q, k, v, st, s); break;
        case 128: launch_one<XT, 128>(write, c, q, k, v, st, s); break;
        case 192: launch_one<XT, 192>(write, c, q, k, v, st, s); break;
        case 256: launch_one<XT, 256>(write, c, q, k, v, st, s); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv8(bool write, const KvCache& c, const KvSeqs& q, void* k, void* v, int xt, const KvStrides& st,
                      hipStream_t s) {
    if (xt == XT_F32) return launch_dim<XT_F32>(write, c, q, k, v, st, s);
    if (xt == XT_F16) return launch_dim<XT_F16>(write, c, q, k, v, st, s);
    return launch_dim<XT_BF16>(write, c, q, k, v, st, s);
}

}  // namespace qg
