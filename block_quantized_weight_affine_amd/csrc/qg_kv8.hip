// qg_kv8.hip -- the 8-bit key/value cache: new tokens coded into their blocks, and read back.
//
// A block is 16 tokens of one head with one scale for K and one for V:
//   d = amax / 127 over the block, code = rint(x / d), value = code * d.
// A block that held tokens before keeps the larger of its scale and the new tokens'; where it grows,
// the earlier codes are coded again as rint(code * d_old / d).
#include <hip/hip_runtime.h>

#include "qg_device.hpp"
#include "qg_internal.hpp"

namespace qg {
namespace {

constexpr float kPer127 = 1.0f / 127.0f;
constexpr int kWaves = 4;

// Two adjacent elements.
template <int XT>
__device__ __forceinline__ void load2(const void* x, int64_t i, float& a, float& b) {
    if constexpr (XT == XT_F32) {
        const float2 t = *(const float2*)((const float*)x + i);
        a = t.x;
        b = t.y;
    } else {
        const uint32_t t = *(const uint32_t*)((const uint16_t*)x + i);
        a = XT == XT_F16 ? f16_to_f32((uint16_t)t) : bf16_to_f32((uint16_t)t);
        b = XT == XT_F16 ? f16_to_f32((uint16_t)(t >> 16)) : bf16_to_f32((uint16_t)(t >> 16));
    }
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

// One wavefront codes one block of one head, K or V.  It holds the block in registers (16 dim values),
// so the new tokens are read once and nothing goes through shared memory:
//   K  a lane takes 16 dims of a token (16 codes = the 16 bytes that lie together in the cache);
//   V  a lane takes two dims of all 16 tokens (two 16-byte runs of the cache).
// Bound by memory traffic for prompts and by latency for single tokens.
template <int XT, int D>
__global__ __launch_bounds__(64 * kWaves) void kv8_write_kernel(KvCache c, KvSeqs q, const void* k, const void* v,
                                                                KvStrides st) {
    const int lane = threadIdx.x & 63;
    int item = blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int s = blockIdx.y;
    const KvSpan sp = kv8_span(q, s);
    const int h = item % c.heads;
    item /= c.heads;
    const bool is_v = item & 1;
    const int p0 = sp.len - sp.n;                    // first new position
    const int blk = (p0 >> 4) + (item >> 1);
    if (sp.n == 0 || 16 * blk >= sp.len) return;
    const int bi = kv8_block(c, q, s, h, blk);
    if (bi < 0) return;
    const int j0 = p0 > 16 * blk ? p0 - 16 * blk : 0;                      // new tokens of the block: j0 .. j1 - 1
    const int j1 = sp.len - 16 * blk < 16 ? sp.len - 16 * blk : 16;
    const bool begun = j0 > 0;
    const int64_t row = (int64_t)sp.r0 + 16 * blk - p0;                    // row of the block's token 0
    float* scale = (is_v ? c.vs : c.ks) + bi;
    const float d_old = begun ? *scale : 0.f;
    int8_t* out = (is_v ? c.vc : c.kc) + (int64_t)bi * (16 * D);
    if (!is_v) {
        constexpr int CH = D / 16, NI = (D + 63) / 64;
        float x[NI][16];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < NI; i++) {
            const int it = lane + 64 * i, tok = it / CH, ch = it % CH;
            if (it < D && tok >= j0 && tok < j1) {
                const int64_t at = (row + tok) * st.k_row + h * st.k_head + 16 * ch;
                float a[8], b[8];
                x_load8<XT>(k, at, a);
                x_load8<XT>(k, at + 8, b);
#pragma unroll
                for (int e = 0; e < 8; e++) x[i][e] = a[e], x[i][8 + e] = b[e];
#pragma unroll
                for (int e = 0; e < 16; e++) top = max(top, abs_bits(x[i][e]));
            }
        }
        const Coding cd = coding(wave_max(top), d_old, begun);
        if (lane == 0) *scale = cd.d;
#pragma unroll
        for (int i = 0; i < NI; i++) {
            const int it = lane + 64 * i, tok = it / CH, ch = it % CH;
            uint4* dst = (uint4*)(out + (ch * 16 + tok) * 16);
            if (it < D && tok >= j0 && tok < j1) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; e++)
                    w[e] = code8(x[i][4 * e] * cd.inv) | code8(x[i][4 * e + 1] * cd.inv) << 8 |
                           code8(x[i][4 * e + 2] * cd.inv) << 16 | code8(x[i][4 * e + 3] * cd.inv) << 24;
                *dst = make_uint4(w[0], w[1], w[2], w[3]);
            } else if (it < D && tok < j0 && cd.ratio != 1.f) {
                const uint4 o = *dst;
                uint32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
                for (int e = 0; e < 4; e++)
                    w[e] = code8(byte_s8(w[e], 0) * cd.ratio) | code8(byte_s8(w[e], 1) * cd.ratio) << 8 |
                           code8(byte_s8(w[e], 2) * cd.ratio) << 16 | code8(byte_s8(w[e], 3) * cd.ratio) << 24;
                *dst = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    } else {
        constexpr int NI = (D / 2 + 63) / 64;
        float x[NI][2][16];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < NI; i++) {
            const int dim = 2 * (lane + 64 * i);
#pragma unroll
            for (int t = 0; t < 16; t++) {
                x[i][0][t] = x[i][1][t] = 0.f;
                if (dim < D && t >= j0 && t < j1)
                    load2<XT>(v, (row + t) * st.v_row + h * st.v_head + dim, x[i][0][t], x[i][1][t]);
                top = max(top, max(abs_bits(x[i][0][t]), abs_bits(x[i][1][t])));
            }
        }
        const Coding cd = coding(wave_max(top), d_old, begun);
        if (lane == 0) *scale = cd.d;
#pragma unroll
        for (int i = 0; i < NI; i++) {
            const int dim = 2 * (lane + 64 * i);
            if (dim >= D) continue;
#pragma unroll
            for (int u = 0; u < 2; u++) {
                uint4* dst = (uint4*)(out + (dim + u) * 16);
                uint32_t w[4] = {0, 0, 0, 0}, old[4] = {0, 0, 0, 0};
                if (begun) {
                    const uint4 o = *dst;
                    old[0] = o.x, old[1] = o.y, old[2] = o.z, old[3] = o.w;
                }
                // earlier tokens, the new ones, and zeros past the sequence's end
#pragma unroll
                for (int t = 0; t < 16; t++) {
                    const uint32_t was = code8(byte_s8(old[t >> 2], t & 3) * cd.ratio);
                    w[t >> 2] |= (t < j0 ? was : code8(x[i][u][t] * cd.inv)) << (8 * (t & 3));
                }
                *dst = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
}

template <int YT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    return (uint32_t)f32_to_16<YT>(a) | (uint32_t)f32_to_16<YT>(b) << 16;
}

// Each value code * scale, rounded once to the output's type.  One wavefront a block, with the lane
// layout of the write kernel, so the stores of a token are one contiguous run.
template <int YT, int D>
__global__ __launch_bounds__(64 * kWaves) void kv8_read_kernel(KvCache c, KvSeqs q, void* k, void* v, KvStrides st) {
    const int lane = threadIdx.x & 63;
    int item = blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int s = blockIdx.y;
    const KvSpan sp = kv8_span(q, s);
    const int h = item % c.heads;
    item /= c.heads;
    const bool is_v = item & 1;
    const int p0 = sp.len - sp.n;
    const int blk = (p0 >> 4) + (item >> 1);
    if (sp.n == 0 || 16 * blk >= sp.len) return;
    const int bi = kv8_block(c, q, s, h, blk);
    const int j0 = p0 > 16 * blk ? p0 - 16 * blk : 0;
    const int j1 = sp.len - 16 * blk < 16 ? sp.len - 16 * blk : 16;
    const int64_t row = (int64_t)sp.r0 + 16 * blk - p0;
    const float d = bi < 0 ? 0.f : (is_v ? c.vs : c.ks)[bi];               // no page: zeros
    const int8_t* in = (is_v ? c.vc : c.kc) + (int64_t)(bi < 0 ? 0 : bi) * (16 * D);
    if (!is_v) {
        constexpr int CH = D / 16, NI = (D + 63) / 64;
#pragma unroll
        for (int i = 0; i < NI; i++) {
            const int it = lane + 64 * i, tok = it / CH, ch = it % CH;
            if (it >= D || tok < j0 || tok >= j1) continue;
            const uint4 o = *(const uint4*)(in + (ch * 16 + tok) * 16);
            const uint32_t w[4] = {o.x, o.y, o.z, o.w};
            const int64_t at = (row + tok) * st.k_row + h * st.k_head + 16 * ch;
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
        constexpr int NI = (D / 2 + 63) / 64;
#pragma unroll
        for (int i = 0; i < NI; i++) {
            const int dim = 2 * (lane + 64 * i);
            if (dim >= D) continue;
            const uint4 o = *(const uint4*)(in + dim * 16), o2 = *(const uint4*)(in + dim * 16 + 16);
            const uint32_t a[4] = {o.x, o.y, o.z, o.w}, b[4] = {o2.x, o2.y, o2.z, o2.w};
#pragma unroll
            for (int t = 0; t < 16; t++) {
                if (t < j0 || t >= j1) continue;
                const float x0 = byte_s8(a[t >> 2], t & 3) * d, x1 = byte_s8(b[t >> 2], t & 3) * d;
                const int64_t at = (row + t) * st.v_row + h * st.v_head + dim;
                if constexpr (YT == XT_F32)
                    *(float2*)((float*)v + at) = make_float2(x0, x1);
                else
                    *(uint32_t*)((uint16_t*)v + at) = pack2<YT>(keep_f32(x0), keep_f32(x1));
            }
        }
    }
}

template <int XT, int D>
void launch_one(bool write, const KvCache& c, const KvSeqs& q, void* k, void* v, const KvStrides& st, hipStream_t s) {
    // blocks that n consecutive tokens touch at most
    const int nblk = (q.max_new + 30) / 16;
    const dim3 grid((uint32_t)(((int64_t)nblk * 2 * c.heads + kWaves - 1) / kWaves), q.seqs);
    if (write)
        kv8_write_kernel<XT, D><<<grid, 64 * kWaves, 0, s>>>(c, q, k, v, st);
    else
        kv8_read_kernel<XT, D><<<grid, 64 * kWaves, 0, s>>>(c, q, k, v, st);
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
