// qg_kv8_block.hpp -- a block of the 8-bit key/value cache in a wavefront's registers: how values become codes, and how
// lanes share a block out.
#pragma once

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

}  // namespace
}  // namespace qg
