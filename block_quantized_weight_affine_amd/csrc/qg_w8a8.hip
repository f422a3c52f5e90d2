// qg_w8a8.hip -- matrix product in 8-bit integers.
//
//   y[t][n] = (sum_k xq[t][k] w[n][k]) * dx[t] * dw[n],  dx[t] = amax_k |x[t][k]| / 127,
//   xq = rint(x / dx).
//
// The sums are exact in 32-bit integers (K <= 2^17), so no order of summation changes a result.
#include <hip/hip_runtime.h>

#include "qg_device.hpp"
#include "qg_internal.hpp"

namespace qg {
namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));

constexpr float kPer127 = 1.0f / 127.0f;

__device__ __forceinline__ uint32_t code8(float x) {
    const float r = __builtin_rintf(x);
    return (uint32_t)(int)__builtin_amdgcn_fmed3f(r, -127.f, 127.f) & 0xffu;
}

// A row's scale from the largest |x| as bits; an infinity makes the row NaN as a whole.
__device__ __forceinline__ float row_scale(uint32_t top) {
    return top >= 0x7f800000u ? __builtin_nanf("") : __uint_as_float(top) * kPer127;
}

// One workgroup codes one row of X: the maximum first, then the codes from a second read (the row is
// in the cache by then).  K % 16 == 0.
template <int XT>
__global__ __launch_bounds__(256) void x_code_kernel(const void* X, int K, int8_t* codes, float* scales) {
    __shared__ uint32_t sh[4];
    const int64_t base = (int64_t)blockIdx.x * K;
    uint32_t top = 0;
    for (int k = 8 * threadIdx.x; k < K; k += 2048) {
        float v[8];
        x_load8<XT>(X, base + k, v);
#pragma unroll
        for (int e = 0; e < 8; e++) top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = top;
    __syncthreads();
    top = max(max(sh[0], sh[1]), max(sh[2], sh[3]));
    const float d = row_scale(top);
    const float inv = d > 0.f ? fminf(1.0f / d, 3.402823466e+38f) : 0.f;
    if (threadIdx.x == 0) scales[blockIdx.x] = d;
    for (int k = 8 * threadIdx.x; k < K; k += 2048) {
        float v[8];
        x_load8<XT>(X, base + k, v);
        uint32_t w[2];
#pragma unroll
        for (int e = 0; e < 2; e++)
            w[e] = code8(v[4 * e] * inv) | code8(v[4 * e + 1] * inv) << 8 | code8(v[4 * e + 2] * inv) << 16 |
                   code8(v[4 * e + 3] * inv) << 24;
        *(uint2*)(codes + base + k) = make_uint2(w[0], w[1]);
    }
}

template <int YT>
__device__ __forceinline__ void store_y(void* Y, int64_t i, float v) {
    if constexpr (YT == XT_F32)
        ((float*)Y)[i] = v;
    else
        ((uint16_t*)Y)[i] = f32_to_16<YT>(keep_f32(v));
}

// 32 x 32 outputs a wavefront, operands straight from memory.
template <int YT>
__global__ __launch_bounds__(256) void w8a8_kernel(W8A8Params p) {
    const int lane = threadIdx.x & 63, r = lane & 31, g = lane >> 5;
    const int wave = threadIdx.x >> 6;
    const int n0 = blockIdx.x * 128 + 32 * wave, t0 = blockIdx.y * 32;
    if (n0 >= p.N) return;
    const int8_t* w = p.w + (int64_t)min(n0 + r, p.N - 1) * p.K + 16 * g;
    const int8_t* x = p.xq + (int64_t)min(t0 + r, p.T - 1) * p.K + 16 * g;
    i32x16_t acc = {};
    for (int k = 0; k < p.K; k += 32) {
        i32x4_t a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
        if (k + 16 * g < p.K) {
            a = *(const i32x4_t*)(w + k);
            b = *(const i32x4_t*)(x + k);
        }
        acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, acc, 0, 0, 0);
    }
    const int t = t0 + r;
    if (t >= p.T) return;
    const float dx = p.xs[t];
#pragma unroll
    for (int i = 0; i < 16; i++) {
        const int n = n0 + 8 * (i >> 2) + 4 * g + (i & 3);
        if (n < p.N) store_y<YT>(p.Y, (int64_t)t * p.N + n, (float)acc[i] * dx * p.ws[n]);
    }
}

}  // namespace

size_t w8a8_workspace(int N, int K, int T) { return ((size_t)T * K + 255) / 256 * 256 + (size_t)T * 4; }

hipError_t launch_w8a8(W8A8Params p, const void* X, int xt, int yt, void* ws, hipStream_t s) {
    p.xq = (const int8_t*)ws;
    float* xs = (float*)((char*)ws + ((size_t)p.T * p.K + 255) / 256 * 256);
    p.xs = xs;
    int8_t* xq = (int8_t*)ws;
    if (xt == XT_F32)
        x_code_kernel<XT_F32><<<p.T, 256, 0, s>>>(X, p.K, xq, xs);
    else if (xt == XT_F16)
        x_code_kernel<XT_F16><<<p.T, 256, 0, s>>>(X, p.K, xq, xs);
    else
        x_code_kernel<XT_BF16><<<p.T, 256, 0, s>>>(X, p.K, xq, xs);
    const dim3 grid((p.N + 127) / 128, (p.T + 31) / 32);
    if (yt == XT_F32)
        w8a8_kernel<XT_F32><<<grid, 256, 0, s>>>(p);
    else if (yt == XT_F16)
        w8a8_kernel<XT_F16><<<grid, 256, 0, s>>>(p);
    else
        w8a8_kernel<XT_BF16><<<grid, 256, 0, s>>>(p);
    return hipGetLastError();
}

}  // namespace qg
