// qg_rope.hpp -- rotary positions: pairs of a head's values turned by the angle position * frequency.
//
//   y_a = m (x_a cos t - x_b sin t),  y_b = m (x_b cos t + x_a sin t),  t = position * freqs[i] of pair i < rot / 2,
//   (a, b) = (i, i + rot/2), or (2 i, 2 i + 1) where interleaved; values from rot on stay as they are.
#pragma once

#include <hip/hip_runtime.h>

#include "qg_device.hpp"
#include "qg_internal.hpp"

namespace qg {
namespace {

// (m cos, m sin) of position * f.  The angle is reduced in 64 bits (as fast as 32 on this card), where a position of 2^24
// leaves an error of 2^-27 radians; the rest of at most an eighth of a turn goes through the series of sin and cos to
// x^9 and x^10, off by less than 2^-28.
__device__ __forceinline__ float2 turn_of(int position, double f, float m) {
    const double turns = (double)position * f * 0.15915494309189535;  // 1 / (2 pi)
    const double quarters = 4.0 * (turns - __builtin_rint(turns));     // -2 .. 2
    const double k = __builtin_rint(quarters);
    const float x = (float)(quarters - k) * 1.57079632679489662f, z = x * x;
    const float s = fmaf(x * z, fmaf(z, fmaf(z, fmaf(z, 2.755731922e-6f, -1.984126984e-4f), 8.333333333e-3f), -1.666666667e-1f), x);
    const float c = fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -2.755731922e-7f, 2.480158730e-5f), -1.388888889e-3f), 4.166666667e-2f), -0.5f), 1.f);
    const int q = (int)k;  // NaN where a frequency is: s and c are NaN too
    const float u = q & 1 ? s : c, v = q & 1 ? c : s;
    return make_float2(m * ((q + 1) & 2 ? -u : u), m * (q & 2 ? -v : v));
}

__device__ __forceinline__ float turned_a(float a, float b, float2 t) { return fmaf(a, t.x, -(b * t.y)); }
__device__ __forceinline__ float turned_b(float a, float b, float2 t) { return fmaf(b, t.x, a * t.y); }

}  // namespace
}  // namespace qg
