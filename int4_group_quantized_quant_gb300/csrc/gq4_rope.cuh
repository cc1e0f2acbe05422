// gq4_rope.cuh -- what the kernels that rotate by position share.
//
// Angles: pos * inv_freq is a 31-bit by 24-bit product; in binary64 its error
// is below 2^-22 of a radian at any position.  It is reduced modulo 2 pi in
// binary64 with a two-term constant (Cody and Waite's reduction) and handed
// to sincosf as a value in [-pi, pi], rounded to f32: 1.2e-7 of a radian.
#pragma once

#include <cstdint>

namespace gq4 {

__device__ __forceinline__ float2 sin_cos_of(int pos, float inv_freq)
{
    const double a = (double)pos * (double)inv_freq;
    const double n = rint(a * 0.15915494309189535);   // 1 / (2 pi)
    double r = fma(n, -6.283185307179586, a);         // 2 pi, high part
    r = fma(n, -2.4492935982947064e-16, r);           // 2 pi, low part
    float s, c;
    sincosf((float)r, &s, &c);
    return make_float2(s, c);
}

// 1 / sqrt(x): the approximation (2 ulp) and a Newton step.
__device__ __forceinline__ float inv_sqrt(float x)
{
    const float r = rsqrtf(x);
    const float e = fmaf(-x * r, r, 1.0f);
    return fabsf(e) < 0.5f ? fmaf(0.5f * r, e, r) : r;   // (x = 0, infinite: r as it is)
}

}  // namespace gq4
