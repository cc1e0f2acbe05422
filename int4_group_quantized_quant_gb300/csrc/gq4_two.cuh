// gq4_two.cuh -- numbers of twice 24 bits as the unevaluated sum of two f32
// (Dekker 1971; Knuth's sum without a condition), for the few values that need
// more than f32's: a warp's operation in 64 bits takes 128 cycles here, one of
// these some 30.  Off by some 2^-46, of values between 2^-70 and 2^70 (below,
// the second parts lose bits).
#pragma once

namespace gq4 {

struct Two {
    float hi, lo;      // |lo| <= 2^-22 |hi|
};

__device__ __forceinline__ Two two_product(float a, float b)
{
    const float p = __fmul_rn(a, b);
    return {p, __fmaf_rn(a, b, -p)};
}

__device__ __forceinline__ Two mul(Two a, Two b)
{
    const Two p = two_product(a.hi, b.hi);
    return {p.hi, __fmaf_rn(a.lo, b.hi, __fmaf_rn(a.hi, b.lo, p.lo))};
}

// |a.hi| >= |b.hi|, or a.hi is 0
__device__ __forceinline__ Two add_smaller(Two a, Two b)
{
    const float s = __fadd_rn(a.hi, b.hi), rest = __fsub_rn(b.hi, __fsub_rn(s, a.hi));
    return {s, __fadd_rn(rest, __fadd_rn(a.lo, b.lo))};
}

__device__ __forceinline__ Two add(Two a, Two b)
{
    const float s = __fadd_rn(a.hi, b.hi), from_b = __fsub_rn(s, a.hi);
    const float rest = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, from_b)), __fsub_rn(b.hi, from_b));
    const float lo = __fadd_rn(rest, __fadd_rn(a.lo, b.lo)), hi = __fadd_rn(s, lo);
    return {hi, __fsub_rn(lo, __fsub_rn(hi, s))};
}

__device__ __forceinline__ Two &operator+=(Two &a, Two b)
{
    return a = add(a, b);
}

// A constant.
constexpr Two two_of(double x)
{
    return {(float)x, (float)(x - (double)(float)x)};
}

}  // namespace gq4
