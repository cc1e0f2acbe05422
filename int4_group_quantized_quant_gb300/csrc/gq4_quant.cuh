// gq4_quant.cuh -- the group-wise quantizer's steps, shared by the kernels that
// write the 4-bit format (the weight quantizer and the key/value cache).
#pragma once

#include <cfloat>
#include <cstdint>

#include "gq4_device.cuh"

namespace gq4 {

__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b)
{
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// min and max that return NaN when either input is NaN, so that a NaN
// anywhere in a group reaches its range.
__device__ __forceinline__ float min_nan(float a, float b)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// min and max over the L consecutive lanes of this lane's segment (segments
// start at multiples of L, L <= 32).  A power of two: an xor butterfly that
// leaves the result in every lane.  Otherwise a tree towards the segment's
// first lane and a broadcast from it; lanes past the last whole segment
// only ever read themselves.
__device__ __forceinline__ void segment_min_max(float &lo, float &hi, int pos, int head, int L)
{
    if ((L & (L - 1)) == 0) {
        for (int off = L >> 1; off > 0; off >>= 1) {
            lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, off));
            hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, off));
        }
        return;
    }
    for (int off = 1; off < L; off <<= 1) {
        const float l2 = __shfl_down_sync(0xffffffffu, lo, off);
        const float h2 = __shfl_down_sync(0xffffffffu, hi, off);
        if (pos + off < L) {
            lo = min_nan(lo, l2);
            hi = max_nan(hi, h2);
        }
    }
    lo = __shfl_sync(0xffffffffu, lo, head);
    hi = __shfl_sync(0xffffffffu, hi, head);
}

__device__ __forceinline__ bool finite_f32(float v)
{
    return fabsf(v) <= FLT_MAX;  // false for NaN and +-inf
}

// Scale, zero and reciprocal of a group from its min and max (NaN when the
// group holds a NaN).  The group is bad when its range is not finite: a NaN,
// an infinity (inf - x, x - (-inf) or inf - inf) or an overflowing
// difference, exactly the groups the oracle rejects value by value.
struct GroupMap {
    float lo, s, r, z;
};

__device__ __forceinline__ GroupMap group_map(float lo, float hi, int &bad)
{
    GroupMap m;
    m.lo = __fadd_rn(lo, 0.0f);  // -0 becomes +0
    hi = __fadd_rn(hi, 0.0f);
    const float d = __fsub_rn(hi, m.lo);
    bad = finite_f32(d) ? 0 : 1;
    float s = __fdiv_rn(d, 15.0f);
    if (s < FLT_MIN) s = 1.0f;
    m.s = s;
    m.r = __frcp_rn(s);
    m.z = __fdiv_rn(-m.lo, s);
    return m;
}

// The 8 codes of one word: t = fl(fl(v - lo) * r) in packed pairs, then
// rounded to the nearest integer, ties to even, by cvt.rni.  (Rounding by
// adding 1.5 * 2^23 is not used: an add after the multiply may be fused into
// one FMA, which rounds the exact product instead of t.)  For a good group
// 0 <= t <= 15 (1 + 4u), so the code needs no clamp.  The eight codes are
// gathered by byte permutes into even and odd codes and merged as nibbles.
__device__ __forceinline__ uint32_t quantize_word(const float (&v)[8], const GroupMap &m)
{
    const f32x2 nlo = pack2(-m.lo, -m.lo), r = pack2(m.r, m.r);
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float2 t = unpack2(mul2(add2(pack2(v[i], v[i + 1]), nlo), r));
        b[i] = (uint32_t)__float2int_rn(t.x);
        b[i + 1] = (uint32_t)__float2int_rn(t.y);
    }
    const uint32_t even = __byte_perm(__byte_perm(b[0], b[2], 0x0040),
                                      __byte_perm(b[4], b[6], 0x0040), 0x5410);
    const uint32_t odd = __byte_perm(__byte_perm(b[1], b[3], 0x0040),
                                     __byte_perm(b[5], b[7], 0x0040), 0x5410);
    return even | (odd << 4);
}

}  // namespace gq4
