// gq4_kv_rope.cu -- a step's rows on their way into the attention, in one pass
// (gq4_kv_rope_append): queries normalised and rotated, keys normalised, rotated
// and quantised into the cache, values quantised.
//
//   y = x / sqrt(mean(x^2) + eps) * gain,  (y_a, y_b) -> rotation by
//   positions[t] * inv_freq[i],  then gq4_quantize's rule per group.
//
// What it saves over gq4_head_norm_rope and gq4_kv_append: a launch, and the
// rotated keys' way to HBM and back (8 bytes per value of k).  Floor: 8 bytes
// per value of q, 4 read and 0.5 + 8/gs written per value of k and v.
//
// A lane holds a word's 8 values, a row takes D/8 lanes, a warp as many rows as
// fit; a CTA takes one token (few tokens: a share of its rows).  All rows of a
// warp are of one kind, so that it goes one way: rows are numbered in units of a
// warp's.  Half-split pairs are read a second time, as two float4s (a first-level
// cache hit), which takes 2 instructions where shuffles take 8.
//
// Codes next to a border.  A key's code is that of its exact value, rounded once
// to f32, as if the rotation were computed in 64 bits: so it does not depend on
// how sums and products were ordered.  The rotation itself is f32; what it
// leaves of a key is off by at most kKeyError (|a| + |b|) for the pair (a, b)
// before the rotation.  Where that could turn a code's rounding -- a value so
// near to the border of two codes -- the warp computes its rows again, the
// values next to a border and next to the group's two ends in 64 bits
// (exact_unit).  With groups of 128 normal values that is one unit in 60.
#include <cstdint>

#include "gq4_kv_internal.h"
#include "gq4_kv_write.cuh"
#include "gq4_rope.cuh"

namespace gq4 {
namespace {

__device__ unsigned int g_kv_rope_error = 0;
constexpr int kRopeAppendThreads = 256, kRopeAppendWarps = kRopeAppendThreads / 32;

// A rotated value's error relative to |a| + |b|, in units of 2^-24 (a rounding):
// the angle's rounding 2, the sine and cosine 2, the gain 1, the products and
// their sum 2, the factor that the row shares 1 (its own error is the same for
// all of the row and moves no code), and 1 that the value in 64 bits is rounded
// by.
constexpr float kKeyError = 9 * 0x1p-24f;
// Of a code's argument (v - lo) r, up to 15, on either side: two roundings and r's two.
constexpr float kCodeError = 8 * 15 * 0x1p-24f;

struct RopeAppendParams {
    gq4_kv_cache c;
    const float *x[3];       // k, v, q
    int ld[3];
    const float *gain[3];    // k's, none, q's (NULL: not normalised)
    float *q_out;
    int ldq_out;
    const int32_t *positions, *slots;
    const float *inv_freq;
    float eps, inv_d;
    int T, q_heads, rot;
    bool interleaved;
    int shift, total;        // log2 of the page size; slots of the pool
    uint32_t page_codes, page_sz;   // bytes per page and head
    int kv_units, units;     // units of k's rows, and of v's; and all (k, v, q)
    int splits;              // CTAs per token
};

enum { kKeyRow, kValueRow, kQueryRow };

// A lane's 8 values and, half-split, their partners.
struct Words {
    float4 v[2], w[2];
};

template <int J>
struct Unit {
    int kind, head;
    bool live;
    const float *row;

    __device__ __forceinline__ Unit(const RopeAppendParams &p, int t, int u, int in_warp)
    {
        constexpr int RPW = 32 / (4 * J);
        kind = u < p.kv_units ? kKeyRow : u < 2 * p.kv_units ? kValueRow : kQueryRow;
        head = (u - kind * p.kv_units) * RPW + in_warp;
        live = in_warp < RPW && head < (kind == kQueryRow ? p.q_heads : p.c.kv_heads);
        row = (kind == kKeyRow ? p.x[0] : kind == kValueRow ? p.x[1] : p.x[2]) +
              (size_t)t * (kind == kKeyRow ? p.ld[0] : kind == kValueRow ? p.ld[1] : p.ld[2]) + (size_t)head * (32 * J);
    }
};

// The partner of value d (a multiple of 4) of a half-split rotation.
__device__ __forceinline__ int partner_of(int d, int half)
{
    return d < half ? d + half : d - half;
}

template <int J>
__device__ __forceinline__ Words load_words_of(const RopeAppendParams &p, const Unit<J> &u, int w)
{
    Words x;
#pragma unroll
    for (int f = 0; f < 2; ++f) {
        const int d = 8 * w + 4 * f;
        x.v[f] = x.w[f] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (u.live) {
            x.v[f] = *reinterpret_cast<const float4 *>(u.row + d);
            if (u.kind != kValueRow && !p.interleaved && d < p.rot)
                x.w[f] = *reinterpret_cast<const float4 *>(u.row + partner_of(d, p.rot >> 1));
        }
    }
    return x;
}

// Sum over a row's lanes, in each of them (lanes of no row: anything).
template <int WPR, typename V>
__device__ __forceinline__ V row_sum(V s, int w, int lane)
{
    if constexpr ((WPR & (WPR - 1)) == 0) {
#pragma unroll
        for (int o = WPR >> 1; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    } else {
#pragma unroll
        for (int o = 1; o < WPR; o <<= 1) {
            const V t = __shfl_down_sync(0xffffffffu, s, o);
            if (w % (2 * o) == 0 && w + o < WPR) s += t;
        }
        s = __shfl_sync(0xffffffffu, s, lane - w);
    }
    return s;
}

__device__ __forceinline__ float4 times(float4 a, float4 b)
{
    return make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w);
}

// The row's values normalised and rotated.  sc: sines and cosines.
template <int J>
__device__ __forceinline__ void turn(const RopeAppendParams &p, int kind, const Words &x, int w, int lane, const float2 *sc,
                                     float (&v)[8])
{
    const float *gain = kind == kKeyRow ? p.gain[0] : p.gain[2];
    float r = 1.0f;
    if (gain) {   // uniform in the warp
        float s[2];
#pragma unroll
        for (int f = 0; f < 2; ++f)
            s[f] = (x.v[f].x * x.v[f].x + x.v[f].y * x.v[f].y) + (x.v[f].z * x.v[f].z + x.v[f].w * x.v[f].w);
        r = inv_sqrt(fmaf(row_sum<4 * J>(s[0] + s[1], w, lane), p.inv_d, p.eps));
    }
    const int half = p.rot >> 1;
#pragma unroll
    for (int f = 0; f < 2; ++f) {
        const int d = 8 * w + 4 * f;
        float4 a = x.v[f], b = x.w[f];
        if (gain && d < 32 * J) a = times(a, __ldg(reinterpret_cast<const float4 *>(gain + d)));
        if (d < p.rot) {
            if (p.interleaved) {
                const float4 s = *reinterpret_cast<const float4 *>(sc + (d >> 1));
                a = make_float4(a.x * s.y - a.y * s.x, a.y * s.y + a.x * s.x, a.z * s.w - a.w * s.z, a.w * s.w + a.z * s.z);
            } else {
                const int other = partner_of(d, half);
                if (gain) b = times(b, __ldg(reinterpret_cast<const float4 *>(gain + other)));
                const float m = d < half ? -1.0f : 1.0f;
                const float4 *s = reinterpret_cast<const float4 *>(sc + min(d, other));
                const float4 s0 = s[0], s1 = s[1];
                a = make_float4(a.x * s0.y + m * b.x * s0.x, a.y * s0.w + m * b.y * s0.z, a.z * s1.y + m * b.z * s1.x,
                                a.w * s1.w + m * b.w * s1.z);
            }
        }
        v[4 * f] = a.x * r;
        v[4 * f + 1] = a.y * r;
        v[4 * f + 2] = a.z * r;
        v[4 * f + 3] = a.w * r;
    }
}

// A group's ends, and how far a code's argument may be off: of the whole row,
// whose values bound every pair (|a| + |b| <= 2 max of the pair as rotated).
template <int J, int L>
struct Group {
    float lo, hi;
    GroupMap m;
    int bad;

    __device__ __forceinline__ Group(const float (&v)[8], int w, int lane)
    {
        lo = hi = v[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) {
            lo = min_nan(lo, v[i]);
            hi = max_nan(hi, v[i]);
        }
        const int pos = w % L;
        segment_min_max(lo, hi, pos, lane - pos, L);
        m = group_map(lo, hi, bad);
    }
    // the largest value of the row
    __device__ __forceinline__ float largest(int w, int lane) const
    {
        constexpr int WPR = 4 * J;
        float a = fmaxf(fabsf(lo), fabsf(hi));
        if constexpr ((WPR & (WPR - 1)) == 0) {
#pragma unroll
            for (int o = L; o < WPR; o <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        } else if constexpr (L < WPR) {
            const int row0 = lane - w;     // (lanes of no row look at lanes that are there)
            const float b = __shfl_sync(0xffffffffu, a, min(row0 + (w + L) % WPR, 31)),
                        c = __shfl_sync(0xffffffffu, a, min(row0 + (w + 2 * L) % WPR, 31));
            a = fmaxf(a, fmaxf(b, c));
        }
        return a;
    }
};

// An argument's distance to a border of two codes: 0.5 less what it is from the
// nearest code.
__device__ __forceinline__ float from_code(float v, const GroupMap &m)
{
    const float t = __fmul_rn(__fsub_rn(v, m.lo), m.r);
    return fabsf(t - rintf(t));
}

__device__ __forceinline__ float code_slack(float largest, const GroupMap &m)
{
    // 2 kKeyError of the largest by the value and by the lower end each, twice that by the scale
    return fmaf(8.0f * kKeyError * largest, m.r, kCodeError);
}

// A unit of key rows whose values next to a border, and to its group's ends, are
// computed in 64 bits.  By the whole warp.
template <int J, int L>
__device__ __noinline__ void exact_unit(const RopeAppendParams &p, int t, int u, int slot, const float2 *sc)
{
    constexpr int D = 32 * J, WPR = 4 * J;
    const int lane = threadIdx.x & 31, in_warp = lane / WPR, w = lane - in_warp * WPR;
    const Unit<J> unit(p, t, u, in_warp);
    const Words x = load_words_of(p, unit, w);
    float v[8];
    turn<J>(p, kKeyRow, x, w, lane, sc, v);
    uint32_t need = 0;
    {
        const Group<J, L> g(v, w, lane);
        const float largest = g.largest(w, lane), slack = code_slack(largest, g.m), near = 4.0f * kKeyError * largest;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (!(from_code(v[i], g.m) <= 0.5f - slack) || v[i] <= g.lo + near || v[i] >= g.hi - near) need |= 1u << i;
        if (!unit.live || g.bad) need = 0;
    }
    const float *gain = p.gain[0];
    double r = 1.0;
    if (gain) {
        double s = 0.0;
#pragma unroll
        for (int f = 0; f < 2; ++f)
            s += (double)x.v[f].x * x.v[f].x + (double)x.v[f].y * x.v[f].y + (double)x.v[f].z * x.v[f].z +
                 (double)x.v[f].w * x.v[f].w;
        r = 1.0 / sqrt(row_sum<WPR>(s, w, lane) / D + (double)p.eps);
    }
    const int half = p.rot >> 1, pos = p.rot > 0 ? __ldg(p.positions + t) : 0;
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
        if (!(need >> i & 1u)) continue;
        const int d = 8 * w + i;
        auto value = [&](int n) { return (double)unit.row[n] * (gain ? (double)__ldg(gain + n) * r : 1.0); };
        double y = value(d);
        if (d < p.rot) {
            const bool first = p.interleaved ? !(d & 1) : d < half;
            const int other = p.interleaved ? d ^ 1 : partner_of(d, half);
            const int at = p.interleaved ? d >> 1 : min(d, other);
            double s, c;
            sincos((double)pos * (double)__ldg(p.inv_freq + at), &s, &c);
            y = y * c + (first ? -s : s) * value(other);
        }
        v[i] = (float)y;
    }
    __syncwarp();
    const Group<J, L> g(v, w, lane);
    const uint32_t word = g.bad ? 0u : quantize_word(v, g.m);
    if (unit.live) write_word<J, L>(p, slot, unit.head, 0, w, word, 0u, g.bad, g.m, &g_kv_rope_error);
}

// J = head_dim / 32; L: lanes per group.
template <int J, int L>
__global__ void __launch_bounds__(kRopeAppendThreads) rope_append_kernel(const __grid_constant__ RopeAppendParams p)
{
    constexpr int WPR = 4 * J;
    __shared__ alignas(16) float2 sc[16 * J];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int in_warp = lane / WPR, w = lane - in_warp * WPR;
    const int t = blockIdx.x / p.splits, part = blockIdx.x - t * p.splits;
    const int slot = __ldg(p.slots + t);
    int u = part * kRopeAppendWarps + warp;
    const int step = p.splits * kRopeAppendWarps;
    Words x;
    if (u < p.units) x = load_words_of(p, Unit<J>(p, t, u, in_warp), w);
    if (p.rot > 0) {
        const int pos = __ldg(p.positions + t);
        for (int i = threadIdx.x; i < p.rot >> 1; i += kRopeAppendThreads) sc[i] = sin_cos_of(pos, __ldg(p.inv_freq + i));
    }
    __syncthreads();
    while (u < p.units) {   // uniform in the warp
        const Unit<J> unit(p, t, u, in_warp);
        float v[8] = {x.v[0].x, x.v[0].y, x.v[0].z, x.v[0].w, x.v[1].x, x.v[1].y, x.v[1].z, x.v[1].w};
        if (unit.kind != kValueRow) turn<J>(p, unit.kind, x, w, lane, sc, v);
        if (unit.kind == kQueryRow) {
            __syncwarp();   // in place: every lane of the row has read before any writes
            if (unit.live) {
                float4 *y = reinterpret_cast<float4 *>(p.q_out + (size_t)t * p.ldq_out + (size_t)unit.head * (32 * J) + 8 * w);
                y[0] = make_float4(v[0], v[1], v[2], v[3]);
                y[1] = make_float4(v[4], v[5], v[6], v[7]);
            }
        } else if (slot >= 0) {
            const Group<J, L> g(v, w, lane);
            bool border = false;
            if (unit.kind == kKeyRow && (p.rot > 0 || p.gain[0])) {
                float far = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) far = fmaxf(far, from_code(v[i], g.m));
                border = !(far <= 0.5f - code_slack(g.largest(w, lane), g.m)) && unit.live && !g.bad;
            }
            if (__any_sync(0xffffffffu, border)) {
                exact_unit<J, L>(p, t, u, slot, sc);
            } else {
                const uint32_t word = g.bad ? 0u : quantize_word(v, g.m);
                const uint32_t other = __shfl_xor_sync(0xffffffffu, word, 4);
                if (unit.live) write_word<J, L>(p, slot, unit.head, unit.kind == kValueRow, w, word, other, g.bad, g.m, &g_kv_rope_error);
            }
        }
        u += step;
        if (u < p.units) x = load_words_of(p, Unit<J>(p, t, u, in_warp), w);
    }
}

}  // namespace

cudaError_t launch_kv_rope_append(const RopeCall &call, const gq4_kv_cache &c, const float *v, int ldv, const int32_t *slots,
                                  cudaStream_t stream)
{
    RopeAppendParams p{};
    p.c = c;
    p.x[0] = call.x[1];
    p.x[1] = v;
    p.x[2] = call.x[0];
    p.ld[0] = call.ldx[1];
    p.ld[1] = ldv;
    p.ld[2] = call.ldx[0];
    p.gain[0] = call.gain[1];
    p.gain[2] = call.gain[0];
    p.q_out = call.y[0];
    p.ldq_out = call.ldy[0];
    p.positions = call.positions;
    p.slots = slots;
    p.inv_freq = call.inv_freq;
    p.eps = call.eps;
    p.inv_d = 1.0f / (float)call.D;
    p.T = call.T;
    p.q_heads = call.heads[0];
    p.rot = call.rot;
    p.interleaved = call.interleaved;
    p.shift = log2_of(c.page_size);
    p.total = c.n_pages * c.page_size;
    p.page_codes = (uint32_t)(c.page_size * c.head_dim / 2);
    p.page_sz = (uint32_t)(c.page_size * (c.head_dim / c.group_size) * 8);
    const int per = 32 / (c.head_dim / 8);
    p.kv_units = (c.kv_heads + per - 1) / per;
    p.units = 2 * p.kv_units + (p.q_heads + per - 1) / per;
    // few tokens: their rows over several CTAs, until the GPU has two each
    p.splits = 1;
    while (p.splits * kRopeAppendWarps < p.units && (long long)call.T * p.splits < 2 * 152) ++p.splits;
    const long long grid = (long long)call.T * p.splits;
    if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
    auto run = [&](auto kern) { kern<<<(unsigned)grid, kRopeAppendThreads, 0, stream>>>(p); };
    switch (c.head_dim * 16 + c.group_size / 32) {
    case 64 * 16 + 1: run(rope_append_kernel<2, 4>); break;
    case 64 * 16 + 2: run(rope_append_kernel<2, 8>); break;
    case 96 * 16 + 1: run(rope_append_kernel<3, 4>); break;
    case 96 * 16 + 3: run(rope_append_kernel<3, 12>); break;
    case 128 * 16 + 1: run(rope_append_kernel<4, 4>); break;
    case 128 * 16 + 2: run(rope_append_kernel<4, 8>); break;
    case 128 * 16 + 4: run(rope_append_kernel<4, 16>); break;
    case 256 * 16 + 1: run(rope_append_kernel<8, 4>); break;
    case 256 * 16 + 2: run(rope_append_kernel<8, 8>); break;
    case 256 * 16 + 4: run(rope_append_kernel<8, 16>); break;
    case 256 * 16 + 8: run(rope_append_kernel<8, 32>); break;
    default: return cudaErrorInvalidValue;
    }
    return cudaGetLastError();
}

cudaError_t read_kv_rope_device_error(unsigned int *bits, bool clear)
{
    cudaError_t err = cudaMemcpyFromSymbol(bits, g_kv_rope_error, sizeof(unsigned int));
    if (err != cudaSuccess || !clear) return err;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_kv_rope_error, &zero, sizeof(unsigned int));
}

}  // namespace gq4
