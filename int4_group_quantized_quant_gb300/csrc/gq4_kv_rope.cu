// gq4_kv_rope.cu -- a step's rows on their way into the attention, in one pass
// (gq4_kv_rope_append): queries normalised and rotated, keys normalised, rotated
// and quantised into the cache, values quantised.
//
//   y = x / sqrt(mean(x^2) + eps) * gain,  (y_a, y_b) -> rotation by
//   positions[t] * inv_freq[i],  then gq4_quantize's rule per group.
//
// What it saves over gq4_head_norm_rope and gq4_kv_append: a launch, and the
// rotated keys' way to HBM and back (8 bytes per value of k).  Floor: 8 bytes
// per value of q, 4 read and 0.5 + 8/gs written per value of k and v.  16381
// tokens, 32 + 8 heads of 128: 118 us, 692 MB at 5.9 TB/s (0.86 of a copy's;
// normalised 127; the two calls 138 and 146), of which the codes' check and
// exact_values are 10; 61 tokens 5.1 us (5.4), of which they are 1.5.  Where the
// queries are few the two calls are as fast: 8 + 8 heads 81 (80), 14 + 2 65 (60).
//
// Two kinds of CTAs take turns in the grid, so that the queries', which wait for
// HBM, and the keys', which are bound by instructions, share an SM.  A CTA of
// queries takes one token (few tokens: a share of its heads): a row is held in
// float4s by 16 lanes (64 values) or 32, pairs of a half-split rotation are
// exchanged by shuffles.  A CTA of keys and values takes a few tokens: a lane
// holds a word's 8 values, a row takes D/8 lanes, a warp as many rows as fit,
// all K or all V; half-split partners are read a second time (a first-level
// cache hit), 2 instructions where shuffles take 8.  (One layout for queries and
// keys, 8 values a lane: 145 us, its loads and stores half a sector each.)  32
// registers a thread and 8 CTAs per SM, at the price of a few spills: 5 CTAs take
// 134 us.
//
// Codes next to a border.  A key's code is that of its value (of the angle in 64
// bits) rounded once to f32: so it does not depend on the order of sums and products.  The
// rotation itself is f32; what it leaves of a key is off by at most key_error
// (|a| + |b|) for the pair (a, b) before the rotation.  Where that could turn a
// code's rounding -- a value so near to the border of two codes -- the warp
// computes its rows again, the values next to a border and next to the group's
// two ends in twice 24 bits (exact_values).  With groups of 128 normal values that
// is one warp's 256 values in 100.  (All of it in 64 bits: 61 tokens 5.7 us.  Set
// aside until the CTA's other rows are written: 120 and 6.9 us.)
#include <cstdint>

#include "gq4_kv_internal.h"
#include "gq4_kv_write.cuh"
#include "gq4_rope.cuh"
#include "gq4_two.cuh"

namespace gq4 {
namespace {

__device__ unsigned int g_kv_rope_error = 0;
constexpr int kRopeAppendThreads = 256, kRopeAppendWarps = kRopeAppendThreads / 32;
constexpr int kRopeTokens = 2;         // tokens of a CTA of keys and values, at most (kv_rows counts on it)

// A rotated value's error relative to |a| + |b|, in units of 2^-24 (a rounding):
// the angle's rounding 1, the sine and cosine 2, the products and their sum 2,
// and 1 that the exact value is rounded by; with a norm the gain 1 and the
// factor that the row shares 1 (its own error is the same for all of the row and
// moves no code).
__device__ __forceinline__ float key_error(bool norm)
{
    return norm ? 8 * 0x1p-24f : 6 * 0x1p-24f;
}
// Mean squares from here on, and with them the factor, are as exact as f32 sums
// are: the squares that it rounds to multiples of 2^-149 are 2^-42 of the sum.
constexpr float kLeastSquare = 0x1p-100f;
// Of a code's argument (v - lo) r, up to 15, on either side: two roundings and r's two.
constexpr float kCodeError = 8 * 15 * 0x1p-24f;

struct RopeAppendParams {
    gq4_kv_cache c;
    const float *q, *k, *v;
    int ldq, ldk, ldv;
    const float *q_gain, *k_gain;   // NULL: not normalised
    float *q_out;
    int ldq_out;
    const int32_t *positions, *slots;
    const float *inv_freq;
    float eps, inv_d;
    int T, q_heads, rot;
    bool interleaved;
    int shift, total;        // log2 of the page size; slots of the pool
    uint32_t page_codes, page_sz;   // bytes per page and head
    int units;               // warps' rows of K of a token, and as many of V
    int q_parts;             // CTAs of queries per token
    int kv_tokens, kv_parts; // tokens per CTA of keys, CTAs per such
    int q_ctas, kv_ctas, turn;      // all of them; CTAs of queries after each of keys
};

// pos * inv_freq less whole quarter turns (n, the nearest), in 64 bits: a 31-bit
// by a 24-bit product, off by less than 2^-22 of a radian at any position, and a
// quarter turn in two terms (Cody and Waite's reduction).
struct Quarter {
    double r;      // [-pi/4, pi/4]
    int n;         // modulo 4

    __device__ __forceinline__ Quarter(int pos, float inv_freq)
    {
        const double a = (double)pos * (double)inv_freq;
        const double whole = 6755399441055744.0;                  // 1.5 2^52: a sum's last bit counts ones
        const double m = fma(a, 0.6366197723675814, whole), k = m - whole;   // 2 / pi
        r = fma(k, -6.123233995736766e-17, fma(k, -1.5707963267948966, a));
        if (fabsf((float)r) >= 1.0f) r = 0.0;          // (angles from 2^50 on, which mean nothing, stay bounded)
        n = __double2loint(m) & 3;
    }
};

// Sine and cosine of x in [-pi/4, pi/4] by their Taylor series, TERMS terms each
// (f32, 5: off by 2^-28 and a rounding or two; f64, 9: by 2^-58), and n quarter
// turns on.
template <int TERMS, typename F>
__device__ __forceinline__ void sin_cos_series(F x, int n, F &s, F &c)
{
    F inverse[2 * TERMS + 1];      // of factorials (constants)
    inverse[0] = F(1);
    double f = 1.0;
#pragma unroll
    for (int i = 1; i <= 2 * TERMS; ++i) {
        f *= i;
        inverse[i] = F(1.0 / f);
    }
    const F y = -x * x;
    F a = inverse[2 * TERMS - 1], b = inverse[2 * TERMS];
#pragma unroll
    for (int i = TERMS - 2; i >= 0; --i) a = fma(a, y, inverse[2 * i + 1]);
#pragma unroll
    for (int i = TERMS - 1; i >= 1; --i) b = fma(b, y, inverse[2 * i]);
    b = fma(b, y, F(1));
    a *= x;
    s = n & 1 ? b : a;
    c = n & 1 ? a : b;
    if (n & 2) s = -s;
    if ((n + 1) & 2) c = -c;
}

// The same in twice 24 bits, off by 2^-46: the terms from 2^-25 of the first on
// in f32.
__device__ __forceinline__ void sin_cos_two(Two x, int n, Two &s, Two &c)
{
    Two y = mul(x, x);
    y = {-y.hi, -y.lo};
    constexpr float tail_a[] = {(float)(1.0 / 39916800), (float)(1.0 / 6227020800.0), (float)(1.0 / 1307674368000.0)};
    constexpr float tail_b[] = {(float)(1.0 / 3628800), (float)(1.0 / 479001600), (float)(1.0 / 87178291200.0)};
    constexpr Two terms_a[] = {two_of(1), two_of(1.0 / 6), two_of(1.0 / 120), two_of(1.0 / 5040), two_of(1.0 / 362880)};
    constexpr Two terms_b[] = {two_of(1), two_of(0.5), two_of(1.0 / 24), two_of(1.0 / 720), two_of(1.0 / 40320)};
    Two a = {__fmaf_rn(__fmaf_rn(tail_a[2], y.hi, tail_a[1]), y.hi, tail_a[0]), 0.0f};
    Two b = {__fmaf_rn(__fmaf_rn(tail_b[2], y.hi, tail_b[1]), y.hi, tail_b[0]), 0.0f};
#pragma unroll
    for (int i = 4; i >= 0; --i) {
        a = add_smaller(terms_a[i], mul(a, y));
        b = add_smaller(terms_b[i], mul(b, y));
    }
    a = mul(a, x);
    s = n & 1 ? b : a;
    c = n & 1 ? a : b;
    if (n & 2) s = {-s.hi, -s.lo};
    if ((n + 1) & 2) c = {-c.hi, -c.lo};
}

// 1 / sqrt(x): f32's, and its series in the rest.
__device__ __forceinline__ Two inv_sqrt_two(Two x)
{
    const float r = inv_sqrt(x.hi);
    const Two q = mul(mul(x, Two{r, 0.0f}), Two{r, 0.0f});
    const float e = __fsub_rn(__fsub_rn(1.0f, q.hi), q.lo);
    return {r, r * __fmaf_rn(0.375f * e, e, 0.5f * e)};
}

// The partner of value d (a multiple of 4) of a half-split rotation.
__device__ __forceinline__ int partner_of(int d, int half)
{
    return d < half ? d + half : d - half;
}

__device__ __forceinline__ float4 times(float4 a, float4 b)
{
    return make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w);
}

__device__ __forceinline__ float square_sum(float4 a)
{
    return (a.x * a.x + a.y * a.y) + (a.z * a.z + a.w * a.w);
}

// A token's rotation with the gain taken in: value d of a row becomes x_d A_d +
// x_d' B_d, d' its partner, A_d = g_d cos and B_d = -+ g_d' sin.
template <int J>
struct alignas(16) Turn {
    float A[32 * J], B[32 * J];
};

// Its angles, for exact_values.
template <int J>
struct Angles {
    double r[16 * J];
    uint8_t n[16 * J];
};

// Pair i of a token's table.  gain: NULL for ones; angles: NULL for none.
template <int J>
__device__ __forceinline__ void make_turn(const RopeAppendParams &p, int pos, int i, const float *gain, Turn<J> &t, Angles<J> *angles)
{
    const Quarter turn(pos, __ldg(p.inv_freq + i));
    if (angles) {
        angles->r[i] = turn.r;
        angles->n[i] = (uint8_t)turn.n;
    }
    float2 sc;
    sin_cos_series<5, float>((float)turn.r, turn.n, sc.x, sc.y);
    const int a = p.interleaved ? 2 * i : i, b = p.interleaved ? 2 * i + 1 : i + (p.rot >> 1);
    const float ga = gain ? __ldg(gain + a) : 1.0f, gb = gain ? __ldg(gain + b) : 1.0f;
    t.A[a] = ga * sc.y;
    t.B[a] = -gb * sc.x;
    t.A[b] = gb * sc.y;
    t.B[b] = ga * sc.x;
}

// Values d .. d + 3 rotated (d < rot); b: their partners.
template <int J>
__device__ __forceinline__ float4 rotated(float4 a, float4 b, int d, const Turn<J> &t)
{
    const float4 A = *reinterpret_cast<const float4 *>(t.A + d), B = *reinterpret_cast<const float4 *>(t.B + d);
    return make_float4(a.x * A.x + b.x * B.x, a.y * A.y + b.y * B.y, a.z * A.z + b.z * B.z, a.w * A.w + b.w * B.w);
}

__device__ __forceinline__ float4 swapped(float4 a)
{
    return make_float4(a.y, a.x, a.w, a.z);
}

// ---------------------------------------------------------------------------
// Queries
// ---------------------------------------------------------------------------

// LPR lanes hold a row, CH float4s each; two rows of a warp under way.
template <int J>
__device__ __forceinline__ void query_rows(const RopeAppendParams &p, int t, int part, const Turn<J> &turn)
{
    constexpr int D4 = 8 * J, LPR = J == 2 ? 16 : 32, CH = J == 8 ? 2 : 1, RPW = 32 / LPR, AHEAD = CH == 1 ? 2 : 1;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & (LPR - 1);
    const int half4 = p.rot >> 3, rot4 = p.rot >> 2;
    const float4 *from = reinterpret_cast<const float4 *>(p.q + (size_t)t * p.ldq);
    float4 *to = reinterpret_cast<float4 *>(p.q_out + (size_t)t * p.ldq_out);
    const float4 *gain = reinterpret_cast<const float4 *>(p.q_gain);
    const int step = kRopeAppendWarps * RPW * p.q_parts;
    bool waited = false;
    // every warp takes the same number of turns (the barrier below)
    for (int row0 = part * kRopeAppendWarps * RPW; row0 < p.q_heads; row0 += AHEAD * step) {
        const int first = row0 + warp * RPW + lane / LPR;
        float4 x[AHEAD][CH];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                x[u][j] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (first + u * step < p.q_heads && l + 32 * j < D4) x[u][j] = from[(first + u * step) * D4 + l + 32 * j];
            }
        if (!waited) __syncthreads();      // the rotation
        waited = true;
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            if (row0 + warp * RPW + u * step >= p.q_heads) break;   // uniform in the warp
            float r = 1.0f;
            if (gain) {
                float s = square_sum(x[u][0]);
#pragma unroll
                for (int j = 1; j < CH; ++j) s += square_sum(x[u][j]);
#pragma unroll
                for (int o = LPR >> 1; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                r = inv_sqrt(fmaf(s, p.inv_d, p.eps));
            }
            float4 y[CH];
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                const int i = l + 32 * j, other = i < half4 ? i + half4 : i - half4;
                float4 b = swapped(x[u][j]);
                if (!p.interleaved) {      // (the whole warp shuffles)
                    b.x = __shfl_sync(0xffffffffu, x[u][0].x, other, LPR);
                    b.y = __shfl_sync(0xffffffffu, x[u][0].y, other, LPR);
                    b.z = __shfl_sync(0xffffffffu, x[u][0].z, other, LPR);
                    b.w = __shfl_sync(0xffffffffu, x[u][0].w, other, LPR);
#pragma unroll
                    for (int n = 1; n < CH; ++n) {
                        const float4 c = make_float4(__shfl_sync(0xffffffffu, x[u][n].x, other), __shfl_sync(0xffffffffu, x[u][n].y, other),
                                                     __shfl_sync(0xffffffffu, x[u][n].z, other), __shfl_sync(0xffffffffu, x[u][n].w, other));
                        if (other >> 5 == n) b = c;
                    }
                }
                y[j] = x[u][j];
                if (i < rot4) y[j] = rotated(y[j], b, 4 * i, turn);
                else if (gain && i < D4) y[j] = times(y[j], __ldg(gain + i));
            }
            __syncwarp();   // in place: every lane of the row has read before any writes
#pragma unroll
            for (int j = 0; j < CH; ++j)
                if (first + u * step < p.q_heads && l + 32 * j < D4)
                    to[(first + u * step) * D4 + l + 32 * j] = gain ? times(y[j], make_float4(r, r, r, r)) : y[j];
        }
    }
}

// ---------------------------------------------------------------------------
// Keys and values
// ---------------------------------------------------------------------------

__device__ __forceinline__ Two shuffled(Two a, int from)
{
    return {__shfl_sync(0xffffffffu, a.hi, from), __shfl_sync(0xffffffffu, a.lo, from)};
}

template <typename V>
__device__ __forceinline__ V shuffled(V a, int from)
{
    return __shfl_sync(0xffffffffu, a, from);
}

// Sum over a row's lanes, in each of them (lanes of no row: anything).
template <int WPR, typename V>
__device__ __forceinline__ V row_sum(V s, int w, int lane)
{
    if constexpr ((WPR & (WPR - 1)) == 0) {
#pragma unroll
        for (int o = WPR >> 1; o > 0; o >>= 1) s += shuffled(s, lane ^ o);
    } else {
#pragma unroll
        for (int o = 1; o < WPR; o <<= 1) {
            const V t = shuffled(s, min(lane + o, 31));
            if (w % (2 * o) == 0 && w + o < WPR) s += t;
        }
        s = shuffled(s, lane - w);
    }
    return s;
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

// How far a code's argument t = 15 (v - lo) / (hi - lo) may be off: v, and lo
// and hi in the parts 1 - t / 15 and t / 15, each by 2 key_error of the row's
// largest.
__device__ __forceinline__ float code_slack(float largest, const GroupMap &m, bool norm)
{
    return fmaf(4.0f * key_error(norm) * largest, m.r, kCodeError);
}

// The 8 codes of a word, as quantize_word's, and how far an argument is from its
// code at most (FAR).  An argument t is rounded by a sum with 1.5 2^23, whose
// last bits are then the code: conversions run at an eighth of the rate.  The
// sum is an FMA with a factor of 1 that the compiler does not see, so that it
// cannot take the product before it in, which would round that instead of t.
template <bool FAR>
__device__ __forceinline__ uint32_t code_word(const float (&v)[8], const GroupMap &m, float &far)
{
    constexpr float kOnes = 12582912.0f;
    float unit = 1.0f;
    asm volatile("" : "+f"(unit));
    const f32x2 nlo = pack2(-m.lo, -m.lo), r = pack2(m.r, m.r), one = pack2(unit, unit), ones = pack2(kOnes, kOnes);
    uint32_t b[8];
    far = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const f32x2 t = mul2(add2(pack2(v[i], v[i + 1]), nlo), r), q = fma2(t, one, ones);
        const float2 c = unpack2(q);
        b[i] = __float_as_uint(c.x);
        b[i + 1] = __float_as_uint(c.y);
        if (FAR) {
            const float2 d = unpack2(add2(add2(q, pack2(-kOnes, -kOnes)), mul2(t, pack2(-unit, -unit))));
            far = fmaxf(far, fmaxf(fabsf(d.x), fabsf(d.y)));
        }
    }
    const uint32_t even = __byte_perm(__byte_perm(b[0], b[2], 0x0040), __byte_perm(b[4], b[6], 0x0040), 0x5410);
    const uint32_t odd = __byte_perm(__byte_perm(b[1], b[3], 0x0040), __byte_perm(b[5], b[7], 0x0040), 0x5410);
    return even | (odd << 4);
}

// A warp's row: its kv head and where it starts.
template <int J>
struct KvRow {
    int head;
    bool live;
    const float *at;

    __device__ __forceinline__ KvRow(const RopeAppendParams &p, int t, int unit, bool value, int in_warp)
    {
        constexpr int RPW = 32 / (4 * J);
        head = unit * RPW + in_warp;
        live = in_warp < RPW && head < p.c.kv_heads;
        at = (value ? p.v : p.k) + (size_t)t * (value ? p.ldv : p.ldk) + head * (32 * J);
    }
};

// Of a unit of key rows, whose values are in v, a lane's 8 in place, those next
// to a border of two codes and to their group's ends, in twice 24 bits; in 64
// where the row's or the group's size would cost the former bits.  lo, hi, r32, slack, near: of
// the lane's group, its ends, its factor and how far its arguments and values may
// be off; largest: of its row; wanted: it has codes.  All values of a normalised
// row whose squares f32 does not hold: it comes as NaN.  By the whole warp.
template <int J>
__device__ __noinline__ void exact_values(const RopeAppendParams &p, int t, int unit, bool wanted, float lo, float hi, float r32,
                                          float slack, float near, float largest, const Angles<J> &angles, float *v)
{
    constexpr int D = 32 * J, WPR = 4 * J;
    const int lane = threadIdx.x & 31, in_warp = lane / WPR, w = lane - in_warp * WPR;
    const KvRow<J> row(p, t, unit, false, in_warp);
    const bool norm = p.k_gain != nullptr;
    v += 8 * lane;
    uint32_t need = 0;
    if (wanted) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = __fmul_rn(__fsub_rn(v[i], lo), r32);
            if (!(fabsf(x - rintf(x)) <= 0.5f - slack) || v[i] <= lo + near || v[i] >= hi - near) need |= 1u << i;
        }
    }
    // (a small group beside larger ones loses its own second parts; one of zeros has none)
    const float size = fmaxf(fabsf(lo), fabsf(hi));
    bool sized = (size >= 0x1p-50f || size == 0.0f) && largest <= 0x1p50f;
    Two r = {1.0f, 0.0f};
    if (norm) {
        Two sum = {0.0f, 0.0f};
        if (row.live) {
#pragma unroll 2
            for (int i = 0; i < 8; ++i) {
                const float x = row.at[8 * w + i];
                sum += two_product(x, x);
            }
        }
        sum = row_sum<WPR>(sum, w, lane);
        sum = add(mul(sum, two_of(1.0 / D)), Two{p.eps, 0.0f});
        sized &= sum.hi >= 0x1p-50f && sum.hi <= 0x1p50f;
        r = inv_sqrt_two(sum);
    }
    const int half = p.rot >> 1;
    auto other_of = [&](int d) { return p.interleaved ? d ^ 1 : partner_of(d, half); };
    auto pair_of = [&](int d) { return p.interleaved ? d >> 1 : min(d, partner_of(d, half)); };
    auto is_first = [&](int d) { return p.interleaved ? !(d & 1) : d < half; };
    if (__all_sync(0xffffffffu, sized || !wanted)) {
#pragma unroll 1
        for (; need; need &= need - 1) {
            const int i = __ffs(need) - 1, d = 8 * w + i;
            auto value = [&](int m) { return norm ? two_product(row.at[m], __ldg(p.k_gain + m)) : Two{row.at[m], 0.0f}; };
            Two y = value(d);
            if (d < p.rot) {
                const double x = angles.r[pair_of(d)];
                const float x_hi = (float)x;
                Two sine, cosine;
                sin_cos_two(Two{x_hi, (float)(x - (double)x_hi)}, angles.n[pair_of(d)], sine, cosine);
                if (is_first(d)) sine = {-sine.hi, -sine.lo};
                y = add(mul(y, cosine), mul(sine, value(other_of(d))));
            }
            y = mul(y, r);
            v[i] = __fadd_rn(y.hi, y.lo);
        }
    } else {
        double factor = 1.0;
        if (norm) {
            double sum = 0.0;
            if (row.live) {
#pragma unroll 1
                for (int i = 0; i < 8; ++i) {
                    const double x = row.at[8 * w + i];
                    sum = fma(x, x, sum);
                }
            }
            sum = fma(row_sum<WPR>(sum, w, lane), 1.0 / D, (double)p.eps);
            factor = inv_sqrt((float)sum);               // (of 0, infinite, NaN)
            if (sum > 0.0 && sum < INFINITY) {
                // of 1 .. 4, which f32 holds, with two Newton steps; the even power of two apart
                const int e = (((__double2hiint(sum) >> 20) & 2047) - 1023) & ~1;
                sum *= __hiloint2double((1023 - e) << 20, 0);
                factor = inv_sqrt((float)sum);
                factor = fma(fma(-0.5 * sum * factor, factor, 0.5), factor, factor);
                factor = fma(fma(-0.5 * sum * factor, factor, 0.5), factor, factor);
                factor *= __hiloint2double((1023 - e / 2) << 20, 0);
            }
        }
#pragma unroll 1
        for (; need; need &= need - 1) {
            const int i = __ffs(need) - 1, d = 8 * w + i;
            auto value = [&](int m) { return (double)row.at[m] * (norm ? (double)__ldg(p.k_gain + m) : 1.0); };
            double y = value(d);
            if (d < p.rot) {
                double sine, cosine;
                sin_cos_series<9, double>(angles.r[pair_of(d)], angles.n[pair_of(d)], sine, cosine);
                y = y * cosine + (is_first(d) ? -sine : sine) * value(other_of(d));
            }
            v[i] = (float)(y * factor);
        }
    }
    __syncwarp();
}

template <int J, int L>
__device__ __forceinline__ void kv_rows(const RopeAppendParams &p, int t0, int part, const Turn<J> *turns, const Angles<J> *angles, float (*scratch)[256])
{
    constexpr int WPR = 4 * J;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int in_warp = lane / WPR, w = lane - in_warp * WPR;
    const int units = min(p.kv_tokens, p.T - t0) * 2 * p.units, step = kRopeAppendWarps * p.kv_parts;
    const int half = p.rot >> 1;
    bool waited = false;
    // every warp takes the same number of turns (the barrier below)
    for (int u0 = part * kRopeAppendWarps; u0 < units; u0 += step) {
        const int u = u0 + warp, n = u >= 2 * p.units, rest = u - n * 2 * p.units, t = t0 + n;
        // a token's units of K and of V, of every second token the other way round: a warp gets both
        const bool value = (rest >= p.units) != (n & 1);
        const int unit = rest >= p.units ? rest - p.units : rest;
        const KvRow<J> row(p, t, unit, value, in_warp);
        const bool in = u < units && row.live;
        const int slot = u < units ? __ldg(p.slots + t) : -1;
        float4 a[2], b[2];
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            const int d = 8 * w + 4 * f;
            a[f] = b[f] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (in) {
                a[f] = *reinterpret_cast<const float4 *>(row.at + d);
                if (!value && !p.interleaved && d < p.rot) b[f] = *reinterpret_cast<const float4 *>(row.at + partner_of(d, half));
            }
        }
        if (!waited) __syncthreads();      // the rotation
        waited = true;
        if (slot < 0) continue;            // uniform in the warp
        if (!value) {
            float r = 1.0f;
            if (p.k_gain) {
                // (squares that f32 does not hold: no number, which exact_values takes)
                const float m = fmaf(row_sum<WPR>(square_sum(a[0]) + square_sum(a[1]), w, lane), p.inv_d, p.eps);
                r = m >= kLeastSquare && m < INFINITY ? inv_sqrt(m) : __int_as_float(0x7fc00000);
            }
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                const int d = 8 * w + 4 * f;
                if (d < p.rot) a[f] = rotated(a[f], p.interleaved ? swapped(a[f]) : b[f], d, turns[n]);
                else if (p.k_gain) a[f] = times(a[f], __ldg(reinterpret_cast<const float4 *>(p.k_gain + d)));
                if (p.k_gain) a[f] = times(a[f], make_float4(r, r, r, r));
            }
        }
        bool exact = value || (p.rot == 0 && !p.k_gain);
#pragma unroll 1
        for (;;) {
            const float v[8] = {a[0].x, a[0].y, a[0].z, a[0].w, a[1].x, a[1].y, a[1].z, a[1].w};
            const Group<J, L> g(v, w, lane);
            float far;
            const uint32_t code = code_word<true>(v, g.m, far);
            if (!exact) {
                const float largest = g.largest(w, lane), slack = code_slack(largest, g.m, p.k_gain != nullptr);
                if (__any_sync(0xffffffffu, !(far <= 0.5f - slack) && row.live)) {
                    // once more with the values that count as they are (without a norm a group that is not finite stays so)
                    float4 *at = reinterpret_cast<float4 *>(scratch[warp] + 8 * lane);
                    at[0] = a[0];
                    at[1] = a[1];
                    exact_values<J>(p, t, unit, row.live && (p.k_gain || !g.bad), g.lo, g.hi, g.m.r, slack,
                                    4.0f * key_error(p.k_gain != nullptr) * largest, largest, angles[n], scratch[warp]);
                    a[0] = at[0];
                    a[1] = at[1];
                    exact = true;
                    continue;
                }
            }
            const uint32_t word = g.bad ? 0u : code, other = __shfl_xor_sync(0xffffffffu, word, 4);
            if (row.live) write_word<J, L>(p, slot, row.head, value, w, word, other, g.bad, g.m, &g_kv_rope_error);
            break;
        }
    }
}

// J = head_dim / 32; L: lanes per group.
template <int J, int L>
__global__ void __launch_bounds__(kRopeAppendThreads, 8) rope_append_kernel(const __grid_constant__ RopeAppendParams p)
{
    __shared__ Turn<J> turns[kRopeTokens];
    __shared__ Angles<J> angles[kRopeTokens];
    __shared__ alignas(16) float scratch[kRopeAppendWarps][256];
    const int turn = blockIdx.x / (p.turn + 1), place = blockIdx.x - turn * (p.turn + 1);
    const bool kv = place == 0;
    const int cta = kv ? turn : turn * p.turn + place - 1;
    if (cta >= (kv ? p.kv_ctas : p.q_ctas)) return;
    const int parts = kv ? p.kv_parts : p.q_parts, per = kv ? p.kv_tokens : 1;
    const int item = parts == 1 ? cta : cta / parts, t0 = item * per, part = cta - item * parts;
    // the tokens' rotations
    const int half = p.rot >> 1, tokens = min(per, p.T - t0);
    for (int i = threadIdx.x; i < tokens * half; i += kRopeAppendThreads) {
        const int n = i >= half;
        make_turn<J>(p, __ldg(p.positions + t0 + n), i - n * half, kv ? p.k_gain : p.q_gain, turns[n],
                     kv ? &angles[n] : nullptr);
    }
    if (kv) kv_rows<J, L>(p, t0, part, turns, angles, scratch);
    else query_rows<J>(p, t0, part, turns[0]);
}

}  // namespace

cudaError_t launch_kv_rope_append(const RopeCall &call, const gq4_kv_cache &c, const float *v, int ldv, const int32_t *slots,
                                  cudaStream_t stream)
{
    RopeAppendParams p{};
    p.c = c;
    p.q = call.x[0];
    p.k = call.x[1];
    p.v = v;
    p.ldq = call.ldx[0];
    p.ldk = call.ldx[1];
    p.ldv = ldv;
    p.q_gain = call.gain[0];
    p.k_gain = call.gain[1];
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
    p.units = (c.kv_heads + per - 1) / per;
    // Few tokens: a token's rows of keys and values, and of queries, over several
    // CTAs, until there are 8 of them, and one, per SM.  One token per CTA where
    // that is a unit for each warp, up to 32 per SM; beyond, the table's making is
    // shared.  us, group 64 (tokens per CTA / CTAs per such): 32 over 8 heads, 1000
    // tokens 11.3 (1/1) and 12.0 (2/1), 16381 122.1 and 118.7; 32 over 32, 500
    // tokens 14.3 (1/3), 16.0 (1/1) and 16.7 (2/1), 4000 65.1 (1/1) and 67.9 (2/1);
    // 14 over 2, 1000 tokens 7.9 (1/1) and 7.5 (2/1).
    auto parts = [](int rows, int ctas, int enough) {
        int n = 1;
        while (n * kRopeAppendWarps < rows && (long long)n * ctas < enough) ++n;
        return n;
    };
    p.kv_tokens = 2 * p.units >= kRopeAppendWarps && call.T <= 32 * 152 ? 1 : kRopeTokens;
    p.kv_parts = parts(2 * p.units * p.kv_tokens, (call.T + p.kv_tokens - 1) / p.kv_tokens, 8 * 152);
    p.q_parts = parts(c.head_dim == 64 ? (p.q_heads + 1) / 2 : p.q_heads, call.T, 152);
    if ((long long)call.T * (p.q_parts + p.kv_parts) > 0x3fffffffll) return cudaErrorInvalidValue;
    p.q_ctas = call.heads[0] > 0 ? call.T * p.q_parts : 0;
    p.kv_ctas = (call.T + p.kv_tokens - 1) / p.kv_tokens * p.kv_parts;
    p.turn = (p.q_ctas + p.kv_ctas - 1) / p.kv_ctas;
    const long long grid = (long long)p.kv_ctas * (p.turn + 1);
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
