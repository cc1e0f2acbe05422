// gq4_rope.cu -- RMSNorm of every query and key head and the rotation by
// position, in one pass (gq4_head_norm_rope).
//
//   y = x / sqrt(mean(x^2) + eps) * gain,  (y_a, y_b) -> rotation by
//   positions[t] * inv_freq[i].
//
// Bound by HBM: 8 bytes per element.  A CTA takes one token and a share of
// its heads: its threads first form the token's rot/2 sines and cosines in
// shared memory (each once for all heads of the CTA; the loads of the rows
// are already in flight), then a row is handled by the smallest power of two
// of lanes that holds it in float4s (16 lanes at 64 dims, 32 at 128, 32
// lanes with 2 or 4 float4 each above).  A half-split pair's partner is
// loaded a second time (a first-level cache hit) rather than shuffled, as
// rot/2 may fall anywhere.
//
// Angles: pos * inv_freq is a 31-bit by 24-bit product; in binary64 its error
// is below 2^-22 of a radian at any position.  It is reduced modulo 2 pi in
// binary64 with a two-term constant (Cody and Waite's reduction) and handed
// to sincosf as a value in [-pi, pi].
#include <cstdint>

#include "gq4_internal.h"

namespace gq4 {
namespace {

constexpr int kRopeThreads = 256;

struct RopeParams {
    RopeCall c;
    int rows;       // q and k heads of a token
    int splits;     // CTAs per token
    int lpr;        // lanes per row
};

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

// A lane's share of one row: its float4s and, half-split, their partners'.
template <int CH>
struct Row {
    float4 v[CH], w[CH];
    float4 *y;
    int side;    // -1: no row
};

template <int CH>
__device__ __forceinline__ Row<CH> load_row(const RopeCall &c, int t, int row, int rows, int l)
{
    Row<CH> x;
    const bool live = row < rows;
    const int s = live && row >= c.heads[0] ? 1 : 0;
    const int h = s ? row - c.heads[0] : row;
    x.side = live ? s : -1;
    x.y = reinterpret_cast<float4 *>(c.y[s] + (size_t)t * c.ldy[s] + (size_t)h * c.D);
    const float4 *in = reinterpret_cast<const float4 *>(c.x[s] + (size_t)t * c.ldx[s] + (size_t)h * c.D);
    const int d4 = c.D >> 2, rot4 = c.rot >> 2, half4 = c.rot >> 3;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int i = l + j * 32;
        x.v[j] = x.w[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (live && i < d4) {
            x.v[j] = in[i];
            if (!c.interleaved && i < rot4) x.w[j] = in[i < half4 ? i + half4 : i - half4];
        }
    }
    return x;
}

__device__ __forceinline__ float4 scaled(float4 a, float r, float4 g)
{
    return make_float4(a.x * r * g.x, a.y * r * g.y, a.z * r * g.z, a.w * r * g.w);
}

// CH: float4 per lane of a row.
template <int CH>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p)
{
    __shared__ float2 sc[GQ4_MAX_HEAD_DIM / 2];
    const RopeCall &c = p.c;
    const int t = blockIdx.x / p.splits, part = blockIdx.x - t * p.splits;
    const int half = c.rot >> 1;
    const int lpr = p.lpr, per = kRopeThreads / lpr;   // rows at once
    const int l = threadIdx.x & (lpr - 1);
    const int stride = per * p.splits;
    const int d4 = c.D >> 2, rot4 = c.rot >> 2, half4 = c.rot >> 3;
    int row = part * per + threadIdx.x / lpr;
    Row<CH> next = load_row<CH>(c, t, row, p.rows, l);
    if (half > 0) {
        const int pos = __ldg(c.positions + t);
        for (int i = threadIdx.x; i < half; i += kRopeThreads) sc[i] = sin_cos_of(pos, __ldg(c.inv_freq + i));
    }
    __syncthreads();
    // every thread takes the same number of turns (the shuffles below); the
    // next row is on its way while this one is worked on
    for (int row0 = part * per; row0 < p.rows; row0 += stride) {
        const Row<CH> x = next;
        row += stride;
        if (row0 + stride < p.rows) next = load_row<CH>(c, t, row, p.rows, l);
        const float4 *gain = reinterpret_cast<const float4 *>(x.side < 0 ? nullptr : c.gain[x.side]);
        float r = 1.0f;
        if (c.gain[0] || c.gain[1]) {  // uniform: the whole warp shuffles
            float s = 0.0f;
#pragma unroll
            for (int j = 0; j < CH; ++j)
                s += x.v[j].x * x.v[j].x + x.v[j].y * x.v[j].y + x.v[j].z * x.v[j].z + x.v[j].w * x.v[j].w;
            for (int o = lpr >> 1; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            r = 1.0f / sqrtf(s / (float)c.D + c.eps);
        }
        __syncwarp();  // in place: every lane of the row has read before any writes
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int i = l + j * 32;
            if (x.side < 0 || i >= d4) continue;
            float4 a = gain ? scaled(x.v[j], r, __ldg(gain + i)) : x.v[j];
            if (i < rot4) {
                if (c.interleaved) {
                    const float2 s0 = sc[2 * i], s1 = sc[2 * i + 1];
                    a = make_float4(a.x * s0.y - a.y * s0.x, a.y * s0.y + a.x * s0.x,
                                    a.z * s1.y - a.w * s1.x, a.w * s1.y + a.z * s1.x);
                } else {
                    const bool first = i < half4;
                    const int other = first ? i + half4 : i - half4, f = 4 * (first ? i : other);
                    const float4 b = gain ? scaled(x.w[j], r, __ldg(gain + other)) : x.w[j];
                    const float m = first ? -1.0f : 1.0f;
                    const float2 s0 = sc[f], s1 = sc[f + 1], s2 = sc[f + 2], s3 = sc[f + 3];
                    a = make_float4(a.x * s0.y + m * b.x * s0.x, a.y * s1.y + m * b.y * s1.x,
                                    a.z * s2.y + m * b.z * s2.x, a.w * s3.y + m * b.w * s3.x);
                }
            }
            x.y[i] = a;
        }
    }
}

}  // namespace

cudaError_t launch_rope(const RopeCall &call, cudaStream_t stream)
{
    RopeParams p{};
    p.c = call;
    p.rows = call.heads[0] + call.heads[1];
    const int d4 = call.D / 4;
    int lpr = 2;
    while (lpr < d4 && lpr < 32) lpr *= 2;
    p.lpr = lpr;
    const int per = kRopeThreads / lpr;
    // few tokens: their heads over several CTAs, until the GPU has two each
    p.splits = 1;
    while (p.splits * per < p.rows && (long long)call.T * p.splits < 2 * 152) ++p.splits;
    const long long grid = (long long)call.T * p.splits;
    if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
    if (d4 <= 32)
        rope_kernel<1><<<(unsigned)grid, kRopeThreads, 0, stream>>>(p);
    else if (d4 <= 64)
        rope_kernel<2><<<(unsigned)grid, kRopeThreads, 0, stream>>>(p);
    else
        rope_kernel<4><<<(unsigned)grid, kRopeThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace gq4
