// gq4_rope.cu -- RMSNorm of every query and key head and the rotation by
// position, in one pass (gq4_head_norm_rope).
//
//   y = x / sqrt(mean(x^2) + eps) * gain,  (y_a, y_b) -> rotation by
//   positions[t] * inv_freq[i].
//
// Bound by HBM: 8 bytes per element, and a float4 in and out per lane.  A
// CTA takes one token and a share of its heads: its threads load their first
// row, form the token's rot/2 sines and cosines in shared memory meanwhile
// (each once for all heads of the CTA), then handle a row with the smallest
// power of two of lanes that holds it in float4s (16 lanes at 64 dims, 32 at
// 128, 32 lanes with 2 or 4 float4 each above).  Half-split pairs are
// exchanged by shuffles within 32 lanes; above 128 dims the partner lies in
// another register of another lane and is loaded a second time (a
// first-level cache hit).
//   8191 tokens of 40 heads of 128: 57 us, 335 MB at 5.9 TB/s (0.87 of a
// copy's).  What counts is few instructions (135 per float4 and warp) and full
// occupancy: 195 instructions took 63 us, and two rows of loads under way per
// thread, at fewer CTAs per SM, 72.
#include <cstdint>

#include "gq4_kv_internal.h"
#include "gq4_rope.cuh"

namespace gq4 {
namespace {

constexpr int kRopeThreads = 256;

struct RopeParams {
    RopeCall c;
    int rows;       // q and k heads of a token
    int splits;     // CTAs per token
    float inv_d;    // 1 / D
};

// A lane's share of one row: its float4s and, half-split above 128 dims,
// their partners'.
template <int CH>
struct Row {
    float4 v[CH], w[CH];
};

template <int CH>
__device__ __forceinline__ Row<CH> load_row(const RopeCall &c, const float *row, bool live, int l)
{
    const float4 *in = reinterpret_cast<const float4 *>(row);
    const int d4 = c.D >> 2, rot4 = c.rot >> 2, half4 = c.rot >> 3;
    Row<CH> x;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int i = l + j * 32;
        x.v[j] = x.w[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (live && i < d4) {
            x.v[j] = in[i];
            if (CH > 1 && !c.interleaved && i < rot4) x.w[j] = in[i < half4 ? i + half4 : i - half4];
        }
    }
    return x;
}

__device__ __forceinline__ float4 scaled(float4 a, float r, float4 g)
{
    return make_float4(a.x * r * g.x, a.y * r * g.y, a.z * r * g.z, a.w * r * g.w);
}

// CH: float4 per lane of a row; LPR: lanes of a row.
template <int CH, int LPR>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p)
{
    constexpr int PER = kRopeThreads / LPR;            // rows at once
    __shared__ alignas(16) float2 sc[GQ4_MAX_HEAD_DIM / 2];
    const RopeCall &c = p.c;
    const int t = blockIdx.x / p.splits, part = blockIdx.x - t * p.splits;
    const int half = c.rot >> 1;
    const int l = threadIdx.x & (LPR - 1);
    const int d4 = c.D >> 2, rot4 = c.rot >> 2, half4 = c.rot >> 3;
    const float *qx = c.x[0] + (size_t)t * c.ldx[0], *kx = c.x[1] + (size_t)t * c.ldx[1];
    float *qy = c.y[0] + (size_t)t * c.ldy[0], *ky = c.y[1] + (size_t)t * c.ldy[1];
    const bool norm = c.gain[0] || c.gain[1];
    bool first_rows = true;
    // every thread takes the same number of turns (the shuffles below)
    for (int row0 = part * PER; row0 < p.rows; row0 += PER * p.splits) {
        const int row = row0 + threadIdx.x / LPR;
        const bool in = row < p.rows, k = row >= c.heads[0];
        const int head = (k ? row - c.heads[0] : row) * c.D;
        const Row<CH> x = load_row<CH>(c, (k ? kx : qx) + head, in, l);
        if (first_rows) {
            if (half > 0) {
                const int pos = __ldg(c.positions + t);
                for (int i = threadIdx.x; i < half; i += kRopeThreads) sc[i] = sin_cos_of(pos, __ldg(c.inv_freq + i));
            }
            __syncthreads();
            first_rows = false;
        }
        const float4 *gain = reinterpret_cast<const float4 *>(k ? c.gain[1] : c.gain[0]);
        float4 *y = reinterpret_cast<float4 *>((k ? ky : qy) + head);
        float r = 1.0f;
        if (norm) {  // uniform: the whole warp shuffles
            float s = 0.0f;
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                const float4 v = x.v[j];
                s += v.x * v.x + v.y * v.y + v.z * v.z + v.w * v.w;
            }
#pragma unroll
            for (int o = LPR >> 1; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            r = inv_sqrt(fmaf(s, p.inv_d, c.eps));
        }
        __syncwarp();  // in place: every lane of the row has read before any writes
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int i = l + j * 32;
            const bool live = in && i < d4, turned = live && i < rot4;
            float4 a = gain && live ? scaled(x.v[j], r, __ldg(gain + i)) : x.v[j];
            if (c.interleaved) {
                if (turned) {
                    const float4 s = reinterpret_cast<const float4 *>(sc)[i];
                    a = make_float4(a.x * s.y - a.y * s.x, a.y * s.y + a.x * s.x,
                                    a.z * s.w - a.w * s.z, a.w * s.w + a.z * s.z);
                }
            } else {
                const bool first = i < half4;
                const int other = first ? i + half4 : i - half4;
                float4 b;
                if (CH == 1) {  // the whole warp shuffles
                    b.x = __shfl_sync(0xffffffffu, a.x, other, LPR);
                    b.y = __shfl_sync(0xffffffffu, a.y, other, LPR);
                    b.z = __shfl_sync(0xffffffffu, a.z, other, LPR);
                    b.w = __shfl_sync(0xffffffffu, a.w, other, LPR);
                } else {
                    b = gain && turned ? scaled(x.w[j], r, __ldg(gain + other)) : x.w[j];
                }
                if (turned) {
                    const float m = first ? -1.0f : 1.0f;
                    const float4 *s = reinterpret_cast<const float4 *>(sc + 4 * (first ? i : other));
                    const float4 s0 = s[0], s1 = s[1];
                    a = make_float4(a.x * s0.y + m * b.x * s0.x, a.y * s0.w + m * b.y * s0.z,
                                    a.z * s1.y + m * b.z * s1.x, a.w * s1.w + m * b.w * s1.z);
                }
            }
            if (live) y[i] = a;
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
    p.inv_d = 1.0f / (float)call.D;
    const int per = kRopeThreads / lpr;
    // few tokens: their heads over several CTAs, until the GPU has two each
    p.splits = 1;
    while (p.splits * per < p.rows && (long long)call.T * p.splits < 2 * 152) ++p.splits;
    const long long grid = (long long)call.T * p.splits;
    if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
    auto run = [&](auto kern) { kern<<<(unsigned)grid, kRopeThreads, 0, stream>>>(p); };
    if (d4 > 64) run(rope_kernel<4, 32>);
    else if (d4 > 32) run(rope_kernel<2, 32>);
    else if (lpr == 32) run(rope_kernel<1, 32>);
    else if (lpr == 16) run(rope_kernel<1, 16>);
    else if (lpr == 8) run(rope_kernel<1, 8>);
    else if (lpr == 4) run(rope_kernel<1, 4>);
    else run(rope_kernel<1, 2>);
    return cudaGetLastError();
}

}  // namespace gq4
