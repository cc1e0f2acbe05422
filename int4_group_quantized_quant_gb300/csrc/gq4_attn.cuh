// gq4_attn.cuh -- what the attention kernels share: a request's rows and keys,
// the base-2 exponential, asynchronous copies into shared memory, groups of
// equal values, and the rows of a prompt that are computed apart.
#pragma once

#include <cstdint>

#include "gq4_device.cuh"
#include "gq4_kv_internal.h"
#include "gq4_kv.cuh"
#include "gq4_tma.cuh"

namespace gq4 {

constexpr unsigned int kAttnBadRequest = 1u << 8;
constexpr unsigned int kAttnGaveUp = 1u << 9;

// One request as the kernels see it.  rows [row0, row0 + n) of q; its
// queries stand at positions len - n .. len - 1.
struct AttnRequest {
    int row0, n, len;
    bool bad;
    // rows to write when the request is bad (those inside T)
    int fill0, fill1;
};

__device__ __forceinline__ AttnRequest attn_request(const AttnCall &p, int b)
{
    AttnRequest r;
    const int q0 = __ldg(p.query_start + b), q1 = __ldg(p.query_start + b + 1);
    r.row0 = q0;
    r.len = __ldg(p.seq_lens + b);
    const long long n = (long long)q1 - q0;
    r.n = n > 0 ? (int)(n < 0x7fffffff ? n : 0x7fffffff) : 0;
    r.fill0 = max(q0, 0);
    r.fill1 = max(min(q1, p.T), r.fill0);
    r.bad = n < 0 || (r.n > 0 && (q0 < 0 || q1 > p.T || n > p.max_query || r.len < 0 || r.len > p.max_len));   // (n < 0: it has no rows)
    return r;
}

// Whether a request with keys is the prompt kernel's.
__device__ __forceinline__ bool prompt_takes(const AttnCall &p, const AttnRequest &r)
{
    return !r.bad && r.len > 0 && (long long)r.n * (p.heads / p.c.kv_heads) >= p.prompt_rows;
}

// First key position that the query at position `last` sees.
__device__ __forceinline__ int attn_first(const AttnCall &p, int last)
{
    return p.window > 0 ? max(0, last + 1 - p.window) : 0;
}

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void cp_async_commit()
{
    asm volatile("cp.async.commit_group;" ::: "memory");
}

template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float quiet_nan()
{
    return __int_as_float(0x7fc00000);
}

constexpr float kLog2e = 1.4426950408889634f;

// 2^k with |x| 2^k in [2^12, 2^13) for the exponent field of x (0: as it is).
__device__ __forceinline__ int scale_exponent(float x)
{
    const int e = (int)((__float_as_uint(x) >> 23) & 255u);
    return x > 0.0f ? min(max(12 + 127 - e, -120), 120) : 0;
}

// log2 of how far apart what shares a power of two may be: two fp16 pieces of
// the largest hold 2^-25 of it, so what is smaller by more would lose digits.
constexpr int kSpread = 12;

// A group of equal values has scale 1, codes 0 and the value in its zero (the
// quantiser's rule), so its scale says nothing of its size: what is held
// against the scale, or sums of codes minus 8 times it, would drown small
// values.  The same value by a scale of its size: (0 - z) 1 = (0 - z / s) s for
// a power of two s with 8 <= |z / s| < 16.
__device__ __forceinline__ float2 equal_values(float2 sz)
{
    const uint32_t bits = __float_as_uint(sz.y) & 0x7fffffffu, e = bits >> 23;
    if (bits == 0) return make_float2(0.0f, 0.0f);
    if (e == 255) return sz;
    const uint32_t s = e > 24 ? e - 3 : 21;
    return make_float2(__uint_as_float(s << 23), sz.y * __uint_as_float((254 - s) << 23));
}

// Threads of the call's last kernel, and what it keeps in shared memory for
// the rows that the prompt kernel left.
constexpr int kJoinThreads = 128;
template <int J>
struct ApartShared {
    float q[kJoinThreads / 32][32 * J];
    uint32_t rows[kPromptTile / 32];
};

// Marks the rows of a tile that see, of some 64 keys, only values less than
// 2^-kSpread of the largest.  By the whole CTA.
template <int J, int G>
__device__ __noinline__ void small_rows(const AttnCall &a, const AttnRequest &rq, const ApartTile &at, int h, uint32_t *rows)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int R = a.heads / a.c.kv_heads, shift = 31 - __clz(a.c.page_size);
    const int row0 = at.tile * kPromptTile, row_hi = min(row0 + kPromptTile, rq.n * R) - 1, pos0 = rq.len - rq.n;
    // keys that some row sees; keys that all rows see
    const int see_hi = pos0 + row_hi / R, all_hi = pos0 + row0 / R;
    const int see_lo = attn_first(a, max(all_hi, -1)), all_lo = attn_first(a, max(see_hi, -1));
    auto size_of = [&](int t) {
        if (t < see_lo || t > see_hi) return 0.0f;
        const int page = __ldg(a.page_table + (size_t)at.request * a.max_pages + (t >> shift));
        if ((uint32_t)page >= (uint32_t)a.c.n_pages) return 0.0f;
        const size_t row = kv_row(a.c, page, h, t & (a.c.page_size - 1));
        const float2 *sz = reinterpret_cast<const float2 *>(a.c.V_sz) + row * G;
        float size = 0.0f;
#pragma unroll 1
        for (int g = 0; g < G; ++g) {
            float2 s = __ldg(sz + g);
            if (s.x == 1.0f) {
                uint32_t any = 0;
                for (int x = 0; x < 8 * (J / G); ++x)
                    any |= reinterpret_cast<const uint16_t *>(a.c.Vq)[row * (8 * J) + (x & 7) * J + g * (J / G) + (x >> 3)];
                if (any == 0) s = equal_values(s);
            }
            const float x = fabsf(s.x) * (G == 1 ? 1.0f : fmaxf(fabsf(s.y), fabsf(15.0f - s.y)));
            if (x < INFINITY) size = fmaxf(size, x);
        }
        return size;
    };
    auto largest = [](float x) { return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x))); };
    for (int k0 = (see_lo / kPromptKeys + warp) * kPromptKeys; k0 <= see_hi; k0 += kPromptKeys * (kJoinThreads / 32)) {
        if (k0 + kPromptKeys - 1 <= all_hi && k0 >= all_lo) continue;
        const int t0 = k0 + lane, t1 = t0 + 32;
        const float v0 = size_of(t0), v1 = size_of(t1);
        const int power = scale_exponent(largest(fmaxf(v0, v1)));
        for (int j = row0 / R; j <= row_hi / R; ++j) {
            const int last = pos0 + j, first = attn_first(a, max(last, -1));
            const float top = largest(fmaxf(t0 <= last && t0 >= first ? v0 : 0.0f, t1 <= last && t1 >= first ? v1 : 0.0f));
            if (top == 0.0f || scale_exponent(top) - power <= kSpread) continue;
            for (int r = max(j * R - row0, 0) + lane; r <= min(j * R + R - 1, row_hi) - row0; r += 32)
                atomicOr(&rows[r >> 5], 1u << (r & 31));
        }
    }
}

// Rows of a prompt tile that its pieces do not hold, in plain f32 over what the
// tile wrote for them: one row per warp and 32 keys at a time, of which a lane
// takes a key and then, of every key, four of the head's values.  Rare, so in
// the call's last kernel: such code in the prompt kernel itself, run or not,
// cost it 1 to 6 % (its roles fill the registers and share the instruction
// cache).  By the whole CTA.
template <int J, int G>
__device__ __noinline__ void apart_rows(const AttnCall &a, const ApartTile &at, int h, ApartShared<J> &s)
{
    constexpr int D = 32 * J, GS = D / G;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b = at.request;
    const int R = a.heads / a.c.kv_heads, shift = 31 - __clz(a.c.page_size);
    // (marks that another call wrote over must not lead out of bounds)
    if ((uint32_t)b >= (uint32_t)a.B) return;
    const AttnRequest rq = attn_request(a, b);
    if (rq.bad || (uint32_t)at.tile >= (uint32_t)((rq.n * R + kPromptTile - 1) / kPromptTile)) return;
    const int32_t *table = a.page_table + (size_t)b * a.max_pages;
    float *q = s.q[warp];
    __syncthreads();
    if (threadIdx.x < kPromptTile / 32) s.rows[threadIdx.x] = at.rows[threadIdx.x];
    __syncthreads();
    if (at.uneven) small_rows<J, G>(a, rq, at, h, s.rows);
    __syncthreads();
    for (int r = warp; r < kPromptTile; r += kJoinThreads / 32) {
        if (!(s.rows[r >> 5] >> (r & 31) & 1u)) continue;
        const int rho = at.tile * kPromptTile + r, j = rho / R, head = h * R + rho - j * R;
        if (rho >= rq.n * R) break;
        const int last = rq.len - rq.n + j, first = attn_first(a, max(last, -1));
        const float *qg = a.q + (size_t)(rq.row0 + j) * a.ldq + (size_t)head * D;
        float x[J], big = 0.0f;        // the row at a size of 1 to 2, undone in its factor
#pragma unroll
        for (int i = 0; i < J; ++i) {
            x[i] = qg[lane + 32 * i];
            if (fabsf(x[i]) < INFINITY) big = fmaxf(big, fabsf(x[i]));
        }
        const uint32_t top_q = __reduce_max_sync(0xffffffffu, __float_as_uint(big));
        const int e = top_q == 0 ? 0 : min(max((int)(top_q >> 23) - 127, -126), 126);
#pragma unroll
        for (int i = 0; i < J; ++i) q[lane + 32 * i] = ldexpf(x[i], -e);
        const float factor = ldexpf(a.scale * kLog2e, e);
        __syncwarp();
        float m = -INFINITY, l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int k0 = first; k0 <= last; k0 += 32) {
            const int t = k0 + lane;
            size_t row = 0;
            bool in = false;
            float w = -INFINITY;
            if (t <= last) {
                const int page = __ldg(table + (t >> shift));
                in = (uint32_t)page < (uint32_t)a.c.n_pages;
                w = quiet_nan();       // a page outside the pool
                if (in) {
                    row = kv_row(a.c, page, h, t & (a.c.page_size - 1));
                    const uint32_t *words = a.c.Kq + row * (4 * J);
                    const float2 *sz = reinterpret_cast<const float2 *>(a.c.K_sz) + row * G;
                    float sum = 0.0f;
#pragma unroll 1
                    for (int x = 0; x < 4 * J; ++x) {
                        const uint32_t word = __ldg(words + k_word_index(x, J));
                        const float2 kz = __ldg(sz + 8 * x / GS);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            sum = fmaf(q[8 * x + i], ((float)(word >> (4 * i) & 15u) - kz.y) * kz.x, sum);
                    }
                    w = sum * factor;
                }
            }
            float top = w;
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            const float mn = fmaxf(m, top), ref = mn == -INFINITY ? 0.0f : mn;
            const float f = exp2_approx(m - ref), p = exp2_approx(w - ref);
            m = mn;
            l = fmaf(l, f, p);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] *= f;
#pragma unroll 1
            for (int x = 0; x < min(32, last - k0 + 1); ++x) {
                const float px = __shfl_sync(0xffffffffu, p, x);
                const size_t rx = __shfl_sync(0xffffffffu, (unsigned long long)row, x);
                if (!__shfl_sync(0xffffffffu, (int)in, x)) {
                    o[0] = o[1] = o[2] = o[3] = quiet_nan();
                    continue;
                }
                if (lane >= 8 * J) continue;
                const uint32_t half = __ldg(reinterpret_cast<const uint16_t *>(a.c.Vq) + rx * (8 * J) + v_half_index(lane, J));
                const float2 vz = __ldg(reinterpret_cast<const float2 *>(a.c.V_sz) + rx * G + 4 * lane / GS);
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = fmaf(px, ((float)(half >> (4 * i) & 15u) - vz.y) * vz.x, o[i]);
            }
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
        const float inv = last < first ? 0.0f : 1.0f / l;
        if (lane < 8 * J)
            *reinterpret_cast<float4 *>(a.out + (size_t)(rq.row0 + j) * a.ldo + (size_t)head * D + 4 * lane) =
                make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
        __syncwarp();
    }
}

}  // namespace gq4
