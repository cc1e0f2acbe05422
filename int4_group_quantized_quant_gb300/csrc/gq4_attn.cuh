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

template <bool MASKS>
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
    if (MASKS && p.tree && n > 32ll * p.tree_words) r.bad = true;
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

// ---- What a row sees in the masked form ----
// Without bits: keys first .. last of the causal rule, and of those up to last
// the first p.sinks.  With them: the same of the keys before the request's new
// ones, at the row's own position (taken as at least the first new token's and
// at most the last's), and new key i where bit i of the row is set.
struct RowSight {
    int first, last;
    int past, len;          // new keys are past .. len - 1
    const uint32_t *bits;   // NULL: none
};

// Of the row of token j of its request.
__device__ __forceinline__ RowSight row_sight(const AttnCall &p, const AttnRequest &r, int j)
{
    RowSight s;
    s.past = r.len - r.n;
    s.len = r.len;
    s.bits = nullptr;
    int at = s.last = s.past + j;
    if (p.tree) {
        s.bits = p.tree + (size_t)(r.row0 + j) * p.tree_words;
        s.last = s.past - 1;
        if (p.window > 0) at = min(max(__ldg(p.positions + r.row0 + j), s.past), s.len - 1);
    }
    s.first = attn_first(p, max(at, -1));
    return s;
}

// Bit x: lo <= k0 + x <= hi.
__device__ __forceinline__ uint32_t range_bits(int k0, int lo, int hi)
{
    const int a = min(max(lo - k0, 0), 32), n = min(hi - k0, 31) + 1 - a;
    return n <= 0 ? 0u : (0xffffffffu >> (32 - n)) << a;
}

// Bit x: the row sees key k0 + x (k0 >= 0).
__device__ __forceinline__ uint32_t sight_bits(const AttnCall &p, const RowSight &s, int k0)
{
    uint32_t seen = range_bits(k0, s.first, s.last);
    if (p.window > 0) seen |= range_bits(k0, 0, min(p.sinks - 1, s.last));
    if (s.bits && k0 + 31 >= s.past) {
        const int o = k0 - s.past, w = o >> 5;     // bits o .. o + 31, from -31 on
        const uint32_t lo = w >= 0 && w < p.tree_words ? __ldg(s.bits + w) : 0u;
        const uint32_t hi = w + 1 >= 0 && w + 1 < p.tree_words ? __ldg(s.bits + w + 1) : 0u;
        seen |= __funnelshift_r(lo, hi, o & 31) & range_bits(k0, max(s.past, 0), s.len - 1);
    }
    return seen;
}

// A tree's rows may all see every key before the new ones, and some the last.
__device__ __forceinline__ void tree_bounds(const AttnCall &p, const AttnRequest &r, int &see_hi, int &all_hi)
{
    if (!p.tree) return;
    see_hi = r.len - 1;
    all_hi = r.len - r.n - 1;
}

// Blocks of `width` keys that hold the first tokens, before the one of see_lo,
// the first key of a window.
__device__ __forceinline__ int lead_blocks(const AttnCall &p, int see_lo, int width)
{
    return p.window > 0 ? min((p.sinks + width - 1) / width, see_lo / width) : 0;
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
template <int J, int G, bool MASKS>
__device__ __noinline__ void small_rows(const AttnCall &a, const AttnRequest &rq, const ApartTile &at, int h, uint32_t *rows)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int R = a.heads / a.c.kv_heads, shift = 31 - __clz(a.c.page_size);
    const int row0 = at.tile * kPromptTile, row_hi = min(row0 + kPromptTile, rq.n * R) - 1, pos0 = rq.len - rq.n;
    // keys that some row sees; keys that all rows see
    int see_hi = pos0 + row_hi / R, all_hi = pos0 + row0 / R;
    if constexpr (MASKS) tree_bounds(a, rq, see_hi, all_hi);
    const int see_lo = attn_first(a, max(MASKS && a.tree ? all_hi + 1 : all_hi, -1)), all_lo = attn_first(a, max(see_hi, -1));
    const int kept = MASKS && a.window > 0 ? a.sinks : 0, lead = MASKS ? lead_blocks(a, see_lo, kPromptKeys) : 0;
    auto size_of = [&](int t) {
        if ((t < see_lo && !(MASKS && t < kept)) || t > see_hi) return 0.0f;
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
    for (int i = warp;; i += kJoinThreads / 32) {
        const int k0 = (MASKS && i < lead ? i : see_lo / kPromptKeys + i - lead) * kPromptKeys;
        if (k0 > see_hi) break;
        if (k0 + kPromptKeys - 1 <= all_hi && k0 >= all_lo) continue;
        const int t0 = k0 + lane, t1 = t0 + 32;
        const float v0 = size_of(t0), v1 = size_of(t1);
        const int power = scale_exponent(largest(fmaxf(v0, v1)));
        for (int j = row0 / R; j <= row_hi / R; ++j) {
            bool in0, in1;
            if constexpr (MASKS) {
                const RowSight s = row_sight(a, rq, j);
                in0 = sight_bits(a, s, k0) >> lane & 1u;
                in1 = sight_bits(a, s, k0 + 32) >> lane & 1u;
            } else {
                const int last = pos0 + j, first = attn_first(a, max(last, -1));
                in0 = t0 <= last && t0 >= first;
                in1 = t1 <= last && t1 >= first;
            }
            const float top = largest(fmaxf(in0 ? v0 : 0.0f, in1 ? v1 : 0.0f));
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
// cache).  By the whole CTA; MASKS: rows row_lo .. row_hi - 1 of the tile.
template <int J, int G, bool MASKS>
__device__ __noinline__ void apart_rows(const AttnCall &a, const ApartTile &at, int h, ApartShared<J> &s, int row_lo = 0,
                                        int row_hi = kPromptTile)
{
    constexpr int D = 32 * J, GS = D / G;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b = at.request;
    const int R = a.heads / a.c.kv_heads, shift = 31 - __clz(a.c.page_size);
    // (marks that another call wrote over must not lead out of bounds)
    if ((uint32_t)b >= (uint32_t)a.B) return;
    const AttnRequest rq = attn_request<MASKS>(a, b);
    if (rq.bad || (uint32_t)at.tile >= (uint32_t)((rq.n * R + kPromptTile - 1) / kPromptTile)) return;
    const int32_t *table = a.page_table + (size_t)b * a.max_pages;
    float *q = s.q[warp];
    __syncthreads();
    if (threadIdx.x < kPromptTile / 32) s.rows[threadIdx.x] = at.rows[threadIdx.x];
    __syncthreads();
    if (at.uneven) small_rows<J, G, MASKS>(a, rq, at, h, s.rows);
    __syncthreads();
    for (int r = (MASKS ? row_lo : 0) + warp; r < (MASKS ? row_hi : kPromptTile); r += kJoinThreads / 32) {
        if (!(s.rows[r >> 5] >> (r & 31) & 1u)) continue;
        const int rho = at.tile * kPromptTile + r, j = rho / R, head = h * R + rho - j * R;
        if (rho >= rq.n * R) break;
        // MASKS: blocks of 32 keys from the first on, those between the first tokens and the window left out
        const RowSight sight = MASKS ? row_sight(a, rq, j) : RowSight{};
        const int last = MASKS ? (a.tree ? rq.len - 1 : sight.last) : rq.len - rq.n + j;
        const int first = MASKS ? (a.tree ? min(sight.first, max(sight.past, 0)) : sight.first) & ~31 : attn_first(a, max(last, -1));
        const int lead = MASKS ? 32 * lead_blocks(a, first, 32) : 0;
        bool some = false;
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
        for (int k = first - lead; k <= last; k += 32) {
            const int k0 = MASKS && k < first ? k - (first - lead) : k, t = k0 + lane;
            const uint32_t seen = MASKS ? sight_bits(a, sight, k0) : 0u;
            if (MASKS && seen == 0) continue;
            some = true;
            size_t row = 0;
            bool in = false;
            float w = -INFINITY;
            if (MASKS ? seen >> lane & 1u : t <= last) {
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
            for (int x = 0; x < (MASKS ? 32 : min(32, last - k0 + 1)); ++x) {
                if (MASKS && !(seen >> x & 1u)) continue;
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
        const float inv = (MASKS ? !some : last < first) ? 0.0f : 1.0f / l;
        if (lane < 8 * J)
            *reinterpret_cast<float4 *>(a.out + (size_t)(rq.row0 + j) * a.ldo + (size_t)head * D + 4 * lane) =
                make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
        __syncwarp();
    }
}

}  // namespace gq4
