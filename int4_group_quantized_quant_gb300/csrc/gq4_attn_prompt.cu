// gq4_attn_prompt.cu -- causal attention over the paged 4-bit cache for
// requests with many query rows (prompts and chunks of prompts), on the
// 5th-generation tensor cores.
//
// A CTA takes 128 query rows of one kv head (tokens times the head's query
// heads, so that a dequantised key serves all of them) and walks the keys in
// tiles of 64:
//   S = Q K^T   (128 x 64, K dimension 128),   P = 2^(S F - m),
//   O = O f + P V   (128 x head_dim, K dimension 64).
// Accuracy.  Every factor is two fp16 pieces (22 bits): x = xh + xl, and a
// product is Ql Kh + Qh Kl + Qh Kh, three MMAs, the small ones first.  Powers
// of two keep the pieces inside fp16: one per CTA for Q, one per key for K
// (undone by the factor F_j of column j), a running one for V.  The tensor
// core cuts its sums rather than rounding them, so a tile's P V starts at
// zero and is added to f32 registers.
//
// Warps: 4 softmax (a thread per row), 8 that add the tiles' P V (a row and
// half of head_dim per thread), 8 that read the cache and write the pieces of
// K and V into shared memory, 1 that issues the MMAs.  Tensor memory (512
// columns): S, P and the tile's O, two slots each, so that the MMA of one
// tile runs under the softmax of another; K and V have two slots too.
// K is stored [key][d] (K-major), V [key][d] as well, which is the MN-major
// form of the second product's B operand: no transposition.
//
// Bound: three times the formula's flops on the fp16 pipe, but the issue
// slots of the dequantising and softmax warps come first.
#include <cuda_fp16.h>

#include <atomic>
#include <cstdint>

#include "gq4_attn.cuh"
#include "gq4_tcgen05.cuh"

namespace gq4 {
namespace {

__device__ unsigned int g_prompt_error = 0;

constexpr int kRows = 128;
constexpr int kTile = 64;                       // keys
constexpr int kSmWarps = 4, kCoWarps = 8, kDqWarps = 8;
constexpr int kCo0 = kSmWarps, kDq0 = kCo0 + kCoWarps, kMma = kDq0 + kDqWarps;
constexpr int kThreads = 32 * (kMma + 1);
constexpr float kSlack = 4.0f;                  // log2 of how far a weight may pass the maximum
constexpr int kPieceBits = 11;                  // P is held times 2^11
constexpr uint32_t kColS = 0, kColP = 128, kColO = 256;
constexpr uint32_t kTmemCols = 512;

struct PromptParams {
    AttnCall a;
};

// Shared memory of a head of DP = 64 or 128 values (96 is padded with zeros).
template <int DP>
struct Mem {
    static constexpr int kBlocks = DP / 64;             // 128-byte columns of 64 fp16
    static constexpr int kQ = kRows * DP * 2;           // bytes of a piece
    static constexpr int kKV = kTile * DP * 2;
    static constexpr int offQ = 0;                      // high, low
    static constexpr int offK = offQ + 2 * kQ;          // [slot][high, low]
    static constexpr int offV = offK + 4 * kKV;
    static constexpr int offF = offV + 4 * kKV;         // F_j [slot][64]
    static constexpr int offFac = offF + 2 * kTile * 4; // row factors [slot][128]
    static constexpr int offInv = offFac + 2 * kRows * 4;   // 1 / l [128]
    static constexpr int offVm = offInv + kRows * 4;    // V's largest per warp [2][8], its factor [2]
    static constexpr int offBar = offVm + 128;
    static constexpr int kBytes = offBar + 256 + 1024;  // and room to align
};

struct Bars {
    uint64_t *k_full, *k_empty, *v_full, *v_empty, *s_full, *s_empty, *p_full, *o_full, *o_empty, *vmax, *fin, *drain;
};

// One MMA, A and B from shared memory (descriptors), D in tensor memory.
__device__ __forceinline__ void tc_mma_ss(uint32_t d_taddr, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_taddr), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// kind::f16 with fp16 A and B, f32 D; b_mn: B is MN-major.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn)
{
    return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// MN-major operand, 128-byte swizzle: 64 values of the MN dimension are one
// 128-byte row, 8 rows (of the K dimension) an atom of 1024 bytes; groups of
// 8 rows are `sbo` bytes apart, blocks of 64 values `lbo`.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr, uint32_t lbo, uint32_t sbo)
{
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(sbo >> 4) << 32) |
           ((uint64_t)1u << 46) | ((uint64_t)2u << 61);
}

// Bounded wait: gives up when another thread of the CTA gave up, or after the
// time limit (recording the error).
__device__ __noinline__ bool bar_wait_slow(uint64_t *bar, uint32_t parity, volatile int *abort)
{
    const unsigned long long t0 = global_timer_ns();
    while (true) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort) return false;
        if (global_timer_ns() - t0 > kWaitLimitNs) {
            *abort = 1;
            atomicOr(&g_prompt_error, kAttnGaveUp);
            return false;
        }
    }
}

__device__ __forceinline__ bool bar_wait(uint64_t *bar, uint32_t parity, volatile int *abort)
{
    return mbar_try_wait(bar, parity) || bar_wait_slow(bar, parity, abort);
}

// The whole warp waits; false in every lane when any gave up.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort)
{
    return __all_sync(0xffffffffu, bar_wait(bar, parity, abort));
}

// Two numbers as their leading fp16 pieces and the rest, each pair packed.
__device__ __forceinline__ void split_pair(float a, float b, uint32_t &hi, uint32_t &lo)
{
    const __half2 h = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h);
    const __half2 r = __floats2half2_rn(a - f.x, b - f.y);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = *reinterpret_cast<const uint32_t *>(&r);
}

// 2^k with |x| 2^k in [2^12, 2^13) for the exponent field of x (0: as it is).
__device__ __forceinline__ int scale_exponent(float x)
{
    const int e = (int)((__float_as_uint(x) >> 23) & 255u);
    return x > 0.0f ? min(max(12 + 127 - e, -120), 120) : 0;
}

__device__ __forceinline__ float pow2(int k)   // |k| <= 126
{
    return __int_as_float((127 + k) << 23);
}

// 8 codes of a word times 2^k: hi[4], lo[4] fp16 pairs of (code - z) s, in
// order.  A nibble at bits 4p is read as 2^23 + 16^p code, so that every
// difference below is exact but the last, which rounds as code - z does.
__device__ __forceinline__ void dequant_word(uint32_t w, float s, float z, uint32_t (&hi)[4], uint32_t (&lo)[4])
{
    const uint32_t magic = kMagicBits;
    const CodePairs c = extract_word(w, magic);
    const f32x2 nm = neg_magic2();
    const ZeroPairs zp = scaled_zero(z);
    const f32x2 s01 = pack2(s, s * 0.0625f), s23 = pack2(s * 0.00390625f, s * 0.000244140625f);
    const f32x2 p[4] = {c.p01, c.p23, c.p45, c.p67};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const f32x2 d = add2(add2(p[i], nm), i & 1 ? zp.nz23 : zp.nz01);
        const f32x2 sc = i & 1 ? s23 : s01;
        f32x2 v;
        asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(d), "l"(sc));
        const float2 f = unpack2(v);
        split_pair(f.x, f.y, hi[i], lo[i]);
    }
}

// A row's S of one tile, from tensor memory: the largest exponent.  Column x
// counts when first <= x <= last.
template <bool MASK>
__device__ __forceinline__ float tile_max(uint32_t s_at, const float4 *F, int last, int first)
{
    float top = -INFINITY;
#pragma unroll
    for (int x = 0; x < kTile / 16; ++x) {
        uint32_t t[16];
        tmem_ld16(s_at + 16 * x, t);
        tmem_wait_ld();
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const float4 f = F[4 * x + y];
            const float v[4] = {__uint_as_float(t[4 * y]) * f.x, __uint_as_float(t[4 * y + 1]) * f.y,
                                __uint_as_float(t[4 * y + 2]) * f.z, __uint_as_float(t[4 * y + 3]) * f.w};
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const int c = 16 * x + 4 * y + n;
                top = fmaxf(top, MASK && (c > last || c < first) ? -INFINITY : v[n]);
            }
        }
    }
    return top;
}

// Its weights 2^(S F - ref), two fp16 pieces of 2^11 times them to tensor
// memory; returns their sum.
template <bool MASK>
__device__ __forceinline__ float tile_weights(uint32_t s_at, uint32_t p_at, const float4 *F, float ref, int last,
                                              int first)
{
    float l = 0.0f;
#pragma unroll
    for (int x = 0; x < kTile / 32; ++x) {
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            uint32_t t[16];
            tmem_ld16(s_at + 32 * x + 16 * z, t);
            tmem_wait_ld();
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const float4 f = F[8 * x + 4 * z + y];
                float v[4] = {fmaf(__uint_as_float(t[4 * y]), f.x, -ref), fmaf(__uint_as_float(t[4 * y + 1]), f.y, -ref),
                              fmaf(__uint_as_float(t[4 * y + 2]), f.z, -ref),
                              fmaf(__uint_as_float(t[4 * y + 3]), f.w, -ref)};
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const int c = 32 * x + 16 * z + 4 * y + n;
                    v[n] = MASK && (c > last || c < first) ? 0.0f : exp2_approx(v[n]);
                }
                l += (v[0] + v[1]) + (v[2] + v[3]);
                split_pair(v[0] * 2048.0f, v[1] * 2048.0f, hi[8 * z + 2 * y], lo[8 * z + 2 * y]);
                split_pair(v[2] * 2048.0f, v[3] * 2048.0f, hi[8 * z + 2 * y + 1], lo[8 * z + 2 * y + 1]);
            }
        }
        tmem_st16(p_at + 16 * x, hi);
        tmem_st16(p_at + 32 + 16 * x, lo);
    }
    return l;
}

template <int NW>
__device__ __forceinline__ int scan_ints(int v, int &total, int *sums)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    int before = 0;
    total = 0;
    for (int i = 0; i < NW; ++i) {
        if (i < warp) before += sums[i];
        total += sums[i];
    }
    return before + inc - v;
}

// J: 32-value blocks of a row, G: scale groups per row, DP: padded head.
template <int J, int G, int DP>
__global__ void __launch_bounds__(kThreads, 1) attn_prompt_kernel(const __grid_constant__ PromptParams p)
{
    constexpr int D = 32 * J, UG = J / G;
    using M = Mem<DP>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t smem_s = smem_addr(smem);
    __shared__ int s_sums[kMma + 1], s_req, s_tile, s_big;
    __shared__ volatile int s_abort;
    __shared__ uint32_t s_tmem;
    const AttnCall &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int H = a.c.kv_heads, R = a.heads / H;

    // ---- this CTA's request and row tile: the last ones (most keys) first ----
    const int h = (int)(blockIdx.x % (unsigned)H);
    {
        auto tiles_of = [&](int b) {
            if (b >= a.B) return 0;
            const AttnRequest r = attn_request(a, b);
            return prompt_takes(a, r) ? (r.n * R + kRows - 1) / kRows : 0;
        };
        int all = 0, mine = 0, before = 0;
        for (int b0 = 0; b0 < a.B; b0 += kThreads) {
            int t;
            mine = tiles_of(b0 + (int)threadIdx.x);
            before = scan_ints<kMma + 1>(mine, t, s_sums);
            all += t;
        }
        const int want = all - 1 - (int)(blockIdx.x / (unsigned)H);
        if (want < 0) return;   // uniform
        int base = 0;
        for (int b0 = 0; b0 < a.B; b0 += kThreads) {
            int t = all;
            if (a.B > kThreads) {
                mine = tiles_of(b0 + (int)threadIdx.x);
                before = scan_ints<kMma + 1>(mine, t, s_sums);
            }
            if (want >= base + before && want < base + before + mine) {
                s_req = b0 + (int)threadIdx.x;
                s_tile = want - (base + before);
            }
            base += t;
            if (base > want) break;   // uniform
        }
    }
    Bars bar;
    {
        uint64_t *b = reinterpret_cast<uint64_t *>(smem + M::offBar);
        bar.k_full = b;
        bar.k_empty = b + 2;
        bar.v_full = b + 4;
        bar.v_empty = b + 6;
        bar.s_full = b + 8;
        bar.s_empty = b + 10;
        bar.p_full = b + 12;
        bar.o_full = b + 14;
        bar.o_empty = b + 16;
        bar.fin = b + 18;
        bar.drain = b + 19;
        bar.vmax = b + 20;
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bar.k_full[s], kDqWarps);
            mbar_init(&bar.k_empty[s], 1);
            mbar_init(&bar.v_full[s], kDqWarps);
            mbar_init(&bar.v_empty[s], 1);
            mbar_init(&bar.s_full[s], 1);
            mbar_init(&bar.s_empty[s], kSmWarps);
            mbar_init(&bar.p_full[s], kSmWarps);
            mbar_init(&bar.o_full[s], 1);
            mbar_init(&bar.o_empty[s], kCoWarps);
        }
        mbar_init(bar.fin, kSmWarps);
        mbar_init(bar.drain, 1);
        mbar_init(bar.vmax, kDqWarps);
        s_abort = 0;
        s_big = 0;
        mbar_fence_init();
    }
    if (warp == kMma) {
        tmem_alloc(&s_tmem, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = s_tmem;
    volatile int *abort = &s_abort;

    const int b = s_req, tile = s_tile;
    const AttnRequest rq = attn_request(a, b);
    const int rows_all = rq.n * R, row0 = tile * kRows;
    const int pos0 = rq.len - rq.n;                        // position of the request's first query
    const int row_hi = min(row0 + kRows, rows_all) - 1;
    // keys that some row sees; keys that all rows see
    const int see_hi = pos0 + row_hi / R, all_hi = pos0 + row0 / R;
    const int see_lo = attn_first(a, max(all_hi, -1)), all_lo = attn_first(a, max(see_hi, -1));
    const int tile_lo = see_lo / kTile;
    const int n_tiles = see_hi >= see_lo ? see_hi / kTile - tile_lo + 1 : 0;

    // ---- Q: two fp16 pieces with one power of two for the CTA ----
    {
        auto row_at = [&](int r) {
            const int rho = row0 + r, j = rho / R;
            return a.q + (size_t)(rq.row0 + j) * a.ldq + (size_t)(h * R + rho - j * R) * D;
        };
        float big = 0.0f;
        for (int i = threadIdx.x; i < kRows * (D / 8); i += kThreads) {
            const int r = i / (D / 8), d8 = i - r * (D / 8);
            if (row0 + r >= rows_all) continue;
            const float4 *q = reinterpret_cast<const float4 *>(row_at(r) + 8 * d8);
            const float4 x = __ldg(q), y = __ldg(q + 1);
            const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
            for (int n = 0; n < 8; ++n)   // an infinity is left to its own row
                if (fabsf(v[n]) < INFINITY) big = fmaxf(big, fabsf(v[n]));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
        if (lane == 0) atomicMax(&s_big, __float_as_int(big));
    }
    __syncthreads();
    const int kq = scale_exponent(__int_as_float(s_big));
    {
        const float up = pow2(kq);
        for (int i = threadIdx.x; i < kRows * (DP / 8); i += kThreads) {
            const int r = i / (DP / 8), d8 = i - r * (DP / 8);
            uint32_t hi[4] = {0u, 0u, 0u, 0u}, lo[4] = {0u, 0u, 0u, 0u};
            if (row0 + r < rows_all && 8 * d8 < D) {
                const int rho = row0 + r, j = rho / R;
                const float4 *q = reinterpret_cast<const float4 *>(a.q + (size_t)(rq.row0 + j) * a.ldq +
                                                                  (size_t)(h * R + rho - j * R) * D + 8 * d8);
                const float4 x = __ldg(q), y = __ldg(q + 1);
                split_pair(x.x * up, x.y * up, hi[0], lo[0]);
                split_pair(x.z * up, x.w * up, hi[1], lo[1]);
                split_pair(y.x * up, y.y * up, hi[2], lo[2]);
                split_pair(y.z * up, y.w * up, hi[3], lo[3]);
            }
            unsigned char *at = smem + M::offQ + (d8 >> 3) * (kRows * 128) + r * 128 + (((d8 & 7) ^ (r & 7)) << 4);
            *reinterpret_cast<uint4 *>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(at + M::kQ) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        // the padding of a 96-value head: zeros in every K and V slot, once
        if constexpr (DP > D) {
            constexpr int per = kTile * (DP - D) / 8;      // 16-byte pieces of one piece's padding
            for (int i = threadIdx.x; i < 8 * per; i += kThreads) {
                const int t = i / per, k = (i - t * per) / ((DP - D) / 8), d8 = D / 8 + (i - t * per) % ((DP - D) / 8);
                *reinterpret_cast<uint4 *>(smem + M::offK + t * M::kKV + (d8 >> 3) * (kTile * 128) + k * 128 +
                                           (((d8 & 7) ^ (k & 7)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
            }
        }
        fence_proxy_async_smem();
    }
    __syncthreads();

    bool ok = true;
    if (warp < kSmWarps) {
        // ===== softmax: a thread per row =====
        const int row = 32 * warp + lane;
        const uint32_t lanes = (uint32_t)(32 * warp) << 16;
        const int last = row0 + row < rows_all ? pos0 + (row0 + row) / R : -1;
        const int first = attn_first(a, max(last, -1));
        float *fac = reinterpret_cast<float *>(smem + M::offFac);
        float m = -INFINITY, l = 0.0f;
        for (int i = 0; i < n_tiles; ++i) {
            const int s = i & 1, k = i >> 1;
            if (!warp_wait(&bar.s_full[s], k & 1, abort)) {
                ok = false;
                break;
            }
            tc_fence_after_sync();
            // two passes over S in tensor memory (the maximum, then the weights)
            // keep the registers few
            const float4 *F = reinterpret_cast<const float4 *>(smem + M::offF) + s * (kTile / 4);
            const int k0 = (tile_lo + i) * kTile;
            const bool masked = k0 + kTile - 1 > all_hi || k0 < all_lo;   // uniform
            const uint32_t s_at = tmem + lanes + kColS + s * kTile, p_at = tmem + lanes + kColP + s * 64;
            const float top = masked ? tile_max<true>(s_at, F, last - k0, first - k0) : tile_max<false>(s_at, F, 0, 0);
            float f = 1.0f;
            if (top > m + kSlack) {
                f = exp2_approx(m - top);
                m = top;
                l *= f;
            }
            const float ref = m == -INFINITY ? 0.0f : m;
            // the tile before last: its factors are read, its P is used up
            if (i >= 2 && !warp_wait(&bar.o_empty[s], (k - 1) & 1, abort)) {
                ok = false;
                break;
            }
            tc_fence_after_sync();
            fac[s * kRows + row] = f;
            l += masked ? tile_weights<true>(s_at, p_at, F, ref, last - k0, first - k0)
                        : tile_weights<false>(s_at, p_at, F, ref, 0, 0);
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.s_empty[s]);
            tmem_wait_st();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.p_full[s]);
        }
        reinterpret_cast<float *>(smem + M::offInv)[row] = m == -INFINITY ? 0.0f : 1.0f / l;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar.fin);
    } else if (warp < kDq0) {
        // ===== the tiles' P V added up: a row and half of the values per thread =====
        constexpr int C = DP / 2;
        const int q4 = warp & 3, half = (warp - kCo0) >> 2;
        const int row = 32 * q4 + lane;
        const uint32_t lanes = (uint32_t)(32 * q4) << 16;
        const float *fac = reinterpret_cast<const float *>(smem + M::offFac);
        const float *vfac = reinterpret_cast<const float *>(smem + M::offVm) + 16;
        const int *vexp = reinterpret_cast<const int *>(smem + M::offVm) + 18;
        float o[C];
#pragma unroll
        for (int d = 0; d < C; ++d) o[d] = 0.0f;
        int e = 0;
        for (int i = 0; i < n_tiles; ++i) {
            const int s = i & 1, k = i >> 1;
            // the factors come with P and with V
            if (!warp_wait(&bar.p_full[s], k & 1, abort) || !warp_wait(&bar.v_full[s], k & 1, abort) ||
                !warp_wait(&bar.o_full[s], k & 1, abort)) {
                ok = false;
                break;
            }
            tc_fence_after_sync();
            const float f = fac[s * kRows + row] * vfac[s];
            e = vexp[s];
#pragma unroll
            for (int x = 0; x < C / 16; ++x) {
                uint32_t t[16];
                tmem_ld16(tmem + lanes + kColO + s * 128 + half * C + 16 * x, t);
                tmem_wait_ld();
#pragma unroll
                for (int y = 0; y < 16; ++y) o[16 * x + y] = fmaf(o[16 * x + y], f, __uint_as_float(t[y]));
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.o_empty[s]);
        }
        if (ok) ok = warp_wait(bar.fin, 0, abort);
        const int rho = row0 + row;
        if (rho < rows_all) {
            const int j = rho / R;
            float *out = a.out + (size_t)(rq.row0 + j) * a.ldo + (size_t)(h * R + rho - j * R) * D + half * C;
            const float inv = ok ? reinterpret_cast<const float *>(smem + M::offInv)[row] * pow2(-kPieceBits)
                                 : quiet_nan();
            const float back = pow2(-e);   // V's power of two
#pragma unroll
            for (int d = 0; d < C; d += 4)
                if (half * C + d < D)
                    *reinterpret_cast<float4 *>(out + d) =
                        make_float4(o[d] * inv * back, o[d + 1] * inv * back, o[d + 2] * inv * back, o[d + 3] * inv * back);
        }
    } else if (warp < kMma) {
        // ===== the cache: codes, scales and zeros to fp16 pieces =====
        // lane: key lane % 8 of the warp's eight, values 32 u + 8 (lane / 8) ..
        // + 7 (eight keys of one shared-memory phase meet eight distinct banks)
        const int w = warp - kDq0, key = 8 * w + (lane & 7), c = lane >> 3;
        const int shift = 31 - __clz(a.c.page_size);
        const int32_t *table = a.page_table + (size_t)b * a.max_pages;
        float *vm = reinterpret_cast<float *>(smem + M::offVm);
        int *vexp = reinterpret_cast<int *>(vm + 18);
        const float Fq = a.scale * kLog2e;
        struct Loaded {
            uint32_t kw[J], vw[J];
            float2 ks[G], vs[G];
            bool here, bad;
        };
        auto fetch = [&](int i) {
            Loaded x;
            const int t = (tile_lo + i) * kTile + key;
            x.here = i < n_tiles && t <= see_hi && t >= see_lo;
            x.bad = false;
            size_t row = 0;
            if (x.here) {
                const int page = __ldg(table + (t >> shift));
                x.bad = (uint32_t)page >= (uint32_t)a.c.n_pages;
                if (!x.bad) row = kv_row(a.c, page, h, t & (a.c.page_size - 1));
            }
            if (x.here && !x.bad) {
                const uint32_t *kp = a.c.Kq + row * (4 * J) + c * J, *vp = a.c.Vq + row * (4 * J) + c * J;
                if constexpr (J == 4) {
                    const uint4 k4 = __ldg(reinterpret_cast<const uint4 *>(kp)), v4 = __ldg(reinterpret_cast<const uint4 *>(vp));
                    x.kw[0] = k4.x; x.kw[1] = k4.y; x.kw[2] = k4.z; x.kw[3] = k4.w;
                    x.vw[0] = v4.x; x.vw[1] = v4.y; x.vw[2] = v4.z; x.vw[3] = v4.w;
                } else {
#pragma unroll
                    for (int u = 0; u < J; ++u) {
                        x.kw[u] = __ldg(kp + u);
                        x.vw[u] = __ldg(vp + u);
                    }
                }
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    x.ks[g] = __ldg(reinterpret_cast<const float2 *>(a.c.K_sz) + row * G + g);
                    x.vs[g] = __ldg(reinterpret_cast<const float2 *>(a.c.V_sz) + row * G + g);
                }
            } else {
#pragma unroll
                for (int u = 0; u < J; ++u) x.kw[u] = x.vw[u] = 0u;
#pragma unroll
                for (int g = 0; g < G; ++g) x.ks[g] = x.vs[g] = make_float2(0.0f, 0.0f);
            }
            return x;
        };
        // the largest |(code - z) s| that the row's scales allow
        auto bound_of = [](const float2 (&sz)[G]) {
            float m = 0.0f;
#pragma unroll
            for (int g = 0; g < G; ++g) m = fmaxf(m, fabsf(sz[g].x) * fmaxf(fabsf(sz[g].y), fabsf(15.0f - sz[g].y)));
            return m;
        };
        auto finite_of = [](const float2 (&sz)[G]) {
            float s = 0.0f;
#pragma unroll
            for (int g = 0; g < G; ++g) s += 0.0f * sz[g].x + 0.0f * sz[g].y;
            return s == 0.0f;
        };
        auto store_row = [&](uint32_t base, int u, const uint32_t (&hi)[4], const uint32_t (&lo)[4]) {
            const int d8 = 4 * u + c;
            const uint32_t at = base + (d8 >> 3) * (kTile * 128) + key * 128 + (((d8 & 7) ^ (key & 7)) << 4);
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(hi[0]), "r"(hi[1]), "r"(hi[2]), "r"(hi[3])
                         : "memory");
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at + M::kKV), "r"(lo[0]), "r"(lo[1]), "r"(lo[2]),
                         "r"(lo[3])
                         : "memory");
        };
        int ve = 120;                                      // V is held times 2^ve
        Loaded cur = fetch(0);
        for (int i = 0; i < n_tiles; ++i) {
            const int s = i & 1, k = i >> 1;
            const Loaded x = cur;
            cur = fetch(i + 1);
            if (x.bad && lane < 8) atomicOr(&g_prompt_error, kAttnBadRequest);
            // ---- K ----
            const float kb = bound_of(x.ks);
            const int kk = kb < INFINITY ? scale_exponent(kb) : 0;
            // a value that is not finite spoils the rows that see it: through the key's factor
            const bool vfine = finite_of(x.vs);
            if (i >= 2 && (!warp_wait(&bar.k_empty[s], (k - 1) & 1, abort) ||
                           !warp_wait(&bar.s_empty[s], (k - 1) & 1, abort))) {
                ok = false;
                break;
            }
            {
                const float up = pow2(kk);
                const uint32_t base = smem_s + M::offK + s * 2 * M::kKV;
#pragma unroll
                for (int u = 0; u < J; ++u) {
                    uint32_t hi[4], lo[4];
                    dequant_word(x.kw[u], x.ks[u / UG].x * up, x.ks[u / UG].y, hi, lo);
                    store_row(base, u, hi, lo);
                }
                if (c == 0) {
                    const float f = ldexpf(Fq, -kq - kk);
                    reinterpret_cast<float *>(smem + M::offF)[s * kTile + key] = x.bad || !vfine ? quiet_nan() : f;
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.k_full[s]);
            // ---- V: a power of two for the tile, never growing ----
            float vb = vfine ? bound_of(x.vs) : 0.0f;
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) vb = fmaxf(vb, __shfl_xor_sync(0xffffffffu, vb, o));
            if (lane == 0) {
                vm[8 * s + w] = vb;
                mbar_arrive(bar.vmax);
            }
            if (!warp_wait(bar.vmax, i & 1, abort)) {
                ok = false;
                break;
            }
#pragma unroll
            for (int y = 0; y < kDqWarps; ++y) vb = fmaxf(vb, vm[8 * s + y]);
            const int ne = vb > 0.0f ? min(ve, scale_exponent(vb < INFINITY ? vb : 1.0f)) : ve;
            const float vf = pow2(max(ne - ve, -126));     // what the sums so far are scaled by
            ve = ne;
            if (i >= 2 && (!warp_wait(&bar.v_empty[s], (k - 1) & 1, abort) ||
                           !warp_wait(&bar.o_empty[s], (k - 1) & 1, abort))) {
                ok = false;
                break;
            }
            {
                const float up = vfine ? pow2(ve) : 0.0f;
                const uint32_t base = smem_s + M::offV + s * 2 * M::kKV;
#pragma unroll
                for (int u = 0; u < J; ++u) {
                    // halves 2c and 2c+1 of block u lie J halves apart
                    uint32_t word;
                    if constexpr (J == 4) word = __byte_perm(x.vw[u / 2], x.vw[2 + u / 2], (u & 1) ? 0x7632 : 0x5410);
                    else if constexpr (J == 2) word = __byte_perm(x.vw[0], x.vw[1], u ? 0x7632 : 0x5410);
                    else
                        word = u == 0   ? __byte_perm(x.vw[0], x.vw[1], 0x7610)
                               : u == 1 ? __byte_perm(x.vw[0], x.vw[2], 0x5432)
                                        : __byte_perm(x.vw[1], x.vw[2], 0x7610);
                    uint32_t hi[4], lo[4];
                    const float z = x.vs[u / UG].y, sv = x.vs[u / UG].x;
                    dequant_word(word, vfine ? sv * up : 0.0f, vfine ? z : 0.0f, hi, lo);
                    store_row(base, u, hi, lo);
                }
                if (w == 0 && lane == 0) {
                    vm[16 + s] = vf;
                    vexp[s] = ve;
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.v_full[s]);
        }
    } else if (lane == 0) {
        // ===== MMA =====
        const uint32_t id_s = idesc_f16_f32(kRows, kTile, false), id_o = idesc_f16_f32(kRows, DP, true);
        const uint32_t qh = smem_s + M::offQ, ql = qh + M::kQ;
        bool any = false;
        auto pv = [&](int i) {
            const int s = i & 1, k = i >> 1;
            if (!bar_wait(&bar.p_full[s], k & 1, abort) || !bar_wait(&bar.v_full[s], k & 1, abort)) return false;
            if (i >= 2 && !bar_wait(&bar.o_empty[s], (k - 1) & 1, abort)) return false;
            tc_fence_after_sync();
            const uint32_t vh = smem_s + M::offV + s * 2 * M::kKV, vl = vh + M::kKV;
            const uint32_t d = tmem + kColO + s * 128, ph = tmem + kColP + s * 64, pl = ph + 32;
#pragma unroll
            for (int x = 0; x < 3; ++x) {
                const uint32_t at = x == 0 ? pl : ph, bt = x == 1 ? vl : vh;
#pragma unroll
                for (int y = 0; y < kTile / 16; ++y)
                    tc_mma_ts(d, at + 8 * y, smem_desc_mn_sw128(bt + 2048 * y, kTile * 128, 1024), id_o,
                              (x | y) != 0 ? 1u : 0u);
            }
            tc_commit(&bar.o_full[s]);
            tc_commit(&bar.v_empty[s]);
            any = true;
            return true;
        };
        for (int i = 0; ok && i < n_tiles; ++i) {
            const int s = i & 1, k = i >> 1;
            ok = bar_wait(&bar.k_full[s], k & 1, abort) && (i < 2 || bar_wait(&bar.s_empty[s], (k - 1) & 1, abort));
            if (!ok) break;
            tc_fence_after_sync();
            const uint32_t kh = smem_s + M::offK + s * 2 * M::kKV, kl = kh + M::kKV;
            const uint32_t d = tmem + kColS + s * kTile;
#pragma unroll
            for (int x = 0; x < 3; ++x) {
                const uint32_t at = x == 0 ? ql : qh, bt = x == 1 ? kl : kh;
#pragma unroll
                for (int y = 0; y < DP / 16; ++y)
                    tc_mma_ss(d, smem_desc_sw128(at + (y >> 2) * (kRows * 128) + (y & 3) * 32, 1024),
                              smem_desc_sw128(bt + (y >> 2) * (kTile * 128) + (y & 3) * 32, 1024), id_s,
                              (x | y) != 0 ? 1u : 0u);
            }
            tc_commit(&bar.s_full[s]);
            tc_commit(&bar.k_empty[s]);
            any = true;
            if (i > 0) ok = pv(i - 1);
        }
        if (ok && n_tiles > 0) ok = pv(n_tiles - 1);
        if (any) {
            // every MMA done before tensor memory and shared memory go
            tc_commit(bar.drain);
            (void)mbar_wait(bar.drain, 0);
        }
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == kMma) tmem_dealloc(tmem, kTmemCols);
}

template <int J, int G, int DP>
cudaError_t launch_prompt_t(const AttnCall &call, cudaStream_t stream)
{
    auto kern = attn_prompt_kernel<J, G, DP>;
    constexpr int smem = Mem<DP>::kBytes;
    int dev = 0;
    cudaError_t err;
    if ((err = cudaGetDevice(&dev)) != cudaSuccess) return err;
    static std::atomic<int> ready_dev{-1};
    if (ready_dev.load(std::memory_order_acquire) != dev) {
        if ((err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess)
            return err;
        ready_dev.store(dev, std::memory_order_release);
    }
    // as many row tiles as the requests can have together, per kv head
    const long long R = call.heads / call.c.kv_heads;
    const long long tiles = (call.T * R + kRows - 1) / kRows + (call.B < call.T ? call.B : call.T);
    const long long grid = tiles * call.c.kv_heads;
    if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
    PromptParams p{};
    p.a = call;
    kern<<<(unsigned)grid, kThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

bool prompt_path_supported(const AttnCall &call)
{
    return call.c.head_dim <= 128;
}

cudaError_t launch_attn_prompt(const AttnCall &call, cudaStream_t stream)
{
    const int G = call.c.head_dim / call.c.group_size;
    switch (call.c.head_dim * 16 + G) {
    case 64 * 16 + 1: return launch_prompt_t<2, 1, 64>(call, stream);
    case 64 * 16 + 2: return launch_prompt_t<2, 2, 64>(call, stream);
    case 96 * 16 + 1: return launch_prompt_t<3, 1, 128>(call, stream);
    case 96 * 16 + 3: return launch_prompt_t<3, 3, 128>(call, stream);
    case 128 * 16 + 1: return launch_prompt_t<4, 1, 128>(call, stream);
    case 128 * 16 + 2: return launch_prompt_t<4, 2, 128>(call, stream);
    case 128 * 16 + 4: return launch_prompt_t<4, 4, 128>(call, stream);
    }
    return cudaErrorInvalidValue;
}

cudaError_t read_prompt_device_error(unsigned int *bits, bool clear)
{
    cudaError_t err = cudaMemcpyFromSymbol(bits, g_prompt_error, sizeof(unsigned int));
    if (err != cudaSuccess || !clear) return err;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_prompt_error, &zero, sizeof(unsigned int));
}

}  // namespace gq4
