// gq4_attn.cu -- causal attention over the paged 4-bit key/value cache
// (gq4_kv_attention), for single tokens and a few rows: the cache is read
// once and the matrix instructions take its codes as they are.
//
// Mathematics.  A query row and the codes of its kv head:
//   w_t = scale * sum_g s_tg (sum_{d in g} q_d c_td - z_tg sum_{d in g} q_d)
//   out = sum_t p_t s_tg (c_td - 8) - sum_t p_t s_tg (z_tg - 8),  p_t = 2^(w_t log2 e - m)
// The codes c enter the warp-level MMA (m16n8k16, f16 inputs, f32 sums) as
// exact fp16 numbers; the other factor is written as two fp16 pieces, which
// take two neighbouring columns of the instruction, so that one thread holds
// both sums.  A query row is a 22-bit fixed-point number 2048 h + l (whole
// numbers, a power of two per row), so that every sum of the first product is
// exact: the tensor core cuts what it cannot hold.  The weights p s are
// xh + xl, 11 bits each (2^-23 relative): a small weight keeps its digits.
// The keys (or, in the second product, the head's values of d) are the 16 rows
// of the instruction and the query rows its 8 columns: 4 rows of two pieces
// each, a full instruction for the four query heads of a kv head, and one
// decode of a code serves all of them.
//   Keys: a word's nibbles i and i+4 are masked in place, an fp16 pair
// c 2^-24 (c 2^-20 for odd i: q is pre-scaled by 1/16 there).
//   Values: nibbles of two tokens are paired by a byte permute, OR-ed with
// 1024 and shifted to c - 8 by one exact fp16 operation (conversion by the
// exponent's bits, as Kim, Henry, Fahim and Awadalla published it in 2022).  Without the 8 the
// sums would carry the codes' mean, several times the result, and its
// rounding.
//   The second product stays in the tensor core for 4 stages (128 keys of a
// warp) and is then added to f32 sums: cut sums of a whole context would be
// off by 2.0e-6 of the result at 125k keys instead of 4.5e-7.
//   A group of equal values (scale 1) is given a scale of its own size first,
// in shared memory: the 8 taken off its codes would drown small ones.
//   The running maximum m moves only when a weight passes 2^4 of it (a vote
// per 32 keys), so that accumulators are rescaled rarely; the scales of the
// values that a row sees likewise share a power of two 2^E, which keeps p s
// inside fp16.
//
// Split.  A stage is 32 keys of one (request, kv head, block of rows), a
// unit; the list of all stages is cut into equal ranges, one per CTA, and
// those into one per warp, whatever the requests' lengths (units of up to 4
// stages are not cut).  So each warp goes its own way through its keys, with
// its own sums, query pieces and copies, and a CTA meets once, at the end: it
// joins its warps' sums of the same unit, and a unit cut by the range of the
// CTA leaves (m, l, sum) in the workspace, which a second kernel joins: no
// atomics, always in order, the same bits every time.  (8 warps that share a
// 256-key step and meet at each unit's end took 62 us where this takes 47.)
// The cut is computed on the device from the lengths, so a captured launch
// follows them.
//
// Copies.  Each warp keeps its own ring of 32-key stages filled by 16-byte
// cp.async: the rows of 16 keys of one page and head are contiguous.  Keys
// are assigned to the instruction's rows so that both products read shared
// memory without bank conflicts (see key_of_row).
//
// Measured in a graph: 48 requests of 500 to 8192 keys, 32 heads over 8 of 128,
// one group: 47 us, 215 MB at 4.6 TB/s; two of 125k keys, two groups: 64 us,
// 319 MB at 5.0 TB/s; 16 drafts of 5 tokens, 16 heads of 64, two groups: 30 us;
// one request of 776 keys: 10 us, of which 2 the ranges, 2 the first loads, 1 a
// stage, 2 the CTA's join and 3 the second kernel.
// Instructions: 675 per stage and warp, 32 of them matrix instructions and 240
// the decoding of codes, issued in 60% of the cycles by the 16 warps that
// registers allow (128 per thread, of which the 4-row form at heads of 128
// spills 92 bytes).
// A row block of a prompt is given all stages up to the request's last key and
// walks past those that it does not see, which the equal cut counts: prompts
// that stay here lose up to half of their time to it.
#include <cuda_fp16.h>

#include <atomic>
#include <cstdint>

#include "gq4_attn.cuh"
#include "gq4_host.h"

namespace gq4 {
namespace {

__device__ unsigned int g_attn_error = 0;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kStageKeys = 32;                    // per warp
constexpr float kSlack = 4.0f;                    // log2 of how far a weight may pass the maximum
constexpr float kRadix = 2048.0f;                 // a query is 2048 h + l, whole numbers
constexpr int kPieceBits = 11;                    // p s <= 2^kSlack is held times 2^11: below 2^15
constexpr int kCarry = 4;                         // stages summed in the tensor core
constexpr int kWholeStages = 4;                   // units of so few stages are one warp's
// What a unit's start costs a warp, in stages, when shares are cut (0 / 2 / 4 take 31.9 / 30.1 / 29.4 us for the
// drafts below, 48.1 / 47.0 / 47.7 for the 48 requests)
constexpr int kStart = 2;
constexpr int kMaxGrid = 304;                     // CTAs (the workspace's slots)

struct SplitParams {
    AttnCall a;
    float *part;        // [grid][2][rows][D + 2] partial sums
    float *head;        // [grid][8 warps][rows][D + 2] a warp's first, cut unit
    int4 *desc;         // [grid][2] the cut unit that starts in this CTA: (first token, rows, kv head,
                        // row block), (last CTA or -1, slot)
    int R;              // query heads per kv head
    int grid;
};

// Key (0..15) that row i of the instruction's A operand takes.  A thread of
// the second product reads the keys of rows 2c, 2c+1, 2c+8, 2c+9: these are
// c, 4 + (c^3), and the same plus 8, so the four lanes of a quad read four
// consecutive keys, and the two rows 2m, 2m+1 of one shared-memory phase of
// the first product lie in different halves of 128 bytes (64-byte rows) or
// in different quarters in fours (32-byte rows).
__device__ __forceinline__ int key_of_row(int i)
{
    const int m = (i >> 1) & 3;
    return (i & 8) + ((i & 1) ? 4 + (m ^ 3) : m);
}

// 16-byte piece of a row, swizzled by its key so that the second product's
// reads (64- and 128-byte rows) meet distinct banks.
template <int J>
__device__ __forceinline__ int swizzle(int key)
{
    return J == 8 ? ((key & 3) << 1) | (key & 1) : J == 4 ? key & 2 : 0;
}

template <int J, int G>
struct Stage {
    static constexpr int kCodes = kStageKeys * 16 * J;    // bytes of 32 rows
    static constexpr int kSz = kStageKeys * 8 * G;
    static constexpr int kBytes = 2 * (kCodes + kSz);
};

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same onto zero.
__device__ __forceinline__ void mma16816_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// x as two fp16 pieces, the leading one in the low half.
__device__ __forceinline__ uint32_t two_pieces(float x)
{
    const float hi = __half2float(__float2half_rn(x));
    const __half2 r = __floats2half2_rn(x, x - hi);
    return *reinterpret_cast<const uint32_t *>(&r);
}

__device__ __forceinline__ uint32_t h2_add(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ uint32_t h2_fma(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

template <uint32_t MASK>
__device__ __forceinline__ uint32_t mask_or(uint32_t x, uint32_t magic)
{
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(x), "n"(MASK), "r"(magic));
    return d;
}

// J consecutive words / halves of a row in shared memory.
template <int J>
__device__ __forceinline__ void load_words(uint32_t s, uint32_t (&w)[J])
{
    if constexpr (J % 4 == 0) {
#pragma unroll
        for (int i = 0; i < J; i += 4)
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                         : "r"(s + 4 * i));
    } else if constexpr (J == 2) {
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(s));
    } else {
#pragma unroll
        for (int i = 0; i < J; ++i) asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[i]) : "r"(s + 4 * i));
    }
}

template <int J>
struct Halves {  // J 16-bit halves as (J + 1) / 2 registers, even ones low
    uint32_t r[(J + 1) / 2];
};

template <int J>
__device__ __forceinline__ Halves<J> load_halves(uint32_t s)
{
    Halves<J> h;
    if constexpr (J == 8) {
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(h.r[0]), "=r"(h.r[1]), "=r"(h.r[2]), "=r"(h.r[3])
                     : "r"(s));
    } else if constexpr (J == 4) {
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(h.r[0]), "=r"(h.r[1]) : "r"(s));
    } else if constexpr (J == 2) {
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(h.r[0]) : "r"(s));
    } else {
        uint16_t a[J];
#pragma unroll
        for (int i = 0; i < J; ++i) asm volatile("ld.shared.u16 %0, [%1];" : "=h"(a[i]) : "r"(s + 2 * i));
#pragma unroll
        for (int i = 0; i < (J + 1) / 2; ++i)
            h.r[i] = a[2 * i] | (2 * i + 1 < J ? (uint32_t)a[2 * i + 1] << 16 : 0u);
    }
    return h;
}

// A lane's J words of a key row; J = 8: two 16-byte pieces whose places differ in bit 4.
template <int J>
__device__ __forceinline__ void load_key(uint32_t at, uint32_t (&w)[J])
{
    if constexpr (J == 8) {
        uint32_t t[4];
        load_words<4>(at, t);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = t[i];
        load_words<4>(at ^ 16u, t);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[4 + i] = t[i];
    } else {
        load_words<J>(at, w);
    }
}

__device__ __forceinline__ float2 lds_f2(uint32_t s)
{
    float2 v;
    asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(s));
    return v;
}

// A request's work: row blocks and key steps.
struct Work {
    int step0, steps;   // stages of kStageKeys keys
    int blocks;         // row blocks of ROWS rows per kv head
    long long total;    // of all its units, with kStart for each one's start
};

template <int ROWS>
__device__ __forceinline__ Work work_of(const AttnCall &p, const AttnRequest &r, int R)
{
    Work w{0, 0, 0, 0};
    if (r.bad || r.n == 0 || r.len == 0 || prompt_takes(p, r)) return w;
    const int first = attn_first(p, max(r.len - r.n, -1));
    w.step0 = first / kStageKeys;
    w.steps = (r.len + kStageKeys - 1) / kStageKeys - w.step0;
    w.blocks = (int)(((long long)r.n * R + ROWS - 1) / ROWS);
    w.total = (long long)w.blocks * p.c.kv_heads * (w.steps + kStart);
    return w;
}

// a / d of nonnegative numbers, in 32 bits where they allow it.
__device__ __forceinline__ long long quotient(long long a, int d)
{
    return (a >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)d) : a / d;
}

__device__ __forceinline__ long long warp_scan(long long v, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// Exclusive prefix of v over the CTA's threads and its total.
__device__ __forceinline__ long long cta_scan(long long v, long long &total, long long *sums)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long inc = warp_scan(v, lane);
    __syncthreads();
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    long long before = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        if (i < warp) before += sums[i];
        total += sums[i];
    }
    return before + inc - v;
}

// 1 / x for a power of two, 2^-126 to 2^126.
__device__ __forceinline__ float inverse_power(float x)
{
    return __uint_as_float(0x7f000000u - __float_as_uint(x));
}

// o += the two pieces' sums, which start again at zero.
template <int NB, int J>
__device__ __forceinline__ void carry(float (&o)[NB][J][4], float (&t0)[NB][J][4], float (&t1)[NB][J][4])
{
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int u = 0; u < J; ++u) {
            o[nb][u][0] += t0[nb][u][0] + t0[nb][u][1];
            o[nb][u][1] += t0[nb][u][2] + t0[nb][u][3];
            o[nb][u][2] += t1[nb][u][0] + t1[nb][u][1];
            o[nb][u][3] += t1[nb][u][2] + t1[nb][u][3];
#pragma unroll
            for (int i = 0; i < 4; ++i) t0[nb][u][i] = t1[nb][u][i] = 0.0f;
        }
}

// A warp's part of a cut unit: the position of the unit's first stage (-1:
// none), and which it is.
struct Segment {
    long long start;
    int length;              // with its start
    int row0, rows;          // the request's first token and its query rows per kv head
    int h, rb;               // kv head, row block
};

// A stage's value groups of equal values, by scales of their size: a lane per
// key.  st: the stage.
template <int J, int G>
__device__ __noinline__ void fit_equal_values(uint32_t st)
{
    using S = Stage<J, G>;
    const int key = threadIdx.x & 31;
    const uint32_t row = st + S::kCodes + key * 16 * J, at = st + 2 * S::kCodes + S::kSz + key * 8 * G;
    __syncwarp();
#pragma unroll 1
    for (int gr = 0; gr < G; ++gr) {
        const float2 sz = lds_f2(at + 8 * gr);
        if (sz.x != 1.0f) continue;
        uint32_t any = 0;
#pragma unroll 1
        for (int x = 0; x < 8 * (J / G); ++x) {
            const int byte = 2 * ((x & 7) * J + gr * (J / G) + (x >> 3));
            uint16_t half;
            asm volatile("ld.shared.u16 %0, [%1];"
                         : "=h"(half)
                         : "r"(row + (((byte >> 4) ^ swizzle<J>(key)) << 4) + (byte & 15))
                         : "memory");
            any |= half;
        }
        if (any != 0) continue;
        const float2 to = equal_values(sz);
        asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(at + 8 * gr), "f"(to.x), "f"(to.y) : "memory");
    }
    __syncwarp();
}

template <int J, int G, int NB, int STAGES, int MINB>
__global__ void __launch_bounds__(kThreads, MINB) attn_split_kernel(const __grid_constant__ SplitParams p)
{
    constexpr int D = 32 * J, ROWS = 4 * NB, UG = J / G;   // UG: 32-value blocks per group
    using S = Stage<J, G>;
    extern __shared__ __align__(128) unsigned char smem[];
    constexpr int kSums = ROWS * (D + 2);   // floats of a unit's sums: [row][D], then m, l of each row
    __shared__ union {
        struct {
            long long sums[kWarps];
            int special;
        } start;
        Segment seg[2 * kWarps];            // a warp's first and last segment, where cut
    } s;
    __shared__ long long s_bound[kWarps + 1];   // where the warps' ranges start and the last ends
    const AttnCall &a = p.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int H = a.c.kv_heads, R = p.R;
    // the requests of a tile of kThreads, until the copies start: the stages up to and with each,
    // and (first token, queries, length, stages of a unit)
    long long *t_end = reinterpret_cast<long long *>(smem);
    int4 *t_req = reinterpret_cast<int4 *>(smem + 8 * kThreads);

    // ---- this CTA's range of stages ----
    if (threadIdx.x == 0) {
        s.start.special = 0;
        p.desc[2 * blockIdx.x + 1] = make_int4(-1, 0, 0, 0);
    }
    __syncthreads();
    long long total = 0;
    // a tile's requests; returns its stages
    auto tile = [&](int b0, bool look) {
        const int b = b0 + threadIdx.x;
        long long mine = 0, t;
        int4 r4 = make_int4(0, 0, 0, 1);
        if (b < a.B) {
            const AttnRequest r = attn_request(a, b);
            const Work w = work_of<ROWS>(a, r, R);
            mine = w.total;
            r4 = make_int4(r.row0, r.n, r.len, max(w.steps, 1));
            if (look && (r.bad || (r.n > 0 && r.len == 0))) s.start.special = 1;
        }
        const long long before = cta_scan(mine, t, s.start.sums);
        t_end[threadIdx.x] = before + mine;
        t_req[threadIdx.x] = r4;
        return t;
    };
    for (int b0 = 0; b0 < a.B; b0 += kThreads) total += tile(b0, true);
    const long long chunk = quotient(total + gridDim.x - 1, (int)gridDim.x);
    const long long raw0 = chunk * blockIdx.x, raw1 = min(raw0 + chunk, total);
    // requests that need no sums: bad ones, and those without keys
    __syncthreads();
    if (s.start.special) {
        for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
            const AttnRequest r = attn_request(a, b);
            if (!r.bad && !(r.n > 0 && r.len == 0)) continue;
            if (r.bad && threadIdx.x == 0) atomicOr(&g_attn_error, kAttnBadRequest);
            const float v = r.bad ? quiet_nan() : 0.0f;
            const int per = a.heads * D;
            for (int row = r.fill0; row < r.fill1; ++row)
                for (int i = threadIdx.x; i < per; i += kThreads) a.out[(size_t)row * a.ldo + i] = v;
        }
    }
    if (raw0 >= raw1) return;
    // this warp's range, from the unit that its first stage belongs to
    long long wb = total, we = total;
    int b = 0, unit = 0, from = 0;    // of the request: (kv head, row block), stage
    AttnRequest rq{};
    Work wk{0, 1, 1, 0};
    {
        const long long n = raw1 - raw0, raw_b = raw0 + n * warp / kWarps, raw_e = raw0 + n * (warp + 1) / kWarps;
        long long base = 0;
        for (int b0 = 0; b0 < a.B && base <= raw1; b0 += kThreads) {   // uniform
            const long long t = a.B > kThreads ? tile(b0, false) : total;
            if (a.B > kThreads) __syncthreads();
            // where a warp starts at the earliest: its place among all stages, within request i
            auto locate = [&](long long raw, int &i, int &u, int &f) {
                const long long rel = raw - base;
                const int block = __ffs(__ballot_sync(0xffffffffu, t_end[lane * 8 + 7] > rel)) - 1;
                i = block * 8 + __ffs(__ballot_sync(0xffffffffu, t_end[block * 8 + (lane & 7)] > rel)) - 1;
                const long long at = rel - (i > 0 ? t_end[i - 1] : 0);
                const int steps = t_req[i].w;
                u = (int)quotient(at, steps + kStart);
                f = (int)(at - (long long)u * (steps + kStart));
                if (steps > kWholeStages) return raw;
                const int whole_from = f;
                f = 0;
                return raw - whole_from;
            };
            int i, u, f;
            if (raw_b >= base && raw_b < base + t) {
                wb = locate(raw_b, i, unit, from);
                const int4 r4 = t_req[i];
                b = b0 + i;
                rq.row0 = r4.x;
                rq.n = r4.y;
                rq.len = r4.z;
                wk = work_of<ROWS>(a, rq, R);
            }
            if (raw_e >= base && raw_e < base + t) we = locate(raw_e, i, u, f);
            base += t;
        }
        if (lane == 0) s_bound[warp] = wb;
        if (threadIdx.x == kThreads - 1) s_bound[kWarps] = we;
    }
    __syncthreads();
    const long long begin = s_bound[0], end = s_bound[kWarps];
    long long pos = wb;
    const uint32_t ring = smem_addr(smem) + (uint32_t)warp * STAGES * S::kBytes;
    float *own = reinterpret_cast<float *>(smem + (size_t)warp * STAGES * S::kBytes);   // when the warp is done
    const uint32_t q_s = smem_addr(smem) + kWarps * STAGES * S::kBytes + warp * NB * J * 512;   // query pieces
    if (lane < 2) s.seg[2 * warp + lane] = Segment{-1, 0, 0, 0, 0, 0};
    // this lane's places in a stage: keys, values (the keys of rows 2c and 2c + 1), scales
    const int ka0 = key_of_row(g), vk0 = c, vk1 = 4 + (c ^ 3);
    const uint32_t kof = J == 8   ? ka0 * 128 + (((2 * c) ^ swizzle<J>(ka0)) << 4)
                         : J == 4 ? ka0 * 64 + ((c ^ swizzle<J>(ka0)) << 4)
                                  : ka0 * 16 * J + 4 * J * c;
    auto v_place = [&](int key) -> uint32_t {
        return S::kCodes + key * 16 * J +
               (J == 8   ? (g ^ swizzle<J>(key)) << 4
                : J == 4 ? (((g >> 1) ^ swizzle<J>(key)) << 4) + (g & 1) * 8
                         : 2 * J * g);
    };
    const uint32_t vof0 = v_place(vk0), vof1 = v_place(vk1);
    const uint32_t sof = 2 * S::kCodes + ka0 * 8 * G;
    // where this lane's first 16-byte piece of 16 rows goes (the next ones 512 bytes on)
    const uint32_t pof = (lane / J) * 16 * J + (((lane % J) ^ swizzle<J>(lane / J)) << 4);
    const int shift = 31 - __clz(a.c.page_size);
    // stretches of 16 rows (640 bytes or more each): a pool holds fewer than 2^32
    const uint32_t page_stretches = (uint32_t)H * (uint32_t)(a.c.page_size >> 4), page_mask = a.c.page_size - 1;
    const uint32_t n_pages = (uint32_t)a.c.n_pages;
    while (pos < we) {
        // its share of the unit: a start of kStart, then the stages
        const int length = wk.steps + kStart, upto = (int)min((long long)length, from + (we - pos));
        const int from_stage = max(from - kStart, 0), iters = max(upto - kStart, 0) - from_stage;
        if (iters == 0) {                                      // the range ends within the start
            pos += upto - from;
            continue;
        }
        const int h = unit / wk.blocks, rb = unit - h * wk.blocks;
        const int rows_all = rq.n * R;
        // keys that some row of the block sees; keys that all of its rows see
        const int row_hi = min(rb * ROWS + ROWS, rows_all) - 1;
        const bool one = rq.n == 1;                            // every row is token 0's
        const int see_hi = rq.len - rq.n + (one ? 0 : row_hi / R);                      // inclusive
        const int all_hi = rq.len - rq.n + (one ? 0 : rb * ROWS / R);
        const int see_lo = attn_first(a, max(all_hi, -1)), all_lo = attn_first(a, see_hi);

        const int32_t *table = a.page_table + (size_t)b * a.max_pages;
        const int key00 = (wk.step0 + from_stage) * kStageKeys;
        // this lane's first 16-byte piece of a page's rows of this head
        const size_t head_row = (size_t)h * a.c.page_size;
        const char *k_at = reinterpret_cast<const char *>(a.c.Kq) + head_row * (D / 2) + 16 * lane;
        const char *v_at = reinterpret_cast<const char *>(a.c.Vq) + head_row * (D / 2) + 16 * lane;
        const char *ks_at = reinterpret_cast<const char *>(a.c.K_sz) + head_row * (8 * G);
        const char *vs_at = reinterpret_cast<const char *>(a.c.V_sz) + head_row * (8 * G);
        // the two pages (16 keys each) of iteration i; -1 where nothing is seen
        auto pages_of = [&](int i) {
            int2 pg = make_int2(-1, -1);
            if (i < iters) {
                const int k0 = key00 + i * kStageKeys;
                if (k0 <= see_hi && k0 + 16 > see_lo) pg.x = __ldg(table + (k0 >> shift));
                if (k0 + 16 <= see_hi && k0 + 32 > see_lo) pg.y = __ldg(table + ((k0 + 16) >> shift));
            }
            return pg;
        };
        auto issue = [&](int i, int slot, int2 pg) {
            const int k0 = key00 + i * kStageKeys;
            if (i < iters && k0 <= see_hi && k0 + 32 > see_lo) {
                const uint32_t st = ring + (uint32_t)slot * S::kBytes;
                const bool ok[2] = {(uint32_t)pg.x < n_pages, (uint32_t)pg.y < n_pages};
                // the two stretches of 16 rows, in the order of the pool
                const uint32_t at[2] = {(uint32_t)pg.x * page_stretches + (((uint32_t)k0 & page_mask) >> 4),
                                        (uint32_t)pg.y * page_stretches + (((uint32_t)(k0 + 16) & page_mask) >> 4)};
                auto codes = [&](int x) {                      // 16 J pieces, contiguous
                    const char *ks = k_at + (uint64_t)at[x] * (8 * D), *vp = v_at + (uint64_t)at[x] * (8 * D);
#pragma unroll
                    for (int j = 0; j < (16 * J + 31) / 32; ++j) {
                        uint32_t dst = st + x * 256 * J;
                        dst += J % 2 == 0 ? pof + 512 * j : (32 * j + lane) * 16;   // (odd J: no swizzle)
                        if (J % 2 == 0 || 32 * j + lane < 16 * J) {
                            cp_async_16(dst, ks + 512 * j);
                            cp_async_16(dst + S::kCodes, vp + 512 * j);
                        }
                    }
                };
                auto scales = [&](auto use) {                  // 16 G pieces each side
#pragma unroll
                    for (int j = 0; j < G; ++j) {
                        const int piece = 32 * j + lane;
                        const int side = piece >= 16 * G, pc = piece - side * 16 * G;
                        const int x = pc >= 8 * G;
                        use(x, st + 2 * S::kCodes + piece * 16,
                            (side ? vs_at : ks_at) + (uint64_t)(x ? at[1] : at[0]) * (128 * G) + (pc - x * 8 * G) * 16);
                    }
                };
                if (ok[0] && ok[1]) {                          // as nearly always: no more questions
                    codes(0);
                    codes(1);
                    scales([](int, uint32_t dst, const char *src) { cp_async_16(dst, src); });
                } else {
                    if (ok[0]) codes(0);
                    if (ok[1]) codes(1);
                    scales([&](int x, uint32_t dst, const char *src) {
                        if (x ? ok[1] : ok[0]) {
                            cp_async_16(dst, src);
                        } else if (x ? k0 + 16 <= see_hi && k0 + 32 > see_lo : k0 <= see_hi && k0 + 16 > see_lo) {
                            // a page outside the pool: NaN rows
                            const float nan = quiet_nan();
                            asm volatile("st.shared.v4.f32 [%0], {%1,%1,%1,%1};" ::"r"(dst), "f"(nan) : "memory");
                            atomicOr(&g_attn_error, kAttnBadRequest);
                        }
                    });
                }
            }
            cp_async_commit();
        };
        // ---- the query rows' values and the first keys on their way ----
        int2 pg = pages_of(0);
        float x[NB][J][8];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const int rho = rb * ROWS + nb * 4 + (g >> 1);     // the row this thread's column holds
            const bool in = rho < rows_all;
            const int j = in && !one ? rho / R : 0, r = in ? rho - j * R : 0;
            const float *q = a.q + (size_t)(rq.row0 + j) * a.ldq + (size_t)(h * R + r) * D + 8 * c;
#pragma unroll
            for (int u = 0; u < J; ++u) {
                float4 v0 = make_float4(0.f, 0.f, 0.f, 0.f), v1 = v0;
                if (in) {
                    v0 = __ldg(reinterpret_cast<const float4 *>(q + 32 * u));
                    v1 = __ldg(reinterpret_cast<const float4 *>(q + 32 * u) + 1);
                }
                x[nb][u][0] = v0.x; x[nb][u][1] = v0.y; x[nb][u][2] = v0.z; x[nb][u][3] = v0.w;
                x[nb][u][4] = v1.x; x[nb][u][5] = v1.y; x[nb][u][6] = v1.z; x[nb][u][7] = v1.w;
            }
        }
#pragma unroll
        for (int i = 0; i < STAGES - 1; ++i) {
            const int2 nx = pages_of(i + 1);
            issue(i, i, pg);
            pg = nx;
        }

        // ---- the query rows as two fp16 pieces, scaled by a power of two per
        // row, in shared memory ----
        __syncwarp();
        float qs[NB][G], F[NB];                                // of row c: sums per group, factor
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            float big = 0.0f;
#pragma unroll
            for (int u = 0; u < J; ++u)
#pragma unroll
                for (int i = 0; i < 8; ++i) big = fmaxf(big, fabsf(x[nb][u][i]));
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
            // 2^k times the row lies in [2^21, 2^22) at its largest
            const int e = (int)((__float_as_uint(big) >> 23) & 255u);
            const int k = big > 0.0f ? min(21 + 127 - e, 120) : 0;
            const float up = exp2f((float)k);
            float sum[G];
#pragma unroll
            for (int gr = 0; gr < G; ++gr) sum[gr] = 0.0f;
            const bool lo = g & 1;
#pragma unroll
            for (int u = 0; u < J; ++u) {
                uint32_t f[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float z[2];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float v = rintf(x[nb][u][i + 4 * y] * up);
                        const float hi = rintf(v * (1.0f / kRadix));
                        sum[u / UG] += v;
                        // odd nibbles are masked at 16 times their value
                        z[y] = (lo ? fmaf(-kRadix, hi, v) : hi) * ((i & 1) ? 0.0625f : 1.0f);
                    }
                    const __half2 pr = __floats2half2_rn(z[0], z[1]);
                    f[i] = *reinterpret_cast<const uint32_t *>(&pr);
                }
                asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(q_s + ((nb * J + u) * 32 + lane) * 16),
                             "r"(f[0]), "r"(f[1]), "r"(f[2]), "r"(f[3])
                             : "memory");
            }
#pragma unroll
            for (int gr = 0; gr < G; ++gr) {
                float t = sum[gr];
                t += __shfl_xor_sync(0xffffffffu, t, 1);
                t += __shfl_xor_sync(0xffffffffu, t, 2);
                qs[nb][gr] = __shfl_sync(0xffffffffu, t, 8 * c) * 0x1p-24f;
            }
            F[nb] = ldexpf(a.scale * kLog2e, 24 - __shfl_sync(0xffffffffu, k, 8 * c));
        }
        __syncwarp();
        int last[NB], first[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const int rc = rb * ROWS + nb * 4 + c;
            last[nb] = rc < rows_all ? rq.len - rq.n + (one ? 0 : rc / R) : -1;
            first[nb] = attn_first(a, last[nb]);
        }

        // o: f32 sums; t: the tensor core's, added to o every kCarry stages
        float o[NB][J][4], t0[NB][J][4], t1[NB][J][4], zs[NB][G], l[NB], m[NB];
        int carried = 0;
        float vs[NB];                                          // a row's 2^(11 - E), E by the values that it sees
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            vs[nb] = 0x1p111f;
            l[nb] = 0.0f;
            m[nb] = -INFINITY;
#pragma unroll
            for (int gr = 0; gr < G; ++gr) zs[nb][gr] = 0.0f;
#pragma unroll
            for (int u = 0; u < J; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[nb][u][i] = t0[nb][u][i] = t1[nb][u][i] = 0.0f;
        }

        int slot = 0, fill = STAGES - 1;
        for (int i = 0; i < iters; ++i) {
            {
                const int2 nx = pages_of(i + STAGES);
                issue(i + STAGES - 1, fill, pg);
                pg = nx;
                if (++fill == STAGES) fill = 0;
            }
            cp_async_wait<STAGES - 1>();
            __syncwarp();
            const int k0 = key00 + i * kStageKeys;
            const uint32_t st = ring + (uint32_t)slot * S::kBytes;
            if (++slot == STAGES) slot = 0;
            if (k0 > see_hi || k0 + kStageKeys <= see_lo) continue;   // uniform in the warp

            // ---- exponents: keys times query rows ----
            float w[2][2][NB];                                 // [16 keys][key row g, g + 8][row]
            {
                uint32_t wa[2][J], wb[2][J];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    load_key<J>(st + kof + 256 * J * x, wa[x]);
                    load_key<J>(st + kof + 256 * J * x + 128 * J, wb[x]);
                }
                float acc[2][NB][4];
#pragma unroll
                for (int u = 0; u < J; ++u) {
                    uint32_t qf[NB][4];
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
                        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                                     : "=r"(qf[nb][0]), "=r"(qf[nb][1]), "=r"(qf[nb][2]), "=r"(qf[nb][3])
                                     : "r"(q_s + ((nb * J + u) * 32 + lane) * 16));
                    const uint32_t m0 = 0x000F000Fu, m1 = 0x00F000F0u;
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint32_t va = wa[x][u], vb = wb[x][u], ha = va >> 8, hb = vb >> 8;
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) {
                            if (u % UG == 0)
                                mma16816_zero(acc[x][nb], va & m0, vb & m0, va & m1, vb & m1, qf[nb][0], qf[nb][1]);
                            else
                                mma16816(acc[x][nb], va & m0, vb & m0, va & m1, vb & m1, qf[nb][0], qf[nb][1]);
                            mma16816(acc[x][nb], ha & m0, hb & m0, ha & m1, hb & m1, qf[nb][2], qf[nb][3]);
                        }
                        if (u % UG == UG - 1) {
                            const int gr = u / UG;
                            const float2 sa = lds_f2(st + sof + (16 * x * G + gr) * 8);
                            const float2 sb = lds_f2(st + sof + ((16 * x + 8) * G + gr) * 8);
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb) {
                                const float ta = fmaf(-sa.y, qs[nb][gr], fmaf(kRadix, acc[x][nb][0], acc[x][nb][1]));
                                const float tb = fmaf(-sb.y, qs[nb][gr], fmaf(kRadix, acc[x][nb][2], acc[x][nb][3]));
                                w[x][0][nb] = gr == 0 ? sa.x * ta : fmaf(sa.x, ta, w[x][0][nb]);
                                w[x][1][nb] = gr == 0 ? sb.x * tb : fmaf(sb.x, tb, w[x][1][nb]);
                            }
                        }
                    }
                }
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        w[x][0][nb] *= F[nb];
                        w[x][1][nb] *= F[nb];
                    }
            }

            // ---- values' scales; what a row does not see ----
            float2 vz[2][2][G];
            bool ones = false;
            auto load_scales = [&] {
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int y = 0; y < 2; ++y)
#pragma unroll
                        for (int gr = 0; gr < G; ++gr) {
                            vz[x][y][gr] = lds_f2(st + sof + S::kSz + ((16 * x + 8 * y) * G + gr) * 8);
                            ones |= vz[x][y][gr].x == 1.0f;
                        }
            };
            load_scales();
            if (__any_sync(0xffffffffu, ones)) {               // rare
                fit_equal_values<J, G>(st);
                load_scales();
            }
            const bool masked = k0 + kStageKeys - 1 > all_hi || k0 < all_lo;   // uniform
            uint32_t hidden = 0;                               // bit (x, y, nb)
            if (masked) {
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int y = 0; y < 2; ++y)
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) {
                            const int key = k0 + 16 * x + ka0 + 8 * y;
                            if (key > last[nb] || key < first[nb]) {
                                hidden |= 1u << ((x * 2 + y) * NB + nb);
                                w[x][y][nb] = -INFINITY;
                            }
                        }
                // scales of keys that none of this thread's rows sees may be rubbish
                constexpr uint32_t kAllRows = (1u << NB) - 1u;
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        if (((hidden >> ((x * 2 + y) * NB)) & kAllRows) == kAllRows) {
#pragma unroll
                            for (int gr = 0; gr < G; ++gr) vz[x][y][gr] = make_float2(0.0f, 0.0f);
                        }
            }
            // ---- the references m and E still hold? ----
            float top[NB], vtop = 0.0f;
            bool move = false;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                top[nb] = fmaxf(fmaxf(w[0][0][nb], w[0][1][nb]), fmaxf(w[1][0][nb], w[1][1][nb]));
                move |= top[nb] > m[nb] + kSlack;
            }
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int gr = 0; gr < G; ++gr) vtop = fmaxf(vtop, fabsf(vz[x][y][gr].x));
            move |= vtop * (NB == 1 ? vs[0] : fmaxf(vs[0], vs[NB - 1])) > (float)(1 << kPieceBits);   // vtop > 2^E
            if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    float t = top[nb];
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
                    const float mn = fmaxf(m[nb], t);
                    const float f = mn > m[nb] ? exp2_approx(m[nb] - mn) : 1.0f;
                    m[nb] = mn;
                    l[nb] *= f;
                    float vt = vtop;
                    if (NB > 1 && masked) {                    // (one row per thread: what it does not see is 0 already)
                        vt = 0.0f;
#pragma unroll 1
                        for (int xy = 0; xy < 4; ++xy)
#pragma unroll
                            for (int gr = 0; gr < G; ++gr)
                                if (!((hidden >> (xy * NB + nb)) & 1u))
                                    vt = fmaxf(vt, fabsf(lds_f2(st + sof + S::kSz + (8 * xy * G + gr) * 8).x));
                    }
                    vt = fmaxf(vt, __shfl_xor_sync(0xffffffffu, vt, 4));
                    vt = fmaxf(vt, __shfl_xor_sync(0xffffffffu, vt, 8));
                    vt = fmaxf(vt, __shfl_xor_sync(0xffffffffu, vt, 16));
                    float fv = 1.0f;
                    const float vref = (float)(1 << kPieceBits) * inverse_power(vs[nb]);
                    if (vt > vref) {
                        const int e = min((int)(__float_as_uint(vt) >> 23) - 126, 127);   // vt < 2^e
                        vs[nb] = __uint_as_float((uint32_t)(127 + kPieceBits - e) << 23);
                        fv = vref * (vs[nb] * (1.0f / (1 << kPieceBits)));
                    }
                    const float fo = f * fv;
#pragma unroll
                    for (int gr = 0; gr < G; ++gr) zs[nb][gr] *= fo;
#pragma unroll
                    for (int u = 0; u < J; ++u)
#pragma unroll
                        for (int i4 = 0; i4 < 4; ++i4) {
                            o[nb][u][i4] *= fo;
                            t0[nb][u][i4] *= fo;
                            t1[nb][u][i4] *= fo;
                        }
                }
            }

            // ---- weights, and the second product group by group ----
            const uint32_t magic = 0x64006400u;   // 1024 in each half
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const float ref = m[nb] == -INFINITY ? 0.0f : m[nb];
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        w[x][y][nb] = exp2_approx(w[x][y][nb] - ref);
                        l[nb] += w[x][y][nb];
                        w[x][y][nb] *= vs[nb];
                    }
            }
            Halves<J> hv[2][4];
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    hv[x][k] = load_halves<J>(st + ((k & 1) ? vof1 : vof0) + (16 * x + 4 * (k & 2)) * 16 * J);
#pragma unroll
            for (int gr = 0; gr < G; ++gr) {
                uint32_t pf[NB][2][2];
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            // (one row per thread: its hidden keys have scale 0 already)
                            const bool hid = NB > 1 && masked && ((hidden >> ((x * 2 + y) * NB + nb)) & 1u);
                            const float ps = hid ? 0.0f : w[x][y][nb] * vz[x][y][gr].x;
                            zs[nb][gr] = hid ? zs[nb][gr] : fmaf(ps, vz[x][y][gr].y - 8.0f, zs[nb][gr]);
                            pf[nb][x][y] = transpose8x8(two_pieces(ps));
                        }
#pragma unroll
                for (int uu = 0; uu < UG; ++uu) {
                    const int u = gr * UG + uu;
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint32_t sel = (u & 1) ? 0x7632u : 0x5410u;
                        const uint32_t x01 = __byte_perm(hv[x][0].r[u / 2], hv[x][1].r[u / 2], sel);
                        const uint32_t x23 = __byte_perm(hv[x][2].r[u / 2], hv[x][3].r[u / 2], sel);
                        const uint32_t y01 = x01 >> 8, y23 = x23 >> 8;
                        const uint32_t m8 = 0xE408E408u;      // -(1024 + 8) in each half
                        const uint32_t s16 = 0x2C002C00u;     // 1/16
                        const uint32_t m72 = 0xD480D480u;     // -72: (1024 + 16 c)/16 - 72 = c - 8
                        const uint32_t a0 = h2_add(mask_or<0x000F000Fu>(x01, magic), m8);
                        const uint32_t a1 = h2_fma(mask_or<0x00F000F0u>(x01, magic), s16, m72);
                        const uint32_t a2 = h2_add(mask_or<0x000F000Fu>(x23, magic), m8);
                        const uint32_t a3 = h2_fma(mask_or<0x00F000F0u>(x23, magic), s16, m72);
                        const uint32_t b0 = h2_add(mask_or<0x000F000Fu>(y01, magic), m8);
                        const uint32_t b1 = h2_fma(mask_or<0x00F000F0u>(y01, magic), s16, m72);
                        const uint32_t b2 = h2_add(mask_or<0x000F000Fu>(y23, magic), m8);
                        const uint32_t b3 = h2_fma(mask_or<0x00F000F0u>(y23, magic), s16, m72);
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) {
                            mma16816(t0[nb][u], a0, a1, a2, a3, pf[nb][x][0], pf[nb][x][1]);
                            mma16816(t1[nb][u], b0, b1, b2, b3, pf[nb][x][0], pf[nb][x][1]);
                        }
                    }
                }
            }
            if (++carried == kCarry) {
                carried = 0;
                carry<NB, J>(o, t0, t1);
            }
            __syncwarp();   // the stage is read: the next copies may land in it
        }
        cp_async_wait<0>();
        __syncwarp();
        carry<NB, J>(o, t0, t1);

        // ---- a whole unit is finished; the sums of a cut one go to the CTA's join ----
        const bool whole = iters == wk.steps, done = pos + (upto - from) >= we;
        float *to = done ? own : p.head + ((size_t)blockIdx.x * kWarps + warp) * kSums;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            float lt = l[nb];
            lt += __shfl_xor_sync(0xffffffffu, lt, 4);
            lt += __shfl_xor_sync(0xffffffffu, lt, 8);
            lt += __shfl_xor_sync(0xffffffffu, lt, 16);
            const int row = nb * 4 + c, rho = rb * ROWS + row;
            float back = inverse_power(vs[nb]);
            if (whole) {
                back *= m[nb] == -INFINITY ? 0.0f : 1.0f / lt;
                const int j = rho / R, r = rho - j * R;
                to = a.out + (size_t)(rq.row0 + j) * a.ldo + (size_t)(h * R + r) * D - row * D;
            } else if (g == 0) {
                to[ROWS * D + 2 * row] = m[nb];
                to[ROWS * D + 2 * row + 1] = lt;
            }
#pragma unroll
            for (int gr = 0; gr < G; ++gr) {
                zs[nb][gr] += __shfl_xor_sync(0xffffffffu, zs[nb][gr], 4);
                zs[nb][gr] += __shfl_xor_sync(0xffffffffu, zs[nb][gr], 8);
                zs[nb][gr] += __shfl_xor_sync(0xffffffffu, zs[nb][gr], 16);
            }
            if (!whole || rho < rows_all) {
#pragma unroll
                for (int u = 0; u < J; ++u) {
                    const float z = zs[nb][u / UG];
                    *reinterpret_cast<float4 *>(to + row * D + 32 * u + 4 * g) =
                        make_float4((o[nb][u][0] - z) * back, (o[nb][u][1] - z) * back, (o[nb][u][2] - z) * back,
                                    (o[nb][u][3] - z) * back);
                }
            }
        }
        if (!whole && lane == 0)
            s.seg[2 * warp + (done ? 1 : 0)] = Segment{pos - from, length, rq.row0, rows_all, h, rb};

        pos += upto - from;
        from = 0;
        if (upto == length && ++unit == wk.blocks * H && pos < we) {
            unit = 0;
            do {                                               // the next request with work
                ++b;
                rq = attn_request(a, b);
                wk = work_of<ROWS>(a, rq, R);
            } while (wk.total == 0);
        }
    }
    __syncthreads();

    // ---- the warps' segments of one unit joined, in order ----
    const long long start_of = lane < 2 * kWarps ? s.seg[lane].start : -1;
    uint32_t left = __ballot_sync(0xffffffffu, start_of >= 0);
    while (left) {
        const Segment seg = s.seg[__ffs(left) - 1];
        const uint32_t mine_of = __ballot_sync(0xffffffffu, start_of == seg.start);
        left &= ~mine_of;
        const long long first = seg.start + kStart;            // its first stage
        const bool whole = first >= begin && seg.start + seg.length <= end;
        const int slot = first > begin ? 1 : 0;
        float *part = p.part + ((size_t)blockIdx.x * 2 + slot) * kSums;
        for (int i = threadIdx.x; i < ROWS * D / 4; i += kThreads) {
            const int row = i / (D / 4), d = 4 * (i - row * (D / 4));
            const int rho = seg.rb * ROWS + row;
            if (rho >= seg.rows) continue;
            auto sums_of = [&](int e) {
                return e & 1 ? reinterpret_cast<const float *>(smem + (size_t)(e >> 1) * STAGES * S::kBytes)
                             : p.head + ((size_t)blockIdx.x * kWarps + (e >> 1)) * kSums;
            };
            float2 ml[2 * kWarps];
            float4 t[2 * kWarps];
            float mt = -INFINITY;
#pragma unroll
            for (int e = 0; e < 2 * kWarps; ++e) {
                ml[e] = make_float2(-INFINITY, 0.0f);
                t[e] = make_float4(0.f, 0.f, 0.f, 0.f);
                if ((mine_of >> e) & 1u) {
                    ml[e] = *reinterpret_cast<const float2 *>(sums_of(e) + ROWS * D + 2 * row);
                    t[e] = *reinterpret_cast<const float4 *>(sums_of(e) + row * D + d);
                }
                mt = fmaxf(mt, ml[e].x);
            }
            const float ref = mt == -INFINITY ? 0.0f : mt;
            float lt = 0.0f;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 2 * kWarps; ++e) {
                const float f = exp2_approx(ml[e].x - ref);
                lt = fmaf(f, ml[e].y, lt);
                v.x = fmaf(f, t[e].x, v.x);
                v.y = fmaf(f, t[e].y, v.y);
                v.z = fmaf(f, t[e].z, v.z);
                v.w = fmaf(f, t[e].w, v.w);
            }
            if (whole) {
                const int j = rho / R, r = rho - j * R;
                const float inv = mt == -INFINITY ? 0.0f : 1.0f / lt;
                *reinterpret_cast<float4 *>(a.out + (size_t)(seg.row0 + j) * a.ldo + (size_t)(seg.h * R + r) * D + d) =
                    make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
            } else {
                *reinterpret_cast<float4 *>(part + (size_t)row * D + d) = v;
                if (d == 0) {
                    part[ROWS * D + 2 * row] = mt;
                    part[ROWS * D + 2 * row + 1] = lt;
                }
            }
        }
        if (threadIdx.x == 0 && !whole && first >= begin) {
            // the unit starts here and goes on in the CTAs up to the one that holds its last stage
            const int last_cta = (int)((uint64_t)(seg.start + seg.length - 1) / (uint64_t)chunk);
            p.desc[2 * blockIdx.x] = make_int4(seg.row0, seg.rows, seg.h, seg.rb);
            p.desc[2 * blockIdx.x + 1] = make_int4(last_cta, slot, 0, 0);
        }
    }
}

// Joins the partial sums of the units that were cut, one CTA for each CTA of
// the first kernel.  J, G: also computes the rows that the prompt kernel left
// (0: there are none).
template <int ROWS, int J, int G>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const __grid_constant__ SplitParams p, int D)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if constexpr (J > 0) {
        // a thread looks at one tile in gridDim.x at a time
        __shared__ ApartShared<J> s;
        for (long long n0 = blockIdx.x; n0 < p.a.n_apart; n0 += (long long)kJoinThreads * gridDim.x) {   // uniform
            const long long n = n0 + (long long)threadIdx.x * gridDim.x;
            bool some = false;
            if (n < p.a.n_apart) {
                const uint4 *at = reinterpret_cast<const uint4 *>(p.a.apart + n);
                const uint4 rows = __ldcg(at), more = __ldcg(at + 1);
                some = (rows.x | rows.y | rows.z | rows.w | more.z) != 0;
            }
            if (!__syncthreads_or(some)) continue;
            for (int x = 0; x < kJoinThreads && n0 + (long long)x * gridDim.x < p.a.n_apart; ++x) {
                const long long m = n0 + (long long)x * gridDim.x;
                const ApartTile &at = p.a.apart[m];
                if ((at.rows[0] | at.rows[1] | at.rows[2] | at.rows[3] | (uint32_t)at.uneven) != 0)
                    apart_rows<J, G>(p.a, at, (int)(m % p.a.c.kv_heads), s);
            }
        }
    }
    const int4 u = __ldcg(p.desc + 2 * blockIdx.x), d = __ldcg(p.desc + 2 * blockIdx.x + 1);
    if (d.x < 0) return;
    const AttnCall &a = p.a;
    const int R = p.R, rows = u.y, h = u.z, rb = u.w;
    const size_t per = (size_t)ROWS * (D + 2);
    auto part_of = [&](int cta) {
        return p.part + ((size_t)cta * 2 + (cta == (int)blockIdx.x ? d.y : 0)) * per;
    };
    for (int i = threadIdx.x; i < ROWS * D / 4; i += kJoinThreads) {
        const int row = i / (D / 4), dd = 4 * (i - row * (D / 4));
        const int rho = rb * ROWS + row;
        if (rho >= rows) continue;
        float m = -INFINITY, l = 0.0f;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        constexpr int kAhead = 8;    // partial sums on their way at once
        for (int cta0 = blockIdx.x; cta0 <= d.x; cta0 += kAhead) {
            float2 ml[kAhead];
            float4 t[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                ml[k] = make_float2(-INFINITY, 0.0f);
                t[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (cta0 + k <= d.x) {
                    const float *pt = part_of(cta0 + k);
                    ml[k] = __ldcg(reinterpret_cast<const float2 *>(pt + (size_t)ROWS * D + 2 * row));
                    t[k] = __ldcg(reinterpret_cast<const float4 *>(pt + (size_t)row * D + dd));
                }
            }
            float mn = m;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) mn = fmaxf(mn, ml[k].x);
            const float ref = mn == -INFINITY ? 0.0f : mn;
            const float fo = exp2_approx(m - ref);
            l *= fo;
            s.x *= fo;
            s.y *= fo;
            s.z *= fo;
            s.w *= fo;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const float fn = exp2_approx(ml[k].x - ref);
                l = fmaf(fn, ml[k].y, l);
                s.x = fmaf(fn, t[k].x, s.x);
                s.y = fmaf(fn, t[k].y, s.y);
                s.z = fmaf(fn, t[k].z, s.z);
                s.w = fmaf(fn, t[k].w, s.w);
            }
            m = mn;
        }
        const int j = rho / R, r = rho - j * R;
        const float inv = m == -INFINITY ? 0.0f : 1.0f / l;
        *reinterpret_cast<float4 *>(a.out + (size_t)(u.x + j) * a.ldo + (size_t)(h * R + r) * D + dd) =
            make_float4(s.x * inv, s.y * inv, s.z * inv, s.w * inv);
    }
}

template <int J, int G, int NB>
cudaError_t launch_split(const AttnCall &call, cudaStream_t stream)
{
    // four query rows and heads of up to 128: registers and shared memory for
    // two CTAs per SM; otherwise one
    constexpr int MINB = NB * J <= 4 ? 2 : 1;
    constexpr int kQ = kWarps * NB * J * 512;
    constexpr int room = (MINB == 2 ? 112 * 1024 : 216 * 1024) - kQ;
    constexpr int fit = room / (kWarps * Stage<J, G>::kBytes);
    constexpr int STAGES = fit < 2 ? 2 : fit > 4 ? 4 : fit;
    static_assert(STAGES * Stage<J, G>::kBytes >= 4 * NB * (32 * J + 2) * 4, "the sums fit the ring");
    auto kern = attn_split_kernel<J, G, NB, STAGES, MINB>;
    constexpr int smem = kWarps * STAGES * Stage<J, G>::kBytes + kQ;
    int dev = 0, sms = 0;
    cudaError_t err;
    if ((err = cudaGetDevice(&dev)) != cudaSuccess) return err;
    static std::atomic<int> ready_dev{-1};
    if (ready_dev.load(std::memory_order_acquire) != dev) {
        if ((err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess)
            return err;
        ready_dev.store(dev, std::memory_order_release);
    }
    if ((err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return err;
    SplitParams p{};
    p.a = call;
    // a stage for every warp at the least
    const int R = call.heads / call.c.kv_heads;
    const long long steps = (call.max_len + kStageKeys - 1) / kStageKeys;
    const long long most_n = call.max_query < call.T ? call.max_query : call.T;
    const long long blocks = (most_n * R + 4 * NB - 1) / (4 * NB);
    const long long units = (call.B < call.T ? call.B : call.T) * blocks * call.c.kv_heads;
    long long grid = (long long)sms * MINB;
    if (grid > kMaxGrid / 2 * MINB) grid = kMaxGrid / 2 * MINB;
    if (grid > (units * steps + kWarps - 1) / kWarps) grid = (units * steps + kWarps - 1) / kWarps;
    if (grid < 1) grid = 1;
    p.grid = (int)grid;
    p.R = R;
    p.desc = static_cast<int4 *>(call.workspace);
    p.part = reinterpret_cast<float *>(static_cast<char *>(call.workspace) + 2 * kMaxGrid * sizeof(int4));
    p.head = p.part + (size_t)grid * 2 * 4 * NB * (32 * J + 2);
    kern<<<(unsigned)grid, kThreads, smem, stream>>>(p);
    if ((err = cudaGetLastError()) != cudaSuccess || ((steps <= kWholeStages || grid <= 1) && call.n_apart == 0))
        return err;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if constexpr (J <= 4)
        if (call.n_apart > 0) return cudaLaunchKernelEx(&cfg, attn_join_kernel<4 * NB, J, G>, p, (int)(32 * J));
    return cudaLaunchKernelEx(&cfg, attn_join_kernel<4 * NB, 0, 0>, p, (int)(32 * J));
}

template <int J, int G>
cudaError_t launch_rows(const AttnCall &call, cudaStream_t stream)
{
    const long long rows = (long long)call.max_query * (call.heads / call.c.kv_heads);
    // 8 rows of 256 values do not fit a thread's registers: blocks of 4 instead
    if constexpr (J < 8)
        if (rows > 4) return launch_split<J, G, 2>(call, stream);
    return launch_split<J, G, 1>(call, stream);
}

}  // namespace

namespace {

// Requests of at least so many query rows per kv head, and calls of so many
// rows in all, are the prompt kernel's.
constexpr int kPromptRows = 48, kPromptTotal = 5120;

// The prompt kernel's CTAs: as many row tiles as its requests can have
// together, per kv head.
long long prompt_ctas(int B, int T, int heads, int kv_heads)
{
    const long long rows = (long long)T * (heads / kv_heads), most = rows / kPromptRows;
    return ((rows + kPromptTile - 1) / kPromptTile + (B < most ? B : most)) * kv_heads;
}

size_t sums_bytes(int D)
{
    // rows of sums of all CTAs: 304 of 8 rows at 64 dims, above that 304 of 4 or 152 of 8
    const size_t rows = D <= 64 ? kMaxGrid * 8 : kMaxGrid * 4;
    return 2 * kMaxGrid * sizeof(int4) + rows * (2 + kWarps) * (size_t)(D + 2) * sizeof(float);
}

}  // namespace

size_t attn_workspace_bytes(int T, int heads, int kv_heads, int D)
{
    static_assert(sizeof(ApartTile) == 32, "a multiple of 16 bytes");
    return sums_bytes(D) + (size_t)prompt_ctas(GQ4_MAX_REQUESTS, T, heads, kv_heads) * sizeof(ApartTile);
}

cudaError_t launch_attn(const AttnCall &in, cudaStream_t stream)
{
    // Requests of many query rows go to the prompt kernel, whose tiles hold
    // 128 rows, if there are enough rows in all to fill its CTAs.  Measured
    // with 4096 keys and more behind 32 heads over 8 of 128, one group:
    // 16 requests of 8 tokens (32 rows each, 4096 in all) 88 us there and 83
    // here, of 12 (48, 6144) 88 and 116, of 16 89 and 150; one request of 64
    // tokens (256, 2048) 90 and 50.  Four groups: of 12 169 and 150, of 16
    // 170 and 197.  (Measured at this shape only; with four groups the border
    // lies somewhat higher, and few rows behind a long past leave SMs idle.)
    AttnCall call = in;
    const long long R = call.heads / call.c.kv_heads;
    const bool prompt = prompt_path_supported(call) && call.max_query * R >= kPromptRows &&
                        (long long)call.T * call.heads >= kPromptTotal;
    call.prompt_rows = prompt ? kPromptRows : 0x7fffffff;
    call.apart = reinterpret_cast<ApartTile *>(static_cast<char *>(call.workspace) + sums_bytes(call.c.head_dim));
    call.n_apart = prompt ? prompt_ctas(call.B, call.T, call.heads, call.c.kv_heads) : 0;
    if (prompt) {
        const cudaError_t err = launch_attn_prompt(call, stream);
        if (err != cudaSuccess) return err;
    }
    const int G = call.c.head_dim / call.c.group_size;
    switch (call.c.head_dim * 16 + G) {
    case 64 * 16 + 1: return launch_rows<2, 1>(call, stream);
    case 64 * 16 + 2: return launch_rows<2, 2>(call, stream);
    case 96 * 16 + 1: return launch_rows<3, 1>(call, stream);
    case 96 * 16 + 3: return launch_rows<3, 3>(call, stream);
    case 128 * 16 + 1: return launch_rows<4, 1>(call, stream);
    case 128 * 16 + 2: return launch_rows<4, 2>(call, stream);
    case 128 * 16 + 4: return launch_rows<4, 4>(call, stream);
    case 256 * 16 + 1: return launch_rows<8, 1>(call, stream);
    case 256 * 16 + 2: return launch_rows<8, 2>(call, stream);
    case 256 * 16 + 4: return launch_rows<8, 4>(call, stream);
    case 256 * 16 + 8: return launch_rows<8, 8>(call, stream);
    }
    return cudaErrorInvalidValue;
}

cudaError_t read_attn_device_error(unsigned int *bits, bool clear)
{
    unsigned int more = 0;
    cudaError_t err = read_prompt_device_error(&more, clear);
    if (err != cudaSuccess) return err;
    err = cudaMemcpyFromSymbol(bits, g_attn_error, sizeof(unsigned int));
    if (err != cudaSuccess) return err;
    *bits |= more;
    if (!clear) return err;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_attn_error, &zero, sizeof(unsigned int));
}

}  // namespace gq4
