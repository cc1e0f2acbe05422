// gq4_attn_prompt.cu -- causal attention over the paged 4-bit cache for
// requests with many query rows (prompts and chunks of prompts), on the
// 5th-generation tensor cores.
//
// A CTA takes 128 query rows of one kv head (tokens times the head's query
// heads, so that a dequantised key serves all of them) and walks the keys in
// tiles of 64:
//   S = Q K^T   (128 x 64, K dimension head_dim),   P = 2^(w - m),
//   O = O f + P V   (128 x head_dim, K dimension 64).
// Two forms, by the scale groups of a row.
//   One group (EXACT): the codes minus 8 are the operands, exact in fp16; the
// scale and zero of key j come off outside the product,
//   w_j = F_j S_j + G_j sum_d q_d,  F_j = scale log2(e) s_j,  G_j = -(z_j - 8) F_j,
//   O = sum_j (p_j s_j) (c_j - 8) - sum_j (p_j s_j)(z_j - 8),
// and Q and p s are two fp16 pieces (22 bits): two MMAs per product.
//   Several groups: the keys and values themselves, (c - z) s, are two pieces
// as well, x = xh + xl, and a product is xl yh + xh yl + xh yh: three MMAs, the
// small ones first.
// Powers of two keep the pieces inside fp16: one per CTA for Q, one per key
// for K (undone by F_j) and for V (undone in P, against the tile's largest).
// Query rows too small for their CTA's power, or whose values are for a tile's
// (some later row's are the large ones), are computed again in plain f32 by the
// call's last kernel (see apart_rows).
// The tensor core cuts its sums rather than rounding them, so a tile's P V
// starts at zero and is added to f32 registers.
//
// Warps: softmax (a thread per row; EXACT: two groups of 4 that take turns at
// the tiles, each with its own maximum), 8 that add the tiles' P V (a row and
// half of head_dim per thread), 1 that fetches the cache's codes, scales and
// zeros into shared memory by cp.async, 1 that makes the factors of its keys
// from them, 4 or 8 that turn the codes into the K and V operands, 2 of which
// a lane issues the MMAs of S and of P V (an MMA's operands cost its thread as
// much time as the MMA takes).  Tensor memory (512 columns): S in four slots,
// whose columns P takes over 16 by 16 as S is read, and the tile's O in two; K
// and V have three slots in shared memory (EXACT; else two), the cache as it
// is four (two).  S runs ahead of P V by as many tiles as it has slots.
// K is stored [key][d] (K-major), V [key][d] as well, which is the MN-major
// form of the second product's B operand: no transposition.
// Measured in a graph, 32 heads over 8 of 128: a prompt of 6007 tokens, one
// group, 664 us (296 GFLOP by the formula, 446 TFLOP/s; twice that in the MMAs,
// 0.46 of the measured bf16 peak); three chunks of 1021 tokens behind 1000 to
// 4096 with a window of 2048, four groups, 459 us (103 GFLOP, 224 TFLOP/s;
// three times that in the MMAs).  Bound by the latency and issue slots of the softmax, adding and
// dequantising warps (issue active in half of the cycles, the tensor pipe in a
// third): a tile takes 2150 cycles, its MMAs 1080; and a CTA starts and ends in
// 18 thousand, of which the queries are 6 and the rows' way out 5.  The roles
// fill the registers and share the instruction cache: code for rare cases costs
// 1 to 6 % here whether it runs or not, so it is the last kernel's.
#include <cuda_fp16.h>

#include <atomic>
#include <cstdint>

#include "gq4_attn.cuh"
#include "gq4_quant.cuh"
#include "gq4_tcgen05.cuh"

namespace gq4 {
namespace {

__device__ unsigned int g_prompt_error = 0;

constexpr int kRows = kPromptTile;
constexpr int kTile = kPromptKeys;
constexpr int kCoWarps = 8;
constexpr int kWarps = 24;                      // all
constexpr int kThreads = 32 * kWarps;
constexpr float kSlack = 4.0f;                  // log2 of how far a weight may pass the maximum
constexpr int kPieceBits = 11;                  // P is held times 2^11
constexpr int kSP = 4;                          // slots of S, which P replaces in place
constexpr int kTab = 8;                         // slots of the key and row tables
constexpr uint32_t kColS = 0, kColO = 256;      // S/P: 64 columns a slot; O: 128, two slots
constexpr uint32_t kTmemCols = 512;

struct PromptParams {
    AttnCall a;
};

// The warps of a form, and its pieces of K and V.
template <bool EXACT>
struct Form {
    static constexpr int kGroups = EXACT ? 2 : 1;               // softmax groups of 4 warps
    static constexpr int kCo0 = 4 * kGroups;                    // first warp that adds
    static constexpr int kDq0 = kCo0 + kCoWarps;                // first that reads the cache
    static constexpr int kCopy = kWarps - 4;                    // fetches the cache; the next warp makes the keys' tables
    static constexpr int kMma = kWarps - 2;                     // issues S; the next warp P V
    static constexpr int kDqWarps = kCopy - kDq0;               // 4 or 8
    static constexpr int kPieces = EXACT ? 1 : 2;
    static constexpr int kTurns = 8 / kDqWarps;                 // keys per thread
    static constexpr int kSlots = EXACT ? 3 : 2;                // of K and of V
    static constexpr int kRaw = EXACT ? 4 : 2;                  // tiles of the cache as it is
};

// Shared memory of a head of DP = 64 or 128 values (96 is padded with zeros).
template <int J, int G, int DP>
struct Mem {
    static constexpr bool EXACT = G == 1;
    static constexpr int kQ = kRows * DP * 2;           // bytes of a piece
    static constexpr int kKV = kTile * DP * 2;
    static constexpr int kSlot = Form<EXACT>::kPieces * kKV;
    static constexpr int offQ = 0;                      // high, low
    static constexpr int offK = offQ + 2 * kQ;          // [slot][pieces]
    static constexpr int offV = offK + Form<EXACT>::kSlots * kSlot;
    static constexpr int offF = offV + Form<EXACT>::kSlots * kSlot;       // per key F, G, s and z - 8, or F and V's power of two, s and the power times P's [slot][4 or 2][64]
    static constexpr int offM = offF + kTab * kTile * (EXACT ? 16 : 8);   // per row: reference, sum p s (z - 8) [2][slot][128]
    static constexpr int offL = offM + kTab * kRows * (EXACT ? 8 : 4);    // per row (reference, sum of weights) [group][128]
    static constexpr int offQs = offL + Form<EXACT>::kGroups * kRows * 8;      // Q's sums over 8 values [128][DP / 8] (EXACT)
    static constexpr int offVm = offQs + (EXACT ? kRows * DP / 2 : 0);   // what undoes P's power of two: the tables', the softmax's [2][slot]
    static constexpr int offBad = offVm + kTab * 8;         // pages outside the pool, by 16 keys [raw slot][4]
    static constexpr int offBar = offBad + 64;
    static constexpr int kRawCodes = kTile * 16 * J, kRawSz = kTile * 8 * G;
    static constexpr int kRawSlot = 2 * (kRawCodes + kRawSz);
    static constexpr int offRaw = offBar + 448;         // [slot](key codes, value codes, key (s, z), value (s, z))
    static constexpr int kBytes = offRaw + Form<EXACT>::kRaw * kRawSlot + 1024;  // and room to align
};

struct Bars {
    uint64_t *k_full, *k_empty, *v_full, *v_empty, *s_full, *sp_empty, *p_full, *o_full, *o_empty, *fin, *drain, *raw_full, *raw_empty;
};

// One MMA, A and B from shared memory, D in tensor memory: the low words of
// the descriptors, which hold the addresses, and their common high word.
// ACC: D += (else D =).
template <bool ACC>
__device__ __forceinline__ void mma_ss(uint32_t d_taddr, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b64 a, {%1, %3};\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}"
        ::"r"(d_taddr), "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "n"(ACC ? 1 : 0)
        : "memory");
}

// The same with A in tensor memory.
template <bool ACC>
__device__ __forceinline__ void mma_ts(uint32_t d_taddr, uint32_t a_taddr, uint32_t b_lo, uint32_t hi, uint32_t idesc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}"
        ::"r"(d_taddr), "r"(a_taddr), "r"(b_lo), "r"(hi), "r"(idesc), "n"(ACC ? 1 : 0)
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
// time limit (recording the error).  try_wait without a time hint leaves the
// thread suspended for as long as the hardware likes, so a waiting warp takes
// few issue slots from the others (with a hint it became a loop of looks and
// sleeps, half of all instructions); the timer is read on long waits only.
__device__ __forceinline__ bool try_wait_once(uint64_t *bar, uint32_t parity)
{
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return done != 0;
}

__device__ __noinline__ bool bar_wait_slow(uint64_t *bar, uint32_t parity, volatile int *abort)
{
    unsigned long long t0 = 0;
    for (unsigned int i = 1;; ++i) {
        if (try_wait_once(bar, parity)) return true;
        if ((i & 15u) == 0u) {
            if (*abort) return false;
            if (t0 == 0) t0 = global_timer_ns();
            if (global_timer_ns() - t0 > kWaitLimitNs) {
                *abort = 1;
                atomicOr(&g_prompt_error, kAttnGaveUp);
                return false;
            }
        }
    }
}

__device__ __forceinline__ bool bar_wait(uint64_t *bar, uint32_t parity, volatile int *abort)
{
    return try_wait_once(bar, parity) || bar_wait_slow(bar, parity, abort);
}

// The whole warp waits; false in every lane when any gave up.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort)
{
    return __all_sync(0xffffffffu, bar_wait(bar, parity, abort));
}

// Wait for the loads, of which v's are the last: v is not to be used before.
template <int N>
__device__ __forceinline__ void tmem_wait_for(uint32_t (&v)[N])
{
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(v[i]));
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&v)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(taddr)
                 : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// Two numbers as their leading fp16 pieces and the rest, each pair packed.
// The rest is one operation, an FMA of fp16 factors onto an f32 number.
__device__ __forceinline__ void split_pair(float a, float b, uint32_t &hi, uint32_t &lo)
{
    float x, y;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(b), "f"(a));
    asm("{\n\t.reg .b16 h, l, m;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "mov.b16 m, 0xBC00;\n\t"            // -1
        "fma.rn.f32.f16 %0, l, m, %3;\n\t"
        "fma.rn.f32.f16 %1, h, m, %4;\n\t}"
        : "=f"(x), "=f"(y)
        : "r"(hi), "f"(a), "f"(b));
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(y), "f"(x));
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
        const float2 f = unpack2(mul2(d, sc));
        split_pair(f.x, f.y, hi[i], lo[i]);
    }
}

__device__ __forceinline__ float lds_f1(uint32_t at)
{
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}

__device__ __forceinline__ float2 lds_f2(uint32_t at)
{
    float2 v;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
    return v;
}

template <int J>
__device__ __forceinline__ void lds_words(uint32_t at, uint32_t (&w)[J])
{
    if constexpr (J == 4) {
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
    } else if constexpr (J == 2) {
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at) : "memory");
    } else {
#pragma unroll
        for (int i = 0; i < J; ++i) asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[i]) : "r"(at + 4 * i) : "memory");
    }
}

// Four consecutive floats as two packed pairs.
__device__ __forceinline__ void lds_pairs(uint32_t at, f32x2 (&v)[2])
{
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(v[0]), "=l"(v[1]) : "r"(at) : "memory");
}

// A softmax thread's row: the reference its weights are taken against (log2),
// and their sum.
struct RowSum {
    float ref, l;
    bool set;        // ref is a maximum seen
};

// The pieces of a tile's first `cols` keys times `by`, a power of two (rarely
// needed).
__device__ __forceinline__ void scale_pieces(uint32_t s_at, int cols, float by)
{
    const __half2 f = __float2half2_rn(by);
    tmem_wait_st();
#pragma unroll 1
    for (int x = 0; x < cols; x += 8) {
        uint32_t u[8];
        tmem_ld8(s_at + x, u);
        tmem_wait_for(u);
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            const __half2 v = __hmul2(*reinterpret_cast<const __half2 *>(&u[n]), f);
            u[n] = *reinterpret_cast<const uint32_t *>(&v);
        }
        tmem_st8(s_at + x, u);
    }
}

// What a tile's weights are made with.
struct TileOf {
    uint32_t s_at, key;     // S in tensor memory; the key tables in shared memory
    f32x2 qsum;             // sum_d q_d, twice
    int last, first;        // column x counts when first <= x <= last
};

// 16 keys, S in t: the weights p_j = 2^(w - ref), two fp16 pieces of them times
// 2^e and the key's s_j or V's power of two (the table holds the product) back
// into the same columns of tensor memory, 8 of leading pieces and 8 of rests.
// When a weight passes 2^kSlack of it the reference moves by a whole power of
// two, by which the pieces of this tile already written are scaled.  From 2^23
// on a whole step may be lost beside the reference: it moves to the largest
// exponent itself there, and the exponents are rounded as numbers of its size
// first, so that the weights and what is summed keep one reference.  l and z:
// sums of the weights and of 2^e p_j s_j (z_j - 8), over even and odd keys.
template <bool EXACT, bool MASK>
__device__ __forceinline__ void keys16(const TileOf &w, int x, uint32_t (&t)[16], RowSum &r, f32x2 &l, f32x2 &z)
{
    float top = -INFINITY;
    const f32x2 base = pack2(-r.ref, -r.ref);
#pragma unroll
    for (int y = 0; y < 16; y += 4) {
        f32x2 f[2], g[2];
        lds_pairs(w.key + 4 * (x + y), f);                          // F
        if (EXACT) lds_pairs(w.key + 4 * (kTile + x + y), g);       // G
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int c = y + 2 * n;
            const f32x2 a = EXACT ? fma2(g[n], w.qsum, base) : base;
            float2 v = unpack2(fma2(pack2(__uint_as_float(t[c]), __uint_as_float(t[c + 1])), f[n], a));
            if (MASK && (x + c > w.last || x + c < w.first)) v.x = -INFINITY;
            if (MASK && (x + c + 1 > w.last || x + c + 1 < w.first)) v.y = -INFINITY;
            top = fmaxf(top, fmaxf(v.x, v.y));
            t[c] = __float_as_uint(v.x);
            t[c + 1] = __float_as_uint(v.y);
        }
    }
    const bool mine = top > (r.set ? kSlack : -INFINITY);
    if (__any_sync(0xffffffffu, mine)) {
        const float most = r.ref + top;
        const bool large = mine && fabsf(most) >= 0x1p23f;
        const float moved = large ? most : r.ref + ceilf(top);
        const float by = large ? moved - r.ref : mine ? ceilf(top) : 0.0f;
        const float up = large ? r.ref : 0.0f, down = large ? moved : by;
        float shrink = mine && r.set ? fminf(by, 48.0f) : 0.0f;   // (2^-48 leaves nothing of pieces below 2^16)
        if (mine) {
            const float f = r.set ? exp2_approx(-by) : 0.0f;   // (0: nothing is summed yet)
            r.l = r.set ? r.l * f : 0.0f;
            l = r.set ? mul2(l, pack2(f, f)) : pack2(0.0f, 0.0f);
            z = r.set ? mul2(z, pack2(f, f)) : pack2(0.0f, 0.0f);
            r.ref = moved;
            r.set = true;
        }
        if (x > 0)
            do {                               // fp16's least power is 2^-24
                scale_pieces(w.s_at, x, exp2_approx(-fminf(fmaxf(shrink, 0.0f), 24.0f)));
                shrink -= 24.0f;
            } while (__any_sync(0xffffffffu, shrink > 0.0f));
#pragma unroll
        for (int y = 0; y < 16; y += 2) {
            const float2 v = unpack2(add2(add2(pack2(__uint_as_float(t[y]), __uint_as_float(t[y + 1])), pack2(up, up)),
                                          pack2(-down, -down)));
            t[y] = __float_as_uint(v.x);
            t[y + 1] = __float_as_uint(v.y);
        }
    }
    uint32_t pc[16];                       // leading pieces, rests
#pragma unroll
    for (int y = 0; y < 16; y += 4) {
        f32x2 s[2], q[2];
        lds_pairs(w.key + 4 * ((EXACT ? 2 : 1) * kTile + x + y), s);        // s, or V's powers of two
        if (EXACT) lds_pairs(w.key + 4 * (3 * kTile + x + y), q);           // z - 8
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int c = y + 2 * n;
            f32x2 p = pack2(exp2_approx(__uint_as_float(t[c])), exp2_approx(__uint_as_float(t[c + 1])));
            l = add2(l, p);
            p = mul2(p, s[n]);
            if (EXACT) z = fma2(p, q[n], z);
            const float2 v = unpack2(p);
            split_pair(v.x, v.y, pc[c / 2], pc[8 + c / 2]);
        }
    }
    tmem_st16(w.s_at + x, pc);
}

// One tile of a row; returns sum_j 2^e p_j s_j (z_j - 8).
template <bool EXACT, bool MASK>
__device__ __forceinline__ float tile_weights(const TileOf &w, RowSum &r)
{
    f32x2 l = pack2(0.0f, 0.0f), z = l;
    uint32_t t[16], next[16];              // one is on its way while the other is worked on
    tmem_ld16(w.s_at, next);
#pragma unroll 1                               // (a small loop: the roles share the instruction cache)
    for (int x = 0; x < kTile; x += 16) {
        tmem_wait_for(next);
#pragma unroll
        for (int y = 0; y < 16; ++y) t[y] = next[y];
        if (x + 16 < kTile) tmem_ld16(w.s_at + x + 16, next);
        keys16<EXACT, MASK>(w, x, t, r, l, z);
    }
    const float2 ls = unpack2(l), zs = unpack2(z);
    r.l += ls.x + ls.y;
    return zs.x + zs.y;
}

// 8 codes of a word minus 8, exact, in the order 0, 4, 1, 5, 2, 6, 3, 7.
__device__ __forceinline__ uint4 exact_word(uint32_t w)
{
    const uint32_t magic = 0x64006400u;      // 1024 in each half
    auto lower = [&](uint32_t x) {           // (1024 + c) - 1032
        uint32_t d, m = 0xE408E408u;
        asm("{\n\t.reg .b32 t;\n\tlop3.b32 t, %1, 0x000F000F, %2, 0xEA;\n\tadd.rn.f16x2 %0, t, %3;\n\t}"
            : "=r"(d) : "r"(x), "r"(magic), "r"(m));
        return d;
    };
    auto upper = [&](uint32_t x) {           // (1024 + 16 c) / 16 - 72
        uint32_t d, s = 0x2C002C00u, m = 0xD480D480u;
        asm("{\n\t.reg .b32 t;\n\tlop3.b32 t, %1, 0x00F000F0, %2, 0xEA;\n\tfma.rn.f16x2 %0, t, %3, %4;\n\t}"
            : "=r"(d) : "r"(x), "r"(magic), "r"(s), "r"(m));
        return d;
    };
    const uint32_t y = w >> 8;
    return make_uint4(lower(w), upper(w), lower(y), upper(y));
}

// Place i of an EXACT operand's group of 8 holds value exact_order(i).
__host__ __device__ constexpr int exact_order(int i)
{
    return (i >> 1) + 4 * (i & 1);
}

// A key's scales and zeros of one side: zeros where the CTA does not see it or
// its page is outside the pool.
template <int G>
struct KeyOf {
    bool bad, finite;
    float bound;             // the largest |(code - z) s| that they allow
    __device__ __forceinline__ int exponent() const { return bound < INFINITY ? scale_exponent(bound) : 0; }
};

template <int G>
__device__ __forceinline__ KeyOf<G> key_of(int see_lo, int see_hi, int t, uint32_t at, uint32_t bad_at, float2 (&sz)[G])
{
    KeyOf<G> k;
    int bad;
    asm volatile("ld.shared.s32 %0, [%1];" : "=r"(bad) : "r"(bad_at) : "memory");
    const bool here = t <= see_hi && t >= see_lo;
    k.bad = here && bad != 0;
    k.bound = 0.0f;
    float f = 0.0f;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        sz[g] = lds_f2(at + 8 * g);
        if (!here || bad != 0) sz[g] = make_float2(0.0f, 0.0f);
        k.bound = fmaxf(k.bound, fabsf(sz[g].x) * fmaxf(fabsf(sz[g].y), fabsf(15.0f - sz[g].y)));
        f += 0.0f * sz[g].x + 0.0f * sz[g].y;
    }
    k.finite = f == 0.0f;
    return k;
}

// One scale group per row: a tile's rows of equal values, as it was copied, by
// scales of their size.  raw: the keys' codes, the values', the keys' scales,
// the values'.
template <int J>
__device__ __noinline__ void fit_equal_rows(uint32_t raw)
{
    const int lane = threadIdx.x & 31;
    __syncwarp();
#pragma unroll 1
    for (int i = lane; i < 2 * kTile; i += 32) {
        const int value = i / kTile, key = i % kTile;
        const uint32_t row = raw + value * kTile * 16 * J + key * 16 * J;
        const uint32_t at = raw + 2 * kTile * 16 * J + value * kTile * 8 + key * 8;
        const float2 sz = lds_f2(at);
        if (sz.x != 1.0f) continue;
        uint32_t any = 0;
#pragma unroll 1
        for (int x = 0; x < 4 * J; ++x) {
            uint32_t word;
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(word) : "r"(row + 4 * x) : "memory");
            any |= word;
        }
        if (any != 0) continue;
        const float2 to = equal_values(sz);
        asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(to.x), "f"(to.y) : "memory");
    }
    __syncwarp();
}

// Several scale groups per row: a power of two is taken from what a key's scales
// and zeros allow, 15 for a group of equal values (scale 1).  Where that leaves
// too few digits for what such rows hold, all rows of the CTA are the last
// kernel's.  zat: the keys' scales, then the values'; keys lo to hi of the tile
// are seen by some row; every: by all.  (The codes are not looked at: a scale
// of 1 by chance is computed there as well, and comes out the same.)
template <int G>
__device__ __noinline__ void leave_equal_rows(uint32_t zat, int lo, int hi, bool every, uint32_t *apart)
{
    constexpr float kLeast = 15.0f / (1 << kSpread);
    const int lane = threadIdx.x & 31;
    bool leave = false, some = false;
    float top = 0.0f;
#pragma unroll 1
    for (int i = lane; i < 2 * kTile; i += 32) {
        const int key = i % kTile;
        bool ones = false;
        float size = 0.0f;
#pragma unroll 1
        for (int g = 0; g < G && key >= lo && key <= hi; ++g) {
            const float2 sz = lds_f2(zat + (i * G + g) * 8);
            ones |= sz.x == 1.0f;
            const float x = fabsf(sz.y);
            size = fmaxf(size, sz.x == 1.0f ? x : fabsf(sz.x) * fmaxf(x, fabsf(15.0f - sz.y)));
        }
        const bool value = i >= kTile;
        if (ones && size > 0.0f && size < kLeast && !(value && every)) leave = true;
        if (value) {
            some |= ones;
            top = fmaxf(top, size);
        }
    }
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
    if (every && __any_sync(0xffffffffu, some) && top > 0.0f && top < kLeast) leave = true;
    if (__any_sync(0xffffffffu, leave) && lane < kRows / 32) apart[lane] = ~0u;
    __syncwarp();
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
    constexpr bool EXACT = G == 1;
    using W = Form<EXACT>;
    using M = Mem<J, G, DP>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t smem_s = smem_addr(smem);
    __shared__ int s_sums[kWarps], s_big, s_small;
    __shared__ volatile int s_req, s_tile;
    __shared__ uint32_t s_apart[kRows / 32];               // a bit per row that is left to the last kernel
    __shared__ int s_uneven;                               // it is to look for rows that see small values only
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
        if (a.B == 1) all = mine = tiles_of(0);
        else for (int b0 = 0; b0 < a.B; b0 += kThreads) {
            int t;
            mine = tiles_of(b0 + (int)threadIdx.x);
            before = scan_ints<kWarps>(mine, t, s_sums);
            all += t;
        }
        const int want = all - 1 - (int)(blockIdx.x / (unsigned)H);
        if (want < 0) {   // uniform
            if (threadIdx.x < kRows / 32) a.apart[blockIdx.x].rows[threadIdx.x] = 0;
            if (threadIdx.x == kRows / 32) a.apart[blockIdx.x].uneven = 0;
            return;
        }
        int base = 0;
        for (int b0 = 0; b0 < a.B; b0 += kThreads) {
            int t = all;
            if (a.B > kThreads) {
                mine = tiles_of(b0 + (int)threadIdx.x);
                before = scan_ints<kWarps>(mine, t, s_sums);
            }
            if (want >= base + before && want < base + before + mine && (a.B > 1 || threadIdx.x == 0)) {
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
        bar.k_empty = b + 4;
        bar.v_full = b + 8;
        bar.v_empty = b + 12;
        bar.o_full = b + 16;
        bar.o_empty = b + 18;
        bar.s_full = b + 20;
        bar.sp_empty = b + 20 + kSP;
        bar.p_full = b + 20 + 2 * kSP;
        bar.fin = b + 20 + 2 * kSP + kTab;
        bar.drain = bar.fin + 1;
        bar.raw_full = bar.fin + 3;
        bar.raw_empty = bar.raw_full + 4;
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < W::kSlots; ++s) {
            mbar_init(&bar.k_full[s], W::kDqWarps + 1);   // and the tables'
            mbar_init(&bar.k_empty[s], 1);
            mbar_init(&bar.v_full[s], W::kDqWarps);
            mbar_init(&bar.v_empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bar.o_full[s], 1);
            mbar_init(&bar.o_empty[s], kCoWarps);
        }
        for (int s = 0; s < kSP; ++s) {
            mbar_init(&bar.s_full[s], 1);
            mbar_init(&bar.sp_empty[s], 1);
        }
        for (int s = 0; s < kTab; ++s) mbar_init(&bar.p_full[s], 4);
        mbar_init(bar.fin, W::kCo0);
        mbar_init(bar.drain, 1);
        mbar_init(bar.drain + 1, 1);
        for (int s = 0; s < W::kRaw; ++s) {
            mbar_init(&bar.raw_full[s], 32);       // every copying thread's copies
            mbar_init(&bar.raw_empty[s], W::kDqWarps + 1);
        }
        s_abort = 0;
        s_big = 0;
        s_small = 0x7f800000;
#pragma unroll
        for (int x = 0; x < kRows / 32; ++x) s_apart[x] = 0;
        s_uneven = 0;
        mbar_fence_init();
    }
    if (warp == W::kMma) {
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

    // ---- Q: two fp16 pieces with one power of two for the CTA, by the softmax
    // and adding warps; the others are under way meanwhile, but the tables need
    // the power (barrier 1) and S the pieces (barrier 2) ----
    constexpr int kStaging = 32 * W::kDq0;
    int kq = 0;
    auto meet = [&](int barrier) {
        if (barrier == 1) asm volatile("bar.sync 1, %0;" ::"n"(kStaging + 32) : "memory");
        else asm volatile("bar.sync 2, %0;" ::"n"(kStaging + 32) : "memory");
    };
    if (warp == W::kCopy + 1) {
        meet(1);
        kq = scale_exponent(__int_as_float(s_big));
    } else if (warp == W::kMma) {
        meet(2);
    } else if (warp < W::kDq0) {
        constexpr int kTurns = (kRows * (DP / 8) + kStaging - 1) / kStaging;
        const int th = (int)threadIdx.x;
        float4 q[kTurns][2];
        float big = 0.0f, small = INFINITY;
        // the largest finite value of a turn's row, whose DP / 8 threads are
        // neighbours (an infinity is left to its own row)
        auto largest = [&](const float4 (&x)[2]) {
            const float v[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (fabsf(v[i]) < INFINITY) m = fmaxf(m, fabsf(v[i]));
#pragma unroll
            for (int o = DP / 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            return m;
        };
#pragma unroll
        for (int n = 0; n < kTurns; ++n) {
            const int i = th + n * kStaging, r = i / (DP / 8), d8 = i - r * (DP / 8);
            q[n][0] = q[n][1] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < kRows && row0 + r < rows_all && 8 * d8 < D) {
                const int rho = row0 + r, j = rho / R;
                const float4 *at = reinterpret_cast<const float4 *>(a.q + (size_t)(rq.row0 + j) * a.ldq +
                                                                   (size_t)(h * R + rho - j * R) * D + 8 * d8);
                q[n][0] = __ldg(at);
                q[n][1] = __ldg(at + 1);
            }
        }
#pragma unroll
        for (int n = 0; n < kTurns; ++n) {
            const int i = th + n * kStaging;
            const float m = largest(q[n]);
            if (i % (DP / 8) == 0 && i < kRows * (DP / 8)) reinterpret_cast<float *>(smem + M::offL)[i / (DP / 8)] = m;
            big = fmaxf(big, m);
            if (m > 0.0f) small = fminf(small, m);
        }
        const unsigned int top = __reduce_max_sync(0xffffffffu, __float_as_uint(big));
        const unsigned int least = __reduce_min_sync(0xffffffffu, __float_as_uint(small));
        if (lane == 0) {
            atomicMax(&s_big, (int)top);
            atomicMin(&s_small, (int)least);
        }
        meet(1);
        kq = scale_exponent(__int_as_float(s_big));
        if (s_small < 0x7f800000 && scale_exponent(__int_as_float(s_small)) - kq > kSpread) {
            // rows of less than 2^-kSpread of the largest would lose digits to it
            const float m = th < kRows ? reinterpret_cast<const float *>(smem + M::offL)[th] : 0.0f;
            if (m > 0.0f && scale_exponent(m) - kq > kSpread) atomicOr(&s_apart[th >> 5], 1u << (th & 31));
        }
        const float up = pow2(kq);
#pragma unroll
        for (int n = 0; n < kTurns; ++n) {
            const int i = th + n * kStaging, r = i / (DP / 8), d8 = i - r * (DP / 8);
            if (r >= kRows) break;
            const float v[8] = {q[n][0].x, q[n][0].y, q[n][0].z, q[n][0].w, q[n][1].x, q[n][1].y, q[n][1].z, q[n][1].w};
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int m = 0; m < 4; ++m)
                split_pair(v[EXACT ? exact_order(2 * m) : 2 * m] * up, v[EXACT ? exact_order(2 * m + 1) : 2 * m + 1] * up,
                           hi[m], lo[m]);
            unsigned char *at = smem + M::offQ + (d8 >> 3) * (kRows * 128) + r * 128 + (((d8 & 7) ^ (r & 7)) << 4);
            *reinterpret_cast<uint4 *>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(at + M::kQ) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            if (EXACT)
                reinterpret_cast<float *>(smem + M::offQs)[r * (DP / 8) + d8] =
                    (((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]))) * up;
        }
        // the padding of a 96-value head: zeros in every K and V slot, once
        if constexpr (DP > D) {
            constexpr int per = kTile * (DP - D) / 8;      // 16-byte pieces of one piece's padding
            for (int i = th; i < 2 * W::kSlots * W::kPieces * per; i += kStaging) {   // K's and V's pieces lie on end
                const int t = i / per, k = (i - t * per) / ((DP - D) / 8), d8 = D / 8 + (i - t * per) % ((DP - D) / 8);
                *reinterpret_cast<uint4 *>(smem + M::offK + t * M::kKV + (d8 >> 3) * (kTile * 128) + k * 128 +
                                           (((d8 & 7) ^ (k & 7)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
            }
        }
        fence_proxy_async_smem();
        meet(2);
    }

    bool ok = true;
    if (warp < W::kCo0) {
        // ===== softmax: a thread per row, a group of 4 warps per tile =====
        const int group = warp >> 2;
        const int row = 32 * (warp & 3) + lane;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const int rho = row0 + row, j = rho / R;
        const int last = rho < rows_all ? pos0 + j : -1;
        const int first = attn_first(a, max(last, -1));
        float qsum = 0.0f;
        if (EXACT) {
#pragma unroll
            for (int d = 0; d < DP / 8; ++d) qsum += reinterpret_cast<const float *>(smem + M::offQs)[row * (DP / 8) + d];
        }
        RowSum r{0.0f, 0.0f, false};
        float *ms = reinterpret_cast<float *>(smem + M::offM);
        for (int i = group; i < n_tiles; i += W::kGroups) {
            const int s = i % kSP, tab = i % kTab;
            if (!warp_wait(&bar.s_full[s], (i / kSP) & 1, abort)) {
                ok = false;
                break;
            }
            tc_fence_after_sync();
            const uint32_t key = smem_s + M::offF + tab * (EXACT ? 16 : 8) * kTile;
            const float undo = lds_f1(smem_s + M::offVm + tab * 4);
            const int k0 = (tile_lo + i) * kTile;
            const bool masked = k0 + kTile - 1 > all_hi || k0 < all_lo;   // uniform
            const TileOf w{tmem + lanes + kColS + s * kTile, key, pack2(qsum, qsum), last - k0, first - k0};
            const float z = masked ? tile_weights<EXACT, true>(w, r) : tile_weights<EXACT, false>(w, r);
            // what the tile's P V is relative to; its power of two apart, which a
            // large reference would swallow
            ms[tab * kRows + row] = r.set ? r.ref : -INFINITY;
            if (row == 0) reinterpret_cast<float *>(smem + M::offVm)[kTab + tab] = undo;
            if (EXACT) ms[(kTab + tab) * kRows + row] = z;
            tmem_wait_st();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.p_full[tab]);
        }
        reinterpret_cast<float2 *>(smem + M::offL)[group * kRows + row] = make_float2(r.set ? r.ref : -INFINITY, r.l);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar.fin);
    } else if (warp < W::kDq0) {
        // ===== the tiles' P V added up: a row and half of the values per thread =====
        constexpr int C = DP / 2;
        const int q4 = warp & 3, half = (warp - W::kCo0) >> 2;
        const int row = 32 * q4 + lane;
        const uint32_t lanes = (uint32_t)(32 * q4) << 16;
        const float *ms = reinterpret_cast<const float *>(smem + M::offM);
        float o[C];
#pragma unroll
        for (int d = 0; d < C; ++d) o[d] = 0.0f;
        float m = -INFINITY, zs = 0.0f;    // o and zs are relative to 2^m
        for (int i = 0; i < n_tiles; ++i) {
            const int s = i & 1, k = i >> 1;
            const int tab = i % kTab;
            // the row's reference comes with P
            if (!warp_wait(&bar.p_full[tab], (i / kTab) & 1, abort) || !warp_wait(&bar.o_full[s], k & 1, abort)) {
                ok = false;
                break;
            }
            tc_fence_after_sync();
            const float undo = reinterpret_cast<const float *>(smem + M::offVm)[kTab + tab];
            const float2 t2 = make_float2(ms[tab * kRows + row], EXACT ? ms[(kTab + tab) * kRows + row] : 0.0f);
            const float mn = fmaxf(m, t2.x), ref = mn == -INFINITY ? 0.0f : mn;
            const float ft = exp2_approx(t2.x - ref) * undo;
            if (__any_sync(0xffffffffu, mn > m)) {
                const float fo = exp2_approx(m - ref);
                zs *= fo;
#pragma unroll
                for (int d = 0; d < C; ++d) o[d] *= fo;
                m = mn;
            }
            zs = fmaf(t2.y, ft, zs);
#pragma unroll
            for (int x = 0; x < C / 8; ++x) {
                uint32_t t[8];
                tmem_ld8(tmem + lanes + kColO + s * 128 + half * C + 8 * x, t);
                tmem_wait_for(t);
#pragma unroll
                for (int y = 0; y < 8; ++y) o[8 * x + y] = fmaf(__uint_as_float(t[y]), ft, o[8 * x + y]);
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.o_empty[s]);
        }
        if (ok) ok = warp_wait(bar.fin, 0, abort);
        // The rows leave by way of shared memory, so that a warp stores whole
        // stretches of them: a thread's own row, 16 bytes at a time, meets 32
        // lines per store (5000 cycles of a CTA instead of 1500).  K and V are
        // not needed any more, unless the kernel gave up.
        constexpr int X = C / 4;           // 16-byte pieces of half a row
        float4 *stage = reinterpret_cast<float4 *>(smem + M::offK) + (warp - W::kCo0) * 32 * X;
        float inv = quiet_nan();
        if (ok) {
            const float2 *gl = reinterpret_cast<const float2 *>(smem + M::offL);
            float l = 0.0f;
#pragma unroll
            for (int x = 0; x < W::kGroups; ++x) {
                const float2 v = gl[x * kRows + row];
                if (v.x != -INFINITY) l = fmaf(v.y, exp2_approx(v.x - m), l);
            }
            inv = m == -INFINITY ? 0.0f : 1.0f / l;
#pragma unroll
            for (int d = 0; d < C; d += 8) {
                float v[8];
#pragma unroll
                for (int n = 0; n < 8; ++n) v[EXACT ? exact_order(n) : n] = (o[d + n] - zs) * inv;
                stage[lane * X + ((d / 4) ^ (lane & 7))] = make_float4(v[0], v[1], v[2], v[3]);
                stage[lane * X + ((d / 4 + 1) ^ (lane & 7))] = make_float4(v[4], v[5], v[6], v[7]);
            }
        }
        __syncwarp();
#pragma unroll
        for (int n = 0; n < X; ++n) {
            const int r = n * (32 / X) + lane / X, x = lane % X;
            const int rho = row0 + 32 * q4 + r, j = rho / R;
            if (rho >= rows_all || half * C + 4 * x >= D) continue;
            *reinterpret_cast<float4 *>(a.out + (size_t)(rq.row0 + j) * a.ldo + (size_t)(h * R + rho - j * R) * D +
                                        half * C + 4 * x) =
                ok ? stage[r * X + (x ^ (r & 7))] : make_float4(inv, inv, inv, inv);
        }
    } else if (warp < W::kCopy) {
        // ===== the cache: codes, scales and zeros to the operands =====
        // lane: key lane % 8 of eight, values 32 u + 8 (lane / 8) .. + 7 (eight
        // keys of one shared-memory phase meet eight distinct banks)
        constexpr int TN = W::kTurns, kStep = 8 * W::kDqWarps;   // keys between a lane's turns
        const int w = warp - W::kDq0, key0 = 8 * w + (lane & 7), c = lane >> 3;
        // this lane's words and its key's scales in a raw slot
        const uint32_t raw0 = smem_s + M::offRaw, raw_w = raw0 + key0 * 16 * J + c * 4 * J, raw_z = raw0 + 2 * M::kRawCodes + key0 * 8 * G;
        // block u of 32 values of key key0 + kStep y: 16-byte piece 4 u + c of
        // its row, swizzled by the key (the same for every turn)
        const uint32_t place0 = key0 * 128 + ((c ^ (key0 & 7)) << 4), place1 = place0 ^ 64u;
        auto place = [&](uint32_t base, int u, int y) {
            return base + ((u & 1) ? place1 : place0) + (u >> 1) * (kTile * 128) + y * kStep * 128;
        };
        auto store16 = [](uint32_t at, uint32_t x0, uint32_t x1, uint32_t x2, uint32_t x3) {
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(x0), "r"(x1), "r"(x2), "r"(x3) : "memory");
        };
        // the 8 value codes of block u, in order (halves 2c and 2c + 1 lie J halves apart)
        auto value_word = [](const uint32_t (&vw)[J], int u) {
            if constexpr (J == 4) return __byte_perm(vw[u / 2], vw[2 + u / 2], (u & 1) ? 0x7632 : 0x5410);
            else if constexpr (J == 2) return __byte_perm(vw[0], vw[1], u ? 0x7632 : 0x5410);
            else
                return u == 0   ? __byte_perm(vw[0], vw[1], 0x7610)
                       : u == 1 ? __byte_perm(vw[0], vw[2], 0x5432)
                                : __byte_perm(vw[1], vw[2], 0x7610);
        };
        const uint32_t bad_at = smem_s + M::offBad;
        int s = 0, phase = 1;              // slot of K and V, parity of the phase before
        for (int i = 0; i < n_tiles; ++i) {
            const int rs = i % W::kRaw;
            const uint32_t raw = (uint32_t)rs * M::kRawSlot;
            if (!warp_wait(&bar.raw_full[rs], (i / W::kRaw) & 1, abort) ||
                (i >= W::kSlots && !warp_wait(&bar.k_empty[s], phase, abort))) {
                ok = false;
                break;
            }
            // ---- K ----
#pragma unroll
            for (int y = 0; y < TN; ++y) {
                uint32_t kw[J];
                lds_words<J>(raw_w + raw + y * kStep * 16 * J, kw);
                const uint32_t base = smem_s + M::offK + s * M::kSlot;
                if constexpr (EXACT) {
#pragma unroll
                    for (int u = 0; u < J; ++u) {
                        const uint4 e = exact_word(kw[u]);
                        store16(place(base, u, y), e.x, e.y, e.z, e.w);
                    }
                } else {
                    float2 ks[G];
                    const KeyOf<G> k = key_of<G>(see_lo, see_hi, (tile_lo + i) * kTile + key0 + kStep * y,
                                                 raw_z + raw + y * kStep * 8 * G, bad_at + rs * 16 + ((key0 + kStep * y) >> 4) * 4, ks);
                    const float up = pow2(k.exponent());
#pragma unroll
                    for (int u = 0; u < J; ++u) {
                        uint32_t hi[4], lo[4];
                        dequant_word(kw[u], ks[u / UG].x * up, ks[u / UG].y, hi, lo);
                        const uint32_t at = place(base, u, y);
                        store16(at, hi[0], hi[1], hi[2], hi[3]);
                        store16(at + M::kKV, lo[0], lo[1], lo[2], lo[3]);
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.k_full[s]);
            // ---- V ----
            if (i >= W::kSlots && !warp_wait(&bar.v_empty[s], phase, abort)) {
                ok = false;
                break;
            }
#pragma unroll
            for (int y = 0; y < TN; ++y) {
                const uint32_t base = smem_s + M::offV + s * M::kSlot;
                uint32_t vw[J];
                lds_words<J>(raw_w + raw + y * kStep * 16 * J + M::kRawCodes, vw);
                float2 vs[G];
                float up = 0.0f;
                if constexpr (!EXACT) {
                    const KeyOf<G> k = key_of<G>(see_lo, see_hi, (tile_lo + i) * kTile + key0 + kStep * y,
                                                 raw_z + raw + y * kStep * 8 * G + M::kRawSz,
                                                 bad_at + rs * 16 + ((key0 + kStep * y) >> 4) * 4, vs);
                    // what is not finite is zero here: the key's factor spoils the rows that see it
                    up = k.finite ? pow2(min(k.exponent(), 80)) : 0.0f;
                    if (!k.finite) {
#pragma unroll
                        for (int g = 0; g < G; ++g) vs[g] = make_float2(0.0f, 0.0f);
                    }
                }
#pragma unroll
                for (int u = 0; u < J; ++u) {
                    const uint32_t word = value_word(vw, u), at = place(base, u, y);
                    if constexpr (EXACT) {
                        const uint4 e = exact_word(word);
                        store16(at, e.x, e.y, e.z, e.w);
                    } else {
                        uint32_t hi[4], lo[4];
                        dequant_word(word, vs[u / UG].x * up, vs[u / UG].y, hi, lo);
                        store16(at, hi[0], hi[1], hi[2], hi[3]);
                        store16(at + M::kKV, lo[0], lo[1], lo[2], lo[3]);
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bar.v_full[s]);
                mbar_arrive(&bar.raw_empty[rs]);
            }
            if (++s == W::kSlots) {
                s = 0;
                phase ^= 1;
            }
        }
    } else if (warp == W::kCopy) {
        // ===== the cache into shared memory: 16 keys of a page are contiguous,
        // 8 lanes' =====
        const int x16 = lane >> 3, l8 = lane & 7;
        const int shift = 31 - __clz(a.c.page_size);
        const int32_t *table = a.page_table + (size_t)b * a.max_pages;
        const size_t head_row = (size_t)h * a.c.page_size;
        const char *k_at = reinterpret_cast<const char *>(a.c.Kq) + head_row * (16 * J) + 16 * l8;
        const char *v_at = reinterpret_cast<const char *>(a.c.Vq) + head_row * (16 * J) + 16 * l8;
        const char *ks_at = reinterpret_cast<const char *>(a.c.K_sz) + head_row * (8 * G) + 16 * l8;
        const char *vs_at = reinterpret_cast<const char *>(a.c.V_sz) + head_row * (8 * G) + 16 * l8;
        const uint32_t page_rows = (uint32_t)(H * a.c.page_size), n_pages = (uint32_t)a.c.n_pages;
        const uint32_t raw_at = smem_s + M::offRaw + x16 * 256 * J + 16 * l8;
        const uint32_t raw_z = smem_s + M::offRaw + 2 * M::kRawCodes + x16 * 128 * G + 16 * l8;
        int *bad = reinterpret_cast<int *>(smem + M::offBad);
        // the page of a tile's block of 16 keys; -2: nothing is seen there
        auto page_of = [&](int i) {
            const int t = (tile_lo + i) * kTile + 16 * x16;
            return i < n_tiles && t <= see_hi && t + 16 > see_lo ? __ldg(table + (t >> shift)) : -2;
        };
        int page = page_of(0);
        for (int i = 0; i < n_tiles; ++i) {
            const int rs = i % W::kRaw, next = page_of(i + 1);
            if (i >= W::kRaw && !warp_wait(&bar.raw_empty[rs], ((i / W::kRaw) - 1) & 1, abort)) {
                ok = false;
                break;
            }
            const bool in = (uint32_t)page < n_pages, out = !in && page != -2;
            if (l8 == 0) {
                bad[rs * 4 + x16] = out;
                if (out) atomicOr(&g_prompt_error, kAttnBadRequest);
            }
            if (in) {
                const uint32_t at = (uint32_t)((tile_lo + i) * kTile + 16 * x16) & (uint32_t)(a.c.page_size - 1);
                const size_t off = (size_t)(uint32_t)page * (page_rows * (16 * J)) + at * (16 * J);
                const size_t zoff = (size_t)(uint32_t)page * (page_rows * (8 * G)) + at * (8 * G);
                const uint32_t dst = raw_at + (uint32_t)rs * M::kRawSlot, zdst = raw_z + (uint32_t)rs * M::kRawSlot;
#pragma unroll
                for (int n = 0; n < 2 * J; ++n) {
                    cp_async_16(dst + 128 * n, k_at + off + 128 * n);
                    cp_async_16(dst + M::kRawCodes + 128 * n, v_at + off + 128 * n);
                }
#pragma unroll
                for (int n = 0; n < G; ++n) {
                    cp_async_16(zdst + 128 * n, ks_at + zoff + 128 * n);
                    cp_async_16(zdst + M::kRawSz + 128 * n, vs_at + zoff + 128 * n);
                }
            }
            page = next;
            cp_async_mbar_arrive(&bar.raw_full[rs]);
        }
        cp_async_commit();
        cp_async_wait<0>();
    } else if (warp < W::kMma) {
        // ===== tables of a tile's keys, two a lane.  They have slots to spare:
        // once the product of the tile kSlots back is done, the softmax of the
        // one 8 back is =====
        const float Fq = ldexpf(a.scale * kLog2e, -kq);
        int slot = 0, phase = 1;
        for (int i = 0; i < n_tiles; ++i) {
            const int rs = i % W::kRaw, tab = i % kTab;
            if (!warp_wait(&bar.raw_full[rs], (i / W::kRaw) & 1, abort) ||
                (i >= W::kSlots && !warp_wait(&bar.k_empty[slot], phase, abort))) {
                ok = false;
                break;
            }
            float vb = 0.0f;
            bool ones = false;             // a scale of 1: a group of equal values, most likely
            if (EXACT) {
                // (nobody else reads the scales of this form)
                const uint32_t raw = smem_s + M::offRaw + (uint32_t)rs * M::kRawSlot, zat = raw + 2 * M::kRawCodes + lane * 8;
#pragma unroll
                for (int y = 0; y < 4; ++y) ones |= lds_f1(zat + (y & 1) * 256 + (y >> 1) * M::kRawSz) == 1.0f;
                if (__any_sync(0xffffffffu, ones)) fit_equal_rows<J>(raw);   // rare
            }
#pragma unroll EXACT ? 2 : 1
            for (int y = 0; y < 2; ++y) {
                const int key = lane + 32 * y, t = (tile_lo + i) * kTile + key;
                const uint32_t zat = smem_s + M::offRaw + 2 * M::kRawCodes + (uint32_t)rs * M::kRawSlot + key * 8 * G;
                const uint32_t bat = smem_s + M::offBad + rs * 16 + (key >> 4) * 4;
                float2 ks[G], vs[G];
                const KeyOf<G> k = key_of<G>(see_lo, see_hi, t, zat, bat, ks),
                               v = key_of<G>(see_lo, see_hi, t, zat + M::kRawSz, bat, vs);
                // a value that is not finite spoils the rows that see it through its key's factor
                const bool spoilt = k.bad || !v.finite;
                float *at = reinterpret_cast<float *>(smem + M::offF) + tab * (EXACT ? 4 : 2) * kTile + key;
                if constexpr (EXACT) {
                    const float F = spoilt ? quiet_nan() : Fq * ks[0].x;
                    at[0] = F;
                    at[kTile] = (8.0f - ks[0].y) * F;
                    at[3 * kTile] = spoilt ? 0.0f : vs[0].y - 8.0f;
                    at[2 * kTile] = spoilt ? 0.0f : vs[0].x;
                    if (!spoilt) vb = fmaxf(vb, fabsf(vs[0].x));
                } else {
                    at[0] = spoilt ? quiet_nan() : Fq * pow2(-k.exponent());
                    // (a row of zeros has no power: any but 0 would be too large beside its neighbours')
#pragma unroll
                    for (int g = 0; g < G; ++g) ones |= ks[g].x == 1.0f || vs[g].x == 1.0f;
                    at[kTile] = v.finite && v.bound > 0.0f ? pow2(-min(v.exponent(), 80)) : 0.0f;
                    if (!spoilt) vb = fmaxf(vb, v.bound);
                }
            }
            __syncwarp();
            if (!EXACT && __any_sync(0xffffffffu, ones)) {   // rare
                const int k0 = (tile_lo + i) * kTile;
                leave_equal_rows<G>(smem_s + M::offRaw + 2 * M::kRawCodes + (uint32_t)rs * M::kRawSlot, see_lo - k0, see_hi - k0,
                                    k0 + kTile - 1 <= all_hi && k0 >= all_lo, s_apart);
            }
            if (lane == 0) mbar_arrive(&bar.raw_empty[rs]);
            // (numbers of one sign order as their bits do)
            const unsigned int top = __reduce_max_sync(0xffffffffu, __float_as_uint(vb));
            // by the tile's largest V (EXACT: its scale), as a power of two: P is
            // held times 2^e, so that 2^kSlack of it is below 2^15
            const int ve = min(scale_exponent(__uint_as_float(top)), 80), e = EXACT ? ve - 2 : ve + kPieceBits;
            float *at = reinterpret_cast<float *>(smem + M::offF) + (tab * (EXACT ? 4 : 2) + (EXACT ? 2 : 1)) * kTile + lane;
            const float by[2] = {at[0], at[32]};
            at[0] = by[0] * pow2(e);
            at[32] = by[1] * pow2(e);
            if (lane == 0) reinterpret_cast<float *>(smem + M::offVm)[tab] = pow2(-e);
            // where some row may not see the largest (uniform)
            const int k0 = (tile_lo + i) * kTile;
            if (k0 + kTile - 1 > all_hi || k0 < all_lo) {
                // (a power of V is 2^-12 of its bound)
                const float least = __uint_as_float(top) * (EXACT ? 0x1p-12f : 0x1p-24f);
                if ((by[0] != 0.0f && fabsf(by[0]) < least) || (by[1] != 0.0f && fabsf(by[1]) < least)) s_uneven = 1;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.k_full[slot]);
            if (++slot == W::kSlots) {
                slot = 0;
                phase ^= 1;
            }
        }
    } else if (lane == 0 && warp == W::kMma) {
        // ===== S = Q K^T: one lane issues =====
        constexpr uint32_t id_s = idesc_f16_f32(kRows, kTile, false);
        constexpr int kProducts = EXACT ? 2 : 3;
        const uint64_t q_d = smem_desc_sw128(smem_s + M::offQ, 1024), k_d = smem_desc_sw128(smem_s + M::offK, 1024);
        const uint32_t hi = (uint32_t)(q_d >> 32), q_lo = (uint32_t)q_d, k_lo = (uint32_t)k_d;
        int slot = 0, phase = 0;
        for (int i = 0; i < n_tiles; ++i) {
            if (!bar_wait(&bar.k_full[slot], phase, abort) ||
                (i >= kSP && !bar_wait(&bar.sp_empty[i % kSP], ((i / kSP) - 1) & 1, abort)))
                break;
            tc_fence_after_sync();
            const uint32_t kh = k_lo + (uint32_t)(slot * (M::kSlot / 16));
            const uint32_t d = tmem + kColS + (i % kSP) * kTile;
#pragma unroll
            for (int x = 0; x < kProducts; ++x)
#pragma unroll
                for (int y = 0; y < DP / 16; ++y) {
                    const uint32_t qa = q_lo + (x == 0 ? M::kQ / 16 : 0) + (y >> 2) * (kRows * 8) + (y & 3) * 2;
                    const uint32_t ka = kh + (!EXACT && x == 1 ? M::kKV / 16 : 0) + (y >> 2) * (kTile * 8) + (y & 3) * 2;
                    if (x == 0 && y == 0) mma_ss<false>(d, qa, ka, hi, id_s);
                    else mma_ss<true>(d, qa, ka, hi, id_s);
                }
            tc_commit(&bar.s_full[i % kSP]);
            tc_commit(&bar.k_empty[slot]);
            if (++slot == W::kSlots) {
                slot = 0;
                phase ^= 1;
            }
        }
        // every MMA done before tensor memory and shared memory go
        tc_commit(bar.drain);
        (void)mbar_wait(bar.drain, 0);
    } else if (lane == 0) {
        // ===== O = P V =====
        constexpr uint32_t id_o = idesc_f16_f32(kRows, DP, true);
        constexpr int kProducts = EXACT ? 2 : 3;
        const uint64_t v_d = smem_desc_mn_sw128(smem_s + M::offV, kTile * 128, 1024);
        const uint32_t hi = (uint32_t)(v_d >> 32), v_lo = (uint32_t)v_d;
        int slot = 0, phase = 0;
        for (int i = 0; i < n_tiles; ++i) {
            const int s = i & 1;
            if (!bar_wait(&bar.v_full[slot], phase, abort) ||
                (i >= 2 && !bar_wait(&bar.o_empty[s], ((i >> 1) - 1) & 1, abort)) ||
                !bar_wait(&bar.p_full[i % kTab], (i / kTab) & 1, abort))
                break;
            tc_fence_after_sync();
            const uint32_t vh = v_lo + (uint32_t)(slot * (M::kSlot / 16));
            const uint32_t d = tmem + kColO + s * 128, ph = tmem + kColS + (i % kSP) * kTile;
#pragma unroll
            for (int x = 0; x < kProducts; ++x)
#pragma unroll
                for (int y = 0; y < kTile / 16; ++y) {
                    const uint32_t pa = ph + (x == 0 ? 8 : 0) + 16 * y;
                    const uint32_t va = vh + (!EXACT && x == 1 ? M::kKV / 16 : 0) + 128 * y;
                    if (x == 0 && y == 0) mma_ts<false>(d, pa, va, hi, id_o);
                    else mma_ts<true>(d, pa, va, hi, id_o);
                }
            tc_commit(&bar.o_full[s]);
            tc_commit(&bar.v_empty[slot]);
            tc_commit(&bar.sp_empty[i % kSP]);
            if (++slot == W::kSlots) {
                slot = 0;
                phase ^= 1;
            }
        }
        tc_commit(bar.drain + 1);
        (void)mbar_wait(bar.drain + 1, 0);
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == W::kMma) tmem_dealloc(tmem, kTmemCols);
    // (the request is read again: in registers for so long it costs the roles)
    if (threadIdx.x < kRows / 32) a.apart[blockIdx.x].rows[threadIdx.x] = s_apart[threadIdx.x];
    if (threadIdx.x == kRows / 32) {
        a.apart[blockIdx.x].request = s_req;
        a.apart[blockIdx.x].tile = s_tile;
        a.apart[blockIdx.x].uneven = s_uneven;
    }
}

template <int J, int G, int DP>
cudaError_t launch_prompt_t(const AttnCall &call, cudaStream_t stream)
{
    auto kern = attn_prompt_kernel<J, G, DP>;
    constexpr int smem = Mem<J, G, DP>::kBytes;
    static_assert(smem + 256 <= 227 * 1024, "shared memory (and the static part)");
    int dev = 0;
    cudaError_t err;
    if ((err = cudaGetDevice(&dev)) != cudaSuccess) return err;
    static std::atomic<int> ready_dev{-1};
    if (ready_dev.load(std::memory_order_acquire) != dev) {
        if ((err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess)
            return err;
        ready_dev.store(dev, std::memory_order_release);
    }
    const long long grid = call.n_apart;
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
