// gq4_kv.cu -- the paged 4-bit key/value cache: its writer (gq4_kv_append),
// its reader (gq4_kv_gather) and a step's book-keeping (gq4_kv_plan).  The
// layout is stated in gq4.h.
#include <cstdint>

#include "gq4_kv_internal.h"
#include "gq4_kv_write.cuh"

namespace gq4 {
namespace {

__device__ unsigned int g_kv_error = 0;
constexpr unsigned int kKvRefused = 1u << 7;

// ---------------------------------------------------------------------------
// Writer.  A lane holds one word's 8 values, a row takes D/8 lanes; a warp
// takes as many rows as fit, so that a group's minimum and maximum are a
// shuffle away.  The K and V rows of a few tokens are one CTA's, numbered in
// 32 bits; a row's loads do not wait for its slot.  Floor: 4 bytes read and
// 0.5 + 8/gs written per value; 16381 tokens of 8 heads of 128 take 30 us
// (153 MB, 5.1 TB/s).  What is left is instructions: 194 per word and warp, a
// quarter of them the group's two divisions and reciprocal (with the lanes of
// a group a run-time number it was 225, and 35 us).
// ---------------------------------------------------------------------------
constexpr int kAppendThreads = 256;
constexpr int kAppendUnroll = 2;   // rows per lane whose loads are issued together

struct AppendParams {
    gq4_kv_cache c;
    const float *x[2];       // k, v
    int ld[2];
    const int32_t *slots;
    int T, tokens;           // all, and per CTA
    int shift;               // log2 of the page size
    int total;               // slots of the pool
    uint32_t page_codes, page_sz;   // bytes per page and head
    uint32_t per_2h;         // divides a CTA's rows by 2 heads
};

// J = head_dim / 32; L: lanes per group.
template <int J, int L>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendParams p)
{
    constexpr int WPR = 4 * J, RPW = 32 / WPR;   // words per row, rows per warp
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int in_warp = lane / WPR, w = lane - in_warp * WPR;
    const int H = p.c.kv_heads;
    const int pos = w % L;
    const int t0 = blockIdx.x * p.tokens;
    const int n_rows = min(p.tokens, p.T - t0) * 2 * H;
    constexpr int kStep = kAppendThreads / 32 * RPW;
    for (int r0 = warp * RPW; r0 < n_rows; r0 += kAppendUnroll * kStep) {
        float4 va[kAppendUnroll], vb[kAppendUnroll];
        int slot[kAppendUnroll], head[kAppendUnroll];
#pragma unroll
        for (int u = 0; u < kAppendUnroll; ++u) {
            const int r = r0 + u * kStep + in_warp;
            slot[u] = -1;
            head[u] = 0;
            va[u] = vb[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (in_warp < RPW && r < n_rows) {
                // rows of a token: its K rows, then its V rows
                const int t = quotient(r, p.per_2h), sh = r - t * 2 * H;
                const bool side = sh >= H;
                const int h = side ? sh - H : sh;
                head[u] = 2 * h + side;
                slot[u] = __ldg(p.slots + t0 + t);
                const float4 *x = reinterpret_cast<const float4 *>(
                    (side ? p.x[1] : p.x[0]) + (size_t)(t0 + t) * (side ? p.ld[1] : p.ld[0]) + h * (32 * J) + 8 * w);
                va[u] = __ldcs(x);
                vb[u] = __ldcs(x + 1);
            }
        }
#pragma unroll
        for (int u = 0; u < kAppendUnroll; ++u) {
            if (r0 + u * kStep >= n_rows) break;   // uniform in the warp
            const float v[8] = {va[u].x, va[u].y, va[u].z, va[u].w, vb[u].x, vb[u].y, vb[u].z, vb[u].w};
            float lo = v[0], hi = v[0];
#pragma unroll
            for (int i = 1; i < 8; ++i) {
                lo = min_nan(lo, v[i]);
                hi = max_nan(hi, v[i]);
            }
            segment_min_max(lo, hi, pos, lane - pos, L);
            int bad;
            const GroupMap m = group_map(lo, hi, bad);
            uint32_t word = bad ? 0u : quantize_word(v, m);
            const int side = head[u] & 1, h = head[u] >> 1;
            // value halves of words w and w + 4 are neighbours: one lane stores
            // the first halves of both, the other the second
            const uint32_t other = __shfl_xor_sync(0xffffffffu, word, 4);
            if (slot[u] < 0) continue;
            write_word<J, L>(p, slot[u], h, side, w, word, other, bad, m, &g_kv_error);
        }
    }
}

// ---------------------------------------------------------------------------
// Reader: a lane dequantises 4 consecutive values (half a word), so that a
// warp stores 512 contiguous bytes at a time; the same 4 of every row that it
// takes.  Bound by HBM writes: 16381 tokens of 8 heads of 128 take 22 us
// (153 MB, 7.0 TB/s) with the codes in L2, just written, and 27 cold.
// ---------------------------------------------------------------------------
struct GatherParams {
    gq4_kv_cache c;
    const int32_t *slots;
    float4 *y[2];
    int T, tokens;           // all, and per CTA
    int shift;
    int total;               // slots of the pool
    uint32_t page_codes, page_sz;   // bytes per page and head
    uint32_t per_h;          // divides a CTA's rows by the heads
};

constexpr int kGatherUnroll = 4;

template <int J>
constexpr int kGatherThreads = J == 3 ? 192 : 256;   // whole rows

// The codes q & 15 and (q >> 4) & 15 as floats: 2^23 + code, less 2^23.
__device__ __forceinline__ f32x2 codes_of(uint32_t q)
{
    return add2(pack2(__uint_as_float((q & 15u) | 0x4b000000u), __uint_as_float(((q >> 4) & 15u) | 0x4b000000u)),
                pack2(-8388608.0f, -8388608.0f));
}

template <int J>
__global__ void __launch_bounds__(kGatherThreads<J>) gather_kernel(const __grid_constant__ GatherParams p)
{
    constexpr int F4 = 8 * J, ROWS = kGatherThreads<J> / F4;   // float4s per row, rows at once
    const int H = p.c.kv_heads, G = 32 * J / p.c.group_size;
    const int side = blockIdx.y;
    const int f = threadIdx.x % F4;
    const uint16_t *half = reinterpret_cast<const uint16_t *>(side ? p.c.Vq : p.c.Kq) +
                           (side ? v_half_index(f, J) : 2 * k_word_index(f >> 1, J) + (f & 1));
    const float2 *sz = reinterpret_cast<const float2 *>(side ? p.c.V_sz : p.c.K_sz) + f * 4 / p.c.group_size;
    const int t0 = blockIdx.x * p.tokens;
    const int n = min(p.tokens, p.T - t0) * H;
    float4 *y = p.y[side] + (size_t)t0 * H * F4 + f;
    for (int r0 = threadIdx.x / F4; r0 < n; r0 += ROWS * kGatherUnroll) {
        int slot[kGatherUnroll];
        uint32_t q[kGatherUnroll];
        float2 m[kGatherUnroll];
#pragma unroll
        for (int u = 0; u < kGatherUnroll; ++u) {
            const int r = r0 + u * ROWS;
            slot[u] = r < n ? __ldg(p.slots + t0 + quotient(r, p.per_h)) : -1;
        }
#pragma unroll
        for (int u = 0; u < kGatherUnroll; ++u) {
            const int r = r0 + u * ROWS, h = r - quotient(r, p.per_h) * H;
            if (slot[u] >= 0 && slot[u] < p.total) {
                const RowAt row(p.c, slot[u], p.shift, h);
                q[u] = *row.in(half, p.page_codes, 2 * F4);
                m[u] = *row.in(sz, p.page_sz, 8 * G);
            }
        }
#pragma unroll
        for (int u = 0; u < kGatherUnroll; ++u) {
            float4 *to = y + (uint32_t)(r0 + u * ROWS) * F4;
            if (slot[u] < 0) continue;
            if (slot[u] >= p.total) {
                const float nan = __int_as_float(0x7fc00000);
                *to = make_float4(nan, nan, nan, nan);
                atomicOr(&g_kv_error, kKvBadSlot);
                continue;
            }
            const f32x2 z = pack2(-m[u].y, -m[u].y), scale = pack2(m[u].x, m[u].x);
            const float2 a = unpack2(mul2(add2(codes_of(q[u]), z), scale));
            const float2 b = unpack2(mul2(add2(codes_of(q[u] >> 8), z), scale));
            __stcs(to, make_float4(a.x, a.y, b.x, b.y));
        }
    }
}

// ---------------------------------------------------------------------------
// Book-keeping.  Every CTA scans all requests' rows and pages itself, a tile
// of 1024 requests at a time in shared memory, and then writes its share of
// the tile's tokens and granted pages: a token finds its request by bisection
// of the tile's first rows.  So no CTA waits for another, unless lengths or
// the count are advanced in place: then the CTAs are one cluster, which meets
// after the tile is read and before it is overwritten.  Latency-bound (a few
// kB): 64 requests of one token 4 us, 2000 requests of up to 256 tokens (257k
// tokens, 2.1 MB written) 10 us.
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;

// Inclusive sum over the CTA's threads, and the total.
__device__ __forceinline__ long long scan_sum(long long v, long long &total, long long *sums)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    if (lane == 31) sums[warp] = v;
    __syncthreads();
    long long s = sums[lane];      // every warp scans the warps' sums itself
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
    }
    total = __shfl_sync(0xffffffffu, s, 31);
    const long long before = __shfl_sync(0xffffffffu, s, (warp + 31) & 31);
    return v + (warp > 0 ? before : 0);
}

// Last i in [0, n) with first[i] <= t, given first[0] <= t.
__device__ __forceinline__ int find_last(const int *first, int n, int t)
{
    int lo = 0, hi = n;            // first[lo] <= t < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

template <bool IN_PLACE>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ PlanCall p, int shift)
{
    __shared__ long long sums[2][32];
    __shared__ int s_row[kPlanThreads], s_page[kPlanThreads], s_past[kPlanThreads], s_had[kPlanThreads];
    __shared__ int s_granted;
    const int cta = blockIdx.x, n_cta = gridDim.x;
    const long long room = (long long)p.max_pages << shift;
    const int avail = min(max(*p.free_count, 0), p.n_free);
    long long rows_before = 0, pages_before = 0;
    if (threadIdx.x == 0) s_granted = 0;
    for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
        const int b = b0 + threadIdx.x, n = min(kPlanThreads, p.B - b0);
        const bool in = b < p.B;
        const int past0 = in ? p.past_lens[b] : 0, new0 = in ? p.new_lens[b] : 0;
        const int past = max(past0, 0), fresh = max(new0, 0);
        bool refused = past0 < 0 || new0 < 0;
        long long rows_in, pages_in;
        const long long row_end = rows_before + scan_sum(fresh, rows_in, sums[0]);
        refused |= (long long)past + fresh > room || (fresh > 0 && row_end > p.T);
        // refused requests aside, past + new stays below 2^31
        const int had = refused ? 0 : (past + p.page - 1) >> shift;
        const int need = refused ? 0 : ((past + fresh + p.page - 1) >> shift) - had;
        const long long page_end = pages_before + scan_sum(need, pages_in, sums[1]);
        if (need > 0 && page_end > avail) refused = true;
        s_row[threadIdx.x] = (int)min(row_end - fresh, (long long)p.T);
        s_page[threadIdx.x] = (int)min(page_end - need, (long long)0x7fffffff);
        s_past[threadIdx.x] = refused ? -1 : past;
        s_had[threadIdx.x] = had;
        if (!refused && need > 0) atomicMax(&s_granted, (int)page_end);
        if (IN_PLACE) {
            asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        } else {
            __syncthreads();
        }
        if (cta == 0 && in) {
            p.query_start[b + 1] = (int)min(row_end, (long long)p.T);
            if (b == 0) p.query_start[0] = 0;
            p.seq_lens[b] = refused ? past : past + fresh;
            if (refused) atomicOr(&g_kv_error, kKvRefused);
        }
        // granted pages of this tile
        const int granted = s_granted;
        const int page_hi = (int)min(pages_before + pages_in, (long long)granted);
        // (unsigned: a stride past the last row or page may pass 2^31)
        const unsigned lead = cta * kPlanThreads + threadIdx.x, step = n_cta * kPlanThreads;
        for (unsigned u = (unsigned)min(pages_before, (long long)granted) + lead; u < (unsigned)page_hi; u += step) {
            const int k = (int)u, i = find_last(s_page, n, k);
            p.page_table[(size_t)(b0 + i) * p.max_pages + s_had[i] + (k - s_page[i])] = p.free_pages[avail - 1 - k];
        }
        // its tokens
        const int row_hi = (int)min(rows_before + rows_in, (long long)p.T);
        for (unsigned u = (unsigned)min(rows_before, (long long)p.T) + lead; u < (unsigned)row_hi; u += step) {
            const int t = (int)u, i = find_last(s_row, n, t);
            int pos = 0, slot = -1;
            if (s_past[i] >= 0) {
                pos = s_past[i] + (t - s_row[i]);
                const int pg = pos >> shift;
                // a granted page from the list itself: its table entry may be another CTA's
                const int id = pg >= s_had[i] ? p.free_pages[avail - 1 - (s_page[i] + pg - s_had[i])]
                                              : p.page_table[(size_t)(b0 + i) * p.max_pages + pg];
                // an id without slots (they would wrap into the pool): a slot outside any
                slot = (unsigned)id < (0x80000000u >> shift) ? (id << shift) + (pos & (p.page - 1)) : 0x7fffffff;
            }
            p.positions[t] = pos;
            p.slots[t] = slot;
        }
        rows_before += rows_in;
        pages_before += pages_in;
        __syncthreads();
    }
    for (unsigned t = (unsigned)min(rows_before, (long long)p.T) + cta * kPlanThreads + threadIdx.x; t < (unsigned)p.T;
         t += n_cta * kPlanThreads) {
        p.positions[t] = 0;
        p.slots[t] = -1;
    }
    if (cta == 0 && threadIdx.x == 0) *p.free_count_out = avail - s_granted;
}

}  // namespace

namespace {

// Tokens per CTA so that each of its threads has `items` of `per_token`.
int tokens_per_cta(int per_token, int items)
{
    const int t = (256 * items + per_token - 1) / per_token;
    return t < 1 ? 1 : t;
}

}  // namespace

cudaError_t launch_kv_append(int T, const gq4_kv_cache &c, const float *k, int ldk, const float *v,
                             int ldv, const int32_t *slots, cudaStream_t stream)
{
    AppendParams p{};
    p.c = c;
    p.x[0] = k;
    p.x[1] = v;
    p.ld[0] = ldk;
    p.ld[1] = ldv;
    p.slots = slots;
    p.T = T;
    p.shift = log2_of(c.page_size);
    p.total = c.n_pages * c.page_size;
    p.page_codes = (uint32_t)(c.page_size * c.head_dim / 2);
    p.page_sz = (uint32_t)(c.page_size * (c.head_dim / c.group_size) * 8);
    p.per_2h = divide_by(2 * c.kv_heads);
    // a lane takes two words of a long prompt; one while tokens are few, so
    // that they spread over the GPU
    p.tokens = tokens_per_cta(2 * c.kv_heads * (c.head_dim / 8), T >= 1024 ? 2 * kAppendUnroll : 1);
    const unsigned grid = (unsigned)((T + p.tokens - 1) / p.tokens);
    auto run = [&](auto kern) { kern<<<grid, kAppendThreads, 0, stream>>>(p); };
    switch (c.head_dim * 16 + c.group_size / 32) {
    case 64 * 16 + 1: run(append_kernel<2, 4>); break;
    case 64 * 16 + 2: run(append_kernel<2, 8>); break;
    case 96 * 16 + 1: run(append_kernel<3, 4>); break;
    case 96 * 16 + 3: run(append_kernel<3, 12>); break;
    case 128 * 16 + 1: run(append_kernel<4, 4>); break;
    case 128 * 16 + 2: run(append_kernel<4, 8>); break;
    case 128 * 16 + 4: run(append_kernel<4, 16>); break;
    case 256 * 16 + 1: run(append_kernel<8, 4>); break;
    case 256 * 16 + 2: run(append_kernel<8, 8>); break;
    case 256 * 16 + 4: run(append_kernel<8, 16>); break;
    case 256 * 16 + 8: run(append_kernel<8, 32>); break;
    default: return cudaErrorInvalidValue;
    }
    return cudaGetLastError();
}

cudaError_t launch_kv_gather(int T, const gq4_kv_cache &c, const int32_t *slots, float *k_out,
                             float *v_out, cudaStream_t stream)
{
    GatherParams p{};
    p.c = c;
    p.slots = slots;
    p.y[0] = reinterpret_cast<float4 *>(k_out);
    p.y[1] = reinterpret_cast<float4 *>(v_out);
    p.T = T;
    p.shift = log2_of(c.page_size);
    p.total = c.n_pages * c.page_size;
    p.page_codes = (uint32_t)(c.page_size * c.head_dim / 2);
    p.page_sz = (uint32_t)(c.page_size * (c.head_dim / c.group_size) * 8);
    p.per_h = divide_by(c.kv_heads);
    p.tokens = tokens_per_cta(c.kv_heads * (c.head_dim / 4), T >= 1024 ? 2 * kGatherUnroll : 1);
    const dim3 grid((unsigned)((T + p.tokens - 1) / p.tokens), 2);
    switch (c.head_dim) {
    case 64: gather_kernel<2><<<grid, kGatherThreads<2>, 0, stream>>>(p); break;
    case 96: gather_kernel<3><<<grid, kGatherThreads<3>, 0, stream>>>(p); break;
    case 128: gather_kernel<4><<<grid, kGatherThreads<4>, 0, stream>>>(p); break;
    default: gather_kernel<8><<<grid, kGatherThreads<8>, 0, stream>>>(p); break;
    }
    return cudaGetLastError();
}

cudaError_t launch_kv_plan(const PlanCall &call, cudaStream_t stream)
{
    const int shift = log2_of(call.page);
    const bool in_place = call.seq_lens == call.past_lens || call.free_count_out == call.free_count;
    // a CTA for every 4096 token rows; in place at most one portable cluster
    const long long want = ((long long)call.T + 4095) / 4096, most = in_place ? 8 : 128;
    const long long grid = want < 1 ? 1 : want > most ? most : want;
    if (!in_place) {
        plan_kernel<false><<<(unsigned)grid, kPlanThreads, 0, stream>>>(call, shift);
        return cudaGetLastError();
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)grid;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, plan_kernel<true>, call, shift);
}

cudaError_t read_kv_device_error(unsigned int *bits, bool clear)
{
    cudaError_t err = cudaMemcpyFromSymbol(bits, g_kv_error, sizeof(unsigned int));
    if (err != cudaSuccess || !clear) return err;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_kv_error, &zero, sizeof(unsigned int));
}

}  // namespace gq4
