// gq4_kv.cu -- the paged 4-bit key/value cache: its writer (gq4_kv_append),
// its reader (gq4_kv_gather) and a step's book-keeping (gq4_kv_plan).  The
// layout is stated in gq4.h.
#include <cstdint>

#include "gq4_internal.h"
#include "gq4_kv.cuh"
#include "gq4_quant.cuh"

namespace gq4 {
namespace {

__device__ unsigned int g_kv_error = 0;
constexpr unsigned int kKvNonFinite = 1u << 3, kKvBadSlot = 1u << 6, kKvRefused = 1u << 7;

// ---------------------------------------------------------------------------
// Writer.  A lane holds one word's 8 values, a row takes D/8 lanes; a warp
// takes as many rows as fit (K and V rows of a token count as rows of their
// own), so that a group's minimum and maximum are a shuffle away.  Bound by
// HBM: 4 bytes read and 0.5 + 8/gs written per value.
// ---------------------------------------------------------------------------
constexpr int kAppendThreads = 256;

struct AppendParams {
    gq4_kv_cache c;
    const float *x[2];       // k, v
    int ld[2];
    const int32_t *slots;
    long long n_rows;        // 2 * T * kv_heads
    int wpr;                 // words (lanes) per row
    int rpw;                 // rows per warp
    int L;                   // lanes per group
};

__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendParams p)
{
    const int lane = threadIdx.x & 31;
    const int in_warp = lane / p.wpr, w = lane - in_warp * p.wpr;
    const long long warp0 = ((long long)blockIdx.x * kAppendThreads + threadIdx.x) >> 5;
    const long long n_warps = ((long long)gridDim.x * kAppendThreads) >> 5;
    const int H = p.c.kv_heads, J = p.c.head_dim / 32, G = p.c.head_dim / p.c.group_size;
    const long long total = (long long)p.c.n_pages * p.c.page_size;
    for (long long r0 = warp0 * p.rpw; r0 < p.n_rows; r0 += n_warps * p.rpw) {
        const long long r = r0 + in_warp;
        const bool in = in_warp < p.rpw && r < p.n_rows;
        const long long th = in ? r >> 1 : 0;
        const int side = (int)(r & 1);
        const int t = (int)(th / H), h = (int)(th - (long long)t * H);
        const int slot = in ? __ldg(p.slots + t) : -1;
        if (in && slot >= total && w == 0) atomicOr(&g_kv_error, kKvBadSlot);
        const bool live = slot >= 0 && slot < total;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.0f;
        if (live) {
            const float4 *x = reinterpret_cast<const float4 *>(p.x[side] + (size_t)t * p.ld[side] +
                                                              (size_t)h * p.c.head_dim + 8 * w);
            const float4 a = __ldcs(x), b = __ldcs(x + 1);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        }
        float lo = v[0], hi = v[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) {
            lo = min_nan(lo, v[i]);
            hi = max_nan(hi, v[i]);
        }
        const int pos = w % p.L;
        segment_min_max(lo, hi, pos, lane - pos, p.L);
        int bad;
        const GroupMap m = group_map(lo, hi, bad);
        if (!live) continue;
        const uint32_t word = bad ? 0u : quantize_word(v, m);
        const int page = slot / p.c.page_size, at = slot - page * p.c.page_size;
        const size_t row = kv_row(p.c, page, h, at);
        if (side == 0) {
            p.c.Kq[row * p.wpr + k_word_index(w, J)] = word;
        } else {
            uint16_t *half = reinterpret_cast<uint16_t *>(p.c.Vq) + row * 2 * p.wpr;
            half[v_half_index(2 * w, J)] = (uint16_t)word;
            half[v_half_index(2 * w + 1, J)] = (uint16_t)(word >> 16);
        }
        if (pos == 0) {
            const float nan = __int_as_float(0x7fc00000);
            float2 *sz = reinterpret_cast<float2 *>(side ? p.c.V_sz : p.c.K_sz);
            sz[row * G + w / p.L] = bad ? make_float2(nan, nan) : make_float2(m.s, m.z);
            if (bad) atomicOr(&g_kv_error, kKvNonFinite);
        }
    }
}

// ---------------------------------------------------------------------------
// Reader: a lane dequantises 4 consecutive values (half a word), a warp
// stores 512 contiguous bytes at a time.
// ---------------------------------------------------------------------------
struct GatherParams {
    gq4_kv_cache c;
    const int32_t *slots;
    float4 *y[2];
    long long n_items;       // float4s per side
    int f4;                  // float4s per row
};

__global__ void __launch_bounds__(256) gather_kernel(const __grid_constant__ GatherParams p)
{
    const int H = p.c.kv_heads, J = p.c.head_dim / 32, G = p.c.head_dim / p.c.group_size;
    const long long total = (long long)p.c.n_pages * p.c.page_size;
    const int side = blockIdx.y;
    const uint16_t *half = reinterpret_cast<const uint16_t *>(side ? p.c.Vq : p.c.Kq);
    const float2 *sz = reinterpret_cast<const float2 *>(side ? p.c.V_sz : p.c.K_sz);
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < p.n_items; i += (long long)gridDim.x * 256) {
        const long long th = i / p.f4;
        const int f = (int)(i - th * p.f4);
        const int t = (int)(th / H), h = (int)(th - (long long)t * H);
        const int slot = __ldg(p.slots + t);
        if (slot < 0) continue;
        if (slot >= total) {
            const float nan = __int_as_float(0x7fc00000);
            p.y[side][i] = make_float4(nan, nan, nan, nan);
            if (f == 0) atomicOr(&g_kv_error, kKvBadSlot);
            continue;
        }
        const int page = slot / p.c.page_size, at = slot - page * p.c.page_size;
        const size_t row = kv_row(p.c, page, h, at);
        const int hi = side ? v_half_index(f, J) : 2 * k_word_index(f >> 1, J) + (f & 1);
        const uint32_t q = half[row * p.f4 + hi];
        const float2 m = sz[row * G + f * 4 / p.c.group_size];
        p.y[side][i] = make_float4(__fmul_rn(__fsub_rn((float)(q & 15u), m.y), m.x),
                                   __fmul_rn(__fsub_rn((float)((q >> 4) & 15u), m.y), m.x),
                                   __fmul_rn(__fsub_rn((float)((q >> 8) & 15u), m.y), m.x),
                                   __fmul_rn(__fsub_rn((float)((q >> 12) & 15u), m.y), m.x));
    }
}

// ---------------------------------------------------------------------------
// Book-keeping: one CTA; a scan over the requests' rows and pages in tiles
// of the CTA's threads, then the requests' tokens and table entries.
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;

// Inclusive sum over the CTA's threads.
__device__ __forceinline__ long long scan_sum(long long v, long long *warp_sums)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    if (warp == 0) {
        long long s = warp_sums[lane];
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += u;
        }
        warp_sums[lane] = s;
    }
    __syncthreads();
    if (warp > 0) v += warp_sums[warp - 1];
    const long long total = warp_sums[31];
    __syncthreads();
    if (threadIdx.x == 0) warp_sums[0] = total;
    __syncthreads();
    return v;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ PlanCall p)
{
    __shared__ long long sums[32];
    const long long room = (long long)p.max_pages * p.page;
    const int avail = min(max(*p.free_count, 0), p.n_free);
    long long rows_before = 0, pages_before = 0;
    int granted = 0;   // pages, the same in every thread
    __shared__ int s_granted;
    if (threadIdx.x == 0) s_granted = 0;
    for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
        const int b = b0 + threadIdx.x;
        const bool in = b < p.B;
        const int past0 = in ? p.past_lens[b] : 0, new0 = in ? p.new_lens[b] : 0;
        const int past = max(past0, 0), fresh = max(new0, 0);
        bool refused = past0 < 0 || new0 < 0;
        const long long row_end = rows_before + scan_sum(fresh, sums);
        const long long rows_total = rows_before + sums[0];
        __syncthreads();
        refused |= (long long)past + fresh > room || row_end > p.T;
        // refused requests aside, past + new stays below 2^31
        const int had = refused ? 0 : (past + p.page - 1) / p.page;
        const int need = refused ? 0 : (past + fresh + p.page - 1) / p.page - had;
        const long long page_end = pages_before + scan_sum(need, sums);
        const long long pages_total = pages_before + sums[0];
        __syncthreads();
        if (need > 0 && page_end > avail) refused = true;
        if (in) {
            const long long start = min(row_end - fresh, (long long)p.T), end = min(row_end, (long long)p.T);
            p.query_start[b + 1] = (int)end;
            if (b == 0) p.query_start[0] = 0;
            p.seq_lens[b] = refused ? past : past + fresh;
            int32_t *table = p.page_table + (size_t)b * p.max_pages;
            const long long page_start = page_end - need;
            if (!refused) {
                for (int j = 0; j < need; ++j) table[had + j] = p.free_pages[avail - 1 - (page_start + j)];
                if (need > 0) atomicMax(&s_granted, (int)page_end);
            } else if (fresh > 0 || past0 < 0 || new0 < 0) {
                atomicOr(&g_kv_error, kKvRefused);
            }
            for (long long t = start; t < end; ++t) {
                const int pos = refused ? 0 : past + (int)(t - start);
                p.positions[t] = pos;
                p.slots[t] = refused ? -1 : table[pos / p.page] * p.page + pos % p.page;
            }
        }
        rows_before = rows_total;
        pages_before = pages_total;
    }
    __syncthreads();
    granted = s_granted;
    for (long long t = min(rows_before, (long long)p.T) + threadIdx.x; t < p.T; t += kPlanThreads) {
        p.positions[t] = 0;
        p.slots[t] = -1;
    }
    if (threadIdx.x == 0) *p.free_count_out = avail - granted;
}

cudaError_t device_sms(int &sms)
{
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    return cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
}

}  // namespace

cudaError_t launch_kv_append(int T, const gq4_kv_cache &c, const float *k, int ldk, const float *v,
                             int ldv, const int32_t *slots, cudaStream_t stream)
{
    int sms = 0;
    cudaError_t err = device_sms(sms);
    if (err != cudaSuccess) return err;
    AppendParams p{};
    p.c = c;
    p.x[0] = k;
    p.x[1] = v;
    p.ld[0] = ldk;
    p.ld[1] = ldv;
    p.slots = slots;
    p.n_rows = 2ll * T * c.kv_heads;
    p.wpr = c.head_dim / 8;
    p.rpw = 32 / p.wpr;
    p.L = c.group_size / 8;
    const long long rows_per_block = (long long)p.rpw * (kAppendThreads / 32);
    const long long want = (p.n_rows + rows_per_block - 1) / rows_per_block, cap = 8ll * sms;
    append_kernel<<<(unsigned)(want < cap ? want : cap), kAppendThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_kv_gather(int T, const gq4_kv_cache &c, const int32_t *slots, float *k_out,
                             float *v_out, cudaStream_t stream)
{
    int sms = 0;
    cudaError_t err = device_sms(sms);
    if (err != cudaSuccess) return err;
    GatherParams p{};
    p.c = c;
    p.slots = slots;
    p.y[0] = reinterpret_cast<float4 *>(k_out);
    p.y[1] = reinterpret_cast<float4 *>(v_out);
    p.f4 = c.head_dim / 4;
    p.n_items = (long long)T * c.kv_heads * p.f4;
    const long long want = (p.n_items + 255) / 256, cap = 8ll * sms;
    gather_kernel<<<dim3((unsigned)(want < cap ? want : cap), 2), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_kv_plan(const PlanCall &call, cudaStream_t stream)
{
    plan_kernel<<<1, kPlanThreads, 0, stream>>>(call);
    return cudaGetLastError();
}

cudaError_t read_kv_device_error(unsigned int *bits, bool clear)
{
    cudaError_t err = cudaMemcpyFromSymbol(bits, g_kv_error, sizeof(unsigned int));
    if (err != cudaSuccess || !clear) return err;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_kv_error, &zero, sizeof(unsigned int));
}

}  // namespace gq4
