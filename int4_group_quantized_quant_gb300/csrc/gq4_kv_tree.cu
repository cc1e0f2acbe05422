// gq4_kv_tree.cu -- the book-keeping of drafted trees: positions and ancestor
// bits from the parents (gq4_kv_tree), and what follows a verification
// (gq4_kv_accept): the accepted rows moved to the end of their request, its
// length, and its surplus pages back on the free list.
#include <cstdint>

#include "gq4_kv_internal.h"
#include "gq4_kv.cuh"

namespace gq4 {
namespace {

__device__ unsigned int g_tree_error = 0;
constexpr unsigned int kTreeRefused = 1u << 10, kAcceptRefused = 1u << 11;
constexpr int kMaxNodes = 32 * GQ4_MAX_TREE_WORDS;

// Whether the planning refused a request: its rows from q0 on, if there are any,
// got no slots, and it has no new tokens though its length counts none.  slots:
// as planned, or NULL (none was refused).
__device__ __forceinline__ bool plan_refused(const int32_t *slots, int T, int q0, long long rows)
{
    return slots && rows > 0 && q0 >= 0 && q0 < T && __ldg(slots + q0) < 0;
}

// ---------------------------------------------------------------------------
// A CTA per request, its parents in shared memory, a thread per node that walks
// up to its root twice: for its depth, and for the bits.  A parent comes before
// its children, so the walk meets the words from the last to the first and one
// register holds the word under way.  Latency-bound, a few kB: 15 nodes 2.4 us,
// 256 trees of up to 60 nodes 3.8 us.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kMaxNodes) tree_kernel(const __grid_constant__ TreeCall p)
{
    __shared__ int16_t up[kMaxNodes];
    const int b = blockIdx.x, i = threadIdx.x;
    const int q0 = __ldg(p.query_start + b), q1 = __ldg(p.query_start + b + 1), len = __ldg(p.seq_lens + b);
    const long long n = (long long)q1 - q0, past = len - n;
    const bool none = plan_refused(p.slots, p.T, q0, n);
    bool bad = none || n < 0 || n > 32 * p.words || q0 < 0 || q1 > p.T || len < 0 || past < 0;
    if (!bad && i < n) {
        const int parent = __ldg(p.parents + q0 + i);
        bad = parent < -1 || parent >= i;
        up[i] = (int16_t)parent;
    }
    if (__syncthreads_or(bad)) {
        if (i == 0 && n != 0 && !none) atomicOr(&g_tree_error, kTreeRefused);
        for (long long row = max(q0, 0) + i; row < min(q1, p.T); row += blockDim.x) {
            p.positions[row] = 0;
            for (int w = 0; w < p.words; ++w) p.bits[row * p.words + w] = 0u;
        }
        return;
    }
    if (i >= n) return;
    int depth = 0;
    for (int j = up[i]; j >= 0; j = up[j]) ++depth;
    const size_t row = (size_t)(q0 + i);
    p.positions[row] = (int)past + depth;
    // steps from the node to where the walk is; it leaves the window at `window`
    // steps, and is back in sight where the position is one of the first
    int j = i, steps = 0;
    for (int w = p.words - 1; w >= 0; --w) {
        uint32_t word = 0;
        for (; j >= 32 * w; j = up[j], ++steps)
            if (p.window <= 0 || steps < p.window || past + depth - steps < p.sinks) word |= 1u << (j & 31);
        p.bits[row * p.words + w] = word;
    }
}

// ---------------------------------------------------------------------------
// Accepting a path.  The first kernel, a CTA per request and share of its
// columns, checks the request and moves its rows: new row path[i] comes to lie
// at row i.  A path rises, so row i is never read after it is written: each
// thread takes a piece of a row (16 bytes of codes, or a scale and zero) along
// the whole path, 8 loads before their stores.  Its verdict is left in the
// workspace for the second kernel, one CTA, which counts the pages left over,
// request after request, and writes the lengths and the list: so lengths and the
// count may be advanced in place.
// ---------------------------------------------------------------------------
constexpr int kMoveThreads = 128, kBookThreads = 1024;
constexpr int kPathTile = 256;

// A request's rows, and whether they can be (before its path is looked at).
// PLANNED: with slots (a form of its own: their load, and the branch around it,
// cost the other 0.4 us).
template <bool PLANNED>
struct Drafted {
    int past, n, len;
    bool none, bad;        // none: the planning refused it, all of its tokens stay

    __device__ __forceinline__ Drafted(const AcceptCall &p, int b, int shift)
    {
        const int q0 = __ldg(p.query_start + b), q1 = __ldg(p.query_start + b + 1);
        const long long rows = (long long)q1 - q0;
        len = __ldg(p.seq_lens + b);
        none = PLANNED && plan_refused(p.slots, p.T, q0, rows);
        bad = !none && (rows < 0 || rows > len || (long long)len > ((long long)p.max_pages << shift) ||
                        (PLANNED && rows > 0 && (q0 < 0 || q1 > p.T)));
        n = none || bad ? 0 : (int)rows;
        past = len - n;
    }
};

template <bool PLANNED>
__global__ void __launch_bounds__(kMoveThreads) accept_move_kernel(const __grid_constant__ AcceptCall p, int shift)
{
    __shared__ int s_from[kPathTile], s_to[kPathTile];   // stretches of a page's rows: page id and row of the page
    const int b = blockIdx.x;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Drafted<PLANNED> r(p, b, shift);
    const int count = r.none ? 0 : __ldg(p.counts + b);
    const int32_t *path = p.path ? p.path + (size_t)b * p.max_path : nullptr;
    const int32_t *table = p.page_table + (size_t)b * p.max_pages;
    bool bad = r.bad || count < 0 || count > r.n || (path && count > p.max_path);
    if (!bad) {
        if (path)
            for (int i = threadIdx.x; i < count; i += kMoveThreads) {
                const int node = __ldg(path + i), before = i > 0 ? __ldg(path + i - 1) : -1;
                bad |= node <= before || node >= r.n;
            }
        if (r.n > 0)
            for (int i = (r.past >> shift) + (int)threadIdx.x; i <= (r.len - 1) >> shift; i += kMoveThreads)
                bad |= (uint32_t)__ldg(table + i) >= (uint32_t)p.c.n_pages;
    }
    bad = __syncthreads_or(bad);
    if (blockIdx.y == 0 && threadIdx.x == 0) p.verdict[b] = bad ? -1 : count;
    if (bad || !path) return;
    // this thread's piece: of a head's row, codes of K and V in 16 bytes, scales and zeros in 8
    const int J = p.c.head_dim / 32, G = p.c.head_dim / p.c.group_size;
    const int per = 2 * J + 2 * G, pieces = per * p.c.kv_heads;
    const uint32_t page_rows = (uint32_t)p.c.kv_heads << shift;
    for (int i0 = 0; i0 < count; i0 += kPathTile) {
        const int tile = min(kPathTile, count - i0);
        for (int i = threadIdx.x; i < tile; i += kMoveThreads) {
            const int from = r.past + __ldg(path + i0 + i), to = r.past + i0 + i, mask = (1 << shift) - 1;
            // (a pool holds fewer than 2^31 rows of one head; the heads come with 64 bits)
            s_from[i] = from == to ? -1 : (__ldg(table + (from >> shift)) << shift) + (from & mask);
            s_to[i] = (__ldg(table + (to >> shift)) << shift) + (to & mask);
        }
        __syncthreads();
        for (int x = blockIdx.y * kMoveThreads + threadIdx.x; x < pieces; x += gridDim.y * kMoveThreads) {
            const int h = x / per, y = x - h * per;
            auto place = [&](char *base, int slot, uint32_t bytes) {
                const size_t row = (size_t)(uint32_t)(slot >> shift) * page_rows + ((uint32_t)h << shift) + (slot & ((1 << shift) - 1));
                return base + row * bytes;
            };
            auto move = [&](auto unit, char *base, uint32_t bytes) {
                using V = decltype(unit);
                constexpr int kAhead = 8;
                for (int i = 0; i < tile; i += kAhead) {
                    V v[kAhead];
                    int from[kAhead];
#pragma unroll
                    for (int k = 0; k < kAhead; ++k) {
                        from[k] = i + k < tile ? s_from[i + k] : -1;
                        if (from[k] >= 0) v[k] = *reinterpret_cast<const V *>(place(base, from[k], bytes));
                    }
#pragma unroll
                    for (int k = 0; k < kAhead; ++k)
                        if (from[k] >= 0) *reinterpret_cast<V *>(place(base, s_to[i + k], bytes)) = v[k];
                }
            };
            if (y < 2 * J)
                move(uint4{}, reinterpret_cast<char *>(y < J ? p.c.Kq : p.c.Vq) + (y < J ? y : y - J) * 16, 16 * J);
            else
                move(uint2{}, reinterpret_cast<char *>(y - 2 * J < G ? p.c.K_sz : p.c.V_sz) + (y - 2 * J - (y - 2 * J < G ? 0 : G)) * 8, 8 * G);
        }
        __syncthreads();
    }
}

template <bool PLANNED>
__global__ void __launch_bounds__(kBookThreads) accept_book_kernel(const __grid_constant__ AcceptCall p, int shift)
{
    __shared__ int s_sums[kBookThreads / 32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int top = min(max(__ldcg(p.free_count), 0), p.n_free);
    long long before = 0;       // pages given back by the requests so far
    for (int b0 = 0; b0 < p.B; b0 += kBookThreads) {
        const int b = b0 + (int)threadIdx.x;
        int back = 0, had = 0;
        if (b < p.B) {
            const Drafted<PLANNED> r(p, b, shift);
            const int verdict = __ldcg(p.verdict + b), len = verdict < 0 ? r.len : r.past + verdict;
            had = (int)(((long long)len + (1 << shift) - 1) >> shift);
            if (verdict < 0) atomicOr(&g_tree_error, kAcceptRefused);
            else back = (int)(((long long)r.len + (1 << shift) - 1) >> shift) - had;
            p.seq_lens_out[b] = len;
        }
        int inc = back;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) s_sums[warp] = inc;
        __syncthreads();
        long long at = before + inc - back, all = 0;
#pragma unroll 8
        for (int i = 0; i < kBookThreads / 32; ++i) {
            if (i < warp) at += s_sums[i];
            all += s_sums[i];
        }
#pragma unroll 1
        for (int i = 0; i < back; ++i) {
            // (unsigned: counts that overflow, of tables that name pages over and over, lead nowhere)
            if ((unsigned long long)(top + at + i) < (unsigned long long)p.n_free) p.free_pages[top + at + i] = __ldg(p.page_table + (size_t)b * p.max_pages + had + i);
            else atomicOr(&g_tree_error, kAcceptRefused);
        }
        before += all;
        __syncthreads();
    }
    if (threadIdx.x == 0) *p.free_count_out = (int)min(top + before, (long long)p.n_free);
}

}  // namespace

cudaError_t launch_kv_tree(const TreeCall &call, cudaStream_t stream)
{
    tree_kernel<<<(unsigned)call.B, 32 * call.words, 0, stream>>>(call);
    return cudaGetLastError();
}

template <bool PLANNED>
static cudaError_t launch_accept(const AcceptCall &call, cudaStream_t stream)
{
    const int shift = log2_of(call.c.page_size);
    // few requests: their columns over several CTAs, until the GPU has one each
    const int pieces = (2 * (call.c.head_dim / 32) + 2 * (call.c.head_dim / call.c.group_size)) * call.c.kv_heads;
    int splits = 1;
    if (call.path)
        while (splits * kMoveThreads < pieces && (long long)call.B * splits < 152) ++splits;
    accept_move_kernel<PLANNED><<<dim3((unsigned)call.B, (unsigned)splits), kMoveThreads, 0, stream>>>(call, shift);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kBookThreads);
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, accept_book_kernel<PLANNED>, call, shift);
}

cudaError_t launch_kv_accept(const AcceptCall &call, cudaStream_t stream)
{
    return call.T >= 0 ? launch_accept<true>(call, stream) : launch_accept<false>(call, stream);
}

cudaError_t read_tree_device_error(unsigned int *bits, bool clear)
{
    cudaError_t err = cudaMemcpyFromSymbol(bits, g_tree_error, sizeof(unsigned int));
    if (err != cudaSuccess || !clear) return err;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_tree_error, &zero, sizeof(unsigned int));
}

}  // namespace gq4
