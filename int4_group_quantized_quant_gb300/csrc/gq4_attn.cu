// gq4_attn.cu -- causal attention over the paged 4-bit key/value cache
// (gq4_kv_attention).
//
// One warp per query row and head, running softmax over the keys one by one.
#include <cstdint>

#include "gq4_internal.h"
#include "gq4_kv.cuh"

namespace gq4 {
namespace {

__device__ unsigned int g_attn_error = 0;
constexpr unsigned int kAttnBad = 1u << 8;

template <int J>
__global__ void __launch_bounds__(128) attn_rows_kernel(const __grid_constant__ AttnCall p)
{
    const int lane = threadIdx.x & 31;
    const int b = blockIdx.y;
    const int h = blockIdx.x * 4 + (threadIdx.x >> 5);
    const int D = 32 * J;
    const int q0 = p.query_start[b], q1 = p.query_start[b + 1], len = p.seq_lens[b];
    if (q1 <= q0 || h >= p.heads) return;
    const int lo_row = max(q0, 0), hi_row = min(q1, p.T);
    const bool bad = q0 < 0 || q1 > p.T || q1 - q0 > p.max_query || len < 0 || len > p.max_len;
    if (bad && lane == 0) atomicOr(&g_attn_error, kAttnBad);
    const int n = q1 - q0, kh = h / (p.heads / p.c.kv_heads), G = D / p.c.group_size;
    const uint32_t *Kq = p.c.Kq;
    const uint16_t *Vh = reinterpret_cast<const uint16_t *>(p.c.Vq);
    const float2 *Ksz = reinterpret_cast<const float2 *>(p.c.K_sz), *Vsz = reinterpret_cast<const float2 *>(p.c.V_sz);
    for (int row = lo_row; row < hi_row; ++row) {
        float *out = p.out + (size_t)row * p.ldo + (size_t)h * D;
        if (bad) {
            for (int u = 0; u < J; ++u) out[32 * u + lane] = __int_as_float(0x7fc00000);
            continue;
        }
        const int last = len - n + (row - q0);
        const int first = p.window > 0 ? max(0, last + 1 - p.window) : 0;
        float q[J], o[J];
        for (int u = 0; u < J; ++u) {
            q[u] = p.q[(size_t)row * p.ldq + (size_t)h * D + 32 * u + lane] * p.scale;
            o[u] = 0.0f;
        }
        float m = -INFINITY, l = 0.0f;
        for (int t = first; t <= last; ++t) {
            const int page = p.page_table[(size_t)b * p.max_pages + t / p.c.page_size];
            if (page < 0 || page >= p.c.n_pages) {
                if (lane == 0) atomicOr(&g_attn_error, kAttnBad);
                l = __int_as_float(0x7fc00000);
                continue;
            }
            const size_t r = kv_row(p.c, page, kh, t % p.c.page_size);
            float w = 0.0f;
            for (int u = 0; u < J; ++u) {
                const float2 s = Ksz[r * G + 32 * u / p.c.group_size];
                const uint32_t x = Kq[r * (D / 8) + (lane >> 3) * J + u] >> (4 * (lane & 7));
                w += q[u] * (((float)(x & 15u) - s.y) * s.x);
            }
            for (int i = 16; i > 0; i >>= 1) w += __shfl_xor_sync(0xffffffffu, w, i);
            const float m2 = fmaxf(m, w);
            const float keep = expf(m - m2), e = expf(w - m2);
            l = l * keep + e;
            for (int u = 0; u < J; ++u) {
                const float2 s = Vsz[r * G + 32 * u / p.c.group_size];
                const uint32_t x = (uint32_t)Vh[r * (D / 4) + (lane >> 2) * J + u] >> (4 * (lane & 3));
                o[u] = o[u] * keep + e * (((float)(x & 15u) - s.y) * s.x);
            }
            m = m2;
        }
        for (int u = 0; u < J; ++u) out[32 * u + lane] = last < first ? 0.0f : o[u] / l;
    }
}

}  // namespace

size_t attn_workspace_bytes(int, int, int, int)
{
    return 256;
}

cudaError_t launch_attn(const AttnCall &p, cudaStream_t stream)
{
    const dim3 grid((unsigned)((p.heads + 3) / 4), (unsigned)p.B);
    switch (p.c.head_dim) {
    case 64: attn_rows_kernel<2><<<grid, 128, 0, stream>>>(p); break;
    case 96: attn_rows_kernel<3><<<grid, 128, 0, stream>>>(p); break;
    case 128: attn_rows_kernel<4><<<grid, 128, 0, stream>>>(p); break;
    default: attn_rows_kernel<8><<<grid, 128, 0, stream>>>(p); break;
    }
    return cudaGetLastError();
}

cudaError_t read_attn_device_error(unsigned int *bits, bool clear)
{
    cudaError_t err = cudaMemcpyFromSymbol(bits, g_attn_error, sizeof(unsigned int));
    if (err != cudaSuccess || !clear) return err;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_attn_error, &zero, sizeof(unsigned int));
}

}  // namespace gq4
