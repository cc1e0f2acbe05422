// gq4_attn.cuh -- what the attention kernels share: a request's rows and keys,
// the base-2 exponential, asynchronous copies into shared memory.
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
    r.bad = r.n > 0 && (q0 < 0 || q1 > p.T || n > p.max_query || r.len < 0 || r.len > p.max_len);
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

}  // namespace gq4
