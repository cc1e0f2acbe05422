// gq4_kv.cuh -- where a row of the paged 4-bit key/value cache and its codes
// lie (the layout stated in gq4.h).
#pragma once

#include <cstddef>
#include <cstdint>

#include "gq4.h"

namespace gq4 {

// Row (page, head, token of the page) of the pool, in 64 bits: a long cache
// passes 2^32 bytes.
__host__ __device__ __forceinline__ size_t kv_row(const gq4_kv_cache &c, int page, int head, int at)
{
    return ((size_t)page * c.kv_heads + head) * (size_t)c.page_size + at;
}

// Where word w (codes 8w .. 8w+7) of a key row, and half h (codes 4h .. 4h+3)
// of a value row are stored; J = head_dim / 32.
__host__ __device__ __forceinline__ int k_word_index(int w, int J)
{
    return (w & 3) * J + (w >> 2);
}

__host__ __device__ __forceinline__ int v_half_index(int h, int J)
{
    return (h & 7) * J + (h >> 3);
}

// r / d for 0 <= r, r d < 2^31, by multiplying with ceil(2^31 / d): that is
// too large by less than d, which adds less than r d / (2^31 d) < 1 / d.
__device__ __forceinline__ int quotient(int r, uint32_t per_d)
{
    return (int)__umulhi(2u * (uint32_t)r, per_d);
}

inline uint32_t divide_by(int d)
{
    return (uint32_t)((0x80000000ull + (uint32_t)d - 1) / (uint32_t)d);
}

// Where a row of the pool lies, in 32-bit steps and one 64-bit sum: the pages
// of all heads are fewer than 2^32 (each is 640 bytes or more).
struct RowAt {
    uint32_t page_head, at;

    __device__ __forceinline__ RowAt(const gq4_kv_cache &c, int slot, int shift, int head)
        : page_head((uint32_t)(slot >> shift) * (uint32_t)c.kv_heads + (uint32_t)head),
          at((uint32_t)slot & (uint32_t)(c.page_size - 1))
    {
    }
    // in an array of `bytes` per row, `page_bytes` per page and head
    template <typename P>
    __device__ __forceinline__ P *in(P *array, uint32_t page_bytes, uint32_t bytes) const
    {
        const char *base = reinterpret_cast<const char *>(array);
        return reinterpret_cast<P *>(const_cast<char *>(base + (uint64_t)page_head * page_bytes + at * bytes));
    }
};

inline int log2_of(int pow2)
{
    int s = 0;
    while ((1 << s) < pow2) ++s;
    return s;
}

}  // namespace gq4
