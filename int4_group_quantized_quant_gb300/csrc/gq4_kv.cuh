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

}  // namespace gq4
