// gq4_kv_write.cuh -- a quantised word on its way into the cache, shared by the
// kernels that write it.
#pragma once

#include "gq4_kv.cuh"
#include "gq4_quant.cuh"

namespace gq4 {

constexpr unsigned int kKvNonFinite = 1u << 3, kKvBadSlot = 1u << 6;

// Word w (codes 8w .. 8w+7) of the row of kv head h in a slot (>= 0), side 0 K
// and 1 V, with its group's scale and zero by the group's first lane.  J =
// head_dim / 32, L: lanes (words) per group.  other: the word of lane w ^ 4 of
// the same row.  P: the pool's steps, as AppendParams has them.
template <int J, int L, typename P>
__device__ __forceinline__ void write_word(const P &p, int slot, int h, int side, int w, uint32_t word, uint32_t other,
                                           int bad, const GroupMap &m, unsigned int *error)
{
    constexpr int WPR = 4 * J, G = WPR / L;
    const int group = w / L, pos = w - group * L;
    if (slot >= p.total) {
        if (w == 0) atomicOr(error, kKvBadSlot);
        return;
    }
    const RowAt row(p.c, slot, p.shift, h);
    if (side == 0) {
        row.in(p.c.Kq, p.page_codes, 4 * WPR)[k_word_index(w, J)] = word;
    } else if constexpr (J % 2 == 0) {
        // value halves of words w and w + 4 are neighbours: one lane stores
        // the first halves of both, the other the second
        const int g = 2 * (w & 3), b = w >> 2;
        const uint32_t both = (b & 1) ? __byte_perm(other, word, 0x7632) : __byte_perm(word, other, 0x5410);
        row.in(p.c.Vq, p.page_codes, 4 * WPR)[((g + (b & 1)) * J + (b & ~1)) >> 1] = both;
    } else {
        uint16_t *half = reinterpret_cast<uint16_t *>(row.in(p.c.Vq, p.page_codes, 4 * WPR));
        half[v_half_index(2 * w, J)] = (uint16_t)word;
        half[v_half_index(2 * w + 1, J)] = (uint16_t)(word >> 16);
    }
    if (pos == 0) {
        const float nan = __int_as_float(0x7fc00000);
        float2 *sz = reinterpret_cast<float2 *>(side ? p.c.V_sz : p.c.K_sz);
        row.in(sz, p.page_sz, 8 * G)[group] = bad ? make_float2(nan, nan) : make_float2(m.s, m.z);
        if (bad) atomicOr(error, kKvNonFinite);
    }
}

}  // namespace gq4
