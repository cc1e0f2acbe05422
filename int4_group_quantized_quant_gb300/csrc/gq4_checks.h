// gq4_checks.h -- argument checks shared by the C entry points: alignment and
// the byte ranges a call reads and writes.
#pragma once

#include <cstddef>
#include <cstdint>

#include "gq4.h"

namespace gq4 {

struct Range {
    uintptr_t lo, hi;     // [lo, hi)
    size_t pitch, width;  // rows of `width` bytes, `pitch` apart; pitch 0: one dense stretch
};

inline Range range_of(const void *p, size_t bytes)
{
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Range{lo, lo + bytes, 0, 0};
}

inline Range rows_of(const void *p, size_t rows, size_t width, size_t pitch)
{
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    if (rows == 0 || width == 0) return Range{lo, lo, 0, 0};
    return Range{lo, lo + (rows - 1) * pitch + width, pitch, width};
}

// Whether two ranges share a byte.  Column blocks of one matrix (rows of the
// same pitch) interleave without sharing any when their columns are apart.
inline bool overlap(Range a, Range b)
{
    if (a.lo == a.hi || b.lo == b.hi) return false;
    if (!(a.lo < b.hi && b.lo < a.hi)) return false;
    if (a.pitch == 0 || a.pitch != b.pitch) return true;
    const uintptr_t first = a.lo < b.lo ? a.lo : b.lo;
    const size_t ca = (a.lo - first) % a.pitch, cb = (b.lo - first) % a.pitch;
    const size_t c = ca > cb ? ca - cb : cb - ca;              // columns apart
    const size_t left = ca > cb ? b.width : a.width;           // width of the left block
    const size_t right = ca > cb ? a.width : b.width;
    return !(left <= c && c + right <= a.pitch);
}

inline bool aligned(const void *p, uintptr_t a)
{
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// Collects the byte ranges of a call and checks them.
struct RangeSet {
    Range in[16];
    int n_in = 0;
    Range out[8];
    int n_out = 0;
    void input(const void *p, size_t bytes)
    {
        if (p && bytes) in[n_in++] = range_of(p, bytes);
    }
    void output(const void *p, size_t bytes)
    {
        if (p && bytes) out[n_out++] = range_of(p, bytes);
    }
    void input_rows(const void *p, size_t rows, size_t width, size_t pitch)
    {
        if (p && rows && width) in[n_in++] = rows_of(p, rows, width, pitch);
    }
    void output_rows(const void *p, size_t rows, size_t width, size_t pitch)
    {
        if (p && rows && width) out[n_out++] = rows_of(p, rows, width, pitch);
    }
    bool disjoint() const
    {
        for (int i = 0; i < n_out; ++i) {
            for (int j = 0; j < n_in; ++j)
                if (overlap(out[i], in[j])) return false;
            for (int j = i + 1; j < n_out; ++j)
                if (overlap(out[i], out[j])) return false;
        }
        return true;
    }
};

}  // namespace gq4

#define GQ4_TRY(expr)                       \
    do {                                    \
        const gq4_status st_ = (expr);      \
        if (st_ != GQ4_OK) return st_;      \
    } while (0)

