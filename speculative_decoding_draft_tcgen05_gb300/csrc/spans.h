// Which bytes the tensors of a call take: for the entry points' checks that
// outputs overlap nothing else. Host code.
#pragma once

#include <stdint.h>

namespace dfl {

// Rows of `width` bytes, [outer, inner] of them, strides in bytes. A plain array is one row; nothing meets a NULL or an empty one.
struct Rows {
    const void *at;
    int64_t width;
    int64_t inner = 1, stride = 0;
    int64_t outer = 1, outer_stride = 0;

    uintptr_t begin() const { return reinterpret_cast<uintptr_t>(at); }
    uintptr_t end() const { return begin() + static_cast<uintptr_t>((outer - 1) * outer_stride + (inner - 1) * stride + width); }
    bool any() const { return at && width > 0 && inner > 0 && outer > 0; }
};

// Whether low < c + k * step < high for a k in [first, last], step >= 0.
inline bool hits(int64_t low, int64_t high, int64_t c, int64_t step, int64_t first, int64_t last)
{
    if (step == 0) return low < c && c < high;
    auto floor_div = [](int64_t a, int64_t b) { return a / b - (a % b < 0 ? 1 : 0); };
    const int64_t k = floor_div(low - c, step) + 1;  // the least k above low
    const int64_t from = k > first ? k : first;
    return from <= last && c + from * step < high;
}

// Whether rows of a share bytes with rows of b. Slices of one buffer, whose strides are equal, may pass one another without
// doing so; with other strides, whatever lies within the same bytes counts as shared.
inline bool meet(const Rows &a, const Rows &b)
{
    if (!a.any() || !b.any() || a.begin() >= b.end() || b.begin() >= a.end()) return false;
    if (a.inner > 1 && b.inner > 1 && a.stride != b.stride) return true;
    if (a.outer > 1 && b.outer > 1 && a.outer_stride != b.outer_stride) return true;
    const int64_t d = static_cast<int64_t>(b.begin() - a.begin());
    // rows of b start d + i * one + j * other bytes behind rows of a, i and j in these ranges
    int64_t one = a.outer > 1 ? a.outer_stride : b.outer_stride, i0 = 1 - a.outer, i1 = b.outer - 1;
    int64_t other = a.inner > 1 ? a.stride : b.stride, j0 = 1 - a.inner, j1 = b.inner - 1;
    if (i1 - i0 > j1 - j0) {  // (the shorter one is walked)
        int64_t t = one;
        one = other, other = t;
        t = i0, i0 = j0, j0 = t;
        t = i1, i1 = j1, j1 = t;
    }
    for (int64_t i = i0; i <= i1; ++i)
        if (hits(-b.width, a.width, d + i * one, other, j0, j1)) return true;
    return false;
}

// Whether rows of a share bytes with one another.
inline bool folds(const Rows &a)
{
    if (!a.any()) return false;
    if ((a.inner > 1 && a.stride < a.width) || (a.outer > 1 && a.outer_stride < a.width)) return true;
    if (a.inner == 1 || a.outer == 1 || a.outer_stride >= (a.inner - 1) * a.stride + a.width || a.stride >= (a.outer - 1) * a.outer_stride + a.width)
        return false;
    const bool by_outer = a.outer <= a.inner;
    const int64_t n = by_outer ? a.outer : a.inner, m = by_outer ? a.inner : a.outer;
    const int64_t one = by_outer ? a.outer_stride : a.stride, other = by_outer ? a.stride : a.outer_stride;
    for (int64_t i = 1; i < n; ++i)
        if (hits(-a.width, a.width, i * one, other, 1 - m, m - 1)) return true;
    return false;
}

}  // namespace dfl
