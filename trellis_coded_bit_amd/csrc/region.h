// Matrices of rows in memory, and whether two of them share a byte (host code).
#pragma once

#include <cstddef>
#include <cstdint>

namespace tcq {

// rows rows of width bytes, stride bytes apart (width <= stride where there are several).  Sums of
// a caller's sizes are taken in 128 bits: none of them wraps.
struct Region {
    using Wide = __int128;
    const char *name;
    const void *p;
    int64_t rows;
    Wide stride, width;
    Wide at() const { return reinterpret_cast<uintptr_t>(p); }
    Wide end() const { return at() + (rows - 1) * stride + width; }
};

inline Region region(const char *name, const void *p, int64_t rows, int64_t ld, int64_t cols,
                     size_t size) {
    const Region::Wide s = size;
    return {name, p, rows, ld * s, cols * s};
}

// Whether a and b share a byte.  Columns of one wider matrix side by side do not, although
// their extents do, so rows are compared: row by row of the one with fewer rows against the first
// row of the other that ends behind its start (one row decides where the strides agree).
inline bool overlap(Region a, Region b) {
    using Wide = Region::Wide;
    if (a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
    if (a.end() <= b.at() || b.end() <= a.at()) return false;
    const auto floor_div = [](Wide n, Wide d) { return n / d - (n % d < 0); };
    if (a.rows > 1 && b.rows > 1 && a.stride == b.stride) {
        // rows j of b and i of a meet where at + (j - i) stride lies in (-b.width, a.width)
        const Wide at = b.at() - a.at();
        Wide t = floor_div(-b.width - at, a.stride) + 1;
        if (t < 1 - a.rows) t = 1 - a.rows;
        return t < b.rows && at + t * a.stride < a.width;
    }
    if (a.rows > b.rows) {
        const Region c = a;
        a = b;
        b = c;
    }
    for (int64_t i = 0; i < a.rows; ++i) {
        const Wide from = a.at() + i * a.stride;
        Wide j = b.rows > 1 ? floor_div(from - b.width - b.at(), b.stride) + 1 : 0;
        if (j < 0) j = 0;
        if (j < b.rows && b.at() + j * b.stride < from + a.width &&
            b.at() + j * b.stride + b.width > from)
            return true;
    }
    return false;
}

}  // namespace tcq
