// The paged cache of keys and values (device code): where a token's codes lie.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "mx_device.h"
#include "tcq_internal.h"

namespace tcq {
namespace cache {

// Sequence s's new rows [begin, end) of the call's rows, and what position row begin has.
struct Span {
    int64_t begin, end, first;
};
__device__ __forceinline__ Span span_of(const CacheBatch &b, int64_t s, int64_t rows) {
    const int64_t at = b.starts[s], to = b.starts[s + 1];
    const int64_t first = static_cast<int64_t>(b.lens[s]) - (to - at);
    Span r;
    r.begin = at < 0 ? 0 : at;
    r.end = to < rows ? to : rows;
    r.first = first + (r.begin - at);
    return r;
}

// How many of the n increasing v are at most x (uniform in a wave), found by 64 probes at a time.
template <typename V>
__device__ __forceinline__ int64_t at_most(const V *v, int64_t n, int64_t x, int lane) {
    int64_t lo = 0;  // the answer is in [lo, lo + n]
    while (n > 0) {
        const int64_t step = (n + 63) / 64;
        const int64_t i = lo + (lane + 1) * step - 1;
        const bool below = i < lo + n && static_cast<int64_t>(v[i]) <= x;
        const int64_t skip = __popcll(__ballot(below)) * step;
        lo += skip;
        n = step - 1 < n - skip ? step - 1 : n - skip;
    }
    return lo;
}

// The sequence that holds row `row` (uniform in a wave).  seqs: none.
__device__ __forceinline__ int64_t sequence_of(const CacheBatch &b, int64_t row, int lane) {
    return row < b.starts[0] ? b.seqs : at_most(b.starts + 1, b.seqs, row, lane);
}

// The page of position pos of sequence s, or -1 where there is none.
__device__ __forceinline__ int64_t page_of(const CacheBatch &b, const CacheShape &c, int64_t s,
                                           int64_t pos) {
    const int64_t i = pos >> c.page_log2;
    if (pos < 0 || i >= b.width) return -1;
    const int64_t p = b.table[s * b.ldt + i];
    return p >= 0 && p < c.pages ? p : -1;
}

// Index of the cache row (page, head, place) that holds position pos.
__device__ __forceinline__ int64_t row_of(const CacheShape &c, int64_t page, int head,
                                          int64_t pos) {
    return ((page * c.heads + head) << c.page_log2) + (pos & ((1ll << c.page_log2) - 1));
}

}  // namespace cache
}  // namespace tcq
