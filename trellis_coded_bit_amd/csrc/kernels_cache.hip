// The paged cache of keys and values: new tokens quantised as they are written (tcq_cache_write),
// and read back (tcq_cache_read).  A row of the cache is one head's vector of one token, in
// groups of 32 along the head's dimension, so a token touches no other token's bytes.
//   Both are bound by memory, or by their launch for a few tokens: a workgroup takes one row
// of the call (a token), looks its sequence and page up once and moves all its heads.
#include <hip/hip_runtime.h>

#include "cache_device.h"
#include "linear_device.h"
#include "mx_device.h"
#include "tcq_internal.h"

namespace tcq {
namespace {

struct CacheMove {
    CacheShape c;
    CacheBatch b;
    int64_t rows;
    const void *k, *v;      // rows x heads x dim, or NULL
    int64_t k_row, k_head, v_row, v_head;
};

constexpr int kMoveThreads = 256;

// Where row `blockIdx.x` of the call lies in the cache: its page (-1: nowhere) and position;
// false behind the last sequence.
__device__ __forceinline__ bool find(const CacheMove &a, int64_t row, int64_t &page,
                                     int64_t &pos) {
    const int64_t s = cache::sequence_of(a.b, row, threadIdx.x & 63);
    if (s >= a.b.seqs) return false;
    const cache::Span sp = cache::span_of(a.b, s, a.rows);
    pos = sp.first + (row - sp.begin);
    page = cache::page_of(a.b, a.c, s, pos);
    return true;
}

// Eight values per thread; four neighbouring lanes share a group.
template <typename T, int FMT>
__global__ __launch_bounds__(kMoveThreads) void cache_write_kernel(CacheMove a) {
    const int per = a.c.dim / 8, total = 2 * a.c.heads * per;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        int64_t page, pos;
        if (!find(a, row, page, pos) || page < 0) continue;
        for (int i = threadIdx.x; i < total; i += kMoveThreads) {
            const bool value = i >= total / 2;
            const int j = value ? i - total / 2 : i;
            const int head = j / per, c = j - head * per;
            const T *x = value ? static_cast<const T *>(a.v) + row * a.v_row + head * a.v_head
                               : static_cast<const T *>(a.k) + row * a.k_row + head * a.k_head;
            const Packed<T> p = *reinterpret_cast<const Packed<T> *>(x + c * 8);
            float f[8];
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                f[k] = static_cast<float>(p.v[k]);
                const uint32_t m = __float_as_uint(f[k]) & 0x7FFFFFFFu;
                top = top > m ? top : m;
            }
            // (dim is a multiple of 32: a group's four lanes are here together)
            const int e = mx::scale_byte<FMT>(mx::group_top(top));
            uint32_t w[2];
            mx::encode8<FMT>(f, e, w);
            const int64_t at = cache::row_of(a.c, page, head, pos);
            uint8_t *q = (value ? a.c.v_codes : a.c.k_codes) + at * mx::bytes<FMT>(a.c.dim) +
                         c * mx::bytes<FMT>(8);
            if constexpr (FMT == TCQ_FP4)
                *reinterpret_cast<uint32_t *>(q) = w[0];
            else
                *reinterpret_cast<uint2 *>(q) = make_uint2(w[0], w[1]);
            if ((c & 3) == 0)
                (value ? a.c.v_scale : a.c.k_scale)[at * (a.c.dim / 32) + c / 4] =
                    static_cast<uint8_t>(e);
        }
    }
}

// Eight values per thread; a token that is nowhere in the cache reads as zeros.
template <typename T, int FMT>
__global__ __launch_bounds__(kMoveThreads) void cache_read_kernel(CacheMove a) {
    const int per = a.c.dim / 8, total = 2 * a.c.heads * per;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        int64_t page, pos;
        if (!find(a, row, page, pos)) continue;
        for (int i = threadIdx.x; i < total; i += kMoveThreads) {
            const bool value = i >= total / 2;
            const int j = value ? i - total / 2 : i;
            const int head = j / per, c = j - head * per;
            T *x = value ? static_cast<T *>(const_cast<void *>(a.v)) + row * a.v_row +
                               head * a.v_head
                         : static_cast<T *>(const_cast<void *>(a.k)) + row * a.k_row +
                               head * a.k_head;
            float f[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (page >= 0) {
                const int64_t at = cache::row_of(a.c, page, head, pos);
                const uint8_t *q = (value ? a.c.v_codes : a.c.k_codes) +
                                   at * mx::bytes<FMT>(a.c.dim) + c * mx::bytes<FMT>(8);
                const float s = mx::scale_of(
                    (value ? a.c.v_scale : a.c.k_scale)[at * (a.c.dim / 32) + c / 4]);
                mx::decode_word<FMT>(reinterpret_cast<const uint32_t *>(q)[0], s, f);
                if constexpr (FMT == TCQ_FP8)
                    mx::decode_word<FMT>(reinterpret_cast<const uint32_t *>(q)[1], s, f + 4);
            }
            Packed<T> p;
#pragma unroll
            for (int k = 0; k < 8; ++k) p.v[k] = static_cast<T>(f[k]);
            *reinterpret_cast<Packed<T> *>(x + c * 8) = p;
        }
    }
}

template <typename T>
hipError_t move(const CacheMove &a, bool write, hipStream_t s) {
    const bool fp4 = a.c.format == TCQ_FP4;
    const auto kern = write ? (fp4 ? cache_write_kernel<T, TCQ_FP4> : cache_write_kernel<T, TCQ_FP8>)
                            : (fp4 ? cache_read_kernel<T, TCQ_FP4> : cache_read_kernel<T, TCQ_FP8>);
    const int64_t most = 1 << 20;
    hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(a.rows < most ? a.rows : most)),
                       dim3(kMoveThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_cache_move(bool write, const CacheShape &c, const CacheBatch &b, int dtype,
                             const CacheRows &k, const CacheRows &v, int64_t rows,
                             hipStream_t s) {
    const CacheMove a{c, b, rows, k.p, v.p, k.row, k.head, v.row, v.head};
    switch (dtype) {
        case TCQ_F32: return move<float>(a, write, s);
        case TCQ_F16: return move<_Float16>(a, write, s);
        default: return move<__bf16>(a, write, s);
    }
}

}  // namespace tcq
