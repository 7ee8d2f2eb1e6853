// The paged cache of keys and values: new tokens quantised as they are written (tcq_cache_write),
// and read back (tcq_cache_read).  A row of the cache is one head's vector of one token, in
// groups of 32 along the head's dimension, so a token touches no other token's bytes.
//   Both are bound by memory, or by their launch for a few tokens: a wave takes one row of the call
// (a token), looks its sequence and page up once, and moves all its heads, four pieces of eight
// values per lane on their way together; a write's are asked for before the lookup.  (Four prompts
// into 4 bits 33 us, back 23, at 3.6 and 5.4 TB/s; a piece of eight values to a thread with its own
// lookup 102 for both; 64 tokens 3.7 and 4.0.)
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
constexpr int kAhead = 4;

// Where row `row` of the call lies in the cache: its page (-1: nowhere) and position, uniform in
// the wave; false behind the last sequence.  64 sequences at most are searched with one access.
__device__ __forceinline__ bool find(const CacheMove &a, int64_t row, int64_t &page,
                                     int64_t &pos) {
    const int lane = threadIdx.x & 63;
    int64_t s;
    if (a.b.seqs <= 64) {
        const int l = lane < a.b.seqs ? lane : static_cast<int>(a.b.seqs) - 1;
        const int from = a.b.starts[l], to = a.b.starts[l + 1], len = a.b.lens[l];
        const int at = __popcll(__ballot(lane < a.b.seqs && to <= row));
        if (at >= a.b.seqs || __builtin_amdgcn_readlane(from, 0) > row) return false;
        s = at;
        const int64_t begin = __builtin_amdgcn_readlane(from, at);
        pos = __builtin_amdgcn_readlane(len, at) -
              (__builtin_amdgcn_readlane(to, at) - begin) + (row - begin);
    } else {
        s = cache::sequence_of(a.b, row, lane);
        if (s >= a.b.seqs) return false;
        const cache::Span sp = cache::span_of(a.b, s, a.rows);
        pos = sp.first + (row - sp.begin);
    }
    page = cache::page_of(a.b, a.c, s, pos);
    return true;
}

// Pieces of eight values of a row: first the keys' heads, then the values'.
struct Piece {
    bool value;
    int head, c;
    __device__ __forceinline__ Piece(int i, int half, int log2) {
        value = i >= half;
        const int j = value ? i - half : i;
        head = j >> log2;
        c = j & ((1 << log2) - 1);
    }
};

template <typename T, int FMT>
__global__ __launch_bounds__(kMoveThreads) void cache_write_kernel(CacheMove a) {
    const int lane = threadIdx.x & 63;
    const int log2 = a.c.dim == 64 ? 3 : (a.c.dim == 128 ? 4 : 5);   // pieces of a vector
    const int half = a.c.heads << log2, total = 2 * half;
    const int64_t waves = static_cast<int64_t>(gridDim.x) * (kMoveThreads / 64);
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * (kMoveThreads / 64) +
                       __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
         row < a.rows; row += waves) {
        auto load = [&](int i) {
            const Piece p(i < total ? i : total - 1, half, log2);
            const T *x = p.value ? static_cast<const T *>(a.v) + row * a.v_row + p.head * a.v_head
                                 : static_cast<const T *>(a.k) + row * a.k_row + p.head * a.k_head;
            return *reinterpret_cast<const Packed<T> *>(x + p.c * 8);
        };
        Packed<T> x[kAhead];
#pragma unroll
        for (int n = 0; n < kAhead; ++n) x[n] = load(n * 64 + lane);
        int64_t page, pos;
        if (!find(a, row, page, pos) || page < 0) continue;
        for (int i0 = 0; i0 < total; i0 += kAhead * 64) {
#pragma unroll
            for (int n = 0; n < kAhead; ++n) {
                const int i = i0 + n * 64 + lane;
                const Packed<T> now = x[n];
                if (i0 + kAhead * 64 < total) x[n] = load(i + kAhead * 64);
                float f[8];
                uint32_t top = 0;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    f[k] = static_cast<float>(now.v[k]);
                    const uint32_t m = __float_as_uint(f[k]) & 0x7FFFFFFFu;
                    top = top > m ? top : m;
                }
                // (total is a multiple of 4, and a group's four lanes hold its four pieces)
                const int e = mx::scale_byte<FMT>(mx::group_top(top));
                uint32_t w[2];
                mx::encode8<FMT>(f, e, w);
                if (i >= total) continue;
                const Piece p(i, half, log2);
                const int64_t at = cache::row_of(a.c, page, p.head, pos);
                uint8_t *q = (p.value ? a.c.v_codes : a.c.k_codes) + at * mx::bytes<FMT>(a.c.dim) +
                             p.c * mx::bytes<FMT>(8);
                if constexpr (FMT == TCQ_FP4)
                    *reinterpret_cast<uint32_t *>(q) = w[0];
                else
                    *reinterpret_cast<uint2 *>(q) = make_uint2(w[0], w[1]);
                if ((p.c & 3) == 0)
                    (p.value ? a.c.v_scale : a.c.k_scale)[at * (a.c.dim / 32) + p.c / 4] =
                        static_cast<uint8_t>(e);
            }
        }
    }
}

// A token that is nowhere in the cache reads as zeros.
template <typename T, int FMT>
__global__ __launch_bounds__(kMoveThreads) void cache_read_kernel(CacheMove a) {
    const int lane = threadIdx.x & 63;
    const int log2 = a.c.dim == 64 ? 3 : (a.c.dim == 128 ? 4 : 5);
    const int half = a.c.heads << log2, total = 2 * half;
    const int64_t waves = static_cast<int64_t>(gridDim.x) * (kMoveThreads / 64);
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * (kMoveThreads / 64) +
                       __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
         row < a.rows; row += waves) {
        int64_t page, pos;
        if (!find(a, row, page, pos)) continue;
        for (int i0 = 0; i0 < total; i0 += kAhead * 64) {
            uint2 q[kAhead];
            int e[kAhead];
#pragma unroll
            for (int n = 0; n < kAhead; ++n) {
                const int i = i0 + n * 64 + lane;
                const Piece p(i < total ? i : total - 1, half, log2);
                q[n] = make_uint2(0u, 0u);
                e[n] = 127;
                if (page < 0) continue;
                const int64_t at = cache::row_of(a.c, page, p.head, pos);
                const uint8_t *c = (p.value ? a.c.v_codes : a.c.k_codes) +
                                   at * mx::bytes<FMT>(a.c.dim) + p.c * mx::bytes<FMT>(8);
                if constexpr (FMT == TCQ_FP4)
                    q[n].x = *reinterpret_cast<const uint32_t *>(c);
                else
                    q[n] = *reinterpret_cast<const uint2 *>(c);
                e[n] = (p.value ? a.c.v_scale : a.c.k_scale)[at * (a.c.dim / 32) + p.c / 4];
            }
#pragma unroll
            for (int n = 0; n < kAhead; ++n) {
                const int i = i0 + n * 64 + lane;
                if (i >= total) continue;
                const Piece p(i, half, log2);
                float f[8];
                const float s = mx::scale_of(e[n]);
                mx::decode_word<FMT>(q[n].x, s, f);
                if constexpr (FMT == TCQ_FP8) mx::decode_word<FMT>(q[n].y, s, f + 4);
                Packed<T> o;
#pragma unroll
                for (int k = 0; k < 8; ++k) o.v[k] = static_cast<T>(f[k]);
                T *x = p.value ? static_cast<T *>(const_cast<void *>(a.v)) + row * a.v_row +
                                     p.head * a.v_head
                               : static_cast<T *>(const_cast<void *>(a.k)) + row * a.k_row +
                                     p.head * a.k_head;
                *reinterpret_cast<Packed<T> *>(x + p.c * 8) = o;
            }
        }
    }
}

template <typename T>
hipError_t move(const CacheMove &a, bool write, hipStream_t s) {
    const bool fp4 = a.c.format == TCQ_FP4;
    const auto kern = write ? (fp4 ? cache_write_kernel<T, TCQ_FP4> : cache_write_kernel<T, TCQ_FP8>)
                            : (fp4 ? cache_read_kernel<T, TCQ_FP4> : cache_read_kernel<T, TCQ_FP8>);
    constexpr int kRows = kMoveThreads / 64;
    hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>((a.rows + kRows - 1) / kRows)),
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
