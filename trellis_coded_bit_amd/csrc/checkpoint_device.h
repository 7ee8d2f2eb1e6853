// 8-bit checkpoints (device code): how threads share rows, and codes back to values.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "linear_device.h"

namespace tcq {

constexpr int kGroup = 32;

// Rows cut into pieces of consecutive values, one per thread and turn.  Global loads and
// stores of any alignment are legal on this hardware, so rows may start anywhere.
struct Pieces {
    uint32_t cpr;      // pieces per row
    int64_t total;     // rows x cpr
};

// Row r and piece c of flat index i (32-bit division where the total allows it).
template <bool SMALL>
__device__ __forceinline__ void split(int64_t i, uint32_t cpr, int64_t &r, uint32_t &c) {
    if constexpr (SMALL) {
        const uint32_t q = static_cast<uint32_t>(i) / cpr;
        r = q;
        c = static_cast<uint32_t>(i) - q * cpr;
    } else {
        r = i / cpr;
        c = static_cast<uint32_t>(i - r * cpr);
    }
}

struct UnpackArgs {
    const int8_t *codes;
    int64_t ldq;
    const uint8_t *scale;
    Pieces ix;
    int64_t cols, ldo, padded;
};

template <typename T>
UnpackArgs unpack_args(const int8_t *codes, int64_t ldq, const uint8_t *scale, int64_t rows,
                       int64_t cols, int64_t ldo, int64_t padded) {
    constexpr int64_t P = 16 / sizeof(T);
    const int64_t cpr = (padded + P - 1) / P;
    return UnpackArgs{codes, ldq, scale, {static_cast<uint32_t>(cpr), rows * cpr}, cols, ldo,
                      padded};
}

// 16 bytes of output per thread (8 values of a 16-bit type, 4 of fp32), so that a wave's
// stores fill whole lines; they bypass the caches (16384 x 14336, call after call: 108 us in bf16
// against 155 with plain stores, 164 against 316 in fp32; 155 in bf16 where the codes come from
// HBM).  out's
// columns cols .. padded - 1 are zeros.  ix.cpr counts the pieces of a padded row.  `block` is
// one of the `blocks` workgroups that share the work.
template <typename T, bool SMALL>
__device__ __forceinline__ void act_unpack(const UnpackArgs &a, T *__restrict__ out,
                                           uint32_t block, uint32_t blocks) {
    constexpr int P = 16 / static_cast<int>(sizeof(T));
    typedef uint32_t Store __attribute__((ext_vector_type(4), aligned(1)));
    const int64_t groups = (a.cols + kGroup - 1) / kGroup;
    for (int64_t i = static_cast<int64_t>(block) * 256 + threadIdx.x; i < a.ix.total;
         i += static_cast<int64_t>(blocks) * 256) {
        int64_t r;
        uint32_t c;
        split<SMALL>(i, a.ix.cpr, r, c);
        const int64_t col = static_cast<int64_t>(c) * P;
        const int left = a.cols - col < P ? static_cast<int>(a.cols - col) : P;  // may be <= 0
        const int8_t *q = a.codes + r * a.ldq + col;
        const int e = left > 0 ? a.scale[r * groups + c / (kGroup / P)] : 0;
        float v[P];
        if (left == P) {
            struct __attribute__((packed)) Words { uint32_t w[P / 4]; };
            const Words t = *reinterpret_cast<const Words *>(q);
#pragma unroll
            for (int k = 0; k < P; ++k)
                v[k] = code_value(static_cast<int8_t>(t.w[k / 4] >> (8 * (k % 4))), e);
        } else {
#pragma unroll
            for (int k = 0; k < P; ++k) v[k] = k < left ? code_value(q[k], e) : 0.0f;
        }
        T *o = out + r * a.ldo + col;
        if (col + P <= a.padded) {
            struct alignas(16) Piece { T v[P]; } s;
#pragma unroll
            for (int k = 0; k < P; ++k) s.v[k] = static_cast<T>(v[k]);
            __builtin_nontemporal_store(__builtin_bit_cast(Store, s),
                                        reinterpret_cast<Store *>(o));
        } else {
#pragma unroll
            for (int k = 0; k < P; ++k)
                if (col + k < a.padded) o[k] = static_cast<T>(v[k]);
        }
    }
}

}  // namespace tcq
