// Microscaled codes back to values (device code).
#pragma once

#include <hip/hip_runtime.h>

#include "checkpoint_device.h"
#include "mx_device.h"
#include "tcq_internal.h"

namespace tcq {

struct MxUnpackArgs {
    const uint8_t *codes;
    int64_t ldq;
    const uint8_t *scale;
    int64_t cols, ldo;
    Pieces ix;          // pieces of 16 bytes of output
    int64_t padded;     // columns cols .. padded - 1 become zeros
    // fp16: values are multiplied by the power of two that brings the largest code of the largest
    // scale byte below 2^16, and its inverse's exponent goes to *shift.down (tops NULL: no)
    MxShift shift;
};

// 16 bytes of output per thread (8 values of a 16-bit type, 4 of fp32), stored past the caches.
template <typename T, int FMT, bool SMALL>
__device__ __forceinline__ void mx_unpack(const MxUnpackArgs &a, T *__restrict__ out,
                                          uint32_t block, uint32_t blocks) {
    constexpr int P = 16 / static_cast<int>(sizeof(T));
    typedef uint32_t Store __attribute__((ext_vector_type(4), aligned(1)));
    const int64_t groups = (a.cols + mx::kGroup - 1) / mx::kGroup;
    int shift = 0;
    if constexpr (__is_same(T, _Float16)) {
        if (a.shift.tops) {
            int top = 0;
#pragma unroll
            for (int k = 0; k < kMxTops; ++k) top = top > a.shift.tops[k] ? top : a.shift.tops[k];
            shift = 127 + 15 - (FMT == TCQ_FP4 ? 2 : 8) - top;
            if (block == 0 && threadIdx.x == 0) *a.shift.down = -shift;
        }
    }
    for (int64_t i = static_cast<int64_t>(block) * 256 + threadIdx.x; i < a.ix.total;
         i += static_cast<int64_t>(blocks) * 256) {
        int64_t r;
        uint32_t c;
        split<SMALL>(i, a.ix.cpr, r, c);
        const int64_t col = static_cast<int64_t>(c) * P;
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = 0.0f;
        if (col < a.cols) {
            // (whole groups of codes are there)
            const uint8_t *q = a.codes + r * a.ldq + static_cast<int64_t>(c) * mx::bytes<FMT>(P);
            const float s = mx::scale_of(a.scale[r * groups + c / (mx::kGroup / P)]);
            if constexpr (FMT == TCQ_FP4 && P == 8) {
                mx::decode_word<FMT>(*reinterpret_cast<const uint32_t *>(q), s, v);
            } else if constexpr (FMT == TCQ_FP4) {
                mx::decode_word<FMT>(*reinterpret_cast<const uint16_t *>(q), s, v);
            } else {
#pragma unroll
                for (int h = 0; h < P / 4; ++h)
                    mx::decode_word<FMT>(reinterpret_cast<const uint32_t *>(q)[h], s, v + 4 * h);
            }
        }
        T *o = out + r * a.ldo + col;
        struct alignas(16) Piece { T v[P]; } st;
#pragma unroll
        for (int k = 0; k < P; ++k)
            st.v[k] = static_cast<T>(
                col + k < a.cols
                    ? (__is_same(T, _Float16) ? __builtin_amdgcn_ldexpf(v[k], shift) : v[k])
                    : 0.0f);
        if (col + P <= a.padded) {
            __builtin_nontemporal_store(__builtin_bit_cast(Store, st),
                                        reinterpret_cast<Store *>(o));
        } else {
#pragma unroll
            for (int k = 0; k < P; ++k)
                if (col + k < a.padded) o[k] = st.v[k];
        }
    }
}

template <typename T>
MxUnpackArgs mx_unpack_args(const MxMatrix &m, int64_t rows, int64_t cols, int64_t ldo,
                            int64_t padded) {
    constexpr int64_t P = 16 / sizeof(T);
    const int64_t cpr = (padded + P - 1) / P;
    return MxUnpackArgs{m.codes, m.ld, m.scale, cols, ldo, {static_cast<uint32_t>(cpr), rows * cpr},
                        padded, MxShift{nullptr, nullptr}};
}

}  // namespace tcq
