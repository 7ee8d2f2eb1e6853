// Microscaled formats (device code): 32 consecutive values of a row share one scale byte e for
// 2^(e - 127), and each is held as a 4-bit (E2M1) or 8-bit (E4M3) floating point code.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "tcq.h"

namespace tcq {
namespace mx {

constexpr int kGroup = 32;

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Bytes of n consecutive codes (n a multiple of 2).
template <int FMT>
constexpr int bytes(int n) {
    return FMT == TCQ_FP4 ? n / 2 : n;
}

// The scale byte of a group whose largest magnitude has the bit pattern top: the exponent field
// less the exponent of the format's largest power of two (4 or 256), so that the largest
// value's code is one of the format's last binade.
template <int FMT>
__device__ __forceinline__ int scale_byte(uint32_t top) {
    const int field = static_cast<int>(top >> 23);
    const int e = field - (FMT == TCQ_FP4 ? 2 : 8);
    return field == 255 ? 255 : (e < 0 ? 0 : e);
}

// The largest of a group's magnitudes, over the four neighbouring lanes that hold it (bit
// patterns order like magnitudes, NaN above infinity).
__device__ __forceinline__ uint32_t group_top(uint32_t top) {
    uint32_t o = __builtin_amdgcn_update_dpp(0, top, 0xB1, 0xF, 0xF, false);  // lanes 1 0 3 2
    top = top > o ? top : o;
    o = __builtin_amdgcn_update_dpp(0, top, 0x4E, 0xF, 0xF, false);           // lanes 2 3 0 1
    return top > o ? top : o;
}

// Codes of x[0 .. 7] under scale byte e: the nearest (ties to even) of x 2^(127 - e), clamped to
// the format's largest value.  The conversions themselves round to nearest even.
template <int FMT>
__device__ __forceinline__ void encode8(const float (&x)[8], int e, uint32_t (&w)[2]) {
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        constexpr float kMost = FMT == TCQ_FP4 ? 6.0f : 448.0f;
        v[k] = __builtin_amdgcn_fmed3f(__builtin_amdgcn_ldexpf(x[k], 127 - e), -kMost, kMost);
    }
    if constexpr (FMT == TCQ_FP4) {
        uint32_t c = 0;
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], 1.0f, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], 1.0f, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], 1.0f, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], 1.0f, 3);
        w[0] = e == 255 ? 0u : c;
        w[1] = 0u;
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            int c = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h], v[4 * h + 1], 0, false);
            c = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2], v[4 * h + 3], c, true);
            w[h] = e == 255 ? 0u : static_cast<uint32_t>(c);
        }
    }
}

// 2^(e - 127) as the conversions take it: they read the exponent field alone, 0 as 2^-127 and
// 255 as NaN.
__device__ __forceinline__ float scale_of(int e) {
    return __uint_as_float(static_cast<uint32_t>(e) << 23);
}

// Values of the codes of one word (8 of fp4, 4 of fp8) times the scale, exact.
template <int FMT>
__device__ __forceinline__ void decode_word(uint32_t w, float s, float *v) {
    f32x2 p[4];
    if constexpr (FMT == TCQ_FP4) {
        p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0);
        p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1);
        p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 2);
        p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 3);
    } else {
        p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, s, false);
        p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, s, true);
    }
#pragma unroll
    for (int k = 0; k < (FMT == TCQ_FP4 ? 4 : 2); ++k) {
        v[2 * k] = p[k][0];
        v[2 * k + 1] = p[k][1];
    }
}

// The same in bf16, two values to a word: exact from 2^-133 up to bf16's largest number.
template <int FMT>
__device__ __forceinline__ void decode_word_bf16(uint32_t w, float s, uint32_t *v) {
    if constexpr (FMT == TCQ_FP4) {
        v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
        v[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
        v[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
        v[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
    } else {
        v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, false));
        v[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, true));
    }
}

// The same in fp16: exact for scales of 2^-23 .. 2^13 (fp4) or 2^-15 .. 2^7 (fp8).
template <int FMT>
__device__ __forceinline__ void decode_word_f16(uint32_t w, float s, uint32_t *v) {
    if constexpr (FMT == TCQ_FP4) {
        v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 0));
        v[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 1));
        v[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 2));
        v[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 3));
    } else {
        v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, s, false));
        v[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, s, true));
    }
}
template <int FMT>
constexpr int kLowF16 = FMT == TCQ_FP4 ? -23 : -15;
template <int FMT>
constexpr int kHighF16 = FMT == TCQ_FP4 ? 13 : 7;

}  // namespace mx
}  // namespace tcq
