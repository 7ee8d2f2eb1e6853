// Element types, activations and checkpoint scales of the coded linear layer (device code).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "tcq.h"

namespace tcq {

// The C ABI's name of an element type.
template <typename T>
constexpr int dtype_of() {
    return sizeof(T) == 4 ? TCQ_F32 : (__is_same(T, _Float16) ? TCQ_F16 : TCQ_BF16);
}

// The activations and their slopes are evaluated in fp32: for fp32 layers (FULL) to a few units
// of the value however small it is, for 16-bit types to 2^-16 of it.  Where exp(-|z|) or
// exp(-z^2 / 2) falls below fp32's smallest normal number it is zero.

// 2^(a c), c a constant and c_low what c lacks: the product's rounding alone would cost
// |a c| 2^-24 of the value, so FULL takes what it lost along.
template <bool FULL>
__device__ __forceinline__ float exp2_product(float a, float c, float c_low, float a_low = 0.0f) {
    const float y = a * c;
    const float r = __builtin_amdgcn_exp2f(y);
    if constexpr (!FULL) return r;
    const float lost =
        __builtin_fmaf(a, c, -y) + __builtin_fmaf(a, c_low, a_low * c);
    return __builtin_fmaf(r, lost * 0.69314718055994531f, r);
}

// s = 1 / (1 + exp(-z)) and n = 1 - s.
template <bool FULL>
__device__ __forceinline__ void sigmoid(float z, float &s, float &n) {
    constexpr float kLog2e = 1.44269504088896340736f, kLow = 1.92596299e-8f;
    if constexpr (FULL) {
        // (from 104 on the exponential is zero; infinities have no remainder)
        const float e = exp2_product<true>(-__builtin_fminf(__builtin_fabsf(z), 104.0f), kLog2e,
                                           kLow);
        const float r = __builtin_amdgcn_rcpf(1.0f + e);
        s = z < 0.0f ? e * r : r;
        n = z < 0.0f ? r : e * r;
    } else {
        s = __builtin_amdgcn_rcpf(1.0f + exp2_product<false>(-z, kLog2e, 0.0f));
        n = 1.0f - s;
    }
}

// Phi(z) and e = exp(-z^2 / 2).  Phi(-x) = e t P(t) with t = 1 / (1 + 0.305 x), x >= 0: P is the
// polynomial of degree 7 with the least relative error over 0 <= x <= 14, 0.95e-7, fitted to
// the scaled complementary error function in 64 bits.  With one degree less the best pole's
// error is 1.3e-6, with 8 3e-8, below fp32's roundings.  The exponential is the one the density
// needs; erfcf takes three times as many instructions.
template <bool FULL>
__device__ __forceinline__ float normal_cdf(float z, float &e) {
    constexpr float kC = -0.72134752044448170368f, kLow = -9.62981495e-9f;
    const float x = __builtin_fabsf(z);
    if constexpr (FULL) {
        const float a = __builtin_fminf(x, 16.0f);  // (the exponential is zero from 14 on)
        const float h = a * a;
        e = exp2_product<true>(h, kC, kLow, __builtin_fmaf(a, a, -h));
    } else {
        e = exp2_product<false>(z * z, kC, 0.0f);
    }
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.305f, x, 1.0f));
    float q = __builtin_fmaf(0.0366991939f, t, -0.1529883249f);
    q = __builtin_fmaf(q, t, 0.1857169113f);
    q = __builtin_fmaf(q, t, -0.0379768429f);
    q = __builtin_fmaf(q, t, 0.1210216853f);
    q = __builtin_fmaf(q, t, 0.1034208643f);
    q = __builtin_fmaf(q, t, 0.1224668173f);
    q = __builtin_fmaf(q, t, 0.1216397326f);
    const float tail = q * t * e;  // Phi(-|z|)
    return z < 0.0f ? tail : 1.0f - tail;
}

// act(z).
template <int ACT, bool FULL>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == TCQ_ACT_RELU) return z < 0.0f ? 0.0f : z;  // NaN stays NaN
    if constexpr (ACT == TCQ_ACT_SILU) {
        float s, n;
        sigmoid<FULL>(z, s, n);
        return z * s;
    }
    if constexpr (ACT == TCQ_ACT_GELU) {
        float e;
        return z * normal_cdf<FULL>(z, e);
    }
    return z;
}

// g act'(z).  relu selects (0 at z <= 0, whatever g holds there), and a NaN z gives NaN as the
// other activations do: a checkpoint's group with an infinity stands for NaN, which must not
// pass for closed units.
template <int ACT, bool FULL>
__device__ __forceinline__ float act_grad(float g, float z) {
    if constexpr (ACT == TCQ_ACT_RELU) return z > 0.0f ? g : (z <= 0.0f ? 0.0f : z);
    if constexpr (ACT == TCQ_ACT_SILU) {
        float s, n;
        sigmoid<FULL>(z, s, n);
        return g * (s * __builtin_fmaf(z, n, 1.0f));
    }
    if constexpr (ACT == TCQ_ACT_GELU) {
        float e;
        const float c = normal_cdf<FULL>(z, e);
        return g * __builtin_fmaf(z, 0.39894228040143268f * e, c);
    }
    return g;
}

// f(std::integral_constant<int, ACT>) for a uniform act.
template <typename F>
__device__ __forceinline__ void with_act(int act, F f) {
    switch (act) {
        case TCQ_ACT_RELU: f(std::integral_constant<int, TCQ_ACT_RELU>{}); break;
        case TCQ_ACT_SILU: f(std::integral_constant<int, TCQ_ACT_SILU>{}); break;
        case TCQ_ACT_GELU: f(std::integral_constant<int, TCQ_ACT_GELU>{}); break;
        default: f(std::integral_constant<int, TCQ_ACT_NONE>{}); break;
    }
}

// Eight (or P) consecutive values at any address: one wide access.
template <typename T, int P = 8>
struct __attribute__((packed)) Packed {
    T v[P];
};

// Value of a checkpoint code q whose group has scale byte e: q 2^(e - 133), exact in fp32;
// e = 255 marks a group that held an infinity or a NaN.
__device__ __forceinline__ float code_value(int q, int e) {
    if (e == 255) return __int_as_float(0x7FC00000);
    return __builtin_amdgcn_ldexpf(static_cast<float>(q), e - 133);
}

}  // namespace tcq
