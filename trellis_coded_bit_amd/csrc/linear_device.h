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

// exp(x) by the hardware's base-2 exponential: relative error about |x| 2^-24.
__device__ __forceinline__ float fast_exp(float x) {
    return __builtin_amdgcn_exp2f(x * 1.44269504088896340736f);
}

__device__ __forceinline__ float sigmoid(float z) {
    return __builtin_amdgcn_rcpf(1.0f + fast_exp(-z));
}

// Phi(z) and e = exp(-z^2 / 2): the rational approximation 7.1.26 of Abramowitz and Stegun,
// Handbook of Mathematical Functions (1964), erf(x) = 1 - (a1 t + ... + a5 t^5) exp(-x^2) with
// t = 1 / (1 + p x) for x >= 0, whose error is at most 1.5e-7 (at most 0.75e-7 in Phi).  The
// exponential is the one the density needs; erff costs three times as many instructions.
__device__ __forceinline__ float normal_cdf(float z, float &e) {
    const float x = __builtin_fabsf(z) * 0.70710678118654752f;
    e = fast_exp(-0.5f * z * z);
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3275911f, x, 1.0f));
    float q = __builtin_fmaf(1.061405429f, t, -1.453152027f);
    q = __builtin_fmaf(q, t, 1.421413741f);
    q = __builtin_fmaf(q, t, -0.284496736f);
    q = __builtin_fmaf(q, t, 0.254829592f);
    const float tail = 0.5f * q * t * e;  // Phi(-|z|)
    return z < 0.0f ? tail : 1.0f - tail;
}

// act(z), in fp32.
template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == TCQ_ACT_RELU) return z < 0.0f ? 0.0f : z;  // NaN stays NaN
    if constexpr (ACT == TCQ_ACT_SILU) return z * sigmoid(z);
    if constexpr (ACT == TCQ_ACT_GELU) {
        float e;
        return z * normal_cdf(z, e);
    }
    return z;
}

// g act'(z), in fp32.  relu selects (0 at z <= 0, whatever g holds there), and a NaN z gives
// NaN as the other activations do: a checkpoint's group with an infinity stands for NaN,
// which must not pass for closed units.
template <int ACT>
__device__ __forceinline__ float act_grad(float g, float z) {
    if constexpr (ACT == TCQ_ACT_RELU) return z > 0.0f ? g : (z <= 0.0f ? 0.0f : z);
    if constexpr (ACT == TCQ_ACT_SILU) {
        const float s = sigmoid(z);
        return g * (s * __builtin_fmaf(z, 1.0f - s, 1.0f));
    }
    if constexpr (ACT == TCQ_ACT_GELU) {
        float e;
        const float c = normal_cdf(z, e);
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
