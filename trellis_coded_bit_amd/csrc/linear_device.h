// Element types, activations and checkpoint scales of the coded linear layer (device code).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "tcq.h"

namespace tcq {

// The C ABI's name of an element type.
template <typename T>
constexpr int dtype_of() {
    return sizeof(T) == 4 ? TCQ_F32 : (__is_same(T, _Float16) ? TCQ_F16 : TCQ_BF16);
}

// act(z), in fp32.
__device__ __forceinline__ float act_value(float z, int act) {
    switch (act) {
        case TCQ_ACT_RELU: return z < 0.0f ? 0.0f : z;  // NaN stays NaN
        case TCQ_ACT_SILU: return z / (1.0f + expf(-z));
        case TCQ_ACT_GELU: return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
        default: return z;
    }
}

// act'(z), in fp32 (relu: 1 for z > 0, else 0).
__device__ __forceinline__ float act_slope(float z, int act) {
    switch (act) {
        case TCQ_ACT_RELU: return z > 0.0f ? 1.0f : 0.0f;
        case TCQ_ACT_SILU: {
            const float s = 1.0f / (1.0f + expf(-z));
            return s * (1.0f + z * (1.0f - s));
        }
        case TCQ_ACT_GELU:
            // Phi(z) + z phi(z)
            return 0.5f * (1.0f + erff(z * 0.70710678118654752f)) +
                   z * (0.39894228040143268f * expf(-0.5f * z * z));
        default: return 1.0f;
    }
}

// Value of a checkpoint code q whose group has scale byte e: q 2^(e - 133), exact in fp32;
// e = 255 marks a group that held an infinity or a NaN.
__device__ __forceinline__ float code_value(int q, int e) {
    if (e == 255) return __int_as_float(0x7FC00000);
    return __builtin_amdgcn_ldexpf(static_cast<float>(q), e - 133);
}

}  // namespace tcq
