// 8-bit activation checkpoints: groups of 32 consecutive values of a row share one scale
// byte e, the exponent field of the group's largest magnitude as an fp32 number, and each
// value is held as an int8 code q standing for q 2^(e - 133):
//     q = clamp(round_half_even(x 2^(133 - e)), -127, 127).
// With a power of two as the scale both directions are exact apart from the one rounding
// to an integer, and every code's value is a bf16 number, so a product can read the
// checkpoint without rounding it again.  e = 255 (an infinity or a NaN in the group) makes
// the whole group NaN.
#include <hip/hip_runtime.h>

#include "linear_device.h"
#include "tcq.h"
#include "tcq_internal.h"

namespace tcq {
namespace {

constexpr int kGroup = 32;

template <typename T>
__global__ __launch_bounds__(256) void act_pack_kernel(const T *__restrict__ X, int64_t rows,
                                                       int64_t cols, int64_t ldx,
                                                       int8_t *__restrict__ codes, int64_t ldq,
                                                       uint8_t *__restrict__ scale) {
    const int64_t groups = (cols + kGroup - 1) / kGroup;
    const int64_t total = rows * groups;
    const int el = threadIdx.x & 31;
    for (int64_t gq = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); gq < total;
         gq += static_cast<int64_t>(gridDim.x) * 8) {
        const int64_t r = gq / groups, g = gq - r * groups;
        const int64_t c = g * kGroup + el;
        const float x = c < cols ? static_cast<float>(X[r * ldx + c]) : 0.0f;
        // magnitudes order like their bit patterns (NaN above infinity)
        uint32_t top = __float_as_uint(x) & 0x7FFFFFFFu;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
            const uint32_t other = __shfl_xor(top, o);
            top = top > other ? top : other;
        }
        const int e = static_cast<int>(top >> 23);
        float q = __builtin_rintf(__builtin_amdgcn_ldexpf(x, 133 - e));
        q = q > 127.0f ? 127.0f : (q < -127.0f ? -127.0f : q);
        if (e == 255) q = 0.0f;
        if (c < cols) codes[r * ldq + c] = static_cast<int8_t>(static_cast<int>(q));
        if (el == 0) scale[gq] = static_cast<uint8_t>(e);
    }
}

template <typename T>
__global__ __launch_bounds__(256) void act_unpack_kernel(const int8_t *__restrict__ codes,
                                                         int64_t ldq,
                                                         const uint8_t *__restrict__ scale,
                                                         int64_t rows, int64_t cols,
                                                         T *__restrict__ out, int64_t ldo,
                                                         int64_t padded) {
    const int64_t groups = (cols + kGroup - 1) / kGroup;
    const int64_t total = rows * padded;
    for (int64_t q = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; q < total;
         q += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t r = q / padded, c = q - r * padded;
        float v = 0.0f;
        if (c < cols) v = code_value(codes[r * ldq + c], scale[r * groups + c / kGroup]);
        out[r * ldo + c] = static_cast<T>(v);
    }
}

unsigned grid_for(int64_t work, int64_t per) {
    int64_t g = (work + per - 1) / per;
    if (g > (1 << 20)) g = 1 << 20;
    return static_cast<unsigned>(g < 1 ? 1 : g);
}

template <typename T>
hipError_t pack(const void *X, int64_t rows, int64_t cols, int64_t ldx, int8_t *codes,
                int64_t ldq, uint8_t *scale, hipStream_t s) {
    const int64_t groups = (cols + kGroup - 1) / kGroup;
    hipLaunchKernelGGL(act_pack_kernel<T>, dim3(grid_for(rows * groups, 8)), dim3(256), 0, s,
                       static_cast<const T *>(X), rows, cols, ldx, codes, ldq, scale);
    return hipGetLastError();
}

template <typename T>
hipError_t unpack(const int8_t *codes, int64_t ldq, const uint8_t *scale, int64_t rows,
                  int64_t cols, void *out, int64_t ldo, int64_t padded, hipStream_t s) {
    hipLaunchKernelGGL(act_unpack_kernel<T>, dim3(grid_for(rows * padded, 256)), dim3(256), 0, s,
                       codes, ldq, scale, rows, cols, static_cast<T *>(out), ldo, padded);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_act_pack(const void *X, int dtype, int64_t rows, int64_t cols, int64_t ldx,
                           int8_t *codes, int64_t ldq, uint8_t *scale, hipStream_t s) {
    switch (dtype) {
        case TCQ_F32: return pack<float>(X, rows, cols, ldx, codes, ldq, scale, s);
        case TCQ_F16: return pack<_Float16>(X, rows, cols, ldx, codes, ldq, scale, s);
        default: return pack<__bf16>(X, rows, cols, ldx, codes, ldq, scale, s);
    }
}

hipError_t launch_act_unpack(const int8_t *codes, int64_t ldq, const uint8_t *scale,
                             int64_t rows, int64_t cols, int dtype, void *out, int64_t ldo,
                             int64_t padded, hipStream_t s) {
    switch (dtype) {
        case TCQ_F32: return unpack<float>(codes, ldq, scale, rows, cols, out, ldo, padded, s);
        case TCQ_F16:
            return unpack<_Float16>(codes, ldq, scale, rows, cols, out, ldo, padded, s);
        default: return unpack<__bf16>(codes, ldq, scale, rows, cols, out, ldo, padded, s);
    }
}

}  // namespace tcq
